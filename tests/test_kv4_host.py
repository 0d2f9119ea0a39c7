"""The 4-bit cache and the rotary variants without a GPU: the oracle against hand-made cases and properties, and the
configs that the library refuses before any device work."""
import math

import numpy as np
import pytest

import oracle
from quantized_moe_decode_gb300 import binding, synth


def _cfg(**kw):
    base = dict(hidden=64, n_heads=2, head_dim=64, n_layers=1, n_dense_layers=1, dense_inter=64, prefix_len=8, ring_len=4)
    base.update(kw)
    return synth.ModelConfig(**base)


# ------------------------------------------------------------------ rotary positions
def test_default_layout_is_the_plain_rotation():
    v = np.random.default_rng(0).standard_normal((3, 64))
    cfg = _cfg()
    for p in (0, 1, 37, 5000):
        assert np.allclose(oracle.rope_cfg(v, p, cfg), oracle.rope(v, p, cfg.rope_theta), atol=1e-12)


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("dims", [0, 2, 20, 64])
def test_scores_depend_on_the_distance_and_other_dimensions_pass(layout, dims):
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((2, 64))
    cfg = _cfg(rope_layout=layout, rope_dims=dims)
    a = oracle.rope_cfg(q, 310, cfg) @ oracle.rope_cfg(k, 300, cfg)
    b = oracle.rope_cfg(q, 10, cfg) @ oracle.rope_cfg(k, 0, cfg)
    assert abs(a - b) < 1e-9
    rd = dims or 64
    assert np.array_equal(oracle.rope_cfg(q, 99, cfg)[rd:], q[rd:])


def test_interleaved_is_the_half_layout_permuted():
    v = np.random.default_rng(2).standard_normal(64)
    order = np.concatenate([np.arange(0, 64, 2), np.arange(1, 64, 2)])
    half = oracle.rope_cfg(v[order], 41, _cfg())
    assert np.allclose(oracle.rope_cfg(v, 41, _cfg(rope_layout=1))[order], half, atol=1e-12)


def test_scaled_frequencies_in_closed_form():
    plain, one = oracle.rope_frequencies(_cfg())
    lin, amp = oracle.rope_frequencies(_cfg(rope_scaling=1, rope_factor=4.0))
    assert one == amp == 1.0 and np.allclose(lin * 4, plain, rtol=1e-15)
    cfg = _cfg(rope_scaling=2, rope_factor=8.0, rope_orig_len=4096)
    inv, amp = oracle.rope_frequencies(cfg)
    assert amp == pytest.approx(0.1 * math.log(8.0) + 1.0)
    turns = 4096 * plain / (2 * math.pi)
    # a pair is left alone or divided in full but for the whole pairs around the two bounds
    fast, slow = np.flatnonzero(turns > 32)[:-1], np.flatnonzero(turns < 1)[1:]
    assert np.allclose(inv[fast], plain[fast], rtol=1e-12) and np.allclose(inv[slow], plain[slow] / 8, rtol=1e-12)
    assert np.all(np.diff(inv / plain) <= 1e-15) and fast.size and slow.size
    assert oracle.rope_frequencies(cfg.replace(rope_mscale=1.5))[1] == 1.5


# ------------------------------------------------------------------ entries
def test_entry_of_hand_made_groups():
    x = np.zeros(96, np.float32)
    x[:32] = np.linspace(-1.5, 1.5, 32)       # step 0.2 over the group
    x[32:64] = 3.0                              # one value: scale 0
    x[64:] = np.arange(32) % 16 * 0.25 - 2.0  # exactly representable
    q, s, m = oracle.kv4_quant(x)
    assert m[0] == np.float16(-1.5) and abs(float(s[0]) - 0.2) <= 0.2 * 2.0 ** -10 and float(s[0]) <= 0.2
    assert q[0] == 0 and q[31] == 15
    assert s[1] == 0 and m[1] == 3.0 and not q[32:64].any()
    assert s[2] == 0.25 and m[2] == -2.0 and np.array_equal(q[64:], np.arange(32) % 16)
    v = oracle.kv4_value(q, s, m)
    assert np.array_equal(v[64:], x[64:]) and np.array_equal(v[32:64], x[32:64])


def test_entry_error_is_half_a_step():
    """|x - value| <= s/2, plus what the top code loses to the scale's rounding toward zero (15 s 2^-10), the
    minimum's rounding (half a step of fp16) and the value's own (2^-11 of it)."""
    x = (np.random.default_rng(3).standard_normal((200, 64)) * np.exp(np.linspace(-3, 3, 200))[:, None]).astype(np.float32)
    q, s, m = oracle.kv4_quant(x)
    v = oracle.kv4_value(q, s, m)
    S, M = np.repeat(s, 32, -1).astype(np.float64), np.repeat(np.abs(m), 32, -1).astype(np.float64)
    assert np.all(np.abs(v - x) <= S * (0.5 + 15 * 2.0 ** -10) + (M + np.abs(x)) * 2.0 ** -11 + 1e-7)
    assert q.max() == 15 and q.min() == 0


def test_entry_extremes_and_what_cannot_be_held():
    x = np.zeros((4, 32), np.float32)
    x[0, 0], x[0, 1] = 65504, -65504
    x[1, 5] = np.nan
    x[2, 5] = np.inf
    x[3, 5] = 7e4
    q, s, m = oracle.kv4_quant(x)
    v = oracle.kv4_value(q, s, m)
    assert np.all(np.isfinite(v[0])) and v[0, 1] == -65504
    assert np.all(np.isnan(v[1:]))


def test_evict_choice_rules():
    w = np.array([0.0, 5, 1, 5, 1, np.nan, 1, 9])
    assert oracle.evict_choice(w, 8, 3, 0).tolist() == [1, 3, 7]
    assert oracle.evict_choice(w, 8, 4, 1).tolist() == [0, 1, 3, 7]
    assert oracle.evict_choice(w, 8, 4, 0).tolist() == [1, 2, 3, 7]      # the lowest of the equal ones
    assert oracle.evict_choice(w, 8, 7, 0).tolist() == [0, 1, 2, 3, 4, 6, 7]  # the NaN goes first
    assert oracle.evict_choice(w, 8, 3, 0, (2, 4)).tolist() == [1, 4, 7]
    assert oracle.evict_choice(w, 8, 0, 0).size == 0


# ------------------------------------------------------------------ configs
@pytest.mark.parametrize("bad", [
    dict(kv_int4=2), dict(kv_int4=1, kv_int8=1), dict(kv_int4=1, head_dim=16, n_heads=4), dict(kv_track=1),
    dict(kv_int4=1, kv_track=-1), dict(rope_layout=2), dict(rope_dims=66), dict(rope_dims=7), dict(rope_dims=-2),
    dict(rope_scaling=3), dict(rope_scaling=1, rope_factor=0.5), dict(rope_scaling=1, rope_factor=float("nan")),
    dict(rope_scaling=2, rope_factor=2.0), dict(rope_scaling=2, rope_factor=2.0, rope_orig_len=64, rope_beta_slow=40.0),
    dict(rope_scaling=2, rope_factor=2.0, rope_orig_len=64, rope_theta=1.0),
    dict(rope_scaling=2, rope_factor=2.0, rope_orig_len=64, rope_mscale=-1.0)])
def test_config_refusals(libuocr, bad):
    with pytest.raises(binding.UocrError) as e:
        binding.Context(_cfg(**bad))
    assert e.value.status == binding.UOCR_E_INVALID_ARG
    assert "invalid config" in str(e.value)


def test_buffers_of_the_wrong_type_are_refused():
    torch = pytest.importorskip("torch")
    with pytest.raises(ValueError):
        binding._buffer(torch.zeros(4, dtype=torch.int16), np.uint8)
    with pytest.raises(ValueError):
        binding._buffer(torch.zeros((4, 4), dtype=torch.uint8).t(), np.uint8)
    p, keep = binding._buffer(torch.zeros(4, dtype=torch.float16), np.float16)
    assert p == keep.data_ptr()
