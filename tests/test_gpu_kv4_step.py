"""Decode steps and prefill with the rotary variants and with the 4-bit cache, against the float64 oracle."""
import numpy as np
import pytest

import oracle
from quantized_moe_decode_gb300 import binding, synth

from helpers import make_ctx, make_oracle
from parity import rel_l2, run_parity

pytestmark = pytest.mark.gpu

# Both sides decide codes in fp32, on keys and values that agree to rounding, so a code may fall one step apart, as with
# int8 activations: the bound per vector is the one that holds there for one step on every code, the median the plain one.
PER_VECTOR, MEDIAN = 2e-2, 2e-3

ROPES = [dict(rope_layout=1), dict(rope_dims=24), dict(rope_layout=1, rope_dims=10, rope_scaling=1, rope_factor=2.0),
         dict(rope_dims=48, rope_scaling=2, rope_factor=4.0, rope_orig_len=16),
         dict(rope_scaling=2, rope_factor=8.0, rope_orig_len=64, rope_beta_fast=8.0, rope_beta_slow=0.5, rope_mscale=1.25)]


def _dense(**kw):
    base = dict(hidden=256, n_heads=4, head_dim=64, n_layers=2, n_dense_layers=2, dense_inter=512, prefix_len=20, ring_len=8,
                max_rows=3)
    base.update(kw)
    return synth.ModelConfig(**base)


@pytest.mark.parametrize("rope", ROPES)
@pytest.mark.parametrize("cache", ["f16", "int8"])
def test_rotary_variants_in_the_step(cuda, rope, cache):
    cfg = _dense(kv_int8=int(cache == "int8"), **rope)
    wl = synth.make_workload("rope", cfg, 3, 10, 300)
    ctx = make_ctx(wl)
    run_parity(ctx, wl, 10, make_oracle(wl))
    ctx.close()


def _int4_oracle(wl):
    return oracle.OracleModel(wl.cfg, wl.tensors, wl.rows, kv_prefix=wl.kv_prefix, sinks=wl.sinks, kv_int4=True)


@pytest.mark.parametrize("kw,rows", [
    (dict(), 3), (dict(use_sink=1, head_dim=32, n_heads=8, **{**ROPES[3], "rope_dims": 28}), 1), (dict(head_dim=128, n_heads=2, prefix_len=70), 20),
    (dict(act_int8=1, kv_track=1, **ROPES[2]), 6)])
def test_int4_decode_steps(cuda, kw, rows):
    torch = cuda
    cfg = _dense(kv_int4=1, max_rows=rows, **kw)
    wl = synth.make_workload("int4", cfg, rows, 12, 301)
    ctx = make_ctx(wl)
    orc = oracle.OracleModel(cfg, wl.tensors, rows, kv_prefix=wl.kv_prefix, sinks=wl.sinks, kv_int4=True,
                             act_int8=bool(cfg.act_int8))
    rels = []
    x = torch.zeros((rows, cfg.hidden), dtype=torch.int16, device="cuda")
    y = torch.zeros((rows, cfg.hidden), dtype=torch.float32, device="cuda")
    for s in range(12):  # past the ring's wrap
        p = wl.start_pos + s
        pos = torch.full((rows,), p, dtype=torch.int32, device="cuda")
        x.copy_(torch.from_numpy(np.ascontiguousarray(wl.step_x[s]).view(np.int16)))
        ctx.uocr_decode_step_embeds(rows, x.data_ptr(), pos.data_ptr(), y.data_ptr())
        ctx.uocr_sync()
        res = orc.step(np.full(rows, p), x=wl.step_x[s])
        got = y.cpu().numpy()
        rels += [rel_l2(got[r], res.hidden[-1][r]) for r in range(rows)]
        # layer 0 sees the same inputs on both sides: the entries' values differ by a step at most
        slot = p if p < cfg.prefix_len else cfg.prefix_len + (p - cfg.prefix_len) % cfg.ring_len
        _, ks, _, _, vs, _ = ctx.uocr_kv_read_i4(0, 0, slot, 1)
        k, v = ctx.uocr_kv_read(0, 0, slot, 1)
        for g, sc, w in ((k, ks, res.k_new[0, 0]), (v, vs, res.v_new[0, 0])):
            one = np.repeat(sc[:, 0].astype(np.float64), 32, -1)
            assert np.all(np.abs(g[:, 0].astype(np.float64) - w) <= 1.05 * one + 2e-3 * np.abs(w) + 1e-4)
    print(f"\nint4 step: worst rel-L2 {max(rels):.2e}, median {np.median(rels):.2e}")
    assert max(rels) <= PER_VECTOR and np.median(rels) <= MEDIAN
    if cfg.kv_track:
        w = torch.zeros(cfg.n_layers, rows, cfg.n_heads, cfg.prefix_len, device="cuda")
        ctx.uocr_kv_weights_read(-1, 0, rows, 0, cfg.prefix_len, w.data_ptr())
        ctx.uocr_sync()
        s = w.sum(-1).cpu().numpy()
        assert np.all(s > 0) and np.all(s < 12)  # twelve queries' weights, some of them on generated tokens
    ctx.close()


@pytest.mark.parametrize("track", [0, 1])
def test_int4_prefill_then_steps(cuda, track):
    torch = cuda
    cfg = _dense(kv_int4=1, kv_track=track, max_rows=2, prefix_len=100, **ROPES[3])
    wl = synth.make_workload("int4_prefill", cfg, 2, 3, 302)
    ctx = binding.Context(cfg, max_rows=2)
    ctx.uocr_load_weights(wl.tensors)
    orc = oracle.OracleModel(cfg, wl.tensors, 2, kv_int4=True)
    rng = np.random.default_rng(4)
    prompt = rng.standard_normal((2, 100, cfg.hidden)).astype(np.float16)
    for r in range(2):
        x = torch.from_numpy(prompt[r].view(np.int16)).cuda()
        ctx.uocr_prefill(r, 100, 0, x_ptr=x.data_ptr())
        ctx.uocr_sync()
    for p in range(100):
        res = orc.step(np.full(2, p), x=prompt[:, p])
    last = ctx.uocr_debug_hidden(2 * cfg.n_layers - 1, 36)[35]
    rels = [rel_l2(last, res.hidden[-1][1])]
    y = torch.zeros((2, cfg.hidden), dtype=torch.float32, device="cuda")
    for s in range(3):
        pos = torch.full((2,), 100 + s, dtype=torch.int32, device="cuda")
        x = torch.from_numpy(np.ascontiguousarray(wl.step_x[s]).view(np.int16)).cuda()
        ctx.uocr_decode_step_embeds(2, x.data_ptr(), pos.data_ptr(), y.data_ptr())
        ctx.uocr_sync()
        res = orc.step(np.full(2, 100 + s), x=wl.step_x[s])
        rels += [rel_l2(y.cpu().numpy()[r], res.hidden[-1][r]) for r in range(2)]
    print(f"\nint4 prefill: rel-L2 {['%.2e' % r for r in rels]}")
    assert max(rels) <= PER_VECTOR
    if track:  # 103 queries of every row and layer gave a weight of one each (what the ring dropped apart)
        w = torch.zeros(2, 2, 4, 108, device="cuda")
        ctx.uocr_kv_weights_read(-1, 0, 2, 0, 108, w.data_ptr())
        ctx.uocr_sync()
        assert np.allclose(w.sum(-1).cpu().numpy(), 103, rtol=1e-4)
    ctx.close()


def test_steps_after_an_eviction(cuda):
    """Evicted in place or into a fresh row, with graphs or without: the same steps."""
    torch = cuda
    cfg = _dense(kv_int4=1, kv_track=1, max_rows=2, prefix_len=64, ring_len=8)
    wl = synth.make_workload("int4_evict", cfg, 2, 6, 303)
    outs = []
    for graphs, dst in ((1, 0), (0, 0), (1, 1)):
        ctx = make_ctx(wl, use_graphs=graphs)
        y = torch.zeros((2, cfg.hidden), dtype=torch.float32, device="cuda")
        got = []
        for s in range(6):
            x = torch.from_numpy(np.ascontiguousarray(np.repeat(wl.step_x[s][:1], 2, 0)).view(np.int16)).cuda()
            pos = torch.tensor([64 + s] * 2, dtype=torch.int32, device="cuda")
            if s == 3:
                ctx.uocr_kv_evict(-1, [0], [dst], 64, 17, 2)
                if dst:  # the ring is not part of an eviction: bring it along
                    for l in range(cfg.n_layers):
                        ctx.uocr_kv_write_i4(1, l, 64, *ctx.uocr_kv_read_i4(0, l, 64, 8))
            ctx.uocr_decode_step_embeds(2, x.data_ptr(), pos.data_ptr(), y.data_ptr())
            ctx.uocr_sync()
            if s >= 3:
                got.append(y[dst].cpu().numpy().copy())
        outs.append(np.stack(got))
        ctx.close()
    assert np.all(np.isfinite(outs[0]))
    assert np.array_equal(outs[0], outs[1]) and np.array_equal(outs[0], outs[2])


def test_prefill_refuses_an_evicted_prefix(cuda):
    torch = cuda
    cfg = _dense(kv_int4=1, kv_track=1, max_rows=2, prefix_len=32)
    wl = synth.make_workload("int4_refuse", cfg, 2, 1, 304)
    ctx = make_ctx(wl)
    x = torch.zeros((40, cfg.hidden), dtype=torch.int16, device="cuda")
    ctx.uocr_kv_evict(1, [0], [0], 20, 5)
    with pytest.raises(binding.UocrError) as e:
        ctx.uocr_prefill(0, 4, 19, x_ptr=x.data_ptr())
    assert e.value.status == binding.UOCR_E_STATE
    ctx.uocr_prefill(0, 4, 20, x_ptr=x.data_ptr())
    ctx.uocr_prefill(1, 4, 0, x_ptr=x.data_ptr())
    ctx.uocr_kv_reset(0, 0)
    ctx.uocr_prefill(0, 40, 0, x_ptr=x.data_ptr())
    ctx.uocr_sync()
    ctx.close()
