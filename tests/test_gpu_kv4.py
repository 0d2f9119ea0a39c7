"""The 4-bit cache's operators on the GPU, through the C ABI, against the float64 oracle: rotary positions and the
append, attention (weights accumulated or not), eviction; their refusals; and runs of them together.

Tolerances.  Entries: the oracle decides in fp32 what the kernels decide in fp32 on bit-equal inputs, so codes, scales
and minima are equal.  Rotated queries: the same fp32 roundings, equal.  Attention: q, the values and the weights enter
with at least 2^-21 relative each, accumulated in fp32 over at most a few thousand terms, with exponentials of 2^-21:
F32 = 2e-5 on the 2-norm and on single values relative to the largest; a 16-bit output adds half a step
(fp16 2^-11, bf16 2^-8 of the value)."""
import numpy as np
import pytest

import oracle
from quantized_moe_decode_gb300 import binding, synth

pytestmark = pytest.mark.gpu

F32 = 2e-5
HALF_STEP = {0: 0.0, 1: 2.0 ** -11, 2: 2.0 ** -8}


def _cfg(**kw):
    base = dict(hidden=64, n_heads=2, head_dim=64, n_layers=1, n_dense_layers=1, dense_inter=64, prefix_len=40,
                ring_len=16, max_rows=4, kv_int4=1)
    base.update(kw)
    if base["n_heads"] * base["head_dim"] % 64:
        base["n_heads"] += 1
    return synth.ModelConfig(**base)


def _dt(torch, dtype):
    return {0: torch.float32, 1: torch.float16, 2: torch.bfloat16}[dtype]


def _entries(rng, shape):
    D = shape[-1]
    code = rng.integers(0, 16, shape).astype(np.uint8)
    s = rng.uniform(0.05, 0.4, shape[:-1] + (D // 32,)).astype(np.float16)
    m = (-7.5 * s.astype(np.float64) + 0.3 * rng.standard_normal(s.shape)).astype(np.float16)
    return code, s, m


def _fill(ctx, cfg, rng, layers=1):
    """Random entries in every slot; their values [layers, rows, 2, nh, SL, D]."""
    SL = cfg.prefix_len + cfg.ring_len
    out = np.zeros((layers, cfg.max_rows, 2, cfg.n_heads, SL, cfg.head_dim))
    for l in range(layers):
        for r in range(cfg.max_rows):
            k, v = (_entries(rng, (cfg.n_heads, SL, cfg.head_dim)) for _ in range(2))
            ctx.uocr_kv_write_i4(r, l, 0, *k, *v)
            out[l, r, 0], out[l, r, 1] = oracle.kv4_value(*k), oracle.kv4_value(*v)
    return out


def _close(got, want, dtype, what=""):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    assert got.shape == want.shape
    step = HALF_STEP[dtype]
    top = max(np.abs(want).max(initial=0.0), 1e-30)
    assert np.all(np.abs(got - want) <= F32 * top + step * np.abs(want) * 1.001 + 2.0 ** -25 * (dtype == 1)), what
    assert np.linalg.norm(got - want) <= (F32 + step) * np.linalg.norm(want), what


def _attend(torch, ctx, cfg, q, positions=None, chunk=None, dtype=0):
    n, qh, D = q.shape
    qd = torch.from_numpy(np.ascontiguousarray(q, np.float32)).cuda()
    out = torch.full((n, qh, D), 7.0, dtype=_dt(torch, dtype), device="cuda")
    if chunk is None:
        pos = torch.tensor(positions, dtype=torch.int32, device="cuda")
        ctx.uocr_attend(0, n, pos.data_ptr(), qh, qd.data_ptr(), out.data_ptr(), dtype)
    else:
        ctx.uocr_attend_chunk(0, chunk[0], chunk[1], n, qh, qd.data_ptr(), out.data_ptr(), dtype)
    ctx.uocr_sync()
    return out.double().cpu().numpy()


def _weights(torch, ctx, cfg, layer=0, rows=None, n=None):
    rows, n = rows or cfg.max_rows, n or cfg.prefix_len + cfg.ring_len
    layers = cfg.n_layers if layer == -1 else 1
    w = torch.full((layers, rows, cfg.n_heads, n), -1.0, device="cuda")
    ctx.uocr_kv_weights_read(layer, 0, rows, 0, n, w.data_ptr())
    ctx.uocr_sync()
    w = w.double().cpu().numpy()
    return w if layer == -1 else w[0]


def _read(ctx, cfg, row, layer=0):
    return ctx.uocr_kv_read_i4(row, layer, 0, cfg.prefix_len + cfg.ring_len)


# ------------------------------------------------------------------ entries
@pytest.mark.parametrize("dim", [32, 64, 128, 256])
def test_entries_round_trip_and_read_as_their_values(cuda, dim):
    rng = np.random.default_rng(dim)
    cfg = _cfg(head_dim=dim, n_heads=3, prefix_len=37, n_layers=2, n_dense_layers=2)
    ctx = binding.Context(cfg, max_rows=3)
    nh = cfg.n_heads
    k, v = (_entries(rng, (nh, 21, dim)) for _ in range(2))
    ctx.uocr_kv_write_i4(1, 1, 7, *k, *v)
    got = ctx.uocr_kv_read_i4(1, 1, 7, 21)
    for a, b in zip(got, k + v):
        assert np.array_equal(a, b)
    assert not any(x.any() for x in ctx.uocr_kv_read_i4(1, 1, 0, 7)) and not any(x.any() for x in ctx.uocr_kv_read_i4(1, 1, 28, 25))
    assert not any(x.any() for x in _read(ctx, cfg, 0, 1)) and not any(x.any() for x in _read(ctx, cfg, 1, 0))
    kd, vd = ctx.uocr_kv_read(1, 1, 7, 21)
    assert np.array_equal(kd, oracle.kv4_value(*k).astype(np.float16))
    assert np.array_equal(vd, oracle.kv4_value(*v).astype(np.float16))
    # a written fp16 vector is quantised as the oracle quantises it
    x = rng.standard_normal((2, nh, 5, dim)).astype(np.float16)
    ctx.uocr_kv_write(2, 0, 30, x[0], x[1])
    got = ctx.uocr_kv_read_i4(2, 0, 30, 5)
    for a, b in zip(got, oracle.kv4_quant(x[0]) + oracle.kv4_quant(x[1])):
        assert np.array_equal(a, b)
    ctx.close()


# ------------------------------------------------------------------ append
CASES = [  # dim, layout, rope_dims, scaling, dtype, group, strided
    (32, 0, 0, 0, 1, 1, False), (32, 1, 6, 1, 0, 8, True), (64, 0, 24, 2, 2, 1, True), (64, 1, 0, 2, 1, 2, False),
    (128, 0, 0, 0, 1, 1, True), (128, 1, 64, 0, 2, 3, False), (128, 0, 2, 1, 0, 1, False), (256, 0, 200, 2, 1, 1, True),
    (256, 1, 0, 0, 0, 4, False)]


def _qkv(torch, rng, n, qh, nh, D, dtype, strided):
    """Device queries, keys, values (views of one buffer when strided) and their fp32 values."""
    dt = _dt(torch, dtype)
    x = torch.from_numpy((rng.standard_normal((n, qh + 2 * nh + 1, D)) * np.exp(0.5 * rng.standard_normal((1, 1, D)))).astype(np.float32)).to(dt).cuda()
    f = x.float().cpu().numpy()
    parts = f[:, :qh], f[:, qh:qh + nh], f[:, qh + nh:qh + 2 * nh]
    if strided:
        ld = (qh + 2 * nh + 1) * D
        e = x.element_size()
        ptrs = x.data_ptr(), x.data_ptr() + qh * D * e, x.data_ptr() + (qh + nh) * D * e
        return ptrs, dict(ld_q=ld, ld_k=ld, ld_v=ld), parts, x
    keep = [x[:, :qh].contiguous(), x[:, qh:qh + nh].contiguous(), x[:, qh + nh:qh + 2 * nh].contiguous()]
    return tuple(t.data_ptr() for t in keep), {}, parts, keep


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("chunk", [False, True])
def test_append_against_the_oracle(cuda, case, chunk):
    torch = cuda
    dim, layout, rd, scaling, dtype, G, strided = case
    rng = np.random.default_rng(dim + 7 * layout + rd + chunk)
    cfg = _cfg(head_dim=dim, n_heads=3, rope_layout=layout, rope_dims=rd, rope_scaling=scaling, rope_factor=4.0,
               rope_orig_len=256, prefix_len=35, ring_len=9, max_rows=5)
    ctx = binding.Context(cfg, max_rows=5)
    nh, P, R = cfg.n_heads, cfg.prefix_len, cfg.ring_len
    before = _fill(ctx, cfg, rng)
    old = [_read(ctx, cfg, r) for r in range(5)]
    n = 29 if chunk else 5
    pos = list(range(13, 13 + n)) if chunk else [0, 34, 35, 43, 100_003]
    rows = [2] * n if chunk else list(range(n))
    ptrs, ld, (fq, fk, fv), keep = _qkv(torch, rng, n, nh * G, nh, dim, dtype, strided)
    q_out = torch.zeros(n, nh * G, dim, device="cuda")
    kval, vval = (torch.zeros(n, nh, dim, dtype=torch.float16, device="cuda") for _ in range(2))
    kw = dict(dtype=dtype, q_heads=nh * G, q_out=q_out.data_ptr(), k_val=kval.data_ptr(), v_val=vval.data_ptr(), **ld)
    if chunk:
        ctx.uocr_kv_append_chunk(0, 2, 13, n, *ptrs, **kw)
    else:
        p = torch.tensor(pos, dtype=torch.int32, device="cuda")
        ctx.uocr_kv_append(0, n, p.data_ptr(), *ptrs, **kw)
    ctx.uocr_sync()
    want_q = np.stack([oracle.rotate_f32(fq[i], pos[i], cfg) for i in range(n)])
    assert np.array_equal(q_out.cpu().numpy(), want_q)
    now = [_read(ctx, cfg, r) for r in range(5)]
    for i in range(n):
        slot = pos[i] if pos[i] < P else P + (pos[i] - P) % R
        want = oracle.kv4_quant(oracle.rotate_f32(fk[i], pos[i], cfg)) + oracle.kv4_quant(fv[i])
        for j, w in enumerate(want):
            assert np.array_equal(now[rows[i]][j][:, slot], w), (i, j)
            old[rows[i]][j][:, slot] = w
        assert np.array_equal(kval[i].double().cpu().numpy(), oracle.kv4_value(*want[:3]))
        assert np.array_equal(vval[i].double().cpu().numpy(), oracle.kv4_value(*want[3:]))
    for r in range(5):  # every other slot as it was
        for a, b in zip(now[r], old[r]):
            assert np.array_equal(a, b)
    assert before.shape[1] == 5 and keep is not None
    ctx.close()


def test_append_of_what_an_entry_cannot_hold_reads_as_nan(cuda):
    torch = cuda
    cfg = _cfg(head_dim=64, n_heads=2, rope_dims=2)
    ctx = binding.Context(cfg, max_rows=1)
    k = torch.randn(3, 2, 64, device="cuda")
    v = torch.randn(3, 2, 64, device="cuda")
    k[0, 0, 40], v[1, 1, 3], v[2, 0, 63] = float("nan"), float("inf"), 1e5
    kval, vval = (torch.zeros(3, 2, 64, dtype=torch.float16, device="cuda") for _ in range(2))
    ctx.uocr_kv_append_chunk(0, 0, 0, 3, 0, k.data_ptr(), v.data_ptr(), dtype=0, k_val=kval.data_ptr(), v_val=vval.data_ptr())
    ctx.uocr_sync()
    kn, vn = kval.isnan().cpu().numpy(), vval.isnan().cpu().numpy()
    want_k, want_v = np.zeros((3, 2, 64), bool), np.zeros((3, 2, 64), bool)
    want_k[0, 0, 32:], want_v[1, 1, :32], want_v[2, 0, 32:] = True, True, True
    assert np.array_equal(kn, want_k) and np.array_equal(vn, want_v)
    ctx.close()


# ------------------------------------------------------------------ attention
@pytest.mark.parametrize("dim", [32, 64, 128, 256])
@pytest.mark.parametrize("group,P,R,sink,dtype", [
    (1, 40, 16, False, 0), (1, 37, 9, True, 1), (2, 0, 5, False, 2), (3, 100, 20, True, 0), (8, 129, 33, False, 1),
    (1, 700, 50, False, 2), (5, 15, 1, True, 1)])
def test_attend_rows(cuda, dim, group, P, R, sink, dtype):
    torch = cuda
    rng = np.random.default_rng(dim + group + P)
    cfg = _cfg(head_dim=dim, n_heads=3, prefix_len=P, ring_len=R, max_rows=7, use_sink=int(sink), kv_track=1)
    ctx = binding.Context(cfg, max_rows=7)
    vals = _fill(ctx, cfg, rng)[0]
    nh = cfg.n_heads
    sinks = rng.standard_normal((1, nh)).astype(np.float32) if sink else None
    if sink:
        ctx.uocr_set_sinks(sinks)
    pos = [0, max(P - 1, 0), P, P + R - 1, P + R, 5 * P + 3 * R + 1, P // 2]
    q = rng.standard_normal((7, nh * group, dim)).astype(np.float32) * 2
    want, w = oracle.attend_kv4(q, vals[:, 0], vals[:, 1], pos, P, R, sinks=None if sinks is None else sinks[0].astype(np.float64))
    _close(_attend(torch, ctx, cfg, q, pos, dtype=dtype), want, dtype)
    _close(_weights(torch, ctx, cfg), w, 0)
    _attend(torch, ctx, cfg, q, pos, dtype=dtype)
    _close(_weights(torch, ctx, cfg), 2 * w, 0)  # the weights add up
    # fewer rows: the others' weights stay
    _attend(torch, ctx, cfg, q[:2], pos[:2], dtype=dtype)
    w[:2] *= 3
    w[2:] *= 2
    _close(_weights(torch, ctx, cfg), w, 0)
    ctx.close()


@pytest.mark.parametrize("n,start,group,P,R,sink", [
    (1, 0, 1, 40, 16, False), (17, 0, 1, 40, 16, True), (56, 0, 2, 40, 16, False), (9, 35, 8, 40, 16, False),
    (70, 60, 1, 131, 8, True), (131, 0, 3, 131, 8, False), (30, 3, 1, 0, 64, False)])
@pytest.mark.parametrize("dim", [32, 64, 128, 256])
def test_attend_chunk_is_causal(cuda, dim, n, start, group, P, R, sink):
    torch = cuda
    rng = np.random.default_rng(dim + n)
    for track in (0, 1):
        cfg = _cfg(head_dim=dim, prefix_len=P, ring_len=R, max_rows=2, use_sink=int(sink), kv_track=track)
        ctx = binding.Context(cfg, max_rows=2)
        vals = _fill(ctx, cfg, rng)[0]
        nh = cfg.n_heads
        sinks = rng.standard_normal((1, nh)).astype(np.float32) if sink else None
        if sink:
            ctx.uocr_set_sinks(sinks)
        q = rng.standard_normal((n, nh * group, dim)).astype(np.float32) * 2
        pos = list(range(start, start + n))
        want, w = oracle.attend_kv4(q, vals[:, 0], vals[:, 1], pos, P, R, causal_row=1,
                                    sinks=None if sinks is None else sinks[0].astype(np.float64))
        dtype = (n + dim) % 3
        _close(_attend(torch, ctx, cfg, q, chunk=(1, start), dtype=dtype), want, dtype)
        if track:
            _close(_weights(torch, ctx, cfg), w, 0)
        ctx.close()


def test_what_a_query_may_not_read_never_reaches_it(cuda):
    """NaN and infinite entries behind the position, in the unwritten ring and in a causal chunk's later tokens."""
    torch = cuda
    rng = np.random.default_rng(5)
    for dim in (32, 128):
        cfg = _cfg(head_dim=dim, prefix_len=50, ring_len=20, max_rows=2, kv_track=1)
        ctx = binding.Context(cfg, max_rows=2)
        vals = _fill(ctx, cfg, rng)[0]
        nh = cfg.n_heads
        bad_from = 23
        c, s, m = _entries(rng, (nh, 70 - bad_from, dim))
        m[:, 0::2], s[:, 1::2] = np.nan, np.inf
        ctx.uocr_kv_write_i4(0, 0, bad_from, c, s, m, c, s, m)
        ctx.uocr_kv_write_i4(1, 0, bad_from, c, s, m, c, s, m)
        q = rng.standard_normal((2, nh, dim)).astype(np.float32)
        want, _ = oracle.attend_kv4(q, vals[:, 0], vals[:, 1], [22, 5], 50, 20)
        _close(_attend(torch, ctx, cfg, q, [22, 5]), want, 0)
        q = rng.standard_normal((30, nh, dim)).astype(np.float32)
        want, _ = oracle.attend_kv4(q, vals[:, 0], vals[:, 1], range(30), 50, 20, causal_row=1)
        got = _attend(torch, ctx, cfg, q, chunk=(1, 0))
        _close(got[:bad_from], want[:bad_from], 0)
        assert np.all(np.isnan(got[bad_from:]))  # a NaN that is read shows
        w = _weights(torch, ctx, cfg)
        assert np.all(np.isfinite(w[0, :, :23]))
        ctx.close()


def test_large_scores_and_equal_scores(cuda):
    torch = cuda
    cfg = _cfg(head_dim=64, prefix_len=300, ring_len=4, max_rows=1, kv_track=1)
    ctx = binding.Context(cfg, max_rows=1)
    rng = np.random.default_rng(6)
    vals = _fill(ctx, cfg, rng)[0]
    for scale in (0.0, 1e-30, 1.0, 300.0, 3e4):
        q = (rng.standard_normal((1, 2, 64)) * scale).astype(np.float32)
        want, _ = oracle.attend_kv4(q, vals[:, 0], vals[:, 1], [299], 300, 4)
        got = _attend(torch, ctx, cfg, q, [299])
        # scores of size S carry 2^-21 S: the weights' relative error follows
        tol = F32 + 64 * scale * 2.0 ** -21
        assert np.abs(got - want).max() <= tol * np.abs(vals[0, 1]).max(), scale
    ctx.close()


# ------------------------------------------------------------------ eviction
def _evict(torch, ctx, cfg, layer, src, dst, n, keep, protect, vals=True):
    layers = cfg.n_layers if layer == -1 else 1
    kept = torch.full((layers, len(src), cfg.n_heads, keep), -1, dtype=torch.int32, device="cuda")
    k, v = (torch.zeros(layers, len(src), cfg.n_heads, keep, cfg.head_dim, dtype=torch.float16, device="cuda") for _ in range(2))
    ctx.uocr_kv_evict(layer, src, dst, n, keep, protect, kept_ptr=kept.data_ptr(),
                      k_val_ptr=k.data_ptr() if vals else 0, v_val_ptr=v.data_ptr() if vals else 0)
    ctx.uocr_sync()
    return kept.cpu().numpy(), k.double().cpu().numpy(), v.double().cpu().numpy()


def _put_weights(torch, ctx, w, layer=0):
    d = torch.from_numpy(np.ascontiguousarray(w, np.float32)).cuda()
    d = d if layer == -1 else d[None]
    ctx.uocr_kv_weights_write(layer, 0, d.shape[1], 0, d.shape[3], d.data_ptr())
    ctx.uocr_sync()


@pytest.mark.parametrize("dim,P,n,keep,protect", [
    (32, 1, 1, 1, 0), (64, 40, 40, 0, 0), (64, 40, 40, 40, 3), (128, 300, 290, 17, 4), (128, 1025, 1025, 512, 0),
    (256, 70, 69, 33, 33), (32, 2000, 1999, 701, 1), (128, 257, 256, 255, 0)])
@pytest.mark.parametrize("in_place", [False, True])
def test_evict_against_the_oracle(cuda, dim, P, n, keep, protect, in_place):
    torch = cuda
    rng = np.random.default_rng(P + keep)
    cfg = _cfg(head_dim=dim, n_heads=2, prefix_len=P, ring_len=6, max_rows=4, kv_track=1, n_layers=2, n_dense_layers=2)
    ctx = binding.Context(cfg, max_rows=4)
    vals = _fill(ctx, cfg, rng, 2)
    SL = P + 6
    w = np.exp(2 * rng.standard_normal((2, 4, 2, SL))).astype(np.float32)
    w = np.round(w * 4) / 4  # many ties
    w[0, 1, 0, ::7] = np.nan
    w[1, 0, 1, ::5] = -0.0
    _put_weights(torch, ctx, w, -1)
    src, dst = [1, 0], ([1, 0] if in_place else [2, 3])
    kept, k, v = _evict(torch, ctx, cfg, -1, src, dst, n, keep, protect)
    after = _weights(torch, ctx, cfg, -1)
    for l in range(2):
        for i, (a, b) in enumerate(zip(src, dst)):
            kr, vr = ctx.uocr_kv_read(b, l, 0, SL)
            for h in range(2):
                want = oracle.evict_choice(w[l, a, h], n, keep, protect)
                assert np.array_equal(kept[l, i, h], want)
                assert np.array_equal(k[l, i, h], vals[l, a, 0, h, want]) and np.array_equal(v[l, i, h], vals[l, a, 1, h, want])
                assert np.array_equal(kr[h, :keep], vals[l, a, 0, h, want].astype(np.float16))
                assert np.array_equal(vr[h, :keep], vals[l, a, 1, h, want].astype(np.float16))
                assert np.array_equal(kr[h, n:], vals[l, b, 0, h, n:].astype(np.float16))  # behind n: as it was
                assert np.array_equal(after[l, b, h, :keep], w[l, a, h, want], equal_nan=True)
                assert not after[l, b, h, keep:n].any()
                assert np.array_equal(after[l, b, h, n:], w[l, b, h, n:], equal_nan=True)
            if not in_place:
                assert np.array_equal(ctx.uocr_kv_read(a, l, 0, SL)[0], vals[l, a, 0].astype(np.float16))
    ctx.close()


@pytest.mark.parametrize("n,keep,protect", [(4097, 1500, 2), (20011, 40, 0), (49153, 30000, 1), (60007, 6001, 7)])
@pytest.mark.parametrize("in_place", [False, True])
def test_evict_of_long_rows(cuda, n, keep, protect, in_place):
    """More entries than shared memory holds weights of; many weights are equal."""
    torch = cuda
    rng = np.random.default_rng(n)
    cfg = _cfg(head_dim=32, n_heads=2, prefix_len=n + 3, ring_len=1, max_rows=2, kv_track=1)
    ctx = binding.Context(cfg, max_rows=2)
    vals = _fill(ctx, cfg, rng)[0]
    w = np.round(rng.random((2, 2, n + 4)) * 500).astype(np.float32)
    _put_weights(torch, ctx, w)
    rd = 0 if in_place else 1
    kept, k, v = _evict(torch, ctx, cfg, 0, [0], [rd], n, keep, protect)
    for h in range(2):
        at = oracle.evict_choice(w[0, h, :n], n, keep, protect)
        assert np.array_equal(kept[0, 0, h], at)
        assert np.array_equal(k[0, 0, h], vals[0, 0, h, at]) and np.array_equal(v[0, 0, h], vals[0, 1, h, at])
        assert np.array_equal(_weights(torch, ctx, cfg)[rd, h, :keep], w[0, h, at])
        assert not np.any(_weights(torch, ctx, cfg)[rd, h, keep:n])
    ctx.close()


def test_attention_skips_what_is_evicted_and_evicts_again(cuda):
    torch = cuda
    rng = np.random.default_rng(8)
    P, R, dim = 90, 12, 128
    cfg = _cfg(head_dim=dim, prefix_len=P, ring_len=R, max_rows=3, kv_track=1)
    nh = cfg.n_heads
    ctx = binding.Context(cfg, max_rows=3)
    vals = _fill(ctx, cfg, rng)[0]
    w = rng.random((3, nh, P + R)).astype(np.float32)
    _put_weights(torch, ctx, w)
    q = rng.standard_normal((3, nh, dim)).astype(np.float32) * 2

    def compacted(state, wts, row, n, keep, protect, hole):
        for h in range(nh):
            at = oracle.evict_choice(wts[row, h], n, keep, protect, hole)
            state[row, :, h, :keep] = state[row][:, h, at]
            wts[row, h, :keep] = wts[row, h, at]
            wts[row, h, keep:n] = 0

    _evict(torch, ctx, cfg, 0, [0, 2], [0, 2], 70, 21, 2)
    w = w.astype(np.float64)
    for r in (0, 2):
        compacted(vals, w, r, 70, 21, 2, (0, 0))
    holes = [(21, 70), (0, 0), (21, 70)]
    for pos in ([75, 75, 89], [P + 3, P, P + 4 * R + 5], [70, 0, 71]):
        want, add = oracle.attend_kv4(q, vals[:, 0], vals[:, 1], pos, P, R, holes)
        _close(_attend(torch, ctx, cfg, q, pos), want, 0)
        w += add
        _close(_weights(torch, ctx, cfg), w, 0)
    # positions inside the evicted prefix are reported
    with pytest.raises(binding.UocrError) as e:
        _attend(torch, ctx, cfg, q, [69, 5, 80])
    assert e.value.status == binding.UOCR_E_POSITION
    w = _weights(torch, ctx, cfg)
    # a second eviction takes from what is left: 21 entries and slots 70..84
    kept, k, v = _evict(torch, ctx, cfg, 0, [0], [1], 85, 30, 0)
    for h in range(nh):
        want = oracle.evict_choice(w[0, h], 85, 30, 0, (21, 70))
        assert np.array_equal(kept[0, 0, h], want) and np.array_equal(k[0, 0, h], vals[0, 0, h, want])
        vals[1, :, h, :30] = vals[0][:, h, want]
    pos = [P + 1, P + 1, P + 1]
    want, _ = oracle.attend_kv4(q, vals[:, 0], vals[:, 1], pos, P, R, [(21, 70), (30, 85), (21, 70)])
    _close(_attend(torch, ctx, cfg, q, pos), want, 0)
    # a chunk goes on behind the evicted prefix
    qc = rng.standard_normal((14, nh, dim)).astype(np.float32)
    want, _ = oracle.attend_kv4(qc, vals[:, 0], vals[:, 1], range(86, 100), P, R, [None, (30, 85), None], causal_row=1)
    _close(_attend(torch, ctx, cfg, qc, chunk=(1, 86)), want, 0)
    ctx.close()


def test_nothing_to_read_gives_zeros(cuda):
    torch = cuda
    cfg = _cfg(prefix_len=20, ring_len=4, max_rows=2, kv_track=1)
    ctx = binding.Context(cfg, max_rows=2)
    rng = np.random.default_rng(9)
    _fill(ctx, cfg, rng)
    _evict(torch, ctx, cfg, 0, [0], [0], 20, 0, 0)
    q = rng.standard_normal((1, cfg.n_heads, 64)).astype(np.float32)
    qd = torch.from_numpy(q).cuda()
    out = torch.full((1, cfg.n_heads, 64), 3.0, device="cuda")
    pos = torch.tensor([11], dtype=torch.int32, device="cuda")
    ctx.uocr_attend(0, 1, pos.data_ptr(), cfg.n_heads, qd.data_ptr(), out.data_ptr(), 0)
    with pytest.raises(binding.UocrError):
        ctx.uocr_sync()  # the position lies in the evicted prefix
    assert not out.any()
    ctx.close()


def test_evicted_slots_refuse_writes_until_reset(cuda):
    torch = cuda
    cfg = _cfg(prefix_len=40, ring_len=8, max_rows=2, kv_track=1)
    ctx = binding.Context(cfg, max_rows=2)
    rng = np.random.default_rng(10)
    _fill(ctx, cfg, rng)
    _evict(torch, ctx, cfg, 0, [0], [0], 30, 10, 0)
    nh, D = cfg.n_heads, cfg.head_dim
    x = np.zeros((nh, 25, D), np.float16)
    e = _entries(rng, (nh, 25, D))
    t = torch.zeros(64, nh, D, device="cuda")
    o = torch.zeros(64, nh, D, device="cuda")
    refused = [lambda: ctx.uocr_kv_write(0, 0, 0, x, x), lambda: ctx.uocr_kv_write_prefix(0, 0, x, x, 9),
               lambda: ctx.uocr_kv_write_i4(0, 0, 14, *e, *e),
               lambda: ctx.uocr_kv_append_chunk(0, 0, 29, 3, 0, t.data_ptr(), t.data_ptr(), dtype=0),
               lambda: ctx.uocr_attend_chunk(0, 0, 0, 3, nh, t.data_ptr(), o.data_ptr(), 0)]
    for call in refused:
        with pytest.raises(binding.UocrError) as err:
            call()
        assert err.value.status == binding.UOCR_E_STATE
    ctx.uocr_kv_write(0, 0, 0, x[:, :10], x[:, :10])          # what is left may be rewritten
    ctx.uocr_kv_append_chunk(0, 0, 30, 3, 0, t.data_ptr(), t.data_ptr(), dtype=0)
    before = _read(ctx, cfg, 0)
    pos = torch.tensor([12, 31], dtype=torch.int32, device="cuda")
    k = torch.randn(2, nh, D, device="cuda")
    ctx.uocr_kv_append(0, 2, pos.data_ptr(), 0, k.data_ptr(), k.data_ptr(), dtype=0)
    with pytest.raises(binding.UocrError) as err:
        ctx.uocr_sync()
    assert err.value.status == binding.UOCR_E_POSITION
    assert all(np.array_equal(a, b) for a, b in zip(before, _read(ctx, cfg, 0)))  # not written
    ctx.uocr_kv_reset(0, 0)
    ctx.uocr_kv_append_chunk(0, 0, 0, 40, 0, t.data_ptr(), t.data_ptr(), dtype=0)
    ctx.uocr_kv_write(0, 0, 0, x, x)
    ctx.uocr_sync()
    ctx.close()


def test_new_entries_start_without_weight_and_reset_clears(cuda):
    torch = cuda
    cfg = _cfg(prefix_len=20, ring_len=8, max_rows=2, kv_track=1)
    ctx = binding.Context(cfg, max_rows=2)
    rng = np.random.default_rng(11)
    _fill(ctx, cfg, rng)
    nh, D = cfg.n_heads, cfg.head_dim
    _put_weights(torch, ctx, np.ones((2, nh, 28)))
    k = torch.randn(4, nh, D, device="cuda")
    pos = torch.tensor([3, 22], dtype=torch.int32, device="cuda")
    ctx.uocr_kv_append(0, 2, pos.data_ptr(), 0, k.data_ptr(), k.data_ptr(), dtype=0)
    ctx.uocr_kv_append_chunk(0, 1, 5, 4, 0, k.data_ptr(), k.data_ptr(), dtype=0)
    x = np.zeros((nh, 2, D), np.float16)
    ctx.uocr_kv_write(0, 0, 10, x, x)
    e = _entries(rng, (nh, 2, D))
    ctx.uocr_kv_write_i4(0, 0, 14, *e, *e)
    want = np.ones((2, nh, 28))
    want[0, :, [3, 10, 11, 14, 15]] = 0
    want[1, :, [22, 5, 6, 7, 8]] = 0
    assert np.array_equal(_weights(torch, ctx, cfg), want)
    ctx.uocr_kv_reset(1, 1)
    want[1, :, 20:] = 0
    assert np.array_equal(_weights(torch, ctx, cfg), want)
    now = _read(ctx, cfg, 1)
    assert not any(a[:, 20:].any() for a in now) and now[0][:, :20].any()
    ctx.uocr_kv_reset(-1, 0)
    assert not _weights(torch, ctx, cfg).any() and not any(a.any() for a in _read(ctx, cfg, 0))
    ctx.close()


# ------------------------------------------------------------------ refusals
def test_refusals(cuda):
    torch = cuda
    t = torch.zeros(64 * 8 * 2 * 64, device="cuda")
    i = torch.zeros(64, dtype=torch.int32, device="cuda")
    p, ip = t.data_ptr(), i.data_ptr()
    f16 = binding.Context(_cfg(kv_int4=0), max_rows=2)
    plain = binding.Context(_cfg(max_rows=2), max_rows=2)
    ctx = binding.Context(_cfg(max_rows=2, kv_track=1), max_rows=2)
    sink = binding.Context(_cfg(max_rows=2, use_sink=1), max_rows=2)
    STATE, ARG = binding.UOCR_E_STATE, binding.UOCR_E_INVALID_ARG
    kw = dict(dtype=0, q_heads=2, q_out=p)
    z8, z16 = np.zeros((2, 3, 64), np.uint8), np.zeros((2, 3, 2), np.float16)
    calls = [
        (STATE, lambda: f16.uocr_attend(0, 1, ip, 2, p, p)), (STATE, lambda: f16.uocr_kv_append(0, 1, ip, p, p, p, **kw)),
        (STATE, lambda: f16.uocr_kv_read_i4(0, 0, 0, 1)), (STATE, lambda: f16.uocr_kv_evict(0, [0], [1], 4, 2)),
        (STATE, lambda: plain.uocr_kv_evict(0, [0], [1], 4, 2)), (STATE, lambda: plain.uocr_kv_weights_read(0, 0, 1, 0, 1, p)),
        (STATE, lambda: sink.uocr_attend(0, 1, ip, 2, p, p)), (STATE, lambda: sink.uocr_attend_chunk(0, 0, 0, 1, 2, p, p)),
        (STATE, lambda: ctx.uocr_kv_read_i8(0, 0, 0, 1)),
        (ARG, lambda: ctx.uocr_attend(1, 1, ip, 2, p, p)), (ARG, lambda: ctx.uocr_attend(-1, 1, ip, 2, p, p)),
        (ARG, lambda: ctx.uocr_attend(0, 0, ip, 2, p, p)), (ARG, lambda: ctx.uocr_attend(0, 3, ip, 2, p, p)),
        (ARG, lambda: ctx.uocr_attend(0, 1, 0, 2, p, p)), (ARG, lambda: ctx.uocr_attend(0, 1, ip, 2, 0, p)),
        (ARG, lambda: ctx.uocr_attend(0, 1, ip, 2, p, 0)), (ARG, lambda: ctx.uocr_attend(0, 1, ip, 3, p, p)),
        (ARG, lambda: ctx.uocr_attend(0, 1, ip, 18, p, p)), (ARG, lambda: ctx.uocr_attend(0, 1, ip, 0, p, p)),
        (ARG, lambda: ctx.uocr_attend(0, 1, ip, 2, p, p, 3)),
        (ARG, lambda: ctx.uocr_attend_chunk(0, 2, 0, 1, 2, p, p)), (ARG, lambda: ctx.uocr_attend_chunk(0, 0, -1, 1, 2, p, p)),
        (ARG, lambda: ctx.uocr_attend_chunk(0, 0, 0, 0, 2, p, p)), (ARG, lambda: ctx.uocr_attend_chunk(0, 0, 50, 7, 2, p, p)),
        (ARG, lambda: ctx.uocr_attend_chunk(0, 0, 2 ** 31 - 1, 2 ** 31 - 1, 2, p, p)),
        (ARG, lambda: ctx.uocr_kv_append(0, 1, ip, p, 0, p, **kw)), (ARG, lambda: ctx.uocr_kv_append(0, 1, ip, 0, p, p, **kw)),
        (ARG, lambda: ctx.uocr_kv_append(0, 1, ip, p, p, p, dtype=3, q_heads=2, q_out=p)),
        (ARG, lambda: ctx.uocr_kv_append(0, 1, ip, p, p, p, dtype=0, q_heads=2)),
        (ARG, lambda: ctx.uocr_kv_append(0, 1, ip, p, p, p, ld_k=127, **kw)),
        (ARG, lambda: ctx.uocr_kv_append(0, 1, ip, p, p, p, ld_q=-128, **kw)),
        (ARG, lambda: ctx.uocr_kv_append(0, 3, ip, p, p, p, **kw)), (ARG, lambda: ctx.uocr_kv_append(0, 1, 0, p, p, p, **kw)),
        (ARG, lambda: ctx.uocr_kv_append_chunk(0, 0, 0, 57, p, p, p, **kw)),
        (ARG, lambda: ctx.uocr_kv_evict(0, [], [], 4, 2)), (ARG, lambda: ctx.uocr_kv_evict(0, [2], [0], 4, 2)),
        (ARG, lambda: ctx.uocr_kv_evict(0, [0, 1], [1, 0], 4, 2)), (ARG, lambda: ctx.uocr_kv_evict(0, [0, 0], [1, 1], 4, 2)),
        (ARG, lambda: ctx.uocr_kv_evict(0, [0], [-1], 4, 2)), (ARG, lambda: ctx.uocr_kv_evict(-2, [0], [1], 4, 2)),
        (ARG, lambda: ctx.uocr_kv_evict(0, [0], [1], 0, 0)), (ARG, lambda: ctx.uocr_kv_evict(0, [0], [1], 41, 2)),
        (ARG, lambda: ctx.uocr_kv_evict(0, [0], [1], 4, 5)), (ARG, lambda: ctx.uocr_kv_evict(0, [0], [1], 4, 2, 3)),
        (ARG, lambda: ctx.uocr_kv_evict(0, [0], [1], 4, -1)),
        (ARG, lambda: ctx.uocr_kv_weights_read(0, 1, 2, 0, 1, p)), (ARG, lambda: ctx.uocr_kv_weights_read(0, 0, 1, 50, 7, p)),
        (ARG, lambda: ctx.uocr_kv_weights_write(1, 0, 1, 0, 1, p)), (ARG, lambda: ctx.uocr_kv_weights_read(0, 0, 1, 0, 1, 0)),
        (ARG, lambda: ctx.uocr_kv_write_i4(0, 0, 54, z8, z16, z16, z8, z16, z16)),
        (ARG, lambda: ctx.uocr_kv_write_i4(2, 0, 0, z8, z16, z16, z8, z16, z16)),
        (ARG, lambda: ctx.uocr_kv_read_i4(0, 0, -1, 1))]
    for k, (status, call) in enumerate(calls):
        with pytest.raises(binding.UocrError) as e:
            call()
        assert e.value.status == status, (k, str(e.value))
    # an eviction inside evicted slots, and of more than is left
    ctx.uocr_kv_evict(0, [0], [0], 30, 10)
    for n, keep in ((20, 5), (31, 12)):
        with pytest.raises(binding.UocrError) as e:
            ctx.uocr_kv_evict(0, [0], [1], n, keep)
        assert e.value.status == ARG
    # a negative position counts as 0 and is reported
    i[0] = -5
    ctx.uocr_attend(0, 1, ip, 2, p, p, 0)
    with pytest.raises(binding.UocrError) as e:
        ctx.uocr_sync()
    assert e.value.status == binding.UOCR_E_POSITION
    for c in (f16, plain, ctx, sink):
        c.close()


# ------------------------------------------------------------------ together
def test_append_attend_evict_as_a_decoder_uses_them(cuda):
    """A prompt in two chunks, decode tokens past a ring wrap, an eviction in between, everything accumulated, on a
    side stream, against the oracle's own cache."""
    torch = cuda
    rng = np.random.default_rng(12)
    P, R, G, dim = 61, 9, 2, 64
    st = torch.cuda.Stream()
    cfg = _cfg(head_dim=dim, n_heads=2, prefix_len=P, ring_len=R, max_rows=2, kv_track=1, rope_layout=1, rope_dims=32,
               rope_scaling=2, rope_factor=4.0, rope_orig_len=32)
    ctx = binding.Context(cfg, max_rows=2, stream=st.cuda_stream)
    nh = cfg.n_heads
    K, V, W = np.zeros((2, nh, P + R, dim)), np.zeros((2, nh, P + R, dim)), np.zeros((2, nh, P + R))
    holes = [(0, 0), (0, 0)]

    def pass_(n, pos, rows, chunk):
        ptrs, ld, (fq, fk, fv), keep = _qkv(torch, rng, n, nh * G, nh, dim, 1, True)
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            q = torch.empty(n, nh * G, dim, device="cuda")
            out = torch.empty(n, nh * G, dim, device="cuda")
            kw = dict(dtype=1, q_heads=nh * G, q_out=q.data_ptr(), **ld)
            if chunk:
                ctx.uocr_kv_append_chunk(0, rows[0], pos[0], n, *ptrs, **kw)
                ctx.uocr_attend_chunk(0, rows[0], pos[0], n, nh * G, q.data_ptr(), out.data_ptr(), 0)
            else:
                p = torch.tensor(pos, dtype=torch.int32, device="cuda")
                ctx.uocr_kv_append(0, n, p.data_ptr(), *ptrs, **kw)
                ctx.uocr_attend(0, n, p.data_ptr(), nh * G, q.data_ptr(), out.data_ptr(), 0)
            got = out.double().cpu().numpy()
        ctx.uocr_sync()
        qr = np.stack([oracle.rotate_f32(fq[i], pos[i], cfg) for i in range(n)])
        for i in range(n):
            s = pos[i] if pos[i] < P else P + (pos[i] - P) % R
            K[rows[i], :, s] = oracle.kv4_value(*oracle.kv4_quant(oracle.rotate_f32(fk[i], pos[i], cfg)))
            V[rows[i], :, s] = oracle.kv4_value(*oracle.kv4_quant(fv[i]))
            W[rows[i], :, s] = 0
        want, add = oracle.attend_kv4(qr, K, V, pos, P, R, holes, causal_row=rows[0] if chunk else None)
        W[:] += add
        _close(got, want, 0)
        assert keep is not None

    for r in range(2):
        pass_(37, list(range(37)), [r] * 37, True)
        pass_(24, list(range(37, 61)), [r] * 24, True)
    for step in range(4):
        pass_(2, [P + step, P + 30 + step], [0, 1], False)
    with torch.cuda.stream(st):
        _close(_weights(torch, ctx, cfg), W, 0)
        w = _weights(torch, ctx, cfg)
        kept, _, _ = _evict(torch, ctx, cfg, 0, [0, 1], [0, 1], P, 20, 3)
    for r in range(2):
        for h in range(nh):
            at = oracle.evict_choice(w[r, h], P, 20, 3)
            assert np.array_equal(kept[0, r, h], at)
            K[r, h, :20], V[r, h, :20], W[r, h, :20] = K[r, h, at], V[r, h, at], W[r, h, at]
            W[r, h, 20:P] = 0
        holes[r] = (20, P)
    for step in range(4, 14):
        pass_(2, [P + step, P + 30 + step], [0, 1], False)
    with torch.cuda.stream(st):
        _close(_weights(torch, ctx, cfg), W, 0)
    ctx.close()


def test_captured_and_replayed_with_new_inputs(cuda):
    torch = cuda
    rng = np.random.default_rng(13)
    st = torch.cuda.Stream()
    cfg = _cfg(prefix_len=33, ring_len=8, max_rows=3, kv_track=1)
    nh, D = cfg.n_heads, cfg.head_dim
    ctxs = [binding.Context(cfg, max_rows=3, stream=s) for s in (st.cuda_stream, 0)]
    for c in ctxs:
        _fill(c, cfg, np.random.default_rng(14))
    x = torch.empty(3, 3 * nh, D, device="cuda")
    pos = torch.zeros(3, dtype=torch.int32, device="cuda")
    q, out = torch.empty(3, nh, D, device="cuda"), torch.empty(3, nh, D, device="cuda")
    q2, out2 = torch.empty_like(q), torch.empty_like(out)

    def call(c, q, out):
        e, b = 4 * nh * D, x.data_ptr()
        c.uocr_kv_append(0, 3, pos.data_ptr(), b, b + e, b + 2 * e, dtype=0, q_heads=nh, ld_q=3 * nh * D, ld_k=3 * nh * D,
                         ld_v=3 * nh * D, q_out=q.data_ptr())
        c.uocr_attend(0, 3, pos.data_ptr(), nh, q.data_ptr(), out.data_ptr(), 0)

    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(st):
        g.capture_begin()
        call(ctxs[0], q, out)
        g.capture_end()
    for step in range(5):
        x.copy_(torch.from_numpy(rng.standard_normal((3, 3 * nh, D)).astype(np.float32)))
        pos.copy_(torch.tensor([step, 30 + step, 60 + 3 * step], dtype=torch.int32))
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            g.replay()
        call(ctxs[1], q2, out2)
        torch.cuda.synchronize()
        assert torch.equal(q, q2) and torch.equal(out, out2)
    assert np.array_equal(_weights(torch, ctxs[0], cfg), _weights(torch, ctxs[1], cfg))
    for c in ctxs:
        c.uocr_sync()
        c.close()


def test_repeated_calls_are_bit_identical(cuda):
    torch = cuda
    rng = np.random.default_rng(15)
    cfg = _cfg(head_dim=128, n_heads=4, prefix_len=900, ring_len=30, max_rows=3, kv_track=1)
    ctx = binding.Context(cfg, max_rows=3)
    _fill(ctx, cfg, rng)
    q = rng.standard_normal((3, 8, 128)).astype(np.float32)
    qc = rng.standard_normal((100, 4, 128)).astype(np.float32)
    runs = []
    for _ in range(3):
        _put_weights(torch, ctx, np.zeros((3, 4, 930)))
        a = _attend(torch, ctx, cfg, q, [929, 400, 5000])
        b = _attend(torch, ctx, cfg, qc, chunk=(1, 800))
        runs.append((a, b, _weights(torch, ctx, cfg)))
    for r in runs[1:]:
        assert all(np.array_equal(u, v) for u, v in zip(r, runs[0]))
    ctx.close()


@pytest.mark.parametrize("dim,group", [(32, 1), (64, 5), (128, 1), (128, 4), (256, 8)])
def test_rows_of_very_different_lengths(cuda, dim, group):
    """Rows from one slot to thousands, some of them evicted to almost nothing, in one call: work is shared out by
    length, so that a row is read by one reader or by many."""
    torch = cuda
    rng = np.random.default_rng(dim)
    P, R = 1500, 40
    cfg = _cfg(head_dim=dim, n_heads=2, prefix_len=P, ring_len=R, max_rows=24, kv_track=1)
    ctx = binding.Context(cfg, max_rows=24)
    vals = _fill(ctx, cfg, rng)[0]
    holes = [(0, 0)] * 24
    w = rng.random((24, 2, P + R)).astype(np.float32)
    _put_weights(torch, ctx, w)
    w = w.astype(np.float64)
    for r, keep in ((3, 0), (4, 1), (11, 17), (23, 0)):
        _evict(torch, ctx, cfg, 0, [r], [r], P, keep, 0, vals=False)
        for h in range(2):
            at = oracle.evict_choice(w[r, h], P, keep, 0)
            vals[r, :, h, :keep] = vals[r][:, h, at]
            w[r, h, :keep] = w[r, h, at]
            w[r, h, keep:P] = 0
        holes[r] = (keep, P)
    for rows in (24, 5, 1):
        pos = [int(p) for p in rng.integers(0, P + 200, 24)]
        pos[0], pos[1], pos[2], pos[5], pos[6] = 1200, 0, 15, 16, P + 3 * R
        for r in (3, 4, 11, 23):
            pos[r] = P + int(rng.integers(0, R))
        q = rng.standard_normal((rows, 2 * group, dim)).astype(np.float32) * 2
        want, add = oracle.attend_kv4(q, vals[:, 0], vals[:, 1], pos, P, R, holes)
        _close(_attend(torch, ctx, cfg, q, pos[:rows]), want, 0)
        w += add
    _close(_weights(torch, ctx, cfg), w, 0)
    ctx.close()


@pytest.mark.parametrize("dim,nh,group,sink,dtype", [(32, 2, 1, False, 0), (32, 4, 8, True, 1), (64, 1, 3, True, 2), (64, 2, 1, False, 0),
                                                     (128, 2, 1, True, 1), (128, 1, 8, False, 0), (256, 1, 2, True, 2), (256, 1, 5, False, 0)])
def test_rows_of_thousands_of_slots(cuda, dim, nh, group, sink, dtype):
    """Rows whose slots many warps share, with short ones among them and evicted ones; repeated calls agree bit for bit."""
    torch = cuda
    rng = np.random.default_rng(dim + group)
    P, R, rows = 3600, 37, 6
    cfg = _cfg(head_dim=dim, n_heads=nh, prefix_len=P, ring_len=R, max_rows=rows, use_sink=int(sink), kv_track=1)
    ctx = binding.Context(cfg, max_rows=rows)
    nh = cfg.n_heads
    vals = _fill(ctx, cfg, rng)[0]
    sinks = rng.standard_normal((1, nh)).astype(np.float32) if sink else None
    if sink:
        ctx.uocr_set_sinks(sinks)
    w = rng.random((rows, nh, P + R)).astype(np.float32)
    _put_weights(torch, ctx, w)
    holes = [(0, 0)] * rows
    for r, keep in ((1, 700), (4, 3)):
        _evict(torch, ctx, cfg, 0, [r], [r], 3000, keep, 0, vals=False)
        for h in range(nh):
            at = oracle.evict_choice(w[r, h, :3000], 3000, keep, 0)
            vals[r, :, h, :keep] = vals[r][:, h, at]
        holes[r] = (keep, 3000)
    pos = [3599, 3400, 0, P + R + 5, 3001, 17]
    q = rng.standard_normal((rows, nh * group, dim)).astype(np.float32) * 2
    want, add = oracle.attend_kv4(q, vals[:, 0], vals[:, 1], pos, P, R, holes, sinks=None if sinks is None else sinks[0].astype(np.float64))
    _put_weights(torch, ctx, np.zeros((rows, nh, P + R)))
    got = _attend(torch, ctx, cfg, q, pos, dtype=dtype)
    _close(got, want, dtype)
    _close(_weights(torch, ctx, cfg), add, 0)
    assert np.array_equal(_attend(torch, ctx, cfg, q, pos, dtype=dtype), got)
    _close(_attend(torch, ctx, cfg, q[:1], pos[:1], dtype=dtype), want[:1], dtype)
    ctx.close()


@pytest.mark.parametrize("dim", [32, 128])
def test_buffers_aligned_to_their_elements_only(cuda, dim):
    """Inputs and outputs one element past a 16-byte boundary give what aligned ones give, bit for bit."""
    torch = cuda
    cfg = _cfg(head_dim=dim, n_heads=2, prefix_len=50, ring_len=9, max_rows=2, kv_track=1)
    rng = np.random.default_rng(dim)

    def off(x):  # a copy that starts one element past an aligned address
        b = torch.empty(x.numel() + 1, dtype=x.dtype, device="cuda")
        b[1:].copy_(x.reshape(-1))
        return b[1:]

    for dtype in (0, 1, 2):
        got = []
        x = [torch.from_numpy(rng.standard_normal((21, h, dim)).astype(np.float32)).to(_dt(torch, dtype)).cuda() for h in (4, 2, 2)]
        for shift in (lambda v: v, off):
            ctx = binding.Context(cfg, max_rows=2)
            ins = [shift(v) for v in x]
            q = shift(torch.zeros(21, 4, dim, device="cuda"))
            k, v, out = shift(torch.zeros(21, 2, dim, device="cuda").half()), shift(torch.zeros(21, 2, dim, device="cuda").half()), \
                shift(torch.zeros(21, 4, dim, device="cuda", dtype=_dt(torch, dtype)))
            ctx.uocr_kv_append_chunk(0, 1, 31, 21, *(t.data_ptr() for t in ins), dtype=dtype, q_heads=4, q_out=q.data_ptr(),
                                     k_val=k.data_ptr(), v_val=v.data_ptr())
            ctx.uocr_attend_chunk(0, 1, 31, 21, 4, q.data_ptr(), out.data_ptr(), dtype)
            pos = torch.tensor([20, 51], dtype=torch.int32, device="cuda")
            one = shift(torch.zeros(2, 4, dim, device="cuda", dtype=_dt(torch, dtype)))
            ctx.uocr_attend(0, 2, pos.data_ptr(), 4, q.data_ptr(), one.data_ptr(), dtype)
            kept = shift(torch.zeros(2, 7, dtype=torch.int32, device="cuda"))
            ke, ve = (shift(torch.zeros(2, 7, dim, device="cuda").half()) for _ in range(2))
            ctx.uocr_kv_evict(0, [1], [0], 49, 7, kept_ptr=kept.data_ptr(), k_val_ptr=ke.data_ptr(), v_val_ptr=ve.data_ptr())
            w = shift(torch.zeros(2, 2, 59, device="cuda"))
            ctx.uocr_kv_weights_read(0, 0, 2, 0, 59, w.data_ptr())
            ctx.uocr_sync()
            got.append([t.reshape(-1).clone() for t in (q, k, v, out, one, kept, ke, ve, w)])
            ctx.close()
        for u, v in zip(*got):
            assert torch.equal(u, v) and u.float().abs().sum() > 0


def _chunk_reference(q, K, V, start, P, R, hole=(0, 0), sinks=None):
    """oracle.attend_kv4 of one row's chunk, by whole products: K, V [nh, slots, D]; (out, weights)."""
    n, qh, D = q.shape
    nh, SL, _ = K.shape
    G = qh // nh
    out, w = np.zeros((n, qh, D)), np.zeros((nh, SL))
    slots = np.arange(SL)
    lim = np.array([p + 1 if p < P else P + min(p - P + 1, R) for p in range(start, start + n)])
    live = (slots[None] < lim[:, None]) & ~((slots >= hole[0]) & (slots < hole[1]))[None]
    for h in range(qh):
        s = np.where(live, np.where(live, q[:, h].astype(np.float64) @ np.nan_to_num(K[h // G]).T, 0) / np.sqrt(D), -np.inf)
        top = s.max(1, keepdims=True)
        if sinks is not None:
            top = np.maximum(top, sinks[h // G])
        e = np.exp(s - top)
        z = e.sum(1, keepdims=True) + (0 if sinks is None else np.exp(sinks[h // G] - top))
        out[:, h] = (e / z) @ np.nan_to_num(V[h // G])
        w[h // G] += (e / z).sum(0)
    return out, w


@pytest.mark.parametrize("dim,nh,n,start,group,P,R,sink,dtype,track,keep", [
    (32, 16, 500, 0, 1, 700, 20, True, 0, 0, None), (64, 10, 250, 131, 3, 380, 9, False, 0, 1, None),
    (128, 8, 1000, 0, 1, 1000, 16, False, 0, 0, None), (128, 12, 641, 333, 1, 900, 128, True, 1, 1, 77),
    (64, 20, 130, 1500, 3, 1600, 40, False, 2, 0, 5), (256, 8, 960, 5, 1, 970, 30, True, 0, 0, None),
    (32, 40, 64, 800, 3, 860, 10, False, 0, 1, 0), (128, 3, 343, 0, 8, 343, 1, False, 0, 0, None)])
def test_attend_long_chunks(cuda, dim, nh, n, start, group, P, R, sink, dtype, track, keep):
    """Enough queries for the kernel that dequantises a block once for 64 of them."""
    torch = cuda
    rng = np.random.default_rng(dim + n)
    cfg = _cfg(head_dim=dim, n_heads=nh, prefix_len=P, ring_len=R, max_rows=1, use_sink=int(sink),
               kv_track=int(track or keep is not None))
    ctx = binding.Context(cfg, max_rows=1)
    nh = cfg.n_heads
    vals = _fill(ctx, cfg, rng)[0]
    sinks = rng.standard_normal((1, nh)).astype(np.float32) if sink else None
    if sink:
        ctx.uocr_set_sinks(sinks)
    hole = (0, 0)
    if keep is not None:
        w = rng.random((1, nh, P + R)).astype(np.float32)
        _put_weights(torch, ctx, w)
        evicted = max(1, start - 10)
        kept, k, v = _evict(torch, ctx, cfg, 0, [0], [0], evicted, keep, 0)
        vals[0, 0, :, :keep], vals[0, 1, :, :keep] = k[0, 0], v[0, 0]
        hole = (keep, evicted)
        _put_weights(torch, ctx, np.zeros((1, nh, P + R)))
    q = rng.standard_normal((n, nh * group, dim)).astype(np.float32) * 2
    want, add = _chunk_reference(q, vals[0, 0], vals[0, 1], start, P, R, hole, None if sinks is None else sinks[0].astype(np.float64))
    _close(_attend(torch, ctx, cfg, q, chunk=(0, start), dtype=dtype), want, dtype)
    if cfg.kv_track:
        _close(_weights(torch, ctx, cfg)[0], add, 0)
    ctx.close()


@pytest.mark.parametrize("dim,nh,n,start,group,P,R", [(32, 64, 640, 0, 1, 640, 20), (64, 48, 700, 9, 1, 720, 3),
                                                      (128, 40, 650, 0, 1, 655, 1), (32, 32, 640, 0, 8, 640, 1)])
def test_attend_chunk_of_many_items(cuda, dim, nh, n, start, group, P, R):
    """More query tiles than SMs: several, some of them in part, to one CTA; last, so many that each has a CTA."""
    torch = cuda
    rng = np.random.default_rng(dim + nh)
    cfg = _cfg(head_dim=dim, n_heads=nh, prefix_len=P, ring_len=R, max_rows=1)
    ctx = binding.Context(cfg, max_rows=1)
    vals = _fill(ctx, cfg, rng)[0]
    q = rng.standard_normal((n, nh * group, dim)).astype(np.float32) * 2
    want, _ = _chunk_reference(q, vals[0, 0], vals[0, 1], start, P, R)
    _close(_attend(torch, ctx, cfg, q, chunk=(0, start)), want, 0)
    ctx.close()


@pytest.mark.parametrize("dim,nh,n,start,P,R,sink,keep", [(32, 64, 300, 1100, 1390, 20, True, None), (32, 64, 700, 1900, 2600, 1, False, 300),
                                                          (128, 40, 520, 1400, 1900, 30, True, 11), (64, 64, 310, 1300, 1700, 9, False, None)])
def test_attend_chunk_after_a_long_prefix(cuda, dim, nh, n, start, P, R, sink, keep):
    """Long items, more of them than SMs: each SM has the end of one, whole ones and the start of another."""
    test_attend_long_chunks(cuda, dim, nh, n, start, 1, P, R, sink, 0, 0, keep)


@pytest.mark.parametrize("dim,nh,n,start", [(128, 16, 300, 0), (64, 16, 200, 1500), (32, 64, 300, 1100), (128, 2, 40, 0)])
def test_captured_chunks_follow_their_inputs(cuda, dim, nh, n, start):
    """A replayed attention of a chunk reads the queries and entries of its time, between other work of the stream."""
    torch = cuda
    rng = np.random.default_rng(dim + n)
    s = torch.cuda.Stream()
    cfg = _cfg(head_dim=dim, n_heads=nh, prefix_len=start + n, ring_len=4, max_rows=1)
    ctx = binding.Context(cfg, max_rows=1, stream=s.cuda_stream)
    nh = cfg.n_heads
    with torch.cuda.stream(s):
        q = torch.zeros(n, nh, dim, device="cuda")
        out = torch.zeros(n, nh, dim, device="cuda")
        twice = torch.zeros_like(out)
        call = lambda: ctx.uocr_attend_chunk(0, 0, start, n, nh, q.data_ptr(), out.data_ptr(), 0)
        vals = _fill(ctx, cfg, rng)[0]
        call()
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            call()
            twice.copy_(out)
            twice.mul_(2)
            call()
        for _ in range(2):
            x = rng.standard_normal((n, nh, dim)).astype(np.float32) * 2
            q.copy_(torch.from_numpy(x))
            g.replay()
            g.replay()
            s.synchronize()
            want, _ = _chunk_reference(x, vals[0, 0], vals[0, 1], start, start + n, 4)
            _close(out.double().cpu().numpy(), want, 0)
            assert torch.equal(twice, 2 * out)
            vals = _fill(ctx, cfg, rng)[0]
            q.mul_(0.5)
            g.replay()
            want, _ = _chunk_reference(x * 0.5, vals[0, 0], vals[0, 1], start, start + n, 4)
            s.synchronize()
            _close(out.double().cpu().numpy(), want, 0)
    ctx.uocr_sync()
    ctx.close()


def test_two_contexts_at_once(cuda):
    """Long chunks and rows of two contexts on two streams, interleaved without a wait between them."""
    torch = cuda
    rng = np.random.default_rng(5)
    todo = []
    for dim, nh, n, start in ((128, 10, 400, 700), (64, 24, 300, 900)):
        s = torch.cuda.Stream()
        cfg = _cfg(head_dim=dim, n_heads=nh, prefix_len=start + n, ring_len=4, max_rows=1)
        ctx = binding.Context(cfg, max_rows=1, stream=s.cuda_stream)
        nh = cfg.n_heads
        vals = _fill(ctx, cfg, rng)[0]
        x = rng.standard_normal((n, nh, dim)).astype(np.float32)
        q = torch.from_numpy(x).cuda()
        out = [torch.zeros(n, nh, dim, device="cuda") for _ in range(6)]
        row = [torch.zeros(1, nh, dim, device="cuda") for _ in range(6)]
        pos = torch.tensor([start + n - 1], dtype=torch.int32, device="cuda")
        want, _ = _chunk_reference(x, vals[0, 0], vals[0, 1], start, start + n, 4)
        todo.append((ctx, n, nh, start, q, out, row, pos, want, s))
    torch.cuda.synchronize()
    for i in range(6):
        for ctx, n, nh, start, q, out, row, pos, want, s in todo:
            ctx.uocr_attend_chunk(0, 0, start, n, nh, q.data_ptr(), out[i].data_ptr(), 0)
            ctx.uocr_attend(0, 1, pos.data_ptr(), nh, q[n - 1].data_ptr(), row[i].data_ptr(), 0)
    for ctx, n, nh, start, q, out, row, pos, want, s in todo:
        ctx.uocr_sync()
        for i in range(6):
            _close(out[i].double().cpu().numpy(), want, 0)
            _close(row[i].double().cpu().numpy(), want[-1:], 0)
        ctx.close()


@pytest.mark.parametrize("dim,nh,n,start,group", [(32, 2, 127, 0, 1), (64, 1, 128, 3, 1), (128, 1, 129, 0, 1),
                                                  (64, 2, 40, 30, 5), (128, 2, 37, 0, 7), (32, 3, 86, 11, 3), (128, 1, 16, 200, 8),
                                                  (64, 1, 65, 0, 2), (32, 2, 50, 0, 6), (128, 3, 32, 1, 4)])
@pytest.mark.parametrize("dtype,shift", [(0, 0), (1, 1), (2, 1), (0, 1), (2, 0)])
def test_attend_chunk_of_any_sharing(cuda, dim, nh, n, start, group, dtype, shift):
    """Around 128 queries per cache head, any number of heads that share one, aligned and shifted pointers."""
    torch = cuda
    rng = np.random.default_rng(dim + n + group)
    cfg = _cfg(head_dim=dim, n_heads=nh, prefix_len=230, ring_len=5, max_rows=1, use_sink=1)
    nh = cfg.n_heads
    ctx = binding.Context(cfg, max_rows=1)
    vals = _fill(ctx, cfg, rng)[0]
    sinks = rng.standard_normal((1, nh)).astype(np.float32)
    ctx.uocr_set_sinks(sinks)
    q = rng.standard_normal((n, nh * group, dim)).astype(np.float32) * 2
    q[n // 2] *= 1e-20
    want, _ = _chunk_reference(q, vals[0, 0], vals[0, 1], start, 230, 5, sinks=sinks[0].astype(np.float64))
    qd = torch.zeros(q.size + 1, device="cuda")[shift:shift + q.size]
    qd.copy_(torch.from_numpy(q).reshape(-1))
    buf = torch.full((q.size + 2,), 7.0, dtype=_dt(torch, dtype), device="cuda")
    out = buf[shift:shift + q.size]
    ctx.uocr_attend_chunk(0, 0, start, n, nh * group, qd.data_ptr(), out.data_ptr(), dtype)
    ctx.uocr_sync()
    _close(out.double().cpu().numpy().reshape(q.shape), want, dtype)
    assert torch.all(buf[shift + q.size:] == 7) and torch.all(buf[:shift] == 7)
    ctx.close()


@pytest.mark.parametrize("dim,nh,n,start,group", [(32, 64, 100, 130, 5), (64, 32, 90, 140, 7), (128, 16, 101, 97, 3), (32, 40, 150, 0, 8),
                                                  (64, 40, 129, 60, 2), (128, 12, 77, 120, 6), (128, 30, 128, 99, 4), (64, 64, 127, 3, 1)])
@pytest.mark.parametrize("dtype,shift", [(0, 1), (1, 0), (2, 1)])
def test_attend_chunk_of_any_sharing_many_heads(cuda, dim, nh, n, start, group, dtype, shift):
    """The same with enough heads for the kernel of long chunks."""
    test_attend_chunk_of_any_sharing(cuda, dim, nh, n, start, group, dtype, shift)


@pytest.mark.parametrize("dim,nh,n,start,group,keep", [(64, 32, 190, 40, 1, None), (32, 40, 64, 240, 3, 17), (128, 16, 96, 200, 2, 0)])
def test_attend_chunk_tracked_on_many_rows_and_heads(cuda, dim, nh, n, start, group, keep):
    test_attend_chunk_tracked_on_many_rows(cuda, dim, nh, n, start, group, keep)


@pytest.mark.parametrize("dim,nh,n,start,group,keep", [(32, 2, 300, 0, 1, None), (64, 2, 150, 160, 2, 9), (128, 2, 310, 0, 1, None),
                                                       (128, 1, 70, 231, 3, 0)])
def test_attend_chunk_tracked_on_many_rows(cuda, dim, nh, n, start, group, keep):
    """A context of many rows accumulates the weights of many queries in one pass."""
    torch = cuda
    rng = np.random.default_rng(dim + n)
    P, R = 310, 6
    cfg = _cfg(head_dim=dim, n_heads=nh, prefix_len=P, ring_len=R, max_rows=24, kv_track=1)
    nh = cfg.n_heads
    ctx = binding.Context(cfg, max_rows=24)
    vals = _fill(ctx, cfg, rng)[0]
    hole = (0, 0)
    w0 = np.zeros((24, nh, P + R), np.float32)
    if keep is not None:
        _put_weights(torch, ctx, rng.random((24, nh, P + R)).astype(np.float32))
        _, k, v = _evict(torch, ctx, cfg, 0, [3], [3], start - 20, keep, 0)
        vals[3, 0, :, :keep], vals[3, 1, :, :keep] = k[0, 0], v[0, 0]
        hole = (keep, start - 20)
        w0 = _weights(torch, ctx, cfg)
    q = rng.standard_normal((n, nh * group, dim)).astype(np.float32) * 2
    want, add = _chunk_reference(q, vals[3, 0], vals[3, 1], start, P, R, hole)
    _close(_attend(torch, ctx, cfg, q, chunk=(3, start)), want, 0)
    w = _weights(torch, ctx, cfg)
    w0 = w0.astype(np.float64)
    w0[3] += add
    _close(w, w0, 0)
    ctx.close()


@pytest.mark.parametrize("dim,nh,n", [(32, 16, 500), (128, 8, 1000), (256, 8, 960)])
def test_long_chunk_never_sees_later_tokens(cuda, dim, nh, n):
    torch = cuda
    rng = np.random.default_rng(dim)
    cfg = _cfg(head_dim=dim, n_heads=nh, prefix_len=n, ring_len=30, max_rows=1)
    ctx = binding.Context(cfg, max_rows=1)
    vals = _fill(ctx, cfg, rng)[0]
    bad = n - 150  # entries from here on: groups that are NaN, infinite or as before
    c, s, m = _entries(rng, (nh, n + 30 - bad, dim))
    m[:, 0::3], s[:, 1::3] = np.nan, np.inf
    ctx.uocr_kv_write_i4(0, 0, bad, c, s, m, c, s, m)
    q = rng.standard_normal((n, nh, dim)).astype(np.float32)
    want, _ = _chunk_reference(q, vals[0, 0], vals[0, 1], 0, n, 30)
    got = _attend(torch, ctx, cfg, q, chunk=(0, 0))
    _close(got[:bad], want[:bad], 0)
    assert np.all(np.isnan(got[bad:]))
    # one dimension group of one value only: the rest of the output stays as it was
    ctx.close()
    ctx = binding.Context(cfg, max_rows=1)
    vals = _fill(ctx, cfg, rng)[0]
    k, ks, km, v, vs, vm = (x.copy() for x in _read(ctx, cfg, 0))
    vm[1, n - 40, 0] = np.nan
    ctx.uocr_kv_write_i4(0, 0, 0, k, ks, km, v, vs, vm)
    want, _ = _chunk_reference(q, vals[0, 0], vals[0, 1], 0, n, 30)
    got = _attend(torch, ctx, cfg, q, chunk=(0, 0))
    assert np.all(np.isnan(got[n - 40:, 1, :32]))
    got[n - 40:, 1, :32] = want[n - 40:, 1, :32]
    _close(got, want, 0)
    ctx.close()
