"""dllm_attention_masked against the formula in 64 bits, element by element.

Tolerance, as for dllm_attention (both sides see the same f16 q, k, v), with A = sum_j w_j |v_j|:
  * a weight 2^(s - m) is rounded to f16 (2^-11 relative; 2^-25 absolute below the normal
    range, against a normaliser of at least 1) and ex2 is good to 2^-21;
  * a score is an f32 sum of dh exact products, off by dh 2^-24 sum|q k| / sqrt(dh); the tanh of the
    cap is good to 2^-20 of the cap; the bias and the other f32 operations on the score to
    2^-22 of the largest magnitude met;  together ds, which moves a weight by ds relative;
  * the normaliser's and the output's f32 sums over Lk + dh terms;
  * an f16 output is rounded once more: 2^-11 of the value, or 2^-25.
So |gpu - ref| <= (2 delta + 2 (Lk + dh) 2^-24) A + 2^-24 Lk max|v| + [f16] (2^-11 |ref| + 2^-25),
delta = 2^-11 + 2^-21 + ds.
"""
import numpy as np
import pytest
import torch

from quantized_int8_gemm_q4_b200 import dllm, synth

pytestmark = pytest.mark.gpu
DH = 128
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("GPU test run without a CUDA device")
    from quantized_int8_gemm_q4_b200 import build
    build.build()
    dllm.load()
    yield
    assert dllm.dllm_get_device_status() == dllm.DLLM_OK


def inputs(Lq, Lk, H, Hkv, *sub, **kw):
    return [torch.from_numpy(a).cuda() for a in synth.attention_inputs(Lq, max(Lk, 1), H, Hkv, DH, 21, *sub, **kw)]


def formula(q, k, v, begin, end, qp, cap, slopes):
    """-> (o f64 [Lq][H][dh], tolerance before the output's rounding)"""
    Lq, H, _ = q.shape
    Lk, g = k.shape[0], H // k.shape[1]
    j = torch.arange(Lk, device="cuda")
    hid = (j < begin[:, None]) | (j >= end[:, None])
    some = (~hid).any(1)
    # what hidden keys hold cannot matter; what no query sees is not looked at
    seen = (~hid).any(0)
    kd, vd = (torch.where(seen[:, None, None], x.double(), 0.0) for x in (k, v))
    o, tol = (torch.zeros(Lq, H, DH, dtype=torch.float64, device="cuda") for _ in range(2))
    vmax = float(vd[torch.isfinite(vd)].abs().max()) if Lk else 0.0
    for h in range(H):
        K, V = kd[:, h // g], vd[:, h // g]
        Q = q[:, h].double()
        s = (Q @ K.T) / DH ** 0.5
        mag = (Q.abs() @ K.abs().T) / DH ** 0.5
        if cap:
            s = cap * torch.tanh(s / cap)
        big = s.abs()
        if slopes is not None:
            b = slopes[h].double() * (qp[:, None] - j).abs()
            s, big = s - b, big + b
        ds = DH * 2.0 ** -24 * mag + cap * 2.0 ** -20 + 2.0 ** -22 * big
        s = s.masked_fill(hid, -INF)[some]
        ds = ds.masked_fill(hid, 0.0)[some].amax(-1, keepdim=True)
        w = torch.softmax(s, -1)
        o[some, h] = w @ V
        delta = 2.0 ** -11 + 2.0 ** -21 + ds
        tol[some, h] = (2 * delta + 2 * (Lk + DH) * 2.0 ** -24) * (w @ V.abs()) + 2.0 ** -24 * Lk * vmax
    return o, tol


def call(q, k, v, Lk, begin=None, end=None, qp=None, cap=0.0, slopes=None, f16=True, stream=None, o=None, ws=None):
    Lq, H, _ = q.shape
    Hkv = k.shape[1]
    dt = torch.float16 if f16 else torch.float32
    if o is None:
        o = torch.full((Lq + 1, H, DH), 7.0, dtype=dt, device="cuda")
    n = dllm.dllm_attention_masked_workspace_bytes(Lq, Lk, H, Hkv)
    if ws is None and n:
        ws = torch.full((n,), 0xff, dtype=torch.uint8, device="cuda")  # NaN where read before written
    i32 = lambda a: None if a is None else a.to(torch.int32)  # noqa: E731
    dllm.dllm_attention_masked(q, q.stride(0), k, k.stride(0), v, v.stride(0), Lq, Lk, H, Hkv, DH, i32(begin), i32(end),
                               i32(qp), cap, slopes, o, dllm.DLLM_F16 if f16 else dllm.DLLM_F32, ws, n, stream)
    return o


def check(q, k, v, begin=None, end=None, qp=None, cap=0.0, slopes=None, f16=True):
    Lq, Lk = q.shape[0], k.shape[0]
    got = call(q, k, v, Lk, begin, end, qp, cap, slopes, f16)
    assert dllm.dllm_get_device_status() == dllm.DLLM_OK
    assert bool((got[Lq:] == 7.0).all())
    got = got[:Lq].double()
    b = torch.zeros(Lq, device="cuda", dtype=torch.int64) if begin is None else begin.clamp(0, Lk)
    e = torch.full((Lq,), Lk, device="cuda") if end is None else end.clamp(0, Lk)
    p = torch.arange(Lq, device="cuda") + Lk - Lq if qp is None else qp
    ref, tol = formula(q, k, v, b, e, p, cap, slopes)
    if f16:
        tol = tol + ref.abs() * 2.0 ** -11 + 2.0 ** -25
    assert bool(torch.isfinite(got).all())
    empty = e <= b
    assert bool((got[empty] == 0).all())
    err = (got - ref).abs()
    bad = err > tol
    assert not bool(bad.any()), (bad.nonzero()[0].tolist(), float((err / tol.clamp_min(1e-300)).max()))


def t(a):
    return torch.as_tensor(np.asarray(a), device="cuda").to(torch.int64)


def documents(lengths, L):
    """Bounds of packed documents; positions past the last are padding (empty)."""
    begin, end, at = np.zeros(L, np.int64), np.zeros(L, np.int64), 0
    for n in lengths:
        begin[at:at + n], end[at:at + n] = at, at + n
        at += n
    return t(begin), t(end)


@pytest.mark.parametrize("f16", [True, False])
@pytest.mark.parametrize("Lq,Lk,H,Hkv", [
    (1, 1, 1, 1), (5, 3, 2, 1), (128, 128, 2, 2), (130, 200, 4, 2), (257, 384, 2, 1), (300, 333, 64, 8),
    (200, 200, 28, 4), (640, 1, 32, 4), (1, 777, 8, 8), (3, 2049, 28, 4), (32, 1500, 8, 1), (19, 260, 130, 1),
    (4, 300, 200, 1),
])
def test_full_intervals(Lq, Lk, H, Hkv, f16):
    check(*inputs(Lq, Lk, H, Hkv, Lq, Lk), f16=f16)


@pytest.mark.parametrize("H,Hkv", [(4, 4), (14, 2), (8, 1)])
@pytest.mark.parametrize("lengths,L", [([1, 1, 1, 1], 4), ([63, 65, 1, 127], 256), ([500, 0, 3, 400], 1000),
                                       ([128, 128, 128], 400), ([700], 1300), ([], 300)])
def test_packed_documents(lengths, L, H, Hkv):
    b, e = documents(lengths, L)
    check(*inputs(L, L, H, Hkv, 3, L), b, e)


@pytest.mark.parametrize("H,Hkv", [(3, 3), (7, 1)])
@pytest.mark.parametrize("prefix", [0, 1, 100, 129, 600])
def test_prefix_then_causal(prefix, H, Hkv):
    L = 600
    check(*inputs(L, L, H, Hkv, 4), None, t(np.maximum(prefix, np.arange(L) + 1)))


@pytest.mark.parametrize("Lq,Lk", [(1, 3001), (17, 3001), (33, 40), (200, 4500)])
def test_last_positions_over_a_kept_prefix(Lq, Lk):
    p = np.arange(Lq) + Lk - Lq
    for H, Hkv in ((8, 8), (28, 4)):
        check(*inputs(Lq, Lk, H, Hkv, 5), None, t(p + 1))


def test_blocks_and_windows():
    L = 900
    i = np.arange(L)
    q, k, v = inputs(L, L, 8, 2, 6)
    check(q, k, v, None, t(np.minimum((i // 48 + 1) * 48, L)))
    for w in (0, 5, 64, 300):
        check(q, k, v, t(i - w), t(i + w + 1))


def test_arbitrary_intervals():
    """Every query its own, some empty, some reversed, some out of range."""
    g = np.random.default_rng(7)
    for Lq, Lk, H, Hkv in ((300, 500, 4, 2), (40, 3000, 2, 2), (260, 1000, 70, 70)):
        check(*inputs(Lq, Lk, H, Hkv, 8), t(g.integers(-100, Lk + 50, Lq)), t(g.integers(-50, Lk + 100, Lq)))


def test_all_empty_and_no_keys():
    q, k, v = inputs(200, 300, 4, 2, 9)
    z = torch.zeros(200, dtype=torch.int64, device="cuda")
    check(q, k, v, z, z)
    check(q, k, v, z + 2 ** 31 - 1, z - 2 ** 31)
    for f16 in (True, False):
        o = call(q, k, v, 0, f16=f16)
        assert bool((o[:200] == 0).all()) and bool((o[200:] == 7).all())


@pytest.mark.parametrize("cap", [2.0 ** -100, 0.5, 5.0, 30.0, 1000.0, 1e9])
@pytest.mark.parametrize("spread", [1.0, 3.0])
def test_capped_scores(cap, spread):
    q, k, v = inputs(150, 400, 6, 3, 10, spread=spread)
    b, e = documents([60, 80], 150)
    check(q, k, v, cap=cap)
    check(q, k, v, b, e, cap=cap)


def test_distance_bias():
    L, H = 500, 8
    slopes = torch.tensor([2.0 ** -(h + 1) for h in range(H)], device="cuda")
    q, k, v = inputs(L, L, H, 2, 11)
    check(q, k, v, slopes=slopes)
    check(q, k, v, None, t(np.arange(L) + 1), slopes=slopes, cap=20.0)
    qq, kk, vv = inputs(20, 3000, H, 4, 12)
    check(qq, kk, vv, slopes=slopes)  # positions Lk - Lq + i
    check(qq, kk, vv, slopes=-slopes / 64)  # a bias that grows
    check(qq, kk, vv, qp=t(np.arange(20) * 140 - 50), slopes=slopes)


@pytest.mark.parametrize("Lq", [250, 420, 700, 900])
def test_cap_and_bias_in_one_to_four_waves(Lq):
    """64 heads x 2, 4, 6 and 8 query tiles; caps that leave scores below and above a third of them."""
    H = 64
    q, k, v = inputs(Lq, Lq, H, H, 24)
    slopes = torch.rand(H, device="cuda") * 0.2
    b, e = documents([Lq // 3, 40, Lq // 2 - 9], Lq)
    check(q, k, v, b, e, cap=5.0)
    check(q, k, v, b, e, cap=30.0, slopes=slopes)
    check(q, k, v, b, e, slopes=slopes)


def test_peaked_rows_and_raised_maxima():
    for Lq, H, Hkv in ((130, 2, 2), (300, 64, 8), (5, 14, 2)):
        check(*inputs(Lq, 640, H, Hkv, 13, spread=4.0))
        q, k, v = inputs(Lq, 700, H, Hkv, 14, key_growth=0.02)
        check(q, k, v)
        check(q, k, v, None, t(np.arange(Lq) * 2 + 1))


def test_what_hidden_keys_hold_does_not_matter():
    """NaN, infinities and the type's lowest value in keys outside the intervals: between two
    documents of one tile, behind the last key, and everywhere for a padded query."""
    bad = [float("nan"), INF, -INF, -65504.0]
    for H, Hkv in ((4, 4), (14, 2), (64, 64)):  # the last: two query tiles per CTA
        L = 400
        q, k, v = inputs(L, L, H, Hkv, 15)
        b, e = documents([30, 0, 50], L)
        b[100:380], e[100:380] = 100, 250  # documents [0, 30), [30, 80), [100, 250); holes between and behind
        b[80:100] = e[80:100] = 0
        b[380:] = e[380:] = 5
        for n, x in enumerate(bad):
            k[80 + n:100:4], v[80 + n:100:4] = x, x
            k[250 + n::4], v[250 + n::4] = x, x
        check(q, k, v, b, e)
        # documents whose own keys are sound next to one that is not: only its queries are lost
        v[40, :, 3] = float("nan")
        o = call(q, k, v, L, b, e)[:L].float()
        lost = torch.zeros(L, dtype=torch.bool, device="cuda")
        lost[30:80] = True
        assert bool(torch.isfinite(o[~lost]).all())
        assert bool((~torch.isfinite(o[lost])).any(-1).all())


@pytest.mark.parametrize("cap", [0.0, 3.0, 50.0])
def test_hidden_keys_do_not_change_a_bit(cap):
    """Hidden keys with scores far above the cap, with scores of zero, and not finite."""
    for L, H, Hkv in ((500, 4, 4), (300, 64, 64), (200, 14, 2)):
        q, k, v = inputs(L, L, H, Hkv, 19)
        b, e = documents([90, 0, 33, 200], L)
        e = torch.maximum(b, e - 7)  # each document's last keys are padding
        seen = torch.zeros(L, dtype=torch.bool, device="cuda")
        for i in range(L):
            seen[int(b[i]):int(e[i])] = True
        sl = torch.rand(H, device="cuda") * 0.1
        outs = []
        for x in (0.0, 300.0, float("nan")):
            k[~seen], v[~seen] = x, x
            outs.append(call(q, k, v, L, b, e, cap=cap, slopes=sl if cap == 3.0 else None)[:L].clone())
        assert bool(torch.isfinite(outs[0].float()).all())
        assert all(torch.equal(o, outs[0]) for o in outs[1:])
    # the document next door: another one's keys do not matter to its rows either
    q, k, v = inputs(256, 256, 2, 2, 20)
    b, e = documents([40, 216], 256)
    want = call(q, k, v, 256, b, e, cap=cap)[:40].clone()
    k[40:] *= 50.0
    assert torch.equal(call(q, k, v, 256, b, e, cap=cap)[:40], want)


@pytest.mark.parametrize("bad", [float("nan"), INF])
def test_attended_keys_of_no_weight_still_count(bad):
    """Scores 360 apart: the far keys' weights underflow in f32, within a CTA and where the key
    range is split over CTAs; a value there that is not finite is still attended."""
    for Lq, Lk, H, Hkv in ((2, 8000, 4, 4), (2, 500, 4, 4), (300, 500, 64, 8)):
        q, k, v = inputs(Lq, Lk, H, Hkv, 23)
        q[:], k[:100], k[100:] = 4.0, 4.0, -4.0
        v[Lk - 300, :, 3] = bad
        o = call(q, k, v, Lk)[:Lq].float()
        assert not bool(torch.isfinite(o[:, :, 3]).any())
        o[:, :, 3] = 0.0
        assert bool(torch.isfinite(o).all())


def test_holes_in_a_long_prefix():
    """Few queries, keys split over CTAs: each query sees one stretch of sound keys between bad ones."""
    Lq, Lk = 8, 4000
    for H, Hkv in ((4, 4), (28, 4)):
        q, k, v = inputs(Lq, Lk, H, Hkv, 18)
        b, e = t(np.arange(Lq) * 480 + 30), t(np.arange(Lq) * 480 + 30 + np.arange(Lq) * 60)
        seen = torch.zeros(Lk, dtype=torch.bool, device="cuda")
        for i in range(Lq):
            seen[int(b[i]):int(e[i])] = True
        k[~seen], v[~seen] = float("nan"), INF
        check(q, k, v, b, e)


@pytest.mark.parametrize("H,Lk", [(32, 19000), (55, 10500)])
def test_long_caches_of_many_heads(H, Lk):
    """Key parts of half an SM each: whole intervals, a stretch in one part, one across several, none."""
    q, k, v = inputs(4, Lk, H, H, 25)
    check(q, k, v)
    b, e = t([Lk - 9, 3000, 17, 50]), t([Lk, 9001, 20, 50])
    slopes = torch.rand(H, device="cuda") * 0.01
    check(q, k, v, b, e)
    check(q, k, v, b, e, cap=20.0, slopes=slopes, qp=t([Lk, 5000, 0, 7]))
    k[9001:Lk - 9], v[9001:Lk - 9] = float("nan"), INF
    check(q, k, v, b, e)
    v[8000, :, 5] = float("nan")  # attended by the second query only
    o = call(q, k, v, Lk, b, e)[:4].float()
    assert not bool(torch.isfinite(o[1, :, 5]).any()) and bool(torch.isfinite(o[[0, 2, 3]]).all())


def test_rows_in_a_fused_buffer_and_a_longer_cache():
    L, H, Hkv = 150, 6, 2
    buf = torch.randn(L, (H + 2 * Hkv) * DH + 64, device="cuda").half()
    q = buf[:, :H * DH].unflatten(1, (H, DH))
    k, v = (buf[:, (H + i * Hkv) * DH:(H + (i + 1) * Hkv) * DH].unflatten(1, (Hkv, DH)) for i in (0, 1))
    check(q, k, v)
    cache = torch.full((2, 1000, Hkv, DH), float("nan"), device="cuda").half()
    cache[0, :L], cache[1, :L] = k, v
    check(q, cache[0], cache[1], None, t(np.full(L, L)))


def test_keys_beyond_32_bit_offsets():
    """A key row 2^20 values wide: the last rows lie past 2^32 values (8 GiB) into the buffer."""
    Lk, W, Lq = 4200, 1 << 20, 3
    buf = torch.empty(Lk * W, dtype=torch.float16, device="cuda")
    k, v = (buf.view(Lk, W)[:, i * DH:(i + 1) * DH].unflatten(1, (1, DH)) for i in (0, 1))
    k.copy_(torch.randn(Lk, 1, DH, device="cuda").half())
    v.copy_(torch.randn(Lk, 1, DH, device="cuda").half())
    q = torch.randn(Lq, 2, DH, device="cuda").half()
    check(q, k, v)
    check(q, k, v, t([4100, 0, 4199]), t([4200, 10, 4200]))


@pytest.mark.parametrize("Lq,Lk,H,Hkv", [(300, 300, 8, 2), (4, 5000, 28, 4)])
def test_streams_graphs_and_a_shared_workspace(Lq, Lk, H, Hkv):
    """Two captured calls that share one workspace, replayed in turn, and calls on two streams with
    a workspace each, give the bits of a call alone."""
    sets = [inputs(Lq, Lk, H, Hkv, 16 + i) for i in (0, 1)]
    want = [call(*s, Lk) for s in sets]
    n = dllm.dllm_attention_masked_workspace_bytes(Lq, Lk, H, Hkv)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    outs = [torch.zeros_like(w) for w in want]
    graphs = []
    for s, o in zip(sets, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(*s, Lk, o=o, ws=ws)
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o[:Lq], w[:Lq]) for o, w in zip(outs, want))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    spaces = [torch.empty_like(ws) for _ in range(2)]
    for o in outs:
        o.zero_()
    torch.cuda.synchronize()
    for _ in range(4):
        for s, st, o, w in zip(sets, streams, outs, spaces):
            call(*s, Lk, o=o, ws=w, stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(o[:Lq], w[:Lq]) for o, w in zip(outs, want))


def test_agrees_with_the_full_attention_entry_point():
    """With every key in every interval the two entry points compute the same attention."""
    q, k, v = inputs(400, 500, 8, 2, 17)
    o = torch.empty(400, 8, DH, device="cuda")
    dllm.dllm_attention(q, k, v, 400, 500, 8, 2, DH, o)
    ref, tol = formula(q, k, v, t(np.zeros(400)), t(np.full(400, 500)), None, 0.0, None)
    got = call(q, k, v, 500, f16=False)[:400]
    assert bool(((o.double() - ref).abs() <= tol).all()) and bool(((got.double() - ref).abs() <= tol).all())


def test_no_queries_is_a_no_op():
    dllm.dllm_attention_masked(None, 256, None, 256, None, 256, 0, 5, 2, 2, DH, None, None, None, 0.0, None, None,
                               dllm.DLLM_F16)
