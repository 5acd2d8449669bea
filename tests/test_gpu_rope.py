"""dllm_qk_rope against the formula in 64 bits, element by element.

Tolerance.  The kernel's angle is off by at most 2^-26 turns (the reduced turns, at most
1/2, rounded to f32) and sincospif by 2 ulp, so cos and sin by less than 2^-22 + 2 * 2^-24 <
2^-21; the rotation's two products and sum and the factor mscale add 4 * 2^-24.  The norm's
f32 sum of dh squares is off by at most dh * 2^-24 relative (half of that after the root),
and its few other operations by 8 * 2^-24.  So before the rounding to f16 an element is off by
E <= mscale (|x1| + |x2|) (2^-20 + [norm] (dh + 8) 2^-24); the rounding adds 2^-11 of the value
(or 2^-25 below the normal range).
"""
import numpy as np
import pytest
import torch

from quantized_int8_gemm_q4_b200 import dllm

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("GPU test run without a CUDA device")
    from quantized_int8_gemm_q4_b200 import build
    build.build()
    dllm.load()
    yield
    assert dllm.dllm_get_device_status() == dllm.DLLM_OK


def pairs(n, layout):
    i = np.arange(n // 2)
    return (2 * i, 2 * i + 1) if layout == dllm.DLLM_ROPE_NORM else (i, i + n // 2)


def formula(x, pos, turns, n, layout, ms, gamma, eps):
    """x f64 [L][heads][dh] -> (y, E) with E the tolerance before the rounding."""
    dh = x.shape[-1]
    x = x.astype(np.float64)
    norm = 0.0
    if gamma is not None:
        x = x * gamma.astype(np.float64) / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
        norm = (dh + 8) * 2.0 ** -24
    y, E = x.copy(), np.abs(x) * norm
    if n:
        t = pos.astype(np.longdouble)[:, None] * turns.astype(np.longdouble)
        a = 2 * np.pi * (t - np.rint(t)).astype(np.float64)
        c, s = (ms * np.cos(a))[:, None], (ms * np.sin(a))[:, None]
        p1, p2 = pairs(n, layout)
        x1, x2 = x[..., p1], x[..., p2]
        y[..., p1], y[..., p2] = x1 * c - x2 * s, x2 * c + x1 * s
        E[..., p1] = E[..., p2] = abs(ms) * (np.abs(x1) + np.abs(x2)) * (2.0 ** -20 + norm)
    return y, E


def check(got, y, E):
    got = got.float().cpu().numpy().astype(np.float64)
    tol = (np.abs(y) + E) * 2.0 ** -11 + 2.0 ** -25 + E
    assert np.all(np.isfinite(got))
    bad = np.abs(got - y) > tol
    assert not bad.any(), (np.argwhere(bad)[0], float(np.max(np.abs(got - y) / tol)))


def run(L, H, Hkv, dh, n, layout, kind=dllm.DLLM_ROPE_PLAIN, pos=None, norm="", with_v=True, seed=0, pad=0, base=1e4):
    g = np.random.default_rng([seed, L, H, dh, n])
    width = (H + 2 * Hkv) * dh + pad
    qkv = torch.from_numpy(g.standard_normal((L, width)).astype(np.float32) * 2).cuda()
    q, k, v = qkv[:, :H * dh], qkv[:, H * dh:(H + Hkv) * dh], qkv[:, (H + Hkv) * dh:(H + 2 * Hkv) * dh]
    turns, ms = dllm.dllm_rope_turns(n, base, kind, 4.0, 2048.0)
    gq = g.uniform(0.5, 1.5, dh).astype(np.float32) if "q" in norm else None
    gk = g.uniform(0.5, 1.5, dh).astype(np.float32) if "k" in norm else None
    dev = lambda a: None if a is None else torch.from_numpy(a).cuda()  # noqa: E731
    # one row more than is written, to see that it stays as it was
    out = [torch.full((L + 1, h, dh), 7.0, dtype=torch.float16, device="cuda") for h in (H, Hkv, Hkv)]
    pd = None if pos is None else torch.from_numpy(np.asarray(pos, np.int32)).cuda()
    dllm.dllm_qk_rope(q, width, k, width, v if with_v else None, width, L, H, Hkv, dh, pd, turns.cuda(), n, layout, ms,
                      dev(gq), dev(gk), 1e-6, out[0], out[1], out[2] if with_v else None)
    assert all(bool((o[L:] == 7.0).all()) for o in out)
    p = np.arange(L) if pos is None else np.asarray(pos)
    host = lambda t, h: t.cpu().numpy().reshape(L, h, dh)  # noqa: E731
    check(out[0][:L], *formula(host(q, H), p, turns.numpy(), n, layout, ms, gq, 1e-6))
    check(out[1][:L], *formula(host(k, Hkv), p, turns.numpy(), n, layout, ms, gk, 1e-6))
    if with_v:
        assert torch.equal(out[2][:L], v.reshape(L, Hkv, dh).half())
    else:
        assert bool((out[2] == 7.0).all())


@pytest.mark.parametrize("layout", [dllm.DLLM_ROPE_NORM, dllm.DLLM_ROPE_NEOX])
@pytest.mark.parametrize("L,H,Hkv,dh,n", [
    (1, 1, 1, 8, 8),        # one position, one lane per head
    (1, 32, 32, 128, 128),  # one position of an 8B model
    (3, 28, 4, 128, 128),   # grouped heads
    (5, 7, 3, 80, 32),      # ten lanes of sixteen, part of the head
    (2, 3, 1, 96, 96),
    (2, 5, 5, 256, 64),     # a full warp per head
    (2, 2, 2, 64, 0),       # no rotation: the rounding alone
    (130, 32, 32, 128, 64),
    (1500, 9, 1, 40, 40),   # all heads of a position in one CTA
])
def test_rope_matches_formula(layout, L, H, Hkv, dh, n):
    run(L, H, Hkv, dh, n, layout)


@pytest.mark.parametrize("norm", ["q", "k", "qk"])
@pytest.mark.parametrize("dh,n,layout", [(128, 128, dllm.DLLM_ROPE_NEOX), (80, 40, dllm.DLLM_ROPE_NORM),
                                         (256, 256, dllm.DLLM_ROPE_NORM), (24, 8, dllm.DLLM_ROPE_NEOX)])
def test_head_norm_in_the_same_pass(norm, dh, n, layout):
    run(19, 12, 4, dh, n, layout, norm=norm, seed=1)


@pytest.mark.parametrize("kind", [dllm.DLLM_ROPE_LINEAR, dllm.DLLM_ROPE_NTK, dllm.DLLM_ROPE_YARN])
def test_scaled_tables(kind):
    run(77, 8, 2, 128, 128, dllm.DLLM_ROPE_NEOX, kind=kind, seed=2)


def test_any_position():
    """Positions to both ends of int32, in no order, some twice."""
    pos = [0, -1, 1, 2 ** 31 - 1, -2 ** 31, 123456789, 5, 5, 1000003]
    for layout in (dllm.DLLM_ROPE_NORM, dllm.DLLM_ROPE_NEOX):
        run(len(pos), 4, 2, 128, 128, layout, pos=pos, seed=3, base=5e5)


def test_without_v_and_with_padded_rows():
    run(40, 6, 2, 64, 32, dllm.DLLM_ROPE_NORM, with_v=False, pad=12, seed=4)


def test_zero_rows_and_large_values():
    """An all-zero head stays zero under the norm; f16 overflow gives infinities, not NaN."""
    x = torch.zeros(2, 3 * 64, device="cuda")
    x[1] = 70000.0
    out = [torch.empty(2, 1, 64, dtype=torch.float16, device="cuda") for _ in range(3)]
    gamma = torch.ones(64, device="cuda")
    turns = dllm.dllm_rope_turns(64, 1e4)[0].cuda()
    args = (x[:, :64], 192, x[:, 64:128], 192, x[:, 128:], 192, 2, 1, 1, 64, None, turns, 64, dllm.DLLM_ROPE_NEOX, 1.0)
    dllm.dllm_qk_rope(*args, gamma, gamma, 1e-6, *out)
    assert bool((out[0][0] == 0).all()) and bool((out[1][0] == 0).all())
    assert bool(torch.isfinite(out[0]).all()) and bool(torch.isinf(out[2][1]).all())


def test_no_positions_is_a_no_op():
    dllm.dllm_qk_rope(None, 128, None, 128, None, 0, 0, 1, 1, 128, None, None, 0, dllm.DLLM_ROPE_NORM, 1.0, None, None,
                      1e-6, None, None, None)


def test_on_another_stream_and_captured():
    """The same bits from a side stream and from a graph replayed on new inputs."""
    L, H, dh = 64, 8, 128
    turns = dllm.dllm_rope_turns(dh, 1e4)[0].cuda()
    x = torch.randn(L, 3 * H * dh, device="cuda")

    def call(out, stream=None):
        W = H * dh
        dllm.dllm_qk_rope(x[:, :W], 3 * W, x[:, W:2 * W], 3 * W, x[:, 2 * W:], 3 * W, L, H, H, dh, None, turns, dh,
                          dllm.DLLM_ROPE_NEOX, 1.0, None, None, 1e-6, *out, stream)

    new = lambda: [torch.zeros(L, H, dh, dtype=torch.float16, device="cuda") for _ in range(3)]  # noqa: E731
    a, b, c = new(), new(), new()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    call(b, s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(c)
    x.mul_(0.5)
    torch.cuda.current_stream().wait_stream(s)
    g.replay()
    call(a)
    torch.cuda.synchronize()
    assert all(torch.equal(u, w) for u, w in zip(a, c))
    s.wait_stream(torch.cuda.current_stream())
    call(b, s)
    s.synchronize()
    assert all(torch.equal(u, w) for u, w in zip(a, b))
