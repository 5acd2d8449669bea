"""dllm_attention_masked on values that are not finite where a query does attend: what comes out does
not depend on how the keys are split, nor on what the rows beside it see."""
import numpy as np
import pytest
import torch

from quantized_int8_gemm_q4_b200 import dllm
from tests import test_gpu_attention_masked as att

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")
# (Lq, Lk, H, Hkv): keys split over CTAs, one query and a few, two CTAs per SM; halves; more tiles than SMs
SHAPES = [(1, 3000, 4, 4), (5, 8200, 28, 4), (1, 19000, 32, 32), (3, 300, 4, 2), (200, 900, 4, 4), (300, 500, 64, 8)]


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("GPU test run without a CUDA device")
    from quantized_int8_gemm_q4_b200 import build
    build.build()
    dllm.load()
    yield
    assert dllm.dllm_get_device_status() == dllm.DLLM_OK


@pytest.mark.parametrize("f16", [True, False])
@pytest.mark.parametrize("Lq,Lk,H,Hkv", SHAPES)
def test_a_query_that_is_not_finite(Lq, Lk, H, Hkv, f16):
    """Its row is NaN, every other one keeps its bits; without keys it gives zeros all the same."""
    q, k, v = att.inputs(Lq, Lk, H, Hkv, 31, Lk)
    i, h = Lq // 2, H - 2
    want = att.call(q, k, v, Lk, f16=f16)[:Lq].clone()
    none = torch.full((Lq,), Lk, device="cuda")
    none[i] = 0
    for bad in (NAN, INF, -INF):
        x = q.clone()
        x[i, h, 5] = bad
        got = att.call(x, k, v, Lk, f16=f16)[:Lq].clone()
        assert bool(torch.isnan(got[i, h]).all())
        got[i, h] = want[i, h]
        assert torch.equal(got, want)
        got = att.call(x, k, v, Lk, end=none, f16=f16)[:Lq]
        assert bool((got[i] == 0).all()) and bool(torch.isfinite(got).all())


@pytest.mark.parametrize("slopes", [False, True])
@pytest.mark.parametrize("Lq,Lk,H,Hkv", SHAPES)
def test_attended_keys_that_are_not_numbers(Lq, Lk, H, Hkv, slopes):
    """One key of a row's many, and all of a row's keys."""
    q, k, v = att.inputs(Lq, Lk, H, Hkv, 32, Lk)
    sl = torch.rand(H, device="cuda") * 0.01 if slopes else None
    g = H // Hkv
    begin, end = torch.zeros(Lq, dtype=torch.int64, device="cuda"), torch.full((Lq,), Lk, device="cuda")
    begin[0], end[0] = 70, 90
    begin[1:], end[1:] = 100, Lk
    for where in (slice(80, 81), slice(70, 90)):
        x = k.clone()
        x[where, Hkv - 1] = NAN
        want = att.call(q, k, v, Lk, begin, end, slopes=sl)[:Lq]
        got = att.call(q, x, v, Lk, begin, end, slopes=sl)[:Lq].clone()
        assert bool(torch.isnan(got[0, H - g:]).all())
        got[0, H - g:] = want[0, H - g:]
        assert torch.equal(got, want)


@pytest.mark.parametrize("Lq,Lk,H,Hkv", SHAPES)
def test_attended_keys_of_score_minus_infinity(Lq, Lk, H, Hkv):
    """They weigh nothing beside others; a row that has no other key has no softmax: NaN."""
    q, k, v = att.inputs(Lq, Lk, H, Hkv, 33, Lk)
    q[:, :, 0] = 4.0
    x = k.clone()
    n = Lk - Lk // 3
    x[:n, :, 0] = -INF
    b, e = torch.full((Lq,), n, device="cuda"), torch.full((Lq,), Lk, device="cuda")
    ref, tol = att.formula(q, k, v, b, e, None, 0.0, None)
    got = att.call(q, x, v, Lk, f16=False)[:Lq].double()
    assert bool(((got - ref).abs() <= tol).all())
    got = att.call(q, x, v, Lk, end=torch.full((Lq,), n - 3, device="cuda"), f16=False)[:Lq]
    assert bool(torch.isnan(got).all())


def documents_beside(Lq, Lk):
    """Intervals that all end inside a block of keys at 40 and begin at 0 or 20: no row sees the block whole."""
    b = torch.where(torch.arange(Lq, device="cuda") % 2 == 0, 0, 20)
    return b, torch.full((Lq,), Lk - 24, device="cuda")


@pytest.mark.parametrize("bad", [NAN, INF, -INF])
@pytest.mark.parametrize("Lq,Lk,H,Hkv", SHAPES)
def test_an_attended_value_costs_its_own_column(Lq, Lk, H, Hkv, bad):
    """Whether the other rows see its block whole, in part or not at all."""
    q, k, v = att.inputs(Lq, Lk, H, Hkv, 34, Lk)
    g = H // Hkv
    some = torch.arange(Lq, device="cuda") % 2 == 0
    for begin, end in ((None, None), documents_beside(Lq, Lk)):
        want = att.call(q, k, v, Lk, begin, end)[:Lq].clone()
        x = v.clone()
        # keys of the first block, a middle one and the last; columns of every part of a row
        for key, col in ((7, 3), (7, 127), (Lk // 2, 64), (Lk - 30, 40), (Lk - 2, 90)):
            x[key, Hkv - 1, col] = bad
        got = att.call(q, k, x, Lk, begin, end)[:Lq].clone()
        lost = torch.zeros_like(got, dtype=torch.bool)
        lost[:, H - g:, 64] = lost[:, H - g:, 40] = True
        if begin is None:
            lost[:, H - g:, 90] = True
        sees7 = torch.ones_like(some) if begin is None else some
        lost[sees7, H - g:, 3] = lost[sees7, H - g:, 127] = True
        assert torch.equal(~torch.isfinite(got), lost)
        got[lost] = want[lost]
        assert torch.equal(got, want)


@pytest.mark.parametrize("Lq,Lk,H,Hkv", SHAPES)
def test_an_attended_value_of_no_weight_costs_its_column(Lq, Lk, H, Hkv):
    """Where its score is minus infinity and that of every key around it."""
    q, k, v = att.inputs(Lq, Lk, H, Hkv, 35, Lk)
    q[:, :, 0] = 4.0
    k[:Lk // 2, :, 0] = -INF
    v[9, :, 3] = NAN
    for begin, end in ((None, None), documents_beside(Lq, Lk)):
        got = att.call(q, k, v, Lk, begin, end)[:Lq]
        sees = torch.zeros(Lq, dtype=torch.bool, device="cuda") if begin is not None else None
        if begin is not None:
            sees = begin == 0
            assert bool(torch.isfinite(got[~sees]).all())
            got = got[sees]
        assert not bool(torch.isfinite(got[:, :, 3]).any())
        assert bool(torch.isfinite(got[:, :, :3]).all()) and bool(torch.isfinite(got[:, :, 4:]).all())


@pytest.mark.parametrize("cap", [1e9, 2.0 ** 99, 2.0 ** 100])
@pytest.mark.parametrize("Lq,Lk,H,Hkv", SHAPES[2:])
def test_a_cap_far_above_the_scores_leaves_them_as_they_are(Lq, Lk, H, Hkv, cap):
    """cap tanh(x / cap) = x to (x / cap)^2 relative.  The kernel's polynomial is good to 2^-22 relative there and
    its scalings to 2^-24 each, together below 2^-20 |x|, which moves a weight by as much: 2 * 2^-20 max|x| max|v|
    beside the tolerance of uncapped scores.  Zeros and scores under a small cap lie outside of it."""
    q, k, v = att.inputs(Lq, Lk, H, Hkv, 36, Lk)
    b, e = torch.full((Lq,), 3, device="cuda"), torch.full((Lq,), Lk - 5, device="cuda")
    ref, tol = att.formula(q, k, v, b, e, None, 0.0, None)
    x = torch.einsum("ihd,jhd->hij", q.double(), k.double().repeat_interleave(H // Hkv, 1)).abs().amax() / att.DH ** 0.5
    tol = tol + 2 * 2.0 ** -20 * x * v.double().abs().amax()
    got = att.call(q, k, v, Lk, b, e, cap=cap, f16=False)[:Lq].double()
    assert bool(((got - ref).abs() <= tol).all())
    small = att.formula(q, k, v, b, e, None, 0.5, None)[0]
    for wrong in (torch.zeros_like(ref), small):
        assert int(((wrong - ref).abs() > tol).sum()) > 100  # one would do
