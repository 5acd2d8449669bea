"""dllm_sample where top_p follows top_k and each limit finds its cut in another way: top_k's by
ranking a bin in every CTA, top_p's by gathering few candidates in the first CTA."""
import numpy as np
import pytest
import torch

from quantized_int8_gemm_q4_b200 import dllm
from tests import test_gpu_sample as smp

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


@pytest.mark.parametrize("R,V", [(160, 60000), (40, 126464), (4, 152064), (200, 9000)])
def test_top_k_of_many_then_top_p_of_few(R, V):
    """Far more than 256 candidates up to top_k's cut, far fewer than 256 up to top_p's; many rows at once and
    again while copies on another stream take SMs, so that the CTAs of a cluster run apart."""
    x, g = smp.logits_of(R, V, 31, spread=1.0)
    x[np.arange(R)[:, None], g.integers(0, V, (R, 12))] = 14 + g.uniform(0, 3, (R, 12))
    k, p, u = g.integers(600, 4000, R), g.uniform(0.5, 0.9, R).astype(np.float32), g.uniform(0, 1, R).astype(np.float32)
    want = []
    for r in range(R):
        w = np.sort(np.exp(x[r].astype(np.float64) - x[r].max()))[::-1][:k[r]]
        assert np.searchsorted(np.cumsum(w), p[r] * w.sum()) < 100  # top_p keeps few
        want.append(smp.define(x[r], 1.0, int(k[r]), float(p[r]), 0.0, float(u[r]))[0])
    d = torch.from_numpy(x).cuda()
    k, p, u = (torch.from_numpy(a).cuda() for a in (k.astype(np.int32), p, u))
    noise, side = torch.zeros(1 << 24, device="cuda"), torch.cuda.Stream()
    token = [torch.full((R,), -7, dtype=torch.int32, device="cuda") for _ in range(12)]
    torch.cuda.synchronize()
    for i, t in enumerate(token):
        if i >= 4:
            with torch.cuda.stream(side):
                noise.add_(1.0)
        dllm.dllm_sample(d, R, V, V, None, k, p, None, u, t, None, None)
    torch.cuda.synchronize()
    assert dllm.dllm_get_device_status() == dllm.DLLM_OK
    for t in token:
        assert t.tolist() == want


def tokens_of(x, T=None, k=None, p=None, mp=None, u=None):
    """The tokens alone: a word of no more than 2^-149 has the confidence 0 in f32."""
    R = len(x)
    f = lambda a, d: np.full(R, d) if a is None else np.asarray(a)  # noqa: E731
    got = smp.run(x, T, k, p, mp, u)[0].tolist()
    T, k, p, mp, u = (f(a, d) for a, d in ((T, 1.0), (k, 0), (p, 1.0), (mp, 0.0), (u, 0.0)))
    T, p, mp, u = (np.float32(a) for a in (T, p, mp, u))
    want = [smp.define(x[r], float(T[r]), int(k[r]), float(p[r]), float(mp[r]), float(u[r]))[0] for r in range(R)]
    assert got == want


@pytest.mark.parametrize("far", [33.0, 40.0, 300.0])
@pytest.mark.parametrize("V", [1, 2, 50, 700, 30001, 160000])
def test_first_and_last_kept_word_however_unlikely(V, far):
    """u at its ends takes the first and the last kept index, also where the kept words before and behind the
    likely ones weigh less than the unit of the masses."""
    u = np.array([0.0, 1.0, -3.0, 7.0, np.nan, 0.0, 1.0, 0.5], np.float32)
    R = len(u)
    for T in (0.1, 1.0, 4.0):
        g = np.random.default_rng([V, int(far)])
        x = (g.standard_normal((R, V)) * 0.1 * T).astype(np.float32)
        x[:, V // 2] = np.float32(far * T)
        x[:, :V // 9:2] = -np.inf  # ruled out: not kept
        if V > 9:
            x[:, V - 3:] = -np.inf
        t = np.full(R, T)
        tokens_of(x, T=t, u=u)
        tokens_of(x, T=t)
        tokens_of(x, T=t, u=u, k=np.array([V, V, 40, 40, 3, 300, 300, 2]))  # by a list of few, and by masses of many
        tokens_of(x, T=t, u=u, p=np.full(R, 0.9))
        tokens_of(x, T=t, u=u, mp=np.full(R, 1e-6))


def test_words_that_weigh_nothing_in_64_bits_are_not_drawn():
    x = np.zeros((3, 5000), np.float32)
    x[:, 77], x[:, 3000], x[:, 4000] = 10.0, 9.5, 9.0
    tokens_of(x, T=np.full(3, 0.01), u=np.array([0.0, 1.0, 0.5]))
    tokens_of(x, T=np.full(3, 0.001), u=np.array([0.0, 1.0, 0.5]))
    tokens_of(x, T=np.full(3, 0.01), u=np.array([0.0, 1.0, 0.5]), k=np.array([100, 3000, 100]))


@pytest.mark.parametrize("R,V", [(6, 900), (6, 40000), (2, 152064)])
def test_words_masked_with_the_lowest_float(R, V):
    """They are finite, weigh nothing and are not drawn, at the first index, the last and where only they follow."""
    low = float(np.finfo(np.float32).min)
    x, g = smp.logits_of(R, V, 37)
    x[:, :7], x[:, V // 3:V // 2], x[:, -9:] = low, low, low
    x[1] = np.where(x[1] == low, -np.inf, x[1])
    x[1, 3] = low
    for u in (np.zeros(R), np.ones(R), g.uniform(0, 1, R)):
        smp.check(x, u=u)
        smp.check(x, k=np.full(R, V - 5), u=u)
        smp.check(x, k=g.integers(1, 400, R), u=u)
        smp.check(x, T=g.uniform(0.3, 2.0, R), p=g.uniform(0.3, 1.0, R), mp=np.full(R, 0.001), u=u)
    x[0] = low  # a row of nothing else: all alike
    smp.check(x[:1], u=np.array([0.3]))
