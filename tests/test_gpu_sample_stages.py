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
