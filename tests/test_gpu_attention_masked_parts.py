"""dllm_attention_masked over long caches at both sides of the rules that cut the keys into parts."""
import pytest
import torch

from quantized_int8_gemm_q4_b200 import dllm
from tests import test_gpu_attention_masked as att

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


@pytest.mark.parametrize("Lq,H,Hkv,lengths", [
    (1, 32, 32, (700, 768, 9000, 12000)), (1, 50, 50, (500, 1100, 2000, 3001)), (3, 40, 40, (2500, 4000)),
    (128, 8, 8, (769, 9000)), (30, 28, 4, (2000, 9001)), (1, 73, 73, (1000, 5000)), (1, 74, 74, (1000, 5000)),
])
def test_parts_of_every_kind(Lq, H, Hkv, lengths):
    """Whole caches, and intervals that leave most parts without a key of a row."""
    for Lk in lengths:
        q, k, v = att.inputs(Lq, Lk, H, Hkv, 41, Lk)
        att.check(q, k, v)
        at = torch.arange(Lq, device="cuda") * (Lk // (2 * Lq))
        att.check(q, k, v, at, at + 70, f16=False)
