"""The rotation, masked attention and sampling entry points on the host: the table of
turns against its formulas, and every refusal, which is decided before any device call."""
import ctypes
import math

import numpy as np
import pytest

from quantized_int8_gemm_q4_b200 import build as nbuild
from quantized_int8_gemm_q4_b200 import dllm


@pytest.fixture(scope="module", autouse=True)
def lib():
    nbuild.build()
    return dllm.load()


def frequencies(n, base, kind, factor, trained, fast, slow):
    f = [base ** (-2 * i / n) for i in range(n // 2)]
    if kind == dllm.DLLM_ROPE_LINEAR:
        return [x / factor for x in f]
    if kind == dllm.DLLM_ROPE_NTK:
        return [(base * factor ** (n / (n - 2))) ** (-2 * i / n) for i in range(n // 2)]
    if kind == dllm.DLLM_ROPE_YARN:
        d = [n / 2 * math.log(trained / (2 * math.pi * b)) / math.log(base) for b in (fast, slow)]
        lo, hi = max(math.floor(d[0]), 0), min(math.ceil(d[1]), n - 1)
        r = [min(max((i - lo) / max(hi - lo, 0.001), 0), 1) for i in range(n // 2)]
        return [x / factor * y + x * (1 - y) for x, y in zip(f, r)]
    return f


@pytest.mark.parametrize("kind", [dllm.DLLM_ROPE_PLAIN, dllm.DLLM_ROPE_LINEAR, dllm.DLLM_ROPE_NTK, dllm.DLLM_ROPE_YARN])
@pytest.mark.parametrize("n,base,factor,trained", [(128, 5e5, 8.0, 4096.0), (64, 1e4, 4.0, 2048.0), (4, 1e6, 1.0, 100.0),
                                                   (32, 1e4, 0.5, 64.0)])
def test_turns(kind, n, base, factor, trained):
    turns, ms = dllm.dllm_rope_turns(n, base, kind, factor, trained, 32.0, 1.0)
    want = np.array(frequencies(n, base, kind, factor, trained, 32.0, 1.0)) / (2 * math.pi)
    assert turns.shape == (n // 2,) and np.allclose(turns.numpy(), want, rtol=1e-14, atol=0)
    yarn = kind == dllm.DLLM_ROPE_YARN and factor > 1
    assert ms == np.float32(0.1 * math.log(factor) + 1 if yarn else 1)


def test_turns_of_an_unrotated_head():
    turns, ms = dllm.dllm_rope_turns(0, 1e4)
    assert turns.numel() == 0 and ms == 1.0


@pytest.mark.parametrize("args", [
    (3, 1e4), (-2, 1e4), (64, 1.0), (64, 0.0), (64, math.inf), (64, math.nan), (64, 1e4, 9), (64, 1e4, 1, 0.0),
    (64, 1e4, 1, -2.0), (64, 1e4, 1, math.nan), (2, 1e4, 2, 4.0), (64, 1e4, 3, 4.0, 0.0), (64, 1e4, 3, 4.0, 4096.0, 1.0, 32.0),
    (64, 1e4, 3, 4.0, 4096.0, 32.0, 0.0), (64, 1e4, 2, 1e300),
])
def test_turns_refused(args):
    with pytest.raises(dllm.DllmError) as e:
        dllm.dllm_rope_turns(*args)
    assert e.value.code == dllm.DLLM_ERR_ARG


P = 1 << 20  # 16-byte aligned, never dereferenced: the checks come first


def refuse(fn, args, names, changes, code):
    a = dict(zip(names, args))
    assert set(changes) <= set(a)
    a.update(changes)
    assert getattr(dllm.load(), fn)(*a.values()) == code


ROPE = ("q ldq k ldk v ldv L H Hkv dh pos turns n_rot layout mscale gamma_q gamma_k eps oq ok ov stream").split()
ROPE_OK = (P, 512, P, 256, P, 256, 4, 4, 2, 128, P, P, 128, 0, 1.0, P, P, 1e-6, P, P, P, None)


@pytest.mark.parametrize("change", [
    dict(L=-1), dict(H=0), dict(Hkv=0), dict(dh=0), dict(dh=100), dict(dh=264), dict(n_rot=-8), dict(n_rot=12),
    dict(n_rot=136), dict(layout=1), dict(ldq=508), dict(ldk=252), dict(ldv=252), dict(mscale=math.inf),
    dict(mscale=math.nan), dict(eps=0.0), dict(eps=math.nan), dict(q=None), dict(k=None), dict(oq=None), dict(ok=None),
    dict(ov=None), dict(turns=None), dict(L=1 << 31), dict(H=65536, ldq=65536 * 128),
])
def test_rope_arguments_refused(change):
    refuse("dllm_qk_rope", ROPE_OK, ROPE, change, dllm.DLLM_ERR_ARG)


@pytest.mark.parametrize("change", [dict(q=P + 4), dict(k=P + 8), dict(v=P + 4), dict(oq=P + 2), dict(ok=P + 8),
                                    dict(ov=P + 8), dict(pos=P + 4), dict(turns=P + 8), dict(gamma_q=P + 4),
                                    dict(gamma_k=P + 4), dict(ldq=513), dict(ldk=258), dict(ldv=257)])
def test_rope_alignment_refused(change):
    refuse("dllm_qk_rope", ROPE_OK, ROPE, change, dllm.DLLM_ERR_ALIGN)


ATT = ("q ldq k ldk v ldv Lq Lk H Hkv dh kv_begin kv_end q_pos softcap slopes o o_type workspace workspace_bytes "
       "stream").split()
ATT_OK = (P, 512, P, 256, P, 256, 4, 9, 4, 2, 128, P, P, P, 0.0, P, P, 1, P, 1 << 30, None)


@pytest.mark.parametrize("change", [
    dict(Lq=-1), dict(Lk=-1), dict(H=0), dict(Hkv=0), dict(H=3), dict(dh=64), dict(o_type=2), dict(softcap=-1.0),
    dict(softcap=math.nan), dict(softcap=math.inf), dict(softcap=1e-31), dict(softcap=2e30), dict(ldq=504), dict(ldk=248), dict(ldv=248), dict(q=None),
    dict(k=None), dict(v=None), dict(o=None), dict(Lq=(1 << 30) + 1), dict(Lk=(1 << 30) + 1), dict(H=65536),
])
def test_attention_arguments_refused(change):
    refuse("dllm_attention_masked", ATT_OK, ATT, change, dllm.DLLM_ERR_ARG)


@pytest.mark.parametrize("change", [dict(q=P + 2), dict(k=P + 8), dict(v=P + 8), dict(o=P + 4), dict(kv_begin=P + 4),
                                    dict(kv_end=P + 4), dict(q_pos=P + 4), dict(slopes=P + 4), dict(ldq=516),
                                    dict(ldk=260), dict(ldv=257)])
def test_attention_alignment_refused(change):
    refuse("dllm_attention_masked", ATT_OK, ATT, change, dllm.DLLM_ERR_ALIGN)


def test_attention_workspace_sizes_refused():
    n = ctypes.c_size_t(0)
    for a in ((-1, 5, 2, 2), (5, -1, 2, 2), (5, 5, 0, 1), (5, 5, 3, 2)):
        assert dllm.load().dllm_attention_masked_workspace_bytes(*a, ctypes.byref(n)) == dllm.DLLM_ERR_ARG
    assert dllm.load().dllm_attention_masked_workspace_bytes(5, 5, 2, 2, None) == dllm.DLLM_ERR_ARG


SMP = "logits R V ldl temperature top_k top_p min_p u token conf entropy stream".split()
SMP_OK = (P, 2, 1000, 1000, P, P, P, P, P, P, P, P, None)


@pytest.mark.parametrize("change", [dict(R=-1), dict(V=0), dict(V=-5), dict(ldl=999), dict(logits=None), dict(token=None),
                                    dict(V=1 << 31, ldl=1 << 31), dict(R=(1 << 27) + 1)])
def test_sample_arguments_refused(change):
    refuse("dllm_sample", SMP_OK, SMP, change, dllm.DLLM_ERR_ARG)


@pytest.mark.parametrize("name", ["logits", "temperature", "top_k", "top_p", "min_p", "u", "token", "conf", "entropy"])
def test_sample_alignment_refused(name):
    refuse("dllm_sample", SMP_OK, SMP, {name: P + 4}, dllm.DLLM_ERR_ALIGN)


def test_empty_calls_succeed_without_a_device():
    refuse("dllm_qk_rope", ROPE_OK, ROPE, dict(L=0, q=None, oq=None), dllm.DLLM_OK)
    refuse("dllm_attention_masked", ATT_OK, ATT, dict(Lq=0, q=None, o=None), dllm.DLLM_OK)
    refuse("dllm_sample", SMP_OK, SMP, dict(R=0, logits=None, token=None), dllm.DLLM_OK)


def test_status_string_of_bad_logits():
    assert "logits" in dllm.status_string(dllm.DLLM_ERR_LOGITS)
