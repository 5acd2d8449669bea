"""The operators of a step in a row, as a denoising loop calls them: RMSNorm -> quantize ->
Q/K/V -> rotation with head norm -> attention over packed requests -> quantize -> O -> final
norm on the requested rows -> output projection -> sampling.  Eagerly and as one captured
graph (with the same bits), and every new stage against its formula on its own inputs."""
import numpy as np
import pytest
import torch

from quantized_int8_gemm_q4_b200 import dllm, synth
from tests import test_gpu_attention_masked as att
from tests import test_gpu_rope as rope
from tests import test_gpu_sample as smp

pytestmark = pytest.mark.gpu
Q4, Q6 = dllm.DLLM_Q4_K, dllm.DLLM_Q6_K


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("GPU test run without a CUDA device")
    from quantized_int8_gemm_q4_b200 import build
    build.build()
    dllm.load()
    yield
    assert dllm.dllm_get_device_status() == dllm.DLLM_OK


class Step:
    """One layer and the output projection over a canvas of packed requests."""

    def __init__(self, M, hidden, H, Hkv, vocab, lengths, rows, seed):
        self.M, self.K, self.H, self.Hkv, self.V = M, hidden, H, Hkv, vocab
        Nq, Nkv = H * 128, Hkv * 128
        w = lambda t, N, K, s: dllm.repack(t, synth.weights(t, N, K, seed, s), N, K)  # noqa: E731
        self.wq, self.wk, self.wv = (w(Q4, n, hidden, i) for i, n in enumerate((Nq, Nkv, Nkv)))
        self.wo, self.w_out = w(Q4, hidden, Nq, 3), w(Q6, vocab, hidden, 4)
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        self.x = dev(synth.activations(M, hidden, seed))
        self.gamma = dev(synth.norm_weights(2, hidden, seed))
        self.gq, self.gk = (0.02 * dev(g) for g in synth.norm_weights(2, 128, seed, 1))  # trained gains keep logits small
        turns, self.ms = dllm.dllm_rope_turns(128, 5e5, dllm.DLLM_ROPE_YARN, 4.0, 2048.0)
        self.turns = turns.cuda()
        begin, end = att.documents(lengths, M)
        self.pos = (torch.arange(M, device="cuda") - begin).to(torch.int32)  # positions restart in every request
        self.begin, self.end = begin.to(torch.int32), end.to(torch.int32)
        self.rows = dev(np.asarray(rows, np.int32))
        R = self.R = len(rows)
        g = np.random.default_rng(seed)
        self.u, self.top_p = dev(g.uniform(0, 1, R).astype(np.float32)), dev(np.full(R, 0.9, np.float32))
        self.t = dev(np.full(R, 300.0, np.float32))
        e = lambda *s, t=torch.float32: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
        self.qkv = e(M, Nq + 2 * Nkv)
        self.q, self.k, self.v = (e(M, h, 128, t=torch.float16) for h in (H, Hkv, Hkv))
        self.o, self.h, self.logits = e(M, H, 128), e(M, hidden), e(R, vocab)
        self.token, self.conf, self.ent = e(R, t=torch.int32), e(R), e(R)
        self.act, self.act_o, self.act_r = dllm.alloc_act(M, hidden), dllm.alloc_act(M, Nq), dllm.alloc_act(R, hidden)
        need = [dllm.dllm_qgemm_workspace_bytes(Q4, Nq + 2 * Nkv, hidden, M), dllm.dllm_qgemm_workspace_bytes(Q4, hidden, Nq, M),
                dllm.dllm_qgemm_workspace_bytes(Q6, vocab, hidden, R)]
        self.ws = dllm.alloc_workspace(max(need + [16]))
        self.att_bytes = dllm.dllm_attention_masked_workspace_bytes(M, M, H, Hkv)
        self.att_ws = dllm.alloc_workspace(self.att_bytes)

    def run(self):
        M, K, H, Hkv = self.M, self.K, self.H, self.Hkv
        Nq, Nkv, ld = H * 128, Hkv * 128, (H + 2 * Hkv) * 128
        wsb = self.ws.numel()
        q, k, v = self.qkv[:, :Nq], self.qkv[:, Nq:Nq + Nkv], self.qkv[:, Nq + Nkv:]
        dllm.dllm_rmsnorm_quantize(self.x, M, K, K, self.gamma[0], 1e-5, None, 0, *self.act)
        dllm.dllm_qkv_qgemm(self.wq, self.wk, self.wv, Q4, Nq, Nkv, K, *self.act, M, q, ld, k, v, ld, self.ws, wsb)
        dllm.dllm_qk_rope(q, ld, k, ld, v, ld, M, H, Hkv, 128, self.pos, self.turns, 128, dllm.DLLM_ROPE_NEOX, self.ms,
                          self.gq, self.gk, 1e-6, self.q, self.k, self.v)
        dllm.dllm_attention_masked(self.q, Nq, self.k, Nkv, self.v, Nkv, M, M, H, Hkv, 128, self.begin, self.end, None,
                                   0.0, None, self.o, dllm.DLLM_F32, self.att_ws, self.att_bytes)
        dllm.dllm_quantize_act(self.o, M, Nq, Nq, *self.act_o)
        dllm.dllm_qgemm(self.wo, Q4, K, Nq, *self.act_o, M, None, 0, self.h, K, self.ws, wsb)
        dllm.dllm_rmsnorm_quantize(self.h, M, K, K, self.gamma[1], 1e-5, self.rows, self.R, *self.act_r)
        dllm.dllm_qgemm(self.w_out, Q6, self.V, K, *self.act_r, self.R, None, 0, self.logits, self.V, self.ws, wsb)
        dllm.dllm_sample(self.logits, self.R, self.V, self.V, self.t, None, self.top_p, None, self.u, self.token,
                         self.conf, self.ent)

    def outputs(self):
        return [t.clone() for t in (self.q, self.k, self.v, self.o, self.logits, self.token, self.conf, self.ent)]


@pytest.mark.parametrize("M,hidden,H,Hkv,vocab,lengths", [
    (48, 512, 4, 2, 1024, [20, 17, 8]),
    (200, 1024, 28, 4, 2048, [1, 130, 60]),   # grouped heads; the last 9 rows are padding
    (700, 512, 32, 32, 1024, [333, 300]),     # two query tiles per CTA
])
def test_a_step_eagerly_and_captured(M, hidden, H, Hkv, vocab, lengths):
    rows = np.random.default_rng(M).permutation(sum(lengths))[:24]
    s = Step(M, hidden, H, Hkv, vocab, lengths, rows, M)
    s.run()
    torch.cuda.synchronize()
    assert dllm.dllm_get_device_status() == dllm.DLLM_OK
    eager = s.outputs()

    # the rotation, on the projections' own outputs
    Nq, Nkv = H * 128, Hkv * 128
    host = s.qkv.cpu().numpy()
    pos = s.pos.cpu().numpy()
    for got, x, gamma in ((s.q, host[:, :Nq], s.gq), (s.k, host[:, Nq:Nq + Nkv], s.gk)):
        rope.check(got, *rope.formula(x.reshape(M, -1, 128), pos, s.turns.cpu().numpy(), 128, dllm.DLLM_ROPE_NEOX, s.ms,
                                      gamma.cpu().numpy(), 1e-6))
    # attention, on the rotation's
    ref, tol = att.formula(s.q, s.k, s.v, s.begin.long(), s.end.long(), None, 0.0, None)
    assert bool(((s.o.double() - ref).abs() <= tol).all())
    assert bool((s.o[sum(lengths):] == 0).all())
    # the tokens, on the output projection's logits
    logits, u = s.logits.cpu().numpy(), s.u.cpu().numpy()
    assert np.isfinite(logits).all() and logits.std() > 0
    for r in range(s.R):
        at, c, h = smp.define(logits[r], 300.0, 0, float(np.float32(0.9)), 0.0, float(u[r]))
        assert int(s.token[r]) == at
        assert abs(float(s.conf[r]) - c) <= 1e-5 * c + 1e-30 and abs(float(s.ent[r]) - h) <= 1e-5 * h + 1e-12

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    for t in (s.qkv, s.q, s.k, s.v, s.o, s.h, s.logits, s.token, s.conf, s.ent):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(eager, s.outputs()))
