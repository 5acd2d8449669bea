"""dllm_sample against the definition in 64 bits: the same token in every row, and the
confidence and entropy within f32 error.

Tolerance of conf and entropy.  The kernel sums at most V / 1024 f32 terms per thread and the
rest in f64: relative error at most (V / 1024 + 8) * 2^-24 of the mass below the largest logit
and of its first moment, plus expf's 2 ulp; both figures are ratios or sums of such terms of one
sign, so 4 (V / 1024 + 16) 2^-24 relative covers them, with the final rounding.
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


def define(row, T, k, p, mp, u):
    l = row.astype(np.float64) - float(row.max())
    greedy = not T > 0
    with np.errstate(invalid="ignore"):
        w = np.exp(l if greedy else np.where(np.isinf(l), -np.inf, l / np.float64(T)))
    order = np.argsort(-row, kind="stable")
    if greedy:
        order = order[:1]
    elif k > 0:
        order = order[:k]
    mp = min(mp, 1.0) if mp > 0 else 0.0
    order = order[w[order] >= mp]
    if not p >= 1:
        p = p if p > 0 else 0.0
        before = np.cumsum(w[order]) - w[order]
        keep = before < p * w[order].sum()
        keep[0] = True
        order = order[keep]
    only = np.zeros_like(w)
    only[order] = w[order]
    mass = np.cumsum(only)
    u = min(u, 1.0) if u > 0 else 0.0
    at = min(int(np.searchsorted(mass, u * mass[-1], side="right")), int(np.flatnonzero(only)[-1]))
    e = np.exp(l)
    pr = e / e.sum()
    return at, pr[at], -(pr[pr > 0] * np.log(pr[pr > 0])).sum()


def run(logits, T=None, k=None, p=None, mp=None, u=None, stream=None):
    R, V = logits.shape
    dev = lambda a, t: None if a is None else torch.from_numpy(np.asarray(a, t)).cuda()  # noqa: E731
    out = (torch.full((R,), -7, dtype=torch.int32, device="cuda"), torch.full((R,), -7.0, device="cuda"),
           torch.full((R,), -7.0, device="cuda"))
    d = torch.from_numpy(np.ascontiguousarray(logits)).cuda()
    dllm.dllm_sample(d, R, V, V, dev(T, np.float32), dev(k, np.int32), dev(p, np.float32), dev(mp, np.float32),
                     dev(u, np.float32), *out, stream)
    return [o.cpu().numpy() for o in out]


def check(logits, T=None, k=None, p=None, mp=None, u=None):
    R, V = logits.shape
    token, conf, ent = run(logits, T, k, p, mp, u)
    f = lambda a, d: np.full(R, d) if a is None else np.asarray(a)  # noqa: E731
    T, k, p, mp, u = (f(np.float32(a) if a is not None and i != 1 else a, d)
                      for i, (a, d) in enumerate(((T, 1.0), (k, 0), (p, 1.0), (mp, 0.0), (u, 0.0))))
    rel = 4 * (V / 1024 + 16) * 2.0 ** -24
    for r in range(R):
        at, c, h = define(logits[r], float(T[r]), int(k[r]), float(p[r]), float(mp[r]), float(u[r]))
        assert token[r] == at, (r, token[r], at)
        assert abs(conf[r] - c) <= rel * c and abs(ent[r] - h) <= rel * h + 1e-12, (r, conf[r], c, ent[r], h)


def logits_of(R, V, seed, spread=2.0):
    g = np.random.default_rng([seed, R, V])
    x = g.standard_normal((R, V)).astype(np.float32) * np.float32(spread)
    for r in range(R):
        n = min(V, 30)
        x[r, g.choice(V, n, replace=False)] = 5 + 4 * g.standard_normal(n)
    return x, g


@pytest.mark.parametrize("V", [1, 2, 31, 33, 1000, 8192, 8193, 16385, 40000, 126464, 152064, 500001])
def test_all_limits(V):
    """Every cluster size, and slices beyond shared memory."""
    R = 12
    x, g = logits_of(R, V, 1)
    x[:, g.integers(0, V, V // 50)] = -np.inf
    x[:, V // 2] = 1.0  # one finite at least
    check(x, T=g.uniform(0.3, 1.6, R), k=g.integers(0, max(2, V // 3), R), p=g.uniform(0.3, 1.0, R),
          mp=g.choice([0.0, 0.001, 0.05], R), u=g.uniform(0, 1, R))


@pytest.mark.parametrize("R,V", [(1, 152064), (3, 126465), (9, 65537), (10, 70000), (2, 800000)])
@pytest.mark.parametrize("spread", [0.3, 3.0])
def test_few_rows_of_large_vocabularies(R, V, spread):
    """Clusters of 16 (up to 9 rows on 148 SMs) and of 8; flat rows, whose limits keep thousands of
    words, and peaked ones, whose limits keep a few."""
    x, g = logits_of(R, V, 9, spread)
    u = g.uniform(0, 1, R)
    check(x, u=u)
    check(x, k=g.integers(1, V, R), p=g.uniform(0.2, 1.0, R), u=u)
    check(x, T=np.full(R, 0.7), k=g.integers(1, 200, R), p=g.uniform(0.2, 1.0, R), u=u)
    check(x, p=g.uniform(0.2, 1.0, R), mp=np.full(R, 1e-4), u=u)
    check(x, T=np.zeros(R), u=u)


@pytest.mark.parametrize("limit", ["none", "k", "p", "mp", "greedy"])
@pytest.mark.parametrize("V", [700, 30001])
def test_each_limit_alone(limit, V):
    R = 40
    x, g = logits_of(R, V, 2, spread=0.5)
    u = g.uniform(0, 1, R)
    check(x, T=np.zeros(R) if limit == "greedy" else None, k=g.integers(1, V + 5, R) if limit == "k" else None,
          p=g.uniform(0.01, 1.0, R) if limit == "p" else None, mp=g.uniform(0, 1, R) if limit == "mp" else None, u=u)


@pytest.mark.parametrize("spread", [0.01, 1.0, 4.0, 30.0])
@pytest.mark.parametrize("V", [1, 7, 5000, 126464])
def test_top_p_alone_from_one_word_to_nearly_all(V, spread):
    """The cut in the first bin, in the middle, and far down the tail, behind words that no bin holds."""
    p = np.array([2.0 ** -24, 0.01, 0.5, 0.9, 0.99, 0.9999, 1 - 2.0 ** -20, 1 - 2.0 ** -24], np.float32)
    R = len(p)
    x, g = logits_of(R, V, 10, spread)
    u = g.uniform(0, 1, R)
    for T in (0.2, 1.0, 5.0):
        check(x, T=np.full(R, T), p=p, u=u)
    check(np.round(x), p=p, u=u)
    x[:, 1::3] = -np.inf
    check(x, T=np.full(R, 0.8), p=p, u=u)


def test_ties_go_to_the_lowest_index():
    """Equal logits at the border of a limit: more than the ranked list holds, and fewer."""
    R, V = 8, 20000
    g = np.random.default_rng(3)
    x = np.round(g.standard_normal((R, V)) * 2).astype(np.float32)  # a dozen distinct values
    u = g.uniform(0, 1, R)
    check(x, k=g.integers(1, V, R), u=u)
    check(x, p=g.uniform(0.05, 0.95, R), u=u)
    check(x, k=g.integers(1, 9000, R), p=g.uniform(0.05, 0.95, R), u=u)
    check(np.zeros((R, V), np.float32), k=g.integers(1, V, R), p=np.full(R, 0.5), u=u)
    check(np.where(x > 3, x, np.float32(-0.0)) * np.float32(1), p=np.full(R, 0.9), u=u)


def test_values_that_crowd_one_bin():
    """A few far values stretch the range, so that nearly all the others share a bin."""
    R, V = 6, 30000
    x, g = logits_of(R, V, 4, spread=0.01)
    x[:, 7], x[:, 11] = 3e38, -3e38
    x[1, 7] = 40.0
    x[2, :] = np.ldexp(np.float32(1), -(np.arange(V) % 140)).astype(np.float32)
    x[3, :] = np.float32(1e-42) * (np.arange(V) % 5)
    x[4, 7] = 1.0
    u = g.uniform(0, 1, R)
    check(x, k=g.integers(1, V, R), u=u)
    check(x, p=np.array([0.5, 0.9, 0.99, 0.7, 0.999, 0.3]), u=u, T=np.array([1, 30, 1, 1, 1, 1e30]))


def test_parameters_at_their_ends():
    V = 3001
    cases = [(0.0, 0, 1.0, 0.0, 0.5), (-1.0, 5, 0.5, 0.0, 0.9), (np.nan, 0, 1.0, 0.0, 0.1), (np.inf, 0, 0.5, 0.0, 0.999),
             (1e-30, 0, 0.9, 0.0, 0.7), (1e30, 7, 1.0, 0.0, 1.0), (1.0, 1, 1.0, 0.0, 1.0), (1.0, V, 0.0, 0.0, 0.99),
             (1.0, -3, -1.0, 0.0, 0.5), (1.0, 0, np.nan, 0.0, 0.5), (1.0, 0, 2.0, 5.0, 0.5), (1.0, 0, 1.0, np.nan, 0.5),
             (1.0, 2 ** 31 - 1, 1.0, 1.0, 0.5), (1.0, 0, 1.0, 0.0, np.nan), (1.0, 0, 1.0, 0.0, 1.0),
             (1.0, 0, 1.0, 0.0, 7.0), (1.0, 0, 1.0, 0.0, -1.0), (1.0, 0, 0.99999994, 0.0, 0.9999999)]
    x, _ = logits_of(len(cases), V, 5)
    T, k, p, mp, u = (np.array(c) for c in zip(*cases))
    check(x, T, k, p, mp, u)


def test_peaked_rows_keep_their_entropy():
    """A row with nearly all its mass on one word: entropy to f32 accuracy, not lost next to 1."""
    x = np.full((4, 5000), -20.0, np.float32)
    x[:, 100] = [0.0, 5.0, 30.0, 60.0]
    check(x, u=np.array([0.0, 0.5, 0.9, 0.99]))


def test_rows_that_cannot_be_sampled():
    x, _ = logits_of(5, 4000, 6)
    x[1, 17], x[2, 3999], x[3] = np.nan, np.inf, -np.inf
    assert dllm.dllm_get_device_status() == dllm.DLLM_OK
    token, conf, ent = run(x, u=np.full(5, 0.3))
    assert dllm.dllm_get_device_status() == dllm.DLLM_ERR_LOGITS
    assert list(token[1:4]) == [-1] * 3 and not conf[1:4].any() and not ent[1:4].any()
    for r in (0, 4):
        at, c, h = define(x[r], 1.0, 0, 1.0, 0.0, float(np.float32(0.3)))
        assert token[r] == at and abs(conf[r] - c) < 1e-5 and abs(ent[r] - h) < 1e-5 * h


def test_row_stride_optional_outputs_and_bounds():
    """A leading dimension beyond V, no conf or entropy, rows behind the last left alone."""
    R, V, ld = 9, 1201, 1300
    x, g = logits_of(R, V, 7)
    buf = torch.full((R, ld), 1e9, device="cuda")
    buf[:, :V] = torch.from_numpy(x).cuda()
    u = torch.from_numpy(g.uniform(0, 1, R).astype(np.float32)).cuda()
    token = torch.full((R + 3,), -7, dtype=torch.int32, device="cuda")
    dllm.dllm_sample(buf, R, V, ld, None, None, None, None, u, token, None, None)
    got = token.cpu().numpy()
    assert list(got[R:]) == [-7] * 3
    assert all(got[r] == define(x[r], 1.0, 0, 1.0, 0.0, float(u[r]))[0] for r in range(R))
    dllm.dllm_sample(None, 0, V, ld, None, None, None, None, None, None, None, None)


def test_two_calls_at_once_and_a_replayed_graph():
    """Calls on two streams at the same time, and a captured call on changed logits."""
    R, V = 64, 60000
    x, g = logits_of(R, V, 8)
    d = torch.from_numpy(x).cuda()
    p, u = torch.full((R,), 0.9, device="cuda"), torch.from_numpy(g.uniform(0, 1, R).astype(np.float32)).cuda()
    new = lambda: (torch.empty(R, dtype=torch.int32, device="cuda"), torch.empty(R, device="cuda"),  # noqa: E731
                   torch.empty(R, device="cuda"))
    outs, streams = [new(), new(), new()], [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        for s, o in zip(streams, outs):
            dllm.dllm_sample(d, R, V, V, None, None, p, None, u, *o, s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs[0], outs[1]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dllm.dllm_sample(d, R, V, V, None, None, p, None, u, *outs[2])
    d.mul_(0.5)
    graph.replay()
    dllm.dllm_sample(d, R, V, V, None, None, p, None, u, *outs[0])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs[0], outs[2]))
