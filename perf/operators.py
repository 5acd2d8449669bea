"""Workloads of a step's operators around its GEMMs: the rotation of queries and keys,
attention under key intervals, and sampling from logits.

A case is one call as a serving program makes it.  run() computes it with elementary
torch operations (own = False) or through the library (own = True).
"""
import math

import numpy as np
import torch

own = False


def listed():
    return [
        # one new position of an 8B model with 32 heads
        dict(name="rope one position", op="rope", L=1, H=32, Hkv=32, dh=128, n_rot=128, layout="norm",
             scaling="plain", qk_norm=False, with_v=True, far=4000),
        # the 128-position canvas of the default step
        dict(name="rope canvas 128", op="rope", L=128, H=32, Hkv=32, dh=128, n_rot=128, layout="norm",
             scaling="plain", qk_norm=False, with_v=True, far=0),
        # grouped heads, normalised, half layout, positions far beyond the trained context
        dict(name="rope norm yarn 1021", op="rope", L=1021, H=28, Hkv=4, dh=128, n_rot=128, layout="neox",
             scaling="yarn", qk_norm=True, with_v=True, far=100000),
        # a batch of canvases in one call, half of each head rotated
        dict(name="rope norm 4096", op="rope", L=4096, H=32, Hkv=32, dh=128, n_rot=64, layout="neox",
             scaling="plain", qk_norm=True, with_v=True, far=0),
        # several requests' canvases packed into one sequence, padded at its end
        dict(name="attention packed 1024", op="attention", Lq=1024, Lk=1024, H=32, Hkv=32, mask="documents", arg=6,
             cap=0.0, bias=False),
        # a long prompt every position sees, the rest causal
        dict(name="attention prefix 4096", op="attention", Lq=4096, Lk=4096, H=32, Hkv=32, mask="prefix", arg=1000,
             cap=0.0, bias=False),
        # one 32-position block denoised over its kept prefix, grouped heads
        dict(name="attention block over 8200", op="attention", Lq=32, Lk=8200, H=28, Hkv=4, mask="blocks", arg=32,
             cap=0.0, bias=False),
        # one position over a long kept prefix
        dict(name="attention one over 20011", op="attention", Lq=1, Lk=20011, H=32, Hkv=32, mask="full", arg=0,
             cap=0.0, bias=False),
        # capped scores with a distance bias over packed requests of odd lengths
        dict(name="attention capped bias 1531", op="attention", Lq=1531, Lk=1531, H=28, Hkv=4, mask="documents",
             arg=3, cap=30.0, bias=True),
        # one requested row of a 152064-word vocabulary
        dict(name="sample 1 row", op="sample", R=1, V=152064, limits="all"),
        # the 32 requested rows of the default step
        dict(name="sample 32 rows", op="sample", R=32, V=126464, limits="p"),
        # every row of two canvases
        dict(name="sample 256 rows", op="sample", R=256, V=126464, limits="all"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "attention", "sample"])
    if op == "rope":
        H, Hkv = rng.choice([(32, 32), (28, 4), (32, 8), (8, 1)])
        dh = rng.choice([64, 80, 96, 128, 256])
        n_rot = rng.choice([dh, dh, dh // 2, 32])
        L = _log_int(rng, 1, min(8192, 4096 * 96 * 128 // ((H + 2 * Hkv) * dh)))
        return dict(op=op, L=L, H=H, Hkv=Hkv, dh=dh, n_rot=n_rot, layout=rng.choice(["norm", "neox"]),
                    scaling=rng.choice(["plain", "linear", "ntk", "yarn"]), qk_norm=rng.random() < 0.5,
                    with_v=rng.random() < 0.8, far=rng.choice([0, 0, 5000, 1000000]))
    if op == "attention":
        H, Hkv = rng.choice([(32, 32), (28, 4), (32, 8), (8, 1)])
        mask = rng.choice(["documents", "prefix", "blocks", "window", "full"])
        if rng.random() < 0.4:  # few queries over a kept prefix
            Lk = _log_int(rng, 64, 20000)
            Lq = min(Lk, _log_int(rng, 1, 64))
        else:
            Lq = Lk = _log_int(rng, 1, 2900)
        arg = {"documents": rng.randint(1, 9), "prefix": rng.randint(0, Lk), "blocks": rng.choice([16, 32, 48, 128]),
               "window": rng.randint(0, 700), "full": 0}[mask]
        return dict(op=op, Lq=Lq, Lk=Lk, H=H, Hkv=Hkv, mask=mask, arg=arg, cap=rng.choice([0.0, 0.0, 30.0, 50.0]),
                    bias=rng.random() < 0.3)
    V = _log_int(rng, 500, 160000)
    return dict(op=op, R=_log_int(rng, 1, min(400, 256 * 126464 // V)), V=V,
                limits=rng.choice(["all", "p", "k", "none"]))


# ------------------------------------------------------------------ what a program has in hand

def _turns(case):
    """Turns per position of each rotated pair, and the factor on cos and sin."""
    n = case["n_rot"]
    base, factor, trained, fast, slow = 500000.0, 8.0, 4096.0, 32.0, 1.0
    i = np.arange(n // 2, dtype=np.float64)
    if case["scaling"] == "ntk":
        base *= factor ** (n / (n - 2))
    f = base ** (-2.0 * i / n)
    if case["scaling"] == "linear":
        f = f / factor
    if case["scaling"] != "yarn":
        return f / (2 * math.pi), 1.0
    at = [n / 2 * math.log(trained / (b * 2 * math.pi)) / math.log(base) for b in (fast, slow)]
    lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), n - 1)
    ramp = np.clip((i - lo) / max(hi - lo, 0.001), 0.0, 1.0)
    return (f / factor * ramp + f * (1 - ramp)) / (2 * math.pi), 0.1 * math.log(factor) + 1.0


def _documents(case):
    """Bounds of arg documents of uneven lengths over the keys; of a whole canvas, the last 3% is padding."""
    n, used = case["arg"], case["Lk"] - (case["Lk"] * 3 // 100 if case["Lq"] == case["Lk"] else 0)
    share = 0.3 + (np.arange(1, n + 1) * 0.6180339887498949) % 1.0
    return np.concatenate([[0], np.round(np.cumsum(share) / share.sum() * used)]).astype(np.int64)


def _intervals(case):
    """Keys [begin, end) of each query; query i sits at key position i + Lk - Lq."""
    Lq, Lk, mask, arg = case["Lq"], case["Lk"], case["mask"], case["arg"]
    at = np.arange(Lq) + Lk - Lq
    begin, end = np.zeros(Lq, np.int64), np.full(Lq, Lk, np.int64)
    if mask == "documents":
        b = _documents(case)
        d = np.searchsorted(b, at, side="right") - 1
        real = d < arg
        begin = np.where(real, b[np.minimum(d, arg)], 0)
        end = np.where(real, b[np.minimum(d + 1, arg)], 0)
    elif mask == "prefix":
        end = np.maximum(arg, at + 1)
    elif mask == "blocks":
        end = np.minimum((at // arg + 1) * arg, Lk)
    elif mask == "window":
        begin, end = np.maximum(at - arg, 0), np.minimum(at + arg + 1, Lk)
    return begin, end


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = dict(case)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    if case["op"] == "rope":
        L, H, Hkv, dh = case["L"], case["H"], case["Hkv"], case["dh"]
        turns, c["mscale"] = _turns(case)
        c["turns"] = torch.from_numpy(turns).cuda()
        c["pos"] = torch.arange(L, device="cuda", dtype=torch.int32) + case["far"]
        # one f32 buffer, as the fused projections can write it
        qkv = normal(L, (H + 2 * Hkv) * dh) * 1.5
        c["ld"] = qkv.stride(0)
        c["q"], c["k"], c["v"] = qkv.split([H * dh, Hkv * dh, Hkv * dh], 1)
        c["gamma_q"], c["gamma_k"] = 0.5 + uniform(dh), 0.5 + uniform(dh)
        c["out"] = {"q": torch.empty(L, H, dh, dtype=torch.float16, device="cuda"),
                    "k": torch.empty(L, Hkv, dh, dtype=torch.float16, device="cuda")}
        if case["with_v"]:
            c["out"]["v"] = torch.empty(L, Hkv, dh, dtype=torch.float16, device="cuda")
    elif case["op"] == "attention":
        Lq, Lk, H, Hkv = case["Lq"], case["Lk"], case["H"], case["Hkv"]
        c["q"] = (normal(Lq, H, 128) * 1.5).half()
        c["k"], c["v"] = (normal(Lk, Hkv, 128) * 1.5).half(), normal(Lk, Hkv, 128).half()
        begin, end = _intervals(case)
        c["begin"], c["end"] = (torch.from_numpy(x.astype(np.int32)).cuda() for x in (begin, end))
        heads = torch.arange(1, H + 1, device="cuda", dtype=torch.float32)
        c["slopes"] = torch.exp2(-8.0 * heads / H) if case["bias"] else None
        c["out"] = torch.empty(Lq, H, 128, dtype=torch.float16, device="cuda")
    else:
        R, V = case["R"], case["V"]
        # a body of unlikely words, a few dozen likely ones, some words ruled out
        logits = normal(R, V) * 2.0
        likely = torch.randint(0, V // 40, (R, 40), generator=g, device="cuda") + torch.arange(40, device="cuda") * (V // 40)
        logits.scatter_(1, likely, 6.0 + 4.0 * normal(R, 40))
        logits[:, torch.randint(0, V, (max(1, V // 1000),), generator=g, device="cuda")] = float("-inf")
        c["logits"], c["u"] = logits, uniform(R)
        c["temperature"], c["top_k"], c["top_p"], c["min_p"] = 0.4 + uniform(R), None, None, None
        if case["limits"] in ("all", "p"):
            c["top_p"] = 0.7 + 0.3 * uniform(R)
        if case["limits"] in ("all", "k"):
            c["top_k"] = torch.randint(1, max(2, V // 20), (R,), generator=g, device="cuda", dtype=torch.int32)
        if case["limits"] == "all":
            c["min_p"] = 0.02 * uniform(R)
            c["temperature"][3::7] = 0.0  # some requests are greedy
        c["out"] = {"token": torch.empty(R, dtype=torch.int32, device="cuda"),
                    "conf": torch.empty(R, device="cuda"), "entropy": torch.empty(R, device="cuda")}
    return c


# ------------------------------------------------------------------ the plain forms

def _plain_rope(c):
    L, dh, n = c["L"], c["dh"], c["n_rot"]
    a = c["pos"].double()[:, None] * c["turns"][None]
    a = 2 * math.pi * (a - a.round())  # far positions: the angle in 64 bits
    cos, sin = (a.cos() * c["mscale"]).float()[:, None], (a.sin() * c["mscale"]).float()[:, None]

    def rotate(x, gamma):
        x = x.reshape(L, -1, dh)
        if c["qk_norm"]:
            x = x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt() * gamma
        r, rest = x[..., :n], x[..., n:]
        if c["layout"] == "norm":
            x1, x2 = r[..., 0::2], r[..., 1::2]
            r = torch.stack([x1 * cos - x2 * sin, x2 * cos + x1 * sin], -1).reshape(L, -1, n)
        else:
            x1, x2 = r[..., :n // 2], r[..., n // 2:]
            r = torch.cat([x1 * cos - x2 * sin, x2 * cos + x1 * sin], -1)
        return torch.cat([r, rest], -1).half()

    out = {"q": rotate(c["q"], c["gamma_q"]), "k": rotate(c["k"], c["gamma_k"])}
    if c["with_v"]:
        out["v"] = c["v"].reshape(L, -1, dh).half()
    return out


def _plain_attention(c):
    Lq, Lk, H, Hkv = c["Lq"], c["Lk"], c["H"], c["Hkv"]
    q = c["q"].float().transpose(0, 1).reshape(Hkv, H // Hkv, Lq, 128)
    k, v = c["k"].float().transpose(0, 1)[:, None], c["v"].float().transpose(0, 1)[:, None]
    s = (q @ k.transpose(-1, -2)) / math.sqrt(128.0)
    if c["cap"]:
        s = c["cap"] * torch.tanh(s / c["cap"])
    j = torch.arange(Lk, device="cuda")
    if c["bias"]:
        far = (torch.arange(Lq, device="cuda")[:, None] + (Lk - Lq) - j[None]).abs()
        s = s - c["slopes"].reshape(Hkv, H // Hkv, 1, 1) * far
    seen = (j[None] >= c["begin"][:, None]) & (j[None] < c["end"][:, None])
    s = torch.where(seen, s, float("-inf"))
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(top == float("-inf"), 0.0, top))
    total = p.sum(-1, keepdim=True)
    o = (p @ v) / torch.where(total == 0, 1.0, total)  # a query without keys gives zeros
    return o.reshape(H, Lq, 128).transpose(0, 1).half()


def _plain_sample(c):
    """Weights and running sums in 64 bits: a token lies next to the border of its interval."""
    V = c["V"]
    l = c["logits"].double()
    top = l.amax(-1, keepdim=True)
    greedy = (c["temperature"] <= 0)[:, None]
    w = torch.exp((l - top) / torch.where(greedy, 1.0, c["temperature"].double()[:, None]))
    order = torch.sort(c["logits"], dim=-1, descending=True, stable=True).indices
    ws = w.gather(1, order)
    rank = torch.arange(V, device="cuda")[None]
    keep = ~greedy | (rank == 0)
    if c["top_k"] is not None:
        keep = keep & (rank < c["top_k"][:, None])
    if c["min_p"] is not None:
        keep = keep & (ws >= c["min_p"].double()[:, None])
    if c["top_p"] is not None:
        upto = torch.where(keep, ws, 0.0).cumsum(-1)
        keep = keep & ((rank == 0) | (upto - ws < c["top_p"].double()[:, None] * upto[:, -1:]))
    kept = torch.zeros_like(keep).scatter(1, order, keep)
    upto = torch.where(kept, w, 0.0).cumsum(-1)
    token = (upto <= c["u"].double()[:, None] * upto[:, -1:]).sum(-1)
    token = torch.minimum(token, torch.where(kept & (w > 0), rank, 0).amax(-1))
    e = torch.exp(l - top)
    total = e.sum(-1)
    entropy = total.log() - torch.where(e > 0, e * (l - top), 0.0).sum(-1) / total
    return {"token": token.int(), "conf": (e.gather(1, token[:, None])[:, 0] / total).float(),
            "entropy": entropy.float()}


def run(c):
    if not own:
        return {"rope": _plain_rope, "attention": _plain_attention, "sample": _plain_sample}[c["op"]](c)
    from quantized_int8_gemm_q4_b200 import dllm
    out = c["out"]
    if c["op"] == "rope":
        ld, norm = c["ld"], c["qk_norm"]
        dllm.dllm_qk_rope(c["q"], ld, c["k"], ld, c["v"] if c["with_v"] else None, ld, c["L"], c["H"], c["Hkv"],
                          c["dh"], c["pos"], c["turns"], c["n_rot"],
                          dllm.DLLM_ROPE_NORM if c["layout"] == "norm" else dllm.DLLM_ROPE_NEOX, c["mscale"],
                          c["gamma_q"] if norm else None, c["gamma_k"] if norm else None, 1e-6, out["q"], out["k"],
                          out.get("v"))
    elif c["op"] == "attention":
        Lq, Lk, H, Hkv = c["Lq"], c["Lk"], c["H"], c["Hkv"]
        if "ws" not in c:  # sized once by the program that makes the calls
            c["ws_bytes"] = dllm.dllm_attention_masked_workspace_bytes(Lq, Lk, H, Hkv)
            c["ws"] = dllm.alloc_workspace(c["ws_bytes"])
        dllm.dllm_attention_masked(c["q"], H * 128, c["k"], Hkv * 128, c["v"], Hkv * 128, Lq, Lk, H, Hkv, 128,
                                   c["begin"], c["end"], None, c["cap"], c["slopes"], out, dllm.DLLM_F16, c["ws"],
                                   c["ws_bytes"])
    else:
        dllm.dllm_sample(c["logits"], c["R"], c["V"], c["V"], c["temperature"], c["top_k"], c["top_p"], c["min_p"],
                         c["u"], out["token"], out["conf"], out["entropy"])
    return out


# ------------------------------------------------------------------ work and definition

def work(case):
    if case["op"] == "rope":
        heads = case["H"] + case["Hkv"] * (2 if case["with_v"] else 1)
        n = case["L"] * heads * case["dh"]
        return {"bytes": 6 * n + 4 * case["L"] + 8 * case["n_rot"] // 2, "flops": 6 * n}
    if case["op"] == "attention":
        begin, end = _intervals(case)
        pairs = int(np.maximum(end - begin, 0).sum())
        # keys that no query sees need not be read
        marks = np.zeros(case["Lk"] + 1, np.int64)
        np.add.at(marks, begin, 1)
        np.add.at(marks, np.maximum(end, begin), -1)
        seen = int((np.cumsum(marks)[:-1] > 0).sum())
        return {"bytes": 256 * (2 * case["Lq"] * case["H"] + 2 * seen * case["Hkv"]) + 8 * case["Lq"],
                "flops": 4 * 128 * case["H"] * pairs}
    return {"bytes": 4 * case["R"] * case["V"] + 32 * case["R"], "flops": 4 * case["R"] * case["V"]}


def exact(case, seed):
    c = prepare(case, seed)
    if case["op"] == "rope":
        L, dh, n = case["L"], case["dh"], case["n_rot"]
        turns = (c["pos"].cpu().numpy().astype(np.longdouble)[:, None] * c["turns"].cpu().numpy())
        angle = torch.from_numpy((2 * math.pi * (turns - np.floor(turns)).astype(np.float64))).cuda()
        turn = torch.polar(torch.full_like(angle, float(np.float32(c["mscale"]))), angle)[:, None]
        out = {}
        for name, gamma in (("q", c["gamma_q"]), ("k", c["gamma_k"])):
            x = c[name].double().reshape(L, -1, dh)
            if case["qk_norm"]:
                x = gamma.double() * x * torch.rsqrt((x * x).sum(-1, keepdim=True) / dh + 1e-6)
            pair = (slice(0, n, 2), slice(1, n, 2)) if case["layout"] == "norm" else (slice(0, n // 2), slice(n // 2, n))
            z = torch.complex(x[..., pair[0]], x[..., pair[1]]) * turn
            y = x.clone()
            y[..., pair[0]], y[..., pair[1]] = z.real, z.imag
            out[name] = y
        if case["with_v"]:
            out["v"] = c["v"].double().reshape(L, -1, dh)
        return out
    if case["op"] == "attention":
        Lq, Lk, H, group = case["Lq"], case["Lk"], case["H"], case["H"] // case["Hkv"]
        begin, end = c["begin"].long(), c["end"].long()
        i, j = torch.arange(Lq, device="cuda") + Lk - Lq, torch.arange(Lk, device="cuda")
        hidden = (j < begin[:, None]) | (j >= end[:, None])
        out = torch.zeros(Lq, H, 128, dtype=torch.float64, device="cuda")
        for h in range(H):
            s = torch.einsum("id,jd->ij", c["q"][:, h].double(), c["k"][:, h // group].double()) / 128 ** 0.5
            if case["cap"]:
                e = torch.exp(-2 * s.abs() / case["cap"])
                s = case["cap"] * s.sign() * (1 - e) / (1 + e)
            if case["bias"]:
                s = s - c["slopes"][h].double() * (i[:, None] - j).abs()
            s = s.masked_fill(hidden, -math.inf)
            some = end > begin
            out[some, h] = torch.softmax(s[some], -1) @ c["v"][:, h // group].double()
        return out
    token, conf, entropy = [], [], []
    rows = c["logits"].cpu().numpy()
    par = {k: None if c[k] is None else c[k].cpu().numpy() for k in ("temperature", "top_k", "top_p", "min_p", "u")}
    for r, row in enumerate(rows):
        l = row.astype(np.float64) - np.float64(row.max())
        t = float(par["temperature"][r])
        w = np.exp(l / t) if t > 0 else (np.arange(len(l)) == int(np.argmax(l))).astype(np.float64)
        if t > 0:
            order = np.argsort(-row, kind="stable")
            if par["top_k"] is not None:
                order = order[:int(par["top_k"][r])]
            if par["min_p"] is not None:
                order = order[w[order] >= float(par["min_p"][r])]
            if par["top_p"] is not None:
                mass = np.cumsum(w[order])
                order = order[:1 + int(np.searchsorted(mass, float(par["top_p"][r]) * mass[-1], side="left"))]
            only = np.zeros_like(w)
            only[order] = w[order]
            w = only
        mass = np.cumsum(w)
        at = int(np.searchsorted(mass, float(par["u"][r]) * mass[-1], side="right"))
        at = min(at, int(np.flatnonzero(w > 0)[-1]))
        p = np.exp(l) / np.exp(l).sum()
        token.append(at)
        conf.append(p[at])
        entropy.append(-(p[p > 0] * np.log(p[p > 0])).sum())
    return {"token": torch.tensor(token, dtype=torch.int32), "conf": torch.tensor(conf, dtype=torch.float64),
            "entropy": torch.tensor(entropy, dtype=torch.float64)}
