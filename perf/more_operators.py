"""Cases that measure routing to experts and low-rank adapters.

Two operators, each in a plain torch form (``own = False``) and through the
library's entry points (``own = True``):

* ``route``: from router logits to experts and gates (``qmm_moe_route``):
  softmax or sigmoid scores, a bias for balance that enters the choice alone,
  groups of experts of which the best stay, the k best experts, gates
  renormalised and scaled;
* ``lora``: y = base + scale_a B_a (A_a x) for rows of many requests at once,
  each with an adapter a of its own or none (``qmm_lora``), beside a shared
  projection whose output is ``base``.

Choices are those of 64-bit scores; experts whose logit is -inf take no part.
"""
import math
import random

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
DEV = "cuda"


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decoded token, the expert layer's 256 experts, bias and scale: latency
        {"name": "route decode 1x256 f32 sigmoid", "op": "route", "dtype": "f32", "T": 1, "E": 256, "k": 8,
         "score": "sigmoid", "bias": True, "groups": 1, "top_groups": 1, "group_score": "max", "renorm": True,
         "scale": 2.5, "masked": 0.0, "pad": 0},
        # one token of each of 60 requests, experts in 8 groups of which 4 stay
        {"name": "route batch 60x256 bf16 groups", "op": "route", "dtype": "bf16", "T": 60, "E": 256, "k": 8,
         "score": "sigmoid", "bias": True, "groups": 8, "top_groups": 4, "group_score": "top2", "renorm": True,
         "scale": 2.5, "masked": 0.0, "pad": 0},
        # a prompt, softmax over few experts, an odd number of them switched off for some tokens
        {"name": "route prompt 2039x60 f16 softmax", "op": "route", "dtype": "f16", "T": 2039, "E": 60, "k": 4,
         "score": "softmax", "bias": False, "groups": 1, "top_groups": 1, "group_score": "max", "renorm": False,
         "scale": 1.0, "masked": 0.1, "pad": 4},
        # prompts of several requests, groups by their best expert
        {"name": "route prompts 8190x160 bf16 softmax groups", "op": "route", "dtype": "bf16", "T": 8190, "E": 160,
         "k": 6, "score": "softmax", "bias": False, "groups": 8, "top_groups": 3, "group_score": "max",
         "renorm": False, "scale": 16.0, "masked": 0.0, "pad": 0},
        # a large batch of prompts
        {"name": "route prompts 32003x256 f32 groups", "op": "route", "dtype": "f32", "T": 32003, "E": 256, "k": 8,
         "score": "sigmoid", "bias": True, "groups": 8, "top_groups": 4, "group_score": "top2", "renorm": True,
         "scale": 2.5, "masked": 0.0, "pad": 0},
        # the largest: many small experts
        {"name": "route prompts 65521x512 f32 softmax", "op": "route", "dtype": "f32", "T": 65521, "E": 512, "k": 10,
         "score": "softmax", "bias": False, "groups": 1, "top_groups": 1, "group_score": "max", "renorm": True,
         "scale": 1.0, "masked": 0.0, "pad": 0},
        # one decoded token beside a square projection: latency
        {"name": "lora decode 1 2048x2048 r16 f32", "op": "lora", "x": "f32", "w": "f16", "y": "f32", "K": 2048,
         "N": 2048, "rank": 16, "mixed": False, "lengths": "one", "T": 1, "adapters": 4, "none": 0.0, "base": True,
         "pad": 0},
        # one token of each of 64 requests, a sixth of them without an adapter, ranks of 16 to 64
        {"name": "lora batch 64 5632x2048 r64 f32", "op": "lora", "x": "f32", "w": "bf16", "y": "f32", "K": 2048,
         "N": 5632, "rank": 64, "mixed": True, "lengths": "one", "T": 64, "adapters": 40, "none": 0.16, "base": True,
         "pad": 0},
        # a batch at the large dense model's width
        {"name": "lora batch 48 8192x8192 r16 bf16", "op": "lora", "x": "bf16", "w": "bf16", "y": "bf16", "K": 8192,
         "N": 8192, "rank": 16, "mixed": False, "lengths": "one", "T": 48, "adapters": 32, "none": 0.0, "base": True,
         "pad": 0},
        # decoded tokens and prompt chunks in one step, an odd rank, odd rows of the projection
        {"name": "lora mix 1013 2051x6144 r24 f16", "op": "lora", "x": "f16", "w": "f16", "y": "f16", "K": 6144,
         "N": 2051, "rank": 24, "mixed": True, "lengths": "mix", "T": 1013, "adapters": 24, "none": 0.1,
         "base": True, "pad": 32},
        # a prompt chunk, the adapter's part alone
        {"name": "lora prompt 2039 8192x5632 r32 f32", "op": "lora", "x": "f32", "w": "f16", "y": "f32", "K": 5632,
         "N": 8192, "rank": 32, "mixed": False, "lengths": "prompt", "T": 2039, "adapters": 4, "none": 0.0,
         "base": False, "pad": 0},
        # the largest: prompts of several requests at the large dense model's width
        {"name": "lora prompts 4093 28672x8192 r64 bf16", "op": "lora", "x": "bf16", "w": "bf16", "y": "bf16",
         "K": 8192, "N": 28672, "rank": 64, "mixed": False, "lengths": "prompt", "T": 4093, "adapters": 8,
         "none": 0.0, "base": True, "pad": 0},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    if rng.random() < 0.45:
        groups = rng.choice([1, 1, 2, 4, 8, 16])
        E = rng.choice([8, 16, 60, 64, 72, 128, 160, 256, 256, 384, 512, rng.randrange(2, 640)])
        E = max(2 * groups, E // groups * groups)
        top = rng.randrange(1, groups + 1)
        return {"op": "route", "dtype": rng.choice(["f32", "f16", "bf16"]), "T": _log(rng, 1, 65521 * 512 // max(E, 512)),
                "E": E, "k": rng.randrange(1, min(16, E // groups * top) + 1), "score": rng.choice(["sigmoid", "softmax"]),
                "bias": rng.random() < 0.5, "groups": groups, "top_groups": top,
                "group_score": rng.choice(["max", "top2"]), "renorm": rng.random() < 0.6,
                "scale": rng.choice([1.0, 2.5, 16.0]), "masked": rng.choice([0.0, 0.0, 0.1, 0.9]),
                "pad": rng.choice([0, 0, 1, 8])}
    x = rng.choice(["f32", "f32", "f16", "bf16"])
    w = {"f32": rng.choice(["f32", "f16", "bf16"]), "f16": "f16", "bf16": "bf16"}[x]
    K = rng.choice([1024, 2048, 4096, 5632, 6144, 8192, 32 * rng.randrange(1, 400)])
    N = rng.choice([1024, 2048, 2560, 5632, 6144, 8192, 28672, rng.randrange(1, 12000)])
    rank = rng.choice([8, 16, 16, 32, 64, 128, rng.randrange(1, 100)])
    lengths = rng.choice(["one", "mix", "prompt"])
    most = 4093 * (8192 + 2 * 28672) * 2 // (2 * (K * SIZE[x] + 2 * N * SIZE[x]))  # bytes, half the largest's
    most = min(most, 4093 * 64 * (8192 + 28672) // (4 * rank * (K + N)))  # products, a quarter of the largest's
    T = _log(rng, 1, max(1, min(200 if lengths == "one" else 6000, most)))
    return {"op": "lora", "x": x, "w": w, "y": x, "K": K, "N": N, "rank": rank, "mixed": rng.random() < 0.4,
            "lengths": lengths, "T": T, "adapters": rng.randrange(1, 49), "none": rng.choice([0.0, 0.0, 0.2]),
            "base": rng.random() < 0.7, "pad": rng.choice([0, 0, 32])}


def _plan(case):
    """Segments [(first row, last + 1, adapter or -1)] and the adapters' ranks; of the case alone."""
    r = random.Random("%d %d %d %s" % (case["T"], case["adapters"], case["rank"], case["lengths"]))
    T, lens = case["T"], []
    if case["lengths"] == "one":
        lens = [1] * T
    elif case["lengths"] == "mix":  # decoded tokens first, then a few chunks; a request without rows among them
        lens = [1] * min(T // 2, 40) + [0]
        while sum(lens) < T:
            lens.append(min(T - sum(lens), r.randrange(1, max(2, T // 2))))
    else:
        cuts = sorted(r.randrange(0, T + 1) for _ in range(min(7, T // 64)))
        lens = [b - a for a, b in zip([0] + cuts, cuts + [T])]
    at, segs = 0, []
    for n in lens:
        segs.append((at, at + n, -1 if r.random() < case["none"] else r.randrange(case["adapters"])))
        at += n
    ranks = [max(1, case["rank"] // r.choice([1, 2, 4])) if case["mixed"] else case["rank"]
             for _ in range(case["adapters"])]
    return segs, ranks


def work(case):
    if case["op"] == "route":
        T, E, k = case["T"], case["E"], case["k"]
        return {"bytes": T * E * SIZE[case["dtype"]] + T * k * 8 + (E * 4 if case["bias"] else 0), "flops": 6 * T * E}
    segs, ranks = _plan(case)
    K, N, w = case["K"], case["N"], SIZE[case["w"]]
    rows = sum(b - a for a, b, i in segs if i >= 0)
    used = {i for a, b, i in segs if i >= 0 and b > a}
    n = rows * K * SIZE[case["x"]] + case["T"] * N * SIZE[case["y"]] * (2 if case["base"] else 1)
    return {"bytes": n + sum(ranks[i] * (K + N) * w for i in used),
            "flops": sum(2 * (b - a) * ranks[i] * (K + N) for a, b, i in segs if i >= 0)}


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device=DEV)

    st = {"case": case}
    if case["op"] == "route":
        T, E, k = case["T"], case["E"], case["k"]
        # trained routers prefer some experts
        logits = randn(T, E) + 0.5 * randn(E)
        if case["masked"]:
            logits[torch.rand(T, E, generator=gen, device=DEV) < case["masked"]] = -math.inf
        buf = torch.full((T, E + case["pad"]), 100.0, device=DEV, dtype=TYPES[case["dtype"]])
        st["logits"] = buf[:, :E]
        st["logits"].copy_(logits)
        st["bias"] = 0.1 * randn(E) if case["bias"] else None
        st["ids"] = torch.zeros(T, k, dtype=torch.int32, device=DEV)
        st["gates"] = torch.zeros(T, k, device=DEV)
    else:
        T, K, N, rank, n = (case[i] for i in ("T", "K", "N", "rank", "adapters"))
        segs, ranks = _plan(case)
        x = randn(T, K)
        x = torch.where(torch.rand(T, K, generator=gen, device=DEV) < 0.01, 20 * x, x)  # outliers, as projections give
        buf = torch.zeros(T, K + case["pad"], device=DEV, dtype=TYPES[case["x"]])
        st["x"] = buf[:, :K]
        st["x"].copy_(x)
        wt = TYPES[case["w"]]
        st["a"] = torch.empty(n, rank, K, device=DEV, dtype=wt)
        st["b"] = torch.empty(n, N, rank, device=DEV, dtype=wt)
        for i in range(n):  # what lies behind a smaller adapter's rank is an older adapter's
            st["a"][i] = randn(rank, K) * K ** -0.5
            st["b"][i] = randn(N, rank) * 0.05
        st["scales"] = 0.5 + 2 * torch.rand(n, generator=gen, device=DEV)
        st["base"] = randn(T, N).to(TYPES[case["y"]]) if case["base"] else None
        st["y"] = torch.empty(T, N, device=DEV, dtype=TYPES[case["y"]])
        st["ranks"] = torch.tensor(ranks, dtype=torch.int32, device=DEV)
        st["start"] = torch.tensor([s[0] for s in segs] + [T], dtype=torch.int32, device=DEV)
        st["adapter"] = torch.tensor([s[2] for s in segs], dtype=torch.int32, device=DEV)
        st["plan"] = segs, ranks  # the scheduler's, on the host
    if own:
        _handles(st)
    return st


def _handles(st):
    """The descriptors that a program makes once for its buffers."""
    from block_quantized_int4_gb300 import qmm
    case = st["case"]
    if case["op"] == "route":
        st["handle"] = qmm.moe_route_op(
            st["logits"], st["ids"], st["gates"], bias=st["bias"],
            score=qmm.ROUTE_SOFTMAX if case["score"] == "softmax" else qmm.ROUTE_SIGMOID,
            n_groups=case["groups"], top_groups=case["top_groups"],
            group_score=qmm.ROUTE_GROUP_MAX if case["group_score"] == "max" else qmm.ROUTE_GROUP_TOP2,
            renormalize=case["renorm"], scale=case["scale"])
    else:
        one = case["lengths"] == "one"
        st["handle"] = qmm.lora_op(st["x"], st["a"], st["b"], st["y"], st["adapter"], base=st["base"],
                                   seg_start=None if one else st["start"], ranks=st["ranks"], scales=st["scales"])


# ------------------------------------------------------------------ the operators
def run(st):
    op = st["case"]["op"]
    if own:
        from block_quantized_int4_gb300 import qmm
        if op == "route":
            qmm.qmm_moe_route(st["handle"])
            return st["ids"], st["gates"]
        qmm.qmm_lora(st["handle"])
        return st["y"]
    return _plain_route(st) if op == "route" else _plain_lora(st)


def _plain_route(st):
    case = st["case"]
    T, E, G = case["T"], case["E"], case["groups"]
    l = st["logits"].double()  # scores next to one another change places in 32 bits
    live = l > -math.inf
    if case["score"] == "softmax":
        e = torch.exp(l - l.amax(-1, keepdim=True).clamp_min(-1e300))
        s = e / e.sum(-1, keepdim=True).clamp_min(1e-300)
    else:
        s = 1 / (1 + torch.exp(-l))
    s = torch.where(live, s, 0.0)
    c = l if st["bias"] is None else s + st["bias"].double()
    c = torch.where(live, c, -1e300)
    if G > 1:
        g = c if case["group_score"] == "max" or st["bias"] is not None else torch.where(live, s, -1e300)
        g = torch.sort(g.view(T, G, E // G), dim=-1, descending=True).values
        if case["group_score"] == "max":
            g = g[..., 0]
        else:  # experts that take no part add nothing
            g = g[..., 0] + torch.where(g[..., 1] > -1e299, g[..., 1], 0.0)
        best = torch.sort(g, dim=-1, descending=True, stable=True).indices[:, :case["top_groups"]]
        kept = torch.zeros(T, G, dtype=torch.bool, device=DEV).scatter_(1, best, True)
        c = torch.where(kept[..., None], c.view(T, G, E // G), -math.inf).view(T, E)
    ids = torch.sort(c, dim=-1, descending=True, stable=True).indices[:, :case["k"]]
    gates = s.gather(1, ids)
    if case["renorm"]:
        gates = gates / gates.sum(-1, keepdim=True).clamp_min(1e-300)
    return ids.to(torch.int32), (gates * case["scale"]).float()


def _plain_lora(st):
    case = st["case"]
    segs, ranks = st["plan"]
    x, a, b = st["x"], st["a"], st["b"]
    y = st["base"].to(torch.float32, copy=True) if case["base"] else torch.zeros(st["y"].shape, device=DEV)
    if case["lengths"] == "one" and case["T"] > 1:  # a row each: gathered adapters, batched products
        at = st["adapter"].long()
        use = at.clamp_min(0)
        h = torch.bmm(a[use].float(), x.float()[..., None])
        h = torch.where(torch.arange(case["rank"], device=DEV) < st["ranks"][use][:, None], h[..., 0], 0.0)
        d = torch.bmm(b[use].float(), h[..., None])[..., 0] * st["scales"][use][:, None]
        return (y + torch.where((at >= 0)[:, None], d, 0.0)).to(st["y"].dtype)
    for first, last, i in segs:
        if i >= 0 and last > first:
            r = ranks[i]
            h = x[first:last].float() @ a[i, :r].float().T
            y[first:last] = y[first:last] + (h @ b[i, :, :r].float().T) * st["scales"][i]
    return y.to(st["y"].dtype)


# ------------------------------------------------------------------ 64 bits, from the definitions
def _exact_route(st):
    """Ranks by counting: the place of an expert is the number of those before it."""
    case = st["case"]
    T, E, G, k = case["T"], case["E"], case["groups"], case["k"]
    ids = torch.empty(T, k, dtype=torch.int32, device=DEV)
    gates = torch.empty(T, k, dtype=torch.float64, device=DEV)

    def place(v):  # [n][m] -> how many of a row come before each: larger ones, and equal ones further left
        m = v.shape[1]
        left = torch.arange(m, device=DEV)[None, :] < torch.arange(m, device=DEV)[:, None]
        a, b = v[:, None, :], v[:, :, None]
        return ((a > b) | ((a == b) & left)).sum(-1)

    step = max(1, (1 << 26) // (E * E))
    for t in range(0, T, step):
        l = st["logits"][t:t + step].double()
        n = l.shape[0]
        out = torch.isneginf(l)
        if case["score"] == "sigmoid":
            p = torch.where(l >= 0, 1 / (1 + torch.exp(-l.abs())), torch.exp(-l.abs()) / (1 + torch.exp(-l.abs())))
        else:
            p = torch.exp(l - torch.logsumexp(l, -1, keepdim=True))
        p = torch.where(out, torch.zeros_like(p), p)
        c = l if st["bias"] is None else p + st["bias"].double()
        allowed = torch.ones(n, E, dtype=torch.bool, device=DEV)
        if G > 1:
            v = c if case["group_score"] == "max" or st["bias"] is not None else p
            v = v.masked_fill(out, -math.inf).reshape(n, G, -1)
            first = v.max(-1)
            score = first.values
            if case["group_score"] == "top2":
                second = v.scatter(-1, first.indices[..., None], -math.inf).amax(-1)
                score = score + second.masked_fill(second == -math.inf, 0.0)
            allowed = (place(score) < case["top_groups"]).repeat_interleave(E // G, 1)
        order = c.masked_fill(out, -1e200).masked_fill(~allowed, -math.inf)
        rank = place(order)
        row, expert = (rank < k).nonzero(as_tuple=True)
        ids[t + row, rank[row, expert]] = expert.to(torch.int32)
        gates[t + row, rank[row, expert]] = p[row, expert]
    total = gates.sum(-1, keepdim=True) if case["renorm"] else torch.ones(T, 1, dtype=torch.float64, device=DEV)
    return ids, torch.where(total > 0, gates / total, torch.zeros_like(gates)) * case["scale"]


def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "route":
        return _exact_route(st)
    y = torch.zeros(case["T"], case["N"], dtype=torch.float64, device=DEV)
    segs, ranks = _plan(case)
    for first, last, i in segs:
        if i >= 0:
            low = torch.einsum("tk,rk->tr", st["x"][first:last].double(), st["a"][i, :ranks[i]].double())
            y[first:last] = torch.einsum("tr,nr->tn", low * st["scales"][i].double(), st["b"][i, :, :ranks[i]].double())
    return y if st["base"] is None else y.add_(st["base"])
