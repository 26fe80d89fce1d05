"""Cases that measure the attention operators over a 4-bit paged cache.

Three operators, each in a plain torch form (``own = False``) and through the
library's entry points (``own = True``):

* ``rope``: RMSNorm of each head and rotary positions in one pass
  (``qmm_rope_heads``);
* ``append``: rotation of keys (and queries), Q4_0 of keys and values, and
  their write into a paged cache (``qmm_kv_append_q4_0``), then the values
  that the written tokens stand for (``qmm_kv_read_q4_0``);
* ``attn``: attention over the paged Q4_0 cache (``qmm_attn_q4_0``).

Cache layout (the library's): a record holds 32 consecutive tokens of one
head, D = 32 * NB values each: K codes [NB][512 bytes], V codes [NB][512
bytes], K scales [NB][64 bytes], V scales [NB][64 bytes].  Token t = 8i + g
(i < 4, g < 8), or t = 8j + 2c + h (j < 4, c < 4, h < 2):

* K codes of block b: the block's 16 Q4_0 bytes (byte m holds value m in its
  low and m + 16 in its high nibble) are four 4-byte words c = 0..3; word c
  of token 8i + g is word (g * 4 + c) * 4 + i of the 512 bytes;
* V codes of block b: the 16-bit unit g of a token holds values g, g + 8,
  g + 16, g + 24 in its nibbles 0..3; unit g of token 8j + 2c + h is unit
  ((g * 4 + c) * 4 + j) * 2 + h of the 512 bytes;
* scales of block b: fp16, that of token 8j + 2c + h at (c * 4 + j) * 2 + h.

The cache is [page][kv head][page_size / 32][record].
"""
import math
import random

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-5
DEV = "cuda"


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decoded token, 32 query heads of 64: latency
        {"name": "rope decode 1x32x64 f32", "op": "rope", "dtype": "f32", "T": 1, "H": 32, "D": 64, "n_rot": 64,
         "pairs": False, "norm": True, "far": 2048, "factor": 1.0},
        # a prompt's queries, half of each head rotated, far positions of a scaled context
        {"name": "rope prompt 4093x64x128 bf16", "op": "rope", "dtype": "bf16", "T": 4093, "H": 64, "D": 128,
         "n_rot": 64, "pairs": True, "norm": True, "far": 131072, "factor": 8.0},
        # one decoded token: 32 query and 4 key/value heads of 64
        {"name": "append decode 1 f32", "op": "append", "dtype": "f32", "T": 1, "Hq": 32, "Hkv": 4, "D": 64,
         "n_rot": 64, "pairs": False, "norm": False, "page": 64, "far": 2048, "factor": 1.0},
        # one token of each of 16 sequences, heads normalised
        {"name": "append batch 16 f32", "op": "append", "dtype": "f32", "T": 16, "Hq": 64, "Hkv": 8, "D": 128,
         "n_rot": 128, "pairs": False, "norm": True, "page": 64, "far": 32768, "factor": 4.0},
        # a prompt chunk
        {"name": "append prompt 2039 bf16", "op": "append", "dtype": "bf16", "T": 2039, "Hq": 64, "Hkv": 8, "D": 128,
         "n_rot": 128, "pairs": False, "norm": False, "page": 64, "far": 8192, "factor": 1.0},
        # a short context, one token: latency
        {"name": "attn 1x1 ctx 301 f32", "op": "attn", "dtype": "f32", "B": 1, "n_q": 1, "Hq": 32, "Hkv": 4, "D": 64,
         "kv": 301, "ragged": False, "causal": True, "window": 0, "page": 64},
        # one sequence of a long context
        {"name": "attn 1x1 ctx 131000 f32", "op": "attn", "dtype": "f32", "B": 1, "n_q": 1, "Hq": 64, "Hkv": 8,
         "D": 128, "kv": 131000, "ragged": False, "causal": True, "window": 0, "page": 64},
        # a batch of sequences of very different lengths
        {"name": "attn 16x1 ragged 32000 bf16", "op": "attn", "dtype": "bf16", "B": 16, "n_q": 1, "Hq": 64, "Hkv": 8,
         "D": 128, "kv": 32000, "ragged": True, "causal": True, "window": 0, "page": 64},
        # five drafted tokens a sequence to verify
        {"name": "attn 4x5 ragged 4001 f32", "op": "attn", "dtype": "f32", "B": 4, "n_q": 5, "Hq": 32, "Hkv": 4,
         "D": 64, "kv": 4001, "ragged": True, "causal": True, "window": 0, "page": 32},
        # a sliding window, three query heads a key head, head size 96
        {"name": "attn 8x1 window 1000 f16", "op": "attn", "dtype": "f16", "B": 8, "n_q": 1, "Hq": 24, "Hkv": 8,
         "D": 96, "kv": 16000, "ragged": True, "causal": True, "window": 1000, "page": 128},
        # a prompt's chunk over what came before it
        {"name": "attn 1x509 ctx 8190 bf16", "op": "attn", "dtype": "bf16", "B": 1, "n_q": 509, "Hq": 64, "Hkv": 8,
         "D": 128, "kv": 8190, "ragged": False, "causal": True, "window": 0, "page": 64},
        # a chunk in the library's own type
        {"name": "attn 2x128 ctx 2048 f32", "op": "attn", "dtype": "f32", "B": 2, "n_q": 128, "Hq": 32, "Hkv": 4,
         "D": 64, "kv": 2048, "ragged": True, "causal": True, "window": 0, "page": 64},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["rope", "append", "attn", "attn"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    D = rng.choice([32, 64, 96, 128, 128, 160, 256])
    if op == "attn":
        B, Hkv = _log(rng, 1, 32), rng.choice([1, 2, 4, 8])
        Hq = Hkv * rng.choice([1, 2, 3, 4, 7, 8, 16])
        n_q = 1 if rng.random() < 0.5 else _log(rng, 2, 512)
        most_kv = 131000 * 8 * 128 // (B * Hkv * D)  # cached bytes as in the long listed context
        most_kv = min(most_kv, 509 * 64 * 128 * 7900 // (B * n_q * Hq * D))  # products as in the listed chunk
        kv = _log(rng, 1, max(1, min(131000, most_kv)))
        return {"op": op, "dtype": dtype, "B": B, "n_q": n_q, "Hq": Hq, "Hkv": Hkv, "D": D, "kv": kv,
                "ragged": rng.random() < 0.7, "causal": rng.random() < 0.8,
                "window": _log(rng, 1, 4000) if rng.random() < 0.25 else 0, "page": rng.choice([32, 64, 128, 256])}
    n_rot = rng.choice([D, D, D // 2, rng.randrange(2, D, 2)])
    case = {"op": op, "dtype": dtype, "D": D, "n_rot": n_rot, "pairs": rng.random() < 0.5,
            "norm": rng.random() < 0.5, "far": _log(rng, 64, 131072), "factor": rng.choice([1.0, 1.0, 4.0, 8.0])}
    if op == "rope":
        H = rng.randrange(1, 65)
        return {**case, "H": H, "T": _log(rng, 1, min(4096, 4093 * 64 * 128 // (2 * H * D)))}
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 3, 4, 7, 8])
    return {**case, "Hq": Hq, "Hkv": Hkv, "page": rng.choice([32, 64, 128, 256]),
            "T": _log(rng, 1, min(4096, 2039 * 80 * 128 // (2 * (Hq + 2 * Hkv) * D)))}


def _lengths(case):
    """Cached tokens of each sequence (the call's own tokens among them); of the case alone."""
    B, kv = case["B"], case["kv"]
    if not case["ragged"]:
        return [kv] * B
    r = random.Random(17 * kv + B)
    return [kv if b == B // 2 else max(1, round(kv * r.random() ** 1.5)) for b in range(B)]


def _visible(case, L):
    """(first, last + 1) key of each query of a sequence of L cached tokens."""
    n, spans = case["n_q"], []
    for i in range(n):
        at = L - n + i
        hi = at + 1 if case["causal"] else L
        lo = at - case["window"] + 1 if case["window"] else 0
        spans.append((max(0, lo), max(0, min(L, hi))))
    return spans


def work(case):
    size = {"f32": 4, "f16": 2, "bf16": 2}[case["dtype"]]
    D = case["D"]
    if case["op"] == "rope":
        n = case["T"] * case["H"] * D
        return {"bytes": 2 * n * size + case["T"] * case["n_rot"] * 4, "flops": 8 * n}
    if case["op"] == "append":
        T, q, kv = case["T"], case["T"] * case["Hq"] * D, case["T"] * case["Hkv"] * D
        # q, k, v and table rows in; q and the cached bytes out; those bytes in again and their values out
        return {"bytes": (2 * q + 2 * kv) * size + T * case["n_rot"] * 4 + 2 * 2 * kv * 0.5625 + 2 * kv * 4,
                "flops": 8 * q + 24 * kv}
    keys = pairs = 0
    for L in _lengths(case):
        spans = [s for s in _visible(case, L) if s[1] > s[0]]
        if spans:
            keys += max(s[1] for s in spans) - min(s[0] for s in spans)
            pairs += sum(s[1] - s[0] for s in spans)
    rows = case["B"] * case["n_q"] * case["Hq"]
    return {"bytes": keys * case["Hkv"] * D * 2 * 0.5625 + 2 * rows * D * size, "flops": 4 * pairs * case["Hq"] * D}


# ------------------------------------------------------------------ inputs
def _pack(codes, scales, value):
    """Codes 0..15 [..., 32 tokens, D] and fp16 scales [..., 32, NB] as a record's (code bytes, scale bytes)."""
    lead, NB = codes.shape[:-2], codes.shape[-1] // 32
    x = codes.to(torch.int32).unflatten(-1, (NB, 32))
    if value:
        x = x.unflatten(-1, (4, 8))  # (n, g): value 8n + g of the block
        unit = x[..., 0, :] | x[..., 1, :] << 4 | x[..., 2, :] << 8 | x[..., 3, :] << 12  # [..., t, NB, g]
        unit = unit.unflatten(-3, (4, 4, 2))  # [..., j, c, h, NB, g]
        n = len(lead)
        unit = unit.permute(*range(n), n + 3, n + 4, n + 1, n, n + 2)  # [..., NB, g, c, j, h]
        raw = torch.where(unit > 32767, unit - 65536, unit).to(torch.int16).contiguous().view(torch.uint8)
    else:
        byte = (x[..., :16] | x[..., 16:] << 4).to(torch.uint8)  # [..., t, NB, 16]
        byte = byte.unflatten(-1, (4, 4)).unflatten(-4, (4, 8))  # [..., i, g, NB, c, 4]
        n = len(lead)
        raw = byte.permute(*range(n), n + 2, n + 1, n + 3, n, n + 4).contiguous()  # [..., NB, g, c, i, 4]
    d = scales.unflatten(-2, (4, 4, 2))  # [..., j, c, h, NB]
    n = len(lead)
    d = d.permute(*range(n), n + 3, n + 1, n, n + 2).contiguous().view(torch.uint8)
    return raw.reshape(*lead, NB * 512), d.reshape(*lead, NB * 64)


def _q4_0(y):
    """Q4_0 of fp32 values [..., D]: codes 0..15 and fp16 scales, IEEE fp32 division, ties away from zero."""
    b = y.unflatten(-1, (-1, 32))
    d = b.abs().amax(-1) / torch.tensor(7.0, device=y.device)
    r = b / torch.where(d > 0, d, 1.0)[..., None]
    q = (torch.trunc(r) + torch.sign(r) * (torch.abs(r - torch.trunc(r)) >= 0.5)).clamp(-8, 7)
    return (q.to(torch.int32) + 8).flatten(-2), d.to(torch.float16)


def _frequencies(case):
    """Turns of each rotated pair in radians a position, and the magnitude of the rotation, in 64 bits: base 10000;
    with a factor, slow pairs are slowed by it and fast ones are kept, with a ramp between (the YaRN method)."""
    n, factor, base, orig = case["n_rot"], case["factor"], 10000.0, 4096
    f = [base ** (-2.0 * i / n) for i in range(n // 2)]
    if factor == 1.0:
        return f, 1.0
    place = lambda turns: n * math.log(orig / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
    lo, hi = max(0.0, math.floor(place(32.0))), min(n / 2 - 1.0, math.ceil(place(1.0)))
    ramp = [min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001))) for i in range(n // 2)]
    return [v * (1 - r) + v / factor * r for v, r in zip(f, ramp)], 0.1 * math.log(factor) + 1.0


def _table(case):
    """cos and sin of every position below `far`, [far][n_rot / 2][2], rounded once from 64 bits."""
    f, m = _frequencies(case)
    a = torch.arange(case["far"], device=DEV, dtype=torch.float64)[:, None] * torch.tensor(f, device=DEV, dtype=torch.float64)
    return torch.stack([m * torch.cos(a), m * torch.sin(a)], -1).float()


def _activations(shape, gen, dtype):
    """Normal values, one in a hundred of them twenty times as large: what a projection's output looks like."""
    x = torch.randn(shape, generator=gen, device=DEV)
    return torch.where(torch.rand(shape, generator=gen, device=DEV) < 0.01, 20 * x, x).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    dtype, D = TYPES[case["dtype"]], case["D"]
    st = {"case": case}
    if case["op"] != "attn":
        T = case["T"]
        st["table"] = _table(case)
        st["pos"] = torch.randint(0, case["far"], (T,), generator=gen, device=DEV, dtype=torch.int32)
        st["k_norm"] = 1 + 0.1 * torch.randn(D, generator=gen, device=DEV) if case["norm"] else None
    if case["op"] == "rope":
        st["x"] = _activations((T, case["H"], D), gen, dtype)
        st["y"] = torch.empty_like(st["x"])
    elif case["op"] == "append":
        Hq, Hkv, page = case["Hq"], case["Hkv"], case["page"]
        qkv = _activations((T, Hq + 2 * Hkv, D), gen, dtype)  # the fused projection's output
        st["q"], st["k"], st["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        st["q_out"] = torch.empty(T, Hq, D, device=DEV, dtype=dtype)
        st["q_norm"] = 1 + 0.1 * torch.randn(D, generator=gen, device=DEV) if case["norm"] else None
        n_pages = -(-T // page) + 3
        pages = torch.randperm(n_pages, generator=gen, device=DEV)
        if T <= 64:  # one token of each of T sequences: anywhere in the cache
            st["slots"] = torch.randperm(n_pages * page, generator=gen, device=DEV)[:T].contiguous()
        else:  # a prompt that starts inside a page
            at = torch.arange(T, device=DEV) + page // 3
            st["slots"] = pages[at // page] * page + at % page
        st["cache"] = torch.zeros(n_pages, Hkv, page // 32, D * 36, dtype=torch.uint8, device=DEV)
        st["k_read"] = torch.empty(T, Hkv, D, device=DEV)
        st["v_read"] = torch.empty(T, Hkv, D, device=DEV)
    else:
        B, n, Hq, Hkv, page = (case[k] for k in ("B", "n_q", "Hq", "Hkv", "page"))
        lengths = _lengths(case)
        each = -(-case["kv"] // page)
        n_pages = sum(-(-L // page) for L in lengths) + 2
        st["q"] = torch.randn(B * n, Hq, D, generator=gen, device=DEV).to(dtype)
        st["out"] = torch.empty_like(st["q"])
        st["cache"] = torch.empty(n_pages, Hkv, page // 32, D * 36, dtype=torch.uint8, device=DEV)
        step = max(1, (1 << 27) // (Hkv * page * D))
        for p in range(0, n_pages, step):
            shape = (min(step, n_pages - p), Hkv, page // 32, 32, D)
            parts = [_pack(*_q4_0(torch.randn(shape, generator=gen, device=DEV)), value) for value in (False, True)]
            st["cache"][p:p + step] = torch.cat([parts[0][0], parts[1][0], parts[0][1], parts[1][1]], -1)
        free = torch.randperm(n_pages, generator=gen, device=DEV).to(torch.int32)
        st["pages"] = torch.full((B, each), -1, dtype=torch.int32, device=DEV)  # unused entries are no pages
        at = 0
        for b, L in enumerate(lengths):
            k = -(-L // page)
            st["pages"][b, :k] = free[at:at + k]
            at += k
        st["kv_len"] = torch.tensor(lengths, dtype=torch.int32, device=DEV)
        st["scale"] = D ** -0.5
    if own:
        _handles(st)
    return st


def _handles(st):
    """The descriptors that a program makes once for its buffers."""
    from block_quantized_int4_gb300 import qmm
    case = st["case"]
    if case["op"] != "attn":
        rope = qmm.rope(st["table"], pairs=case["pairs"])
    if case["op"] == "rope":
        st["rope_op"] = qmm.rope_op(st["x"], st["y"], st["pos"], rope, norm_w=st["k_norm"], norm_eps=EPS)
    elif case["op"] == "append":
        cache = qmm.kv_cache(st["cache"], case["page"])
        st["append_op"] = qmm.kv_append_op(cache, st["k"], st["v"], st["slots"], pos=st["pos"], rope=rope, q=st["q"],
                                           q_out=st["q_out"], k_norm=st["k_norm"], q_norm=st["q_norm"], norm_eps=EPS)
        st["read_op"] = qmm.kv_read_op(cache, st["slots"], st["k_read"], st["v_read"])
    else:
        cache = qmm.kv_cache(st["cache"], case["page"])
        st["attn_op"] = qmm.attn_op(cache, st["q"], st["pages"], st["kv_len"], st["out"], max_kv=case["kv"],
                                    max_q=case["n_q"], scale=st["scale"], causal=case["causal"],
                                    window=case["window"])


# ------------------------------------------------------------------ the operators
def run(st):
    op = st["case"]["op"]
    if own:
        from block_quantized_int4_gb300 import qmm
        if op == "rope":
            qmm.qmm_rope_heads(st["rope_op"])
            return st["y"]
        if op == "append":
            qmm.qmm_kv_append_q4_0(st["append_op"])
            qmm.qmm_kv_read_q4_0(st["read_op"])
            return st["q_out"], st["k_read"], st["v_read"]
        qmm.qmm_attn_q4_0(st["attn_op"])
        return st["out"]
    return {"rope": _plain_rope, "append": _plain_append, "attn": _plain_attn}[op](st)


def _rotate(x, gamma, table, pos, n_rot, pairs):
    """Norm and rotation of x [T][H][D], in x's precision."""
    if gamma is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * gamma.to(x.dtype)
    cs = table[pos.long()].to(x.dtype)[:, None]  # [T][1][n_rot / 2][2]
    c, s = cs[..., 0], cs[..., 1]
    rot, rest = x[..., :n_rot], x[..., n_rot:]
    if pairs:
        a, b = rot[..., 0::2], rot[..., 1::2]
        rot = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    else:
        a, b = rot[..., :n_rot // 2], rot[..., n_rot // 2:]
        rot = torch.cat([a * c - b * s, b * c + a * s], -1)
    return torch.cat([rot, rest], -1)


def _plain_rope(st):
    case = st["case"]
    y = _rotate(st["x"].float(), st["k_norm"], st["table"], st["pos"], case["n_rot"], case["pairs"])
    return y.to(st["x"].dtype)


def _scatter(cache, slots, codes, scales, value, NB):
    """Writes tokens' codes [T][H][D] and scales [T][H][NB] into the cache."""
    Hkv, groups, rec = cache.shape[1:]
    T = slots.shape[0]
    page, at = slots // (groups * 32), slots % (groups * 32)
    base = (page[:, None] * Hkv + torch.arange(Hkv, device=DEV)) * groups + (at // 32)[:, None]
    base = base * rec  # [T][H]: the record's first byte
    t = at % 32
    j, c, h = t // 8, t // 2 % 4, t % 2
    blk, unit = torch.arange(NB, device=DEV), torch.arange(8, device=DEV)
    x = codes.unflatten(-1, (NB, 32))
    flat = cache.view(-1)
    if value:
        x = x.unflatten(-1, (4, 8))
        u = torch.stack([x[..., 0, :] | x[..., 1, :] << 4, x[..., 2, :] | x[..., 3, :] << 4], -1).to(torch.uint8)
        where = ((unit * 4 + c[:, None]) * 4 + j[:, None]) * 2 + h[:, None]  # [T][8]
        where = (NB * 512 + blk[:, None] * 512 + where[:, None, :] * 2)[..., None] + torch.arange(2, device=DEV)
    else:
        u = (x[..., :16] | x[..., 16:] << 4).to(torch.uint8)
        m = torch.arange(16, device=DEV)
        where = (((t % 8)[:, None] * 4 + m // 4) * 4 + (t // 8)[:, None]) * 4 + m % 4  # [T][16]
        where = blk[:, None] * 512 + where[:, None, :]
    flat[base.view(T, Hkv, *[1] * (where.dim() - 1)) + where[:, None]] = u
    d = scales.contiguous().view(torch.uint8).unflatten(-1, (NB, 2))
    where = NB * (1088 if value else 1024) + blk[:, None] * 64 + (((c * 4 + j) * 2 + h) * 2)[:, None, None] + torch.arange(2, device=DEV)
    flat[base[..., None, None] + where[:, None]] = d


def _values(cache, D):
    """Every token's K and V values, fp32 [pages][H][page_size][D] each."""
    NB = D // 32
    lead = cache.shape[:-1]
    n = len(lead)
    k, v, kd, vd = cache.split([NB * 512, NB * 512, NB * 64, NB * 64], -1)
    k = k.reshape(*lead, NB, 8, 4, 4, 4).permute(*range(n), n + 3, n + 1, n, n + 2, n + 4)  # [..., i, g, NB, c, 4]
    k = k.reshape(*lead, 32, NB, 16)
    k = torch.cat([k & 15, k >> 4], -1)
    v = v.reshape(*lead, NB, 8, 4, 4, 2, 2).permute(*range(n), n + 3, n + 2, n + 4, n, n + 5, n + 1)  # [..., j, c, h, NB, 2, g]
    v = torch.stack([v & 15, v >> 4], -2).reshape(*lead, 32, NB, 32)  # values: (byte, nibble, g)
    out = []
    for codes, d in ((k, kd), (v, vd)):
        d = d.contiguous().view(torch.float16).reshape(*lead, NB, 4, 4, 2).permute(*range(n), n + 2, n + 1, n + 3, n)
        val = (codes.float() - 8) * d.float().reshape(*lead, 32, NB, 1)
        out.append(val.reshape(*lead[:-1], lead[-1] * 32, D))
    return out


def _plain_append(st):
    case = st["case"]
    NB, D, page = case["D"] // 32, case["D"], case["page"]
    q = _rotate(st["q"].float(), st["q_norm"], st["table"], st["pos"], case["n_rot"], case["pairs"])
    # codes jump where a value crosses a border between two of them: keys in 64 bits, rounded once
    k = _rotate(st["k"].double(), st["k_norm"], st["table"], st["pos"], case["n_rot"], case["pairs"]).float()
    slots = st["slots"]
    _scatter(st["cache"], slots, *_q4_0(k), False, NB)
    _scatter(st["cache"], slots, *_q4_0(st["v"].float()), True, NB)
    kv = _values(st["cache"], D)
    k_read, v_read = (x[slots // page, :, slots % page] for x in kv)
    return q.to(st["q"].dtype), k_read, v_read


def _plain_attn(st):
    case = st["case"]
    B, n, Hq, Hkv, D, kv = (case[k] for k in ("B", "n_q", "Hq", "Hkv", "D", "kv"))
    k, v = (x[st["pages"].clamp_min(0).long()] for x in _values(st["cache"], D))  # [B][each][H][page][D]
    k, v = (x.transpose(1, 2).flatten(2, 3)[:, :, :kv] for x in (k, v))  # [B][H][kv][D]
    q = st["q"].float().view(B, n, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    s = (q @ k.transpose(-1, -2) * st["scale"]).view(B, Hkv, Hq // Hkv, n, kv)
    L = st["kv_len"].long()[:, None, None]
    key, at = torch.arange(kv, device=DEV), L - n + torch.arange(n, device=DEV)[:, None]  # [B][n][1]
    seen = (key < L) & (key > at - case["window"] if case["window"] else key >= 0)
    if case["causal"]:
        seen = seen & (key <= at)
    seen = seen[:, None, None]
    s = s.masked_fill(~seen, -math.inf)
    top = s.amax(-1, keepdim=True).clamp_min(-3e38)
    p = torch.exp(s - top)
    p = p / p.sum(-1, keepdim=True).clamp_min(1e-38)
    o = p.view(B, Hkv, -1, kv) @ v.masked_fill(~(key < L)[..., None], 0.0)
    o = o.view(B, Hkv, Hq // Hkv, n, D).permute(0, 3, 1, 2, 4).reshape(B * n, Hq, D)
    return o.to(st["q"].dtype)


# ------------------------------------------------------------------ 64 bits, from the definitions
def _exact_heads(x, gamma, st):
    """Complex rotation of the normalised heads, in 64 bits."""
    case = st["case"]
    x = x.double()
    if gamma is not None:
        x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / case["D"] + EPS) * gamma.double()
    turn = torch.view_as_complex(st["table"].double()).index_select(0, st["pos"].long()).unsqueeze(1)
    half = case["n_rot"] // 2
    i = torch.arange(half, device=DEV)
    first, second = (2 * i, 2 * i + 1) if case["pairs"] else (i, i + half)
    z = torch.complex(x[..., first], x[..., second]) * turn
    y = x.clone()
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_q4_0(y):
    """The values that Q4_0 of y stands for: block scales from fp32 division, nearest code with ties away from zero."""
    T, H, D = y.shape
    b = y.float().reshape(T, H, D // 32, 32)
    d = torch.div(b.abs().max(-1, keepdim=True).values, torch.full((), 7.0, device=DEV))
    code = torch.div(b, d.clamp_min(1e-45)).double()
    code = torch.copysign(torch.floor(code.abs() + 0.5), code).clamp(-8.0, 7.0)
    return (code * d.half().double()).reshape(T, H, D)


def _exact_values(cache, D):
    """K and V of every token by their places in the layout, 64 bits [pages][H][page_size][D]."""
    P, H, groups, rec = cache.shape
    NB = D // 32
    tok, val = torch.arange(32, device=DEV)[:, None], torch.arange(D, device=DEV)[None]
    b, e = val // 32, val % 32
    byte = b * 512 + (((tok % 8) * 4 + e % 16 // 4) * 4 + tok // 8) * 4 + e % 4
    k = cache[..., byte] >> (4 * (e // 16)) & 15
    unit = (((e % 8) * 4 + tok // 2 % 4) * 4 + tok // 8) * 2 + tok % 2
    v = cache[..., NB * 512 + b * 512 + unit * 2 + e // 16] >> (4 * (e // 8 % 2)) & 15
    half = cache.view(torch.float16)
    d = b * 32 + ((tok // 2 % 4) * 4 + tok // 8) * 2 + tok % 2
    kd, vd = half[..., NB * 512 + d], half[..., NB * 544 + d]
    return [((x.double() - 8) * s.double()).reshape(P, H, groups * 32, D) for x, s in ((k, kd), (v, vd))]


def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "rope":
        return _exact_heads(st["x"], st["k_norm"], st)
    if case["op"] == "append":
        return (_exact_heads(st["q"], st["q_norm"], st), _exact_q4_0(_exact_heads(st["k"], st["k_norm"], st)),
                _exact_q4_0(st["v"].double()))
    B, n, Hq, Hkv, D = (case[k] for k in ("B", "n_q", "Hq", "Hkv", "D"))
    out = torch.zeros(B, n, Hq, D, dtype=torch.float64, device=DEV)
    q = st["q"].double().view(B, n, Hq, D)
    for seq, L in enumerate(_lengths(case)):
        used = st["pages"][seq, :-(-L // case["page"])].long()
        k, v = (x.transpose(0, 1).reshape(Hkv, -1, D)[:, :L] for x in _exact_values(st["cache"][used], D))
        lo, hi = (torch.tensor(x, device=DEV)[:, None] for x in zip(*_visible(case, L)))
        j = torch.arange(L, device=DEV)
        hidden = (j < lo) | (j >= hi)
        for head in range(Hq):
            s = (q[seq, :, head] @ k[head * Hkv // Hq].T) * st["scale"]
            p = torch.softmax(s.masked_fill(hidden, -math.inf), -1).masked_fill(hidden, 0.0)
            out[seq, :, head] = p @ v[head * Hkv // Hq]
    return out.view(B * n, Hq, D)
