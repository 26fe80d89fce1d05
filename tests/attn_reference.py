"""Plain 64-bit forms of the attention operators, and the cache layout of
include/qmm.h written out place by place (numpy, no library code)."""
import numpy as np


def record_bytes(D):
    return 36 * D


def places(D):
    """Where the cache keeps a token's values, from a record's first byte:
    (K byte, K nibble), (V byte, V nibble) [32][D] each, and the byte of the
    K and V scales [32][D / 32]."""
    NB = D // 32
    tok, val = np.arange(32)[:, None], np.arange(D)[None]
    b, e = val // 32, val % 32
    i, g = tok // 8, tok % 8
    j, c, h = tok // 8, tok // 2 % 4, tok % 2
    word = (g * 4 + e % 16 // 4) * 4 + i
    k = (b * 512 + word * 4 + e % 4, np.broadcast_to(e // 16, (32, D)))
    unit = ((e % 8 * 4 + c) * 4 + j) * 2 + h
    v = (NB * 512 + b * 512 + unit * 2 + e // 16, np.broadcast_to(e // 8 % 2, (32, D)))
    s = (c * 4 + j) * 2 + h
    blk = np.arange(NB)[None]
    return k, v, NB * 1024 + blk * 64 + 2 * s, NB * 1088 + blk * 64 + 2 * s


def cache_values(cache, D):
    """fp64 K and V [pages][heads][page_size][D] of cache bytes [pages][heads][groups][36 D]."""
    (kb, kn), (vb, vn), ks, vs = places(D)
    out = []
    for byte, nib, sc in ((kb, kn, ks), (vb, vn, vs)):
        q = (cache[..., byte] >> (4 * nib)) & 15
        d = (cache[..., sc].astype(np.uint16) | cache[..., sc + 1].astype(np.uint16) << 8).view(np.float16)
        with np.errstate(invalid="ignore", over="ignore"):
            val = (q.astype(np.float64) - 8) * np.repeat(d.astype(np.float64), 32, -1)
        P, H, G = cache.shape[:3]
        out.append(val.reshape(P, H, G * 32, D))
    return out


def random_cache(P, H, page, D, rng, scale=0.3):
    """Random cache bytes: every nibble value, fp16 scales around `scale`, of both signs."""
    cache = rng.integers(0, 256, (P, H, page // 32, record_bytes(D)), dtype=np.uint8)
    d = (scale * rng.uniform(0.2, 1.0, (P, H, page // 32, 2 * D)) * rng.choice([-1, 1], (P, H, page // 32, 2 * D)))
    n = D // 32 * 64
    cache[..., -2 * n:] = d[..., :n].astype(np.float16).view(np.uint8)
    return cache


def rotate(x, gamma, eps, table, pos, n_rot, pairs):
    """Norm and rotation of x [T][H][D], fp64."""
    x = np.asarray(x, np.float64)
    if gamma is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(gamma, np.float64)
    y = x.copy()
    if n_rot:
        cs = np.asarray(table, np.float64)[np.asarray(pos)][:, None]
        c, s = cs[..., 0], cs[..., 1]
        lo = slice(0, n_rot, 2) if pairs else slice(0, n_rot // 2)
        hi = slice(1, n_rot, 2) if pairs else slice(n_rot // 2, n_rot)
        y[..., lo] = x[..., lo] * c - x[..., hi] * s
        y[..., hi] = x[..., hi] * c + x[..., lo] * s
    return y


def q4_0_values(y):
    """What Q4_0 of fp32 values stands for: IEEE fp32 divisions, ties away from zero, fp16 scales."""
    y = np.asarray(y, np.float32)
    b = y.reshape(*y.shape[:-1], -1, 32)
    d = np.abs(b).max(-1) / np.float32(7)
    with np.errstate(invalid="ignore", divide="ignore"):
        r = (b / d[..., None]).astype(np.float64)
    r = np.where(d[..., None] > 0, r, 0)
    q = np.clip(np.copysign(np.floor(np.abs(r) + 0.5), r), -8, 7)
    return (q * d.astype(np.float16).astype(np.float64)[..., None]).reshape(y.shape)


def attention(q, k, v, n_kv, scale, causal, window, seen_keys=None):
    """fp64 attention of one sequence: q [n][Hq][D]; k, v [Hkv][n_kv or more][D]; seen_keys: a mask of keys
    that count at all.  Returns out and, for tolerances, sum_j p_j |v_j|, max_j |s_j| and the number of keys
    seen [n][Hq][1 or D]."""
    n, Hq, D = q.shape
    G = Hq // k.shape[0]
    out, mag = np.zeros((n, Hq, D)), np.zeros((n, Hq, D))
    top, seen_n = np.zeros((n, Hq, 1)), np.zeros((n, Hq, 1))
    j = np.arange(n_kv)
    for i in range(n):
        p = n_kv - n + i
        seen = (j <= p) if causal else np.ones(n_kv, bool)
        if window:
            seen = seen & (j > p - window)
        if seen_keys is not None:
            seen = seen & seen_keys
        if not seen.any():
            continue
        for h in range(Hq):
            kk, vv = k[h // G, :n_kv][seen], v[h // G, :n_kv][seen]
            s = scale * (kk @ q[i, h])
            w = np.exp(s - s.max())
            w /= w.sum()
            out[i, h], mag[i, h] = w @ vv, w @ np.abs(vv)
            top[i, h], seen_n[i, h] = np.abs(s).max(), seen.sum()
    return out, mag, top, seen_n
