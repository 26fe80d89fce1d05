"""qmm_attn_q4_0 against attention in 64 bits over the cache's own values.

Tolerances, for an output o = sum_j p_j v_j with m = sum_j p_j |v_j| and N
keys seen, u = 2^-24 (half a step of fp32):

* a score: q as two fp16 parts is off by u |q|, a block's sum of 32 products
  and the seed by at most 34 roundings of its partial sums, whose size is at
  most sum |q| d (15 + 8), the sum over blocks and the two scalings by NB + 3;
  so |ds| <= (37 + NB) 2 u X with X = |scale| max_j sum_e |q_e| d_j 23.  The
  tensor core may truncate where fp32 rounds: 2 u a step.  Its exponential's
  argument and reference cost 2 u (|s| + 40) more, ex2.approx 4 u.
* the sums over N keys, fp32 in steps of at least 16 keys a lane: at most
  (N / 16 + 64) 2 u of m for the numerator and the denominator each.
* weights: 2 u as two parts, 2^-12 (fp16's half step 2^-11 relative / 2 with
  the bound taken whole: 2^-11) as one part; 2^-38 of the largest weight times
  the largest |v| where the part is subnormal.
* 16-bit outputs: half a step of their type.
* bf16 with many rows a key/value head: k and v as fp16 (2^-11 each, so a score
  is off by up to 2^-11 |scale| sum_e |q_e k_je| <= 2^-11 X 8 / 23).
"""
import numpy as np
import pytest
import torch

import attn_reference as R
from parity import lib
from oracle import oracle as O

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def _np(t):
    return t.detach().double().cpu().numpy()


class Case:
    """Sequences over a shuffled page table; whatever no query sees is NaN scales, unused pages entries are junk."""

    def __init__(self, qmm, lens, nqs, Hq, Hkv, D, page, dtype="f32", causal=True, window=0, seed=0, scale=None,
                 strided=False, q_start=None, extra_kv=0, cache_scale=0.3):
        rng = np.random.default_rng(seed)
        self.qmm, self.lens, self.nqs, self.D, self.page = qmm, lens, nqs, D, page
        self.Hq, self.Hkv, self.causal, self.window = Hq, Hkv, causal, window
        self.scale = D ** -0.5 if scale is None else scale
        self.dtype = TYPES[dtype]
        each = [-(-L // page) for L in lens]
        P = sum(each) + 2
        cache = R.random_cache(P, Hkv, page, D, rng, cache_scale)
        order = rng.permutation(P)
        table = np.full((len(lens), max(each + [1]) + 1 + extra_kv), -123456, np.int32)
        used = np.zeros((P, page), bool)
        at = 0
        for b, L in enumerate(lens):
            table[b, :each[b]] = order[at:at + each[b]]
            at += each[b]
            used[table[b, np.arange(L) // page], np.arange(L) % page] = True
        self.values = R.cache_values(cache, D)
        (_, _), (_, _), ks, vs = R.places(D)
        groups = used.reshape(P, page // 32, 32)
        for p, gr, t in zip(*np.nonzero(~groups)):  # tokens that nobody may look at
            for s in (ks[t], vs[t]):
                cache[p, :, gr, s], cache[p, :, gr, s + 1] = 0xFF, 0x7F
        self.table = table
        T = sum(nqs)
        q = rng.standard_normal((T, Hq, D))
        q[rng.random(q.shape) < 0.02] *= 8
        self.q = torch.tensor(q, dtype=torch.float32).to(self.dtype).to(DEV)
        if strided:
            base = torch.full((T, Hq + 3, D + strided), float("nan"), dtype=self.dtype, device=DEV)
            base[:, 1:Hq + 1, strided:] = self.q
            self.q = base[:, 1:Hq + 1, strided:]
        self.cache_t = torch.tensor(cache, device=DEV)
        self.cache = qmm.kv_cache(self.cache_t, page)
        self.pages = torch.tensor(table, device=DEV)
        self.kv_len = torch.tensor(lens, dtype=torch.int32, device=DEV)
        self.max_q = max(nqs + [1])
        uniform = all(n == nqs[0] for n in nqs)
        self.q_start = None if uniform and q_start is None else torch.tensor(
            np.r_[0, np.cumsum(nqs)], dtype=torch.int32, device=DEV)

    def op(self, out=None, **kw):
        kw = {"max_q": self.max_q, "max_kv": max(self.lens + [1]), "scale": self.scale, "causal": self.causal,
              "window": self.window, "q_start": self.q_start, **kw}
        return self.qmm.attn_op(self.cache, self.q, self.pages, self.kv_len, out=out, **kw)

    def run(self, **kw):
        out = torch.full((self.q.shape[0], self.Hq, self.D), float("nan"), dtype=self.dtype, device=DEV)
        op = self.op(out, **kw)
        if op._keep[-1] is not None:
            op._keep[-1].fill_(0xFF)  # a workspace may hold anything
        self.qmm.qmm_attn_q4_0(op)
        return out

    def reference(self, hide=None):
        K, V = self.values
        parts = []
        at = 0
        for b, (L, n) in enumerate(zip(self.lens, self.nqs)):
            pg = self.table[b, np.arange(L) // self.page]
            k, v = (x[pg, :, np.arange(L) % self.page].transpose(1, 0, 2) for x in (K, V))
            q = _np(self.q[at:at + n])
            at += n
            out, mag, top, seen = R.attention(q, k, v, L, self.scale, self.causal, self.window,
                                              None if hide is None else hide(b, L))
            d = np.abs(k).reshape(*k.shape[:2], self.D // 32, 32).max(-1).max((0, 1), initial=0)  # >= the scale
            X = abs(self.scale) * (np.abs(q) * np.repeat(d, 32)).sum(-1, keepdims=True) * 23
            big = np.abs(v).max(initial=0)
            parts.append((out, mag, top, seen, X, np.full(seen.shape, big)))
        return [np.concatenate(x) for x in zip(*parts)]

    def check(self, out, hide=None):
        ref, mag, top, N, X, big = self.reference(hide)
        u = 2.0 ** -24
        NB = self.D // 32
        ds = (37 + NB) * 2 * u * X + 2 * u * (top + 40) + 4 * u
        rel = 2 * ds + 2 * (N / 16 + 64) * 2 * u + 2 * u
        tol = mag * rel + N * 2.0 ** -38 * big
        if self.dtype != torch.float32:
            half = torch.finfo(self.dtype).eps / 2
            if self.dtype == torch.bfloat16 and self.max_q * self.Hq // self.Hkv >= 32 and self.D <= 128:
                tol = tol + mag * 2.0 ** -11 * (2 * X * 8 / 23 + 1)
            tol = (tol + mag * 2.0 ** -11) * (1 + half) + np.abs(ref) * half + 2.0 ** -25
        err = np.abs(_np(out) - ref)
        assert np.isfinite(err).all()
        assert (err <= tol + 1e-30).all(), (np.max(err / (tol + 1e-30)), np.abs(ref).max())
        assert (_np(out)[(N == 0)[..., 0]] == 0).all()  # rows that see nothing
        norm = np.linalg.norm(ref)
        # root mean square: fp32 2^-18 (64 u; the bound above is linear in every rounding)
        assert np.linalg.norm(err) <= norm * (2.0 ** -18 if self.dtype == torch.float32
                                              else torch.finfo(self.dtype).eps / 2 + 2.0 ** -11) + 1e-30
        assert self.qmm.qmm_last_device_error() == 0


@pytest.mark.parametrize("D", [32, 64, 96, 128, 160, 192, 224, 256])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_one_token(D, dtype):
    qmm = lib()
    c = Case(qmm, [1, 31, 32, 33, 700, 0, 129], [1] * 7, 6, 2, D, 32, dtype, seed=D)
    c.check(c.run())


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 4), (3, 1), (8, 1), (9, 1), (16, 1), (17, 1), (40, 1), (64, 8)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_head_groups(Hq, Hkv, dtype):
    qmm = lib()
    c = Case(qmm, [300, 45], [1, 1], Hq, Hkv, 64, 64, dtype, seed=Hq)
    c.check(c.run())


@pytest.mark.parametrize("lens,nqs,causal,window", [
    ([40, 7, 100], [5, 7, 3], True, 0),            # a prompt of its own length among them
    ([3, 0, 5, 1], [6, 4, 5, 0], True, 0),         # more queries than keys: rows that see nothing; none at all
    ([3, 0, 5, 64], [6, 4, 5, 2], False, 0),
    ([500, 1000, 33], [1, 2, 33], True, 1),
    ([500, 1000, 33], [1, 2, 33], True, 70),
    ([500, 1000, 33], [4, 2, 33], False, 70),
    ([2000], [1], True, 100000),
    ([90], [90], True, 0),
    ([777, 64], [70, 64], True, 129),
])
@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_masks_and_lengths(lens, nqs, causal, window, dtype):
    qmm = lib()
    c = Case(qmm, lens, nqs, 6, 2, 64, 32, dtype, causal, window, seed=len(lens) + window, q_start=True)
    c.check(c.run())


@pytest.mark.parametrize("n,L,Hq,Hkv,D,page,dtype", [
    (3, 900, 8, 1, 128, 64, "f32"), (17, 400, 8, 2, 128, 96, "bf16"), (65, 300, 5, 1, 96, 32, "f16"),
    (130, 200, 4, 2, 32, 128, "f32"), (33, 500, 16, 1, 256, 64, "bf16"), (20, 300, 3, 3, 160, 32, "f32"),
])
def test_chunks(n, L, Hq, Hkv, D, page, dtype):
    qmm = lib()
    c = Case(qmm, [L, L // 2, n], [n] * 3, Hq, Hkv, D, page, dtype, seed=n)
    c.check(c.run())


@pytest.mark.parametrize("D", [32, 64, 96, 128])
@pytest.mark.parametrize("lens,nqs,causal,window,Hq,Hkv,page", [
    ([200], [64], True, 0, 1, 1, 32),                      # one tile, half of it
    ([300, 128], [64, 64], True, 0, 4, 1, 64),             # two tiles
    ([150, 64, 5], [100, 64, 5], True, 0, 6, 2, 32),       # more than one row block; fewer keys than queries
    ([3, 700, 0, 257], [130, 40, 64, 1], True, 0, 4, 2, 96),
    ([700, 90], [70, 90], True, 100, 3, 1, 32),            # a window
    ([700, 90], [70, 90], False, 33, 3, 1, 128),
    ([130, 127], [80, 80], False, 0, 8, 8, 32),
    ([1, 128, 129, 127], [64, 64, 64, 64], True, 0, 2, 1, 32),
])
def test_many_rows(D, lens, nqs, causal, window, Hq, Hkv, page):
    qmm = lib()
    c = Case(qmm, lens, nqs, Hq, Hkv, D, page, "bf16", causal, window, seed=D + len(lens), q_start=True)
    c.check(c.run())


def test_many_rows_of_sequences_without_keys():
    """Items with nothing to attend to between others: zeros, every time (such an item writes its rows with
    no products between its warps)."""
    qmm = lib()
    for D in (32, 64, 128):
        c = Case(qmm, [0, 3, 0, 300, 0], [130, 64, 128, 40, 64], 4, 2, D, 96, "bf16", seed=D, q_start=True)
        first = c.run()
        c.check(first)
        for _ in range(20):
            assert torch.equal(first, c.run())


def test_many_rows_of_many_keys():
    """Few row blocks and long contexts: items are cut over the CTAs, a CTA holds parts of several."""
    qmm = lib()
    c = Case(qmm, [2000, 40, 1500], [64] * 3, 2, 1, 64, 64, "bf16", seed=21)
    first = c.run()
    c.check(first)
    for _ in range(3):
        assert torch.equal(first, c.run())
    c = Case(qmm, [1000, 900], [64] * 2, 8, 4, 32, 32, "bf16", False, 0, seed=22)
    c.check(c.run())


def test_many_rows_strided_quantized_and_missing_pages():
    qmm = lib()
    qmm.qmm_last_device_error()
    c = Case(qmm, [400, 300], [70, 70], 4, 2, 64, 32, "bf16", strided=1, seed=23)
    base = torch.full((140, 9, 65), 7.0, dtype=c.dtype, device=DEV)
    out = base[:, 2:6, 1:]
    qmm.qmm_attn_q4_0(c.op(out))
    c.check(out)
    base[:, 2:6, 1:] = 7.0
    assert (base == 7.0).all()
    yq = torch.full((140, 256), 99, dtype=torch.int8, device=DEV)
    yd = torch.full((140, 8), 99, dtype=torch.int16, device=DEV)
    plain = torch.empty(140, 4, 64, dtype=c.dtype, device=DEV)
    qmm.qmm_attn_q4_0(c.op(plain, yq=yq, yd=yd))
    # bf16 of the fp32 output that was quantized: off by half a bf16 step and half a code (and fp16's step in d)
    d = yd.view(torch.float16).double()[:, :, None].expand(-1, -1, 32).reshape(140, 256)
    off = (yq.double() * d - plain.double().view(140, 256)).abs()
    assert (off <= 0.5 * d + plain.double().view(140, 256).abs() * (2.0 ** -8 + 2.0 ** -10)).all()
    c.pages[0, 3] = c.cache.n_pages
    out = c.run()
    assert qmm.qmm_last_device_error() == 10
    c.check(out, lambda b, L: np.ones(L, bool) if b else np.arange(L) // 32 != 3)


MAY_GROW = 1 << 18  # a max_kv that calls for the kernel of many rows, whatever the lengths are


@pytest.mark.parametrize("D", [32, 64, 96, 128])
@pytest.mark.parametrize("lens,nqs,causal,window,Hq,Hkv,page", [
    ([200], [64], True, 0, 1, 1, 32),
    ([300, 128], [64, 64], True, 0, 4, 1, 64),
    ([150, 64, 5], [100, 64, 5], True, 0, 6, 2, 32),
    ([3, 700, 0, 257], [130, 40, 64, 1], True, 0, 4, 2, 96),
    ([700, 90], [70, 90], True, 100, 3, 1, 32),
    ([700, 90], [70, 90], False, 33, 3, 1, 128),
    ([130, 127], [80, 80], False, 0, 8, 8, 32),
    ([1, 128, 129, 127], [64, 64, 64, 64], True, 0, 2, 1, 32),
    ([2000, 40, 1500], [64] * 3, True, 0, 2, 1, 64),
])
def test_many_rows_that_may_see_many_keys(D, lens, nqs, causal, window, Hq, Hkv, page):
    qmm = lib()
    c = Case(qmm, lens, nqs, Hq, Hkv, D, page, "bf16", causal, window, seed=D + len(lens), q_start=True,
             extra_kv=MAY_GROW // page)
    c.check(c.run(max_kv=MAY_GROW))


@pytest.mark.parametrize("D", [32, 64, 96, 128])
def test_many_rows_of_many_items(D):
    """Row blocks enough for every CTA, of few keys or none, whole."""
    qmm = lib()
    lens, nqs = [0, 3, 129, 300, 70], [130, 64, 128, 40, 70]
    for causal, window in ((True, 0), (False, 0), (True, 50)):
        c = Case(qmm, lens * 14, nqs * 14, 4, 2, D, 96, "bf16", causal, window, seed=D + window, q_start=True)
        first = c.run()
        c.check(first)
        for _ in range(10):
            assert torch.equal(first, c.run())


def test_many_rows_without_keys_that_may_see_many():
    qmm = lib()
    for D in (32, 64, 128):
        c = Case(qmm, [0, 3, 0, 300, 0], [130, 64, 128, 40, 64], 4, 2, D, 96, "bf16", seed=D, q_start=True,
                 extra_kv=MAY_GROW // 96)
        first = c.run(max_kv=MAY_GROW)
        c.check(first)
        for _ in range(20):
            assert torch.equal(first, c.run(max_kv=MAY_GROW))


def test_many_rows_may_grow_strided_quantized_and_missing_pages():
    qmm = lib()
    qmm.qmm_last_device_error()
    c = Case(qmm, [400, 300], [70, 70], 4, 2, 64, 32, "bf16", strided=1, seed=23, extra_kv=MAY_GROW // 32)
    base = torch.full((140, 9, 65), 7.0, dtype=c.dtype, device=DEV)
    out = base[:, 2:6, 1:]
    qmm.qmm_attn_q4_0(c.op(out, max_kv=MAY_GROW))
    c.check(out)
    base[:, 2:6, 1:] = 7.0
    assert (base == 7.0).all()
    yq = torch.full((140, 256), 99, dtype=torch.int8, device=DEV)
    yd = torch.full((140, 8), 99, dtype=torch.int16, device=DEV)
    plain = torch.empty(140, 4, 64, dtype=c.dtype, device=DEV)
    qmm.qmm_attn_q4_0(c.op(plain, yq=yq, yd=yd, max_kv=MAY_GROW))
    # bf16 of the fp32 output that was quantized: off by half a bf16 step and half a code (and fp16's step in d)
    d = yd.view(torch.float16).double()[:, :, None].expand(-1, -1, 32).reshape(140, 256)
    off = (yq.double() * d - plain.double().view(140, 256)).abs()
    assert (off <= 0.5 * d + plain.double().view(140, 256).abs() * (2.0 ** -8 + 2.0 ** -10)).all()
    c.pages[0, 3] = c.cache.n_pages
    out = c.run(max_kv=MAY_GROW)
    assert qmm.qmm_last_device_error() == 10
    c.check(out, lambda b, L: np.ones(L, bool) if b else np.arange(L) // 32 != 3)


@pytest.mark.parametrize("D", [32, 64, 96, 128, 160, 192, 224, 256])
@pytest.mark.parametrize("dtype,n,L,Hq,Hkv,page,window", [
    ("f32", 5, 300, 8, 1, 64, 0), ("f16", 5, 300, 8, 1, 96, 40), ("bf16", 5, 300, 8, 1, 32, 0),
    ("f32", 33, 200, 3, 1, 32, 50), ("f16", 17, 130, 4, 2, 64, 0),
])
def test_wide_blocks(D, dtype, n, L, Hq, Hkv, page, window):
    """Calls that may see so many keys that 16 rows share a CTA."""
    qmm = lib()
    c = Case(qmm, [L, 0, L // 2, n, 1], [n, 1, n, n, 0], Hq, Hkv, D, page, dtype, True, window, seed=n + D,
             q_start=True, extra_kv=4 * MAY_GROW // page)
    c.check(c.run(max_kv=4 * MAY_GROW))


@pytest.mark.parametrize("D", [32, 64, 96, 128, 160, 192, 224, 256])
@pytest.mark.parametrize("dtype,lens,n,window", [
    ("f32", [4096], 1, 0), ("bf16", [4090, 1, 0, 129], 1, 0), ("f16", [1200, 1300], 1, 1000), ("f32", [2000], 9, 0),
    ("f32", [257], 1, 0), ("bf16", [130], 3, 0),
])
def test_clusters(D, dtype, lens, n, window):
    """Few items of few keys: a cluster of up to 16 CTAs an item, some of them with nothing to do."""
    qmm = lib()
    c = Case(qmm, lens, [n] * len(lens), 8, 1, D, 64, dtype, True, window, seed=D + n)
    first = c.run()
    c.check(first)
    for _ in range(3):
        assert torch.equal(first, c.run())


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
def test_wide_blocks_of_many_items(dtype, D):
    """As many items as CTAs, of few keys or none, whole."""
    qmm = lib()
    lens, nqs = [0, 3, 129, 300, 70], [3, 2, 5, 9, 4]
    for causal, window in ((True, 0), (False, 50)):
        c = Case(qmm, lens * 40, nqs * 40, 12, 4, D, 96, dtype, causal, window, seed=D + window, q_start=True)
        c.check(c.run())


@pytest.mark.parametrize("longest", [1536, 2048])
@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_wide_blocks_on_clusters(dtype, longest):
    """Half as many items as CTAs, and few enough keys that two CTAs share each."""
    qmm = lib()
    rng = np.random.default_rng(9)
    lens = [int(x) for x in rng.integers(0, longest, 57)]
    lens[:4] = [longest, longest - 1, 0, 1]
    c = Case(qmm, lens, [4] * 57, 16, 4, 64, 64, dtype, seed=31, q_start=True)
    first = c.run()
    c.check(first)
    for _ in range(3):
        assert torch.equal(first, c.run())


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_long_context(dtype):
    qmm = lib()
    c = Case(qmm, [20000, 9001, 1], [1] * 3, 4, 1, 64, 256, dtype, seed=5)
    c.check(c.run())


def test_many_sequences():
    qmm = lib()
    rng = np.random.default_rng(1)
    lens = [int(x) for x in rng.integers(0, 400, 300)]
    c = Case(qmm, lens, [1] * 300, 2, 1, 32, 32, "f32", seed=6)
    c.check(c.run())
    c = Case(qmm, lens[:150], [int(x) for x in rng.integers(0, 4, 150)], 2, 1, 32, 32, "bf16", seed=7)
    c.check(c.run())


@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0])
def test_scales_of_scores(scale):
    qmm = lib()
    c = Case(qmm, [333, 64], [2, 2], 4, 2, 64, 32, "f32", scale=scale, seed=8)
    c.check(c.run())


@pytest.mark.parametrize("cache_scale", [1e-6, 3e-4, 100.0])
def test_magnitudes_of_the_cache(cache_scale):
    qmm = lib()
    c = Case(qmm, [333, 64], [2, 2], 4, 2, 64, 32, "f32", scale=0.1 / cache_scale, seed=9, cache_scale=cache_scale)
    ref = c.reference()[0]
    err = np.linalg.norm(_np(c.run()) - ref) / np.linalg.norm(ref)
    assert err <= 2.0 ** -18, err


@pytest.mark.parametrize("strided,dtype", [(8, "bf16"), (1, "bf16"), (1, "f32"), (4, "f32")])
def test_strided_heads(strided, dtype):
    qmm = lib()
    c = Case(qmm, [100, 300], [2, 2], 6, 2, 64, 32, dtype, strided=strided, seed=10)
    base = torch.full((4, 9, 64 + strided), 7.0, dtype=c.dtype, device=DEV)
    out = base[:, 2:8, strided:]
    qmm.qmm_attn_q4_0(c.op(out))
    c.check(out)
    base[:, 2:8, strided:] = 7.0
    assert (base == 7.0).all()  # nothing else is written


def test_q8_0_output():
    qmm = lib()
    c = Case(qmm, [500, 64, 0, 30], [1] * 4, 8, 2, 128, 64, "f32", seed=11)
    out = torch.empty(4, 8, 128, device=DEV)
    yq = torch.full((4, 1024), 99, dtype=torch.int8, device=DEV)
    yd = torch.full((4, 32), 99, dtype=torch.int16, device=DEV)
    qmm.qmm_attn_q4_0(c.op(out, yq=yq, yd=yd))
    c.check(out)
    q, d = O.quantize_q8_0(out.view(4, 1024).cpu().numpy())
    assert np.array_equal(yq.cpu().numpy(), q) and np.array_equal(yd.cpu().numpy().view(np.uint16), d)
    yq2, yd2 = torch.empty_like(yq), torch.empty_like(yd)
    qmm.qmm_attn_q4_0(c.op(None, yq=yq2, yd=yd2))
    assert torch.equal(yq, yq2) and torch.equal(yd, yd2)


def test_results_do_not_change_from_call_to_call():
    qmm = lib()
    for dtype, nq in (("f32", 1), ("bf16", 9)):
        c = Case(qmm, [5000, 77, 1200], [nq] * 3, 8, 2, 64, 64, dtype, seed=12)
        first = c.run()
        for _ in range(3):
            assert torch.equal(first, c.run())


def test_graph_replay_and_another_stream():
    qmm = lib()
    c = Case(qmm, [3000, 50], [1, 1], 8, 2, 64, 64, "f32", seed=13)
    want = c.run()
    out = torch.zeros_like(want)
    op = c.op(out)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        qmm.qmm_attn_q4_0(op)
    s.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qmm.qmm_attn_q4_0(op)
    # another step: the lengths and queries are read at replay
    c.kv_len.copy_(torch.tensor([2999, 17], dtype=torch.int32))
    c.lens = [2999, 17]
    c.q.mul_(-0.5)
    graph.replay()
    torch.cuda.synchronize()
    c.check(out)


def test_pages_and_lengths_out_of_range():
    """Bad entries are found on the device, counted as unseen and reported; the other rows are right."""
    qmm = lib()
    qmm.qmm_last_device_error()
    c = Case(qmm, [700, 300], [1, 2], 4, 2, 64, 32, "f32", seed=14, q_start=True)
    c.pages[0, 3], c.pages[0, 9] = c.cache.n_pages, -1
    out = c.run()
    assert qmm.qmm_last_device_error() == 10

    def hide(b, L):
        pg = np.arange(L) // 32
        return np.ones(L, bool) if b else (pg != 3) & (pg != 9)
    c.check(out, hide)
    # a length above max_kv is clamped to it
    c = Case(qmm, [700, 300], [1, 1], 4, 2, 64, 32, "f32", seed=15)
    c.kv_len[1] = 1 << 30
    c.lens = [700, 700]
    c.table[1] = c.table[0]
    c.pages.copy_(torch.tensor(c.table))
    out = c.run(max_kv=700)
    assert qmm.qmm_last_device_error() == 10
    c.check(out)
    c.kv_len[1] = -5
    c.lens = [700, 0]
    out = c.run(max_kv=700)
    assert qmm.qmm_last_device_error() == 10
    c.check(out)
    # query rows past the end
    c = Case(qmm, [100, 100], [2, 2], 4, 2, 64, 32, "f32", seed=16, q_start=True)
    c.q_start[2] = 1000
    out = c.run()
    assert qmm.qmm_last_device_error() == 10
    c.check(out)


def test_cache_offsets_beyond_32_bits():
    """A cache of more than 2^32 bytes: pages at its far end."""
    qmm = lib()
    D, page, Hkv, P = 128, 256, 8, 20000  # 36,864 * 8 bytes a page: 5.9 GB
    data = torch.empty(P, Hkv, page // 32, 36 * D, dtype=torch.uint8, device=DEV)
    rng = np.random.default_rng(17)
    pages = [P - 1, 3, P - 7]
    small = R.random_cache(3, Hkv, page, D, rng)
    for i, p in enumerate(pages):
        data[p] = torch.tensor(small[i], device=DEV)
    c = Case(qmm, [700], [1], 16, Hkv, D, page, "f32", seed=18)
    c.values = R.cache_values(small, D)
    c.table = np.array([[0, 1, 2]], np.int32)
    c.pages = torch.tensor([pages], dtype=torch.int32, device=DEV)
    c.cache = qmm.kv_cache(data, page)
    c.check(c.run())
    slots = torch.tensor([(P - 2) * page + 5], device=DEV)
    x = torch.randn(1, Hkv, D, device=DEV)
    qmm.qmm_kv_append_q4_0(qmm.kv_append_op(c.cache, x, x, slots))
    k = torch.empty(1, Hkv, D, device=DEV)
    qmm.qmm_kv_read_q4_0(qmm.kv_read_op(c.cache, slots, k=k))
    assert np.array_equal(_np(k), R.q4_0_values(_np(x)))


def test_empty_calls():
    qmm = lib()
    c = Case(qmm, [10], [1], 2, 1, 32, 32, "f32")
    none = torch.empty(0, 2, 32, device=DEV)
    empty = torch.empty(0, dtype=torch.int32, device=DEV)
    qmm.qmm_attn_q4_0(qmm.attn_op(c.cache, none, c.pages[:0], empty, none, max_q=1, max_kv=32))
    # a sequence without queries, and a batch where nothing is cached
    c = Case(qmm, [0, 0], [1, 1], 2, 1, 32, 32, "f32")
    assert (c.run(max_kv=0) == 0).all()
