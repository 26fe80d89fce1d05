"""qmm_attn_q4_0 where the size of the cached scales decides what is kept:
scales of v on both sides of a power of two whose exponent bits share none
(2 is 10000, 1 is 01111), a few large ones among ordinary ones, and large
ones throughout.  fp32 rows carry 22 bits of the weights whatever the scales:
the bounds of test_gpu_attn.py (elementwise, and 2^-18 root mean square)."""
import numpy as np
import pytest

from parity import lib
from test_gpu_attn import MAY_GROW, Case

pytestmark = pytest.mark.gpu


def _scales(lens, page, D, draw, keys=None):
    """Factors of a cache's scales [pages][1][records][K: D, V: D], V's drawn, K's `keys` or a third."""
    P = sum(-(-L // page) for L in lens) + 2
    s = np.full((P, 1, page // 32, 2 * D), 0.3 if keys is None else keys)
    s[..., D:] = draw((P, 1, page // 32, D))
    return s


@pytest.mark.parametrize("top", [2.2, 3.0, 8.0, 40.0, 3000.0, 60000.0])
@pytest.mark.parametrize("lens,n,Hq,Hkv,D", [([4096], 1, 4, 1, 64), ([700, 33], 3, 8, 1, 128), ([9000, 500], 1, 6, 2, 96),
                                             ([600], 17, 4, 1, 32)])
def test_scales_of_v_over_powers_of_two(top, lens, n, Hq, Hkv, D):
    """Scales between a fifth of `top` and `top`."""
    qmm = lib()
    c = Case(qmm, lens, [n] * len(lens), Hq, Hkv, D, 64, "f32", seed=int(top),
             cache_scale=_scales(lens, 64, D, lambda shape: np.full(shape, top)))
    c.check(c.run())


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("lens,n,D", [([4096], 1, 64), ([20000], 1, 64), ([300, 1000], 9, 128)])
def test_few_large_scales_of_v(dtype, lens, n, D):
    """One block in a hundred 20 times as large, as a projection's outliers make them."""
    qmm = lib()
    rng = np.random.default_rng(len(lens) + n)
    c = Case(qmm, lens, [n] * len(lens), 8, 1, D, 64, dtype, seed=n,
             cache_scale=_scales(lens, 64, D, lambda shape: np.where(rng.random(shape) < 0.01, 8.0, 0.4)))
    c.check(c.run())


def test_a_long_diffuse_softmax_over_scales_around_two():
    """Nearly equal weights: each is small beside the reference, and its low part with it."""
    qmm = lib()
    lens = [30000]
    c = Case(qmm, lens, [1], 2, 1, 64, 256, "f32", seed=2, scale=0.02,
             cache_scale=_scales(lens, 256, 64, lambda shape: np.full(shape, 3.0)))
    c.check(c.run())


@pytest.mark.parametrize("top", [6000.0, 60000.0])
@pytest.mark.parametrize("max_kv", [None, MAY_GROW])
@pytest.mark.parametrize("lens,nqs,Hq,Hkv,D", [([300, 128], [64, 64], 4, 1, 64), ([700, 0, 90], [130, 5, 90], 2, 1, 128),
                                               ([2000], [64], 2, 1, 32)])
def test_values_beyond_fp16(top, max_kv, lens, nqs, Hq, Hkv, D):
    """Cached values d q above 65504 (d itself is fp16), in some records or all, in calls of few and of many keys."""
    qmm = lib()
    rng = np.random.default_rng(len(lens))
    for share in (0.02, 1.0):
        def draw(shape):
            return np.where(rng.random(shape[:3] + (1,)) < share, top, 0.5) * np.ones(shape)
        s = _scales(lens, 64, D, draw)
        s[..., :D] = draw(s.shape)[..., :D]
        c = Case(qmm, lens, nqs, Hq, Hkv, D, 64, "bf16", seed=D, q_start=True, scale=0.3 / top,
                 extra_kv=0 if max_kv is None else max_kv // 64, cache_scale=s)
        c.check(c.run(**({} if max_kv is None else {"max_kv": max_kv})))


@pytest.mark.parametrize("D", [32, 128])
@pytest.mark.parametrize("share", [0.1, 1.0])
def test_values_beyond_fp16_in_whole_items(D, share):
    """As many items as fill the tensor-memory kernel's CTAs, some with large scales and some without, and no keys."""
    qmm = lib()
    rng = np.random.default_rng(D)
    lens, nqs = [0, 3, 129, 300, 70] * 14, [130, 64, 128, 40, 70] * 14
    s = _scales(lens, 96, D, lambda shape: np.where(rng.random(shape[:3] + (1,)) < share, 60000.0, 0.5) * np.ones(shape))
    s[..., :D] = s[..., D:]
    c = Case(qmm, lens, nqs, 4, 2, D, 96, "bf16", seed=D, q_start=True, scale=0.3 / 60000, cache_scale=s)
    first = c.run()
    assert qmm.qmm_debug_attn_plan(c.op(first)) == (qmm.ATTN_TMEM, qmm.ATTN_WHOLE)
    c.check(first)
    for _ in range(5):
        assert np.array_equal(first.float().cpu().numpy(), c.run().float().cpu().numpy())
