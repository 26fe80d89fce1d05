"""qmm_attn_q4_0: what a row's output owes to the row alone, and how near the
16-bit types come to their own rounding."""
import numpy as np
import pytest
import torch

import attn_reference as R
from parity import lib
from test_gpu_attn import DEV, MAY_GROW, Case, _np

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("dtype,lens,n,Hq,Hkv,D,max_kv", [
    ("f32", [300, 45], 1, 8, 1, 64, None), ("f16", [300, 45], 3, 8, 2, 128, None), ("bf16", [300, 45], 5, 8, 1, 96, None),
    ("f32", [9000, 45], 1, 8, 1, 64, None), ("bf16", [300, 200], 70, 4, 2, 64, MAY_GROW),
    ("bf16", [300, 200], 70, 4, 2, 128, MAY_GROW), ("f16", [700], 40, 4, 1, 64, None)])
def test_rows_that_are_not_finite_stay_by_themselves(bad, dtype, lens, n, Hq, Hkv, D, max_kv):
    """A query row with a NaN or an infinity gives NaN, and every other row the bits it has without it."""
    qmm = lib()
    kw = {} if max_kv is None else {"max_kv": max_kv}
    c = Case(qmm, lens, [n] * len(lens), Hq, Hkv, D, 32, dtype, seed=n,
             extra_kv=0 if max_kv is None else max_kv // 32)
    want = c.run(**kw)
    rows = [(0, 1), (c.q.shape[0] - 1, Hq - 1), (c.q.shape[0] // 2, 0)]
    for t, h in rows:
        c.q[t, h, (7 * t + h) % D] = bad
    out = c.run(**kw)
    hit = torch.zeros(out.shape[:2], dtype=torch.bool, device=out.device)
    for t, h in rows:
        hit[t, h] = True
    assert torch.isnan(out[hit]).all()
    assert torch.equal(out[~hit], want[~hit])
    assert qmm.qmm_last_device_error() == 0


@pytest.mark.parametrize("lens,nqs,Hq,Hkv,D,window", [
    ([4096], [1], 8, 1, 64, 0), ([1000, 700], [1, 1], 24, 8, 96, 500), ([20000], [1], 4, 1, 128, 0),
    ([300, 200], [40, 40], 4, 1, 64, 0)])
def test_fp16_outputs_are_rounded_once(lens, nqs, Hq, Hkv, D, window):
    """fp16 rows carry q exactly and the weights as fp32 rows do, so what is left beside fp16's own rounding of the
    output is far below it: of an error e = r + k (r the rounding, uniform; k the rest, 2^-18 relative as for fp32
    rows against r's about 2^-12.8), |e| <= |r| + |k| <= 1.03 |r|."""
    qmm = lib()
    c = Case(qmm, lens, nqs, Hq, Hkv, D, 64, "f16", True, window, seed=D)
    ref = c.reference()[0]
    out = _np(c.run())
    rounding = np.linalg.norm(ref.astype(np.float16).astype(np.float64) - ref)
    assert np.linalg.norm(out - ref) <= 1.03 * rounding, np.linalg.norm(out - ref) / rounding


@pytest.mark.parametrize("dtype,ratio", [(torch.float16, 1.03), (torch.bfloat16, 1.03)])
def test_long_sums_have_no_drift(dtype, ratio):
    """524288 keys of one CTA (more sequences than CTAs find room, which share their pages), nearly equal weights: the
    sum's own error stays far below the output's rounding, as above."""
    qmm = lib()
    B, L, D, page, scale = 460, 1 << 19, 32, 256, 0.05
    small = R.random_cache(L // page, 1, page, D, np.random.default_rng(5))
    small[..., -4 * D:] = np.abs(small[..., -4 * D:].view(np.float16)).view(np.uint8)
    K, V = (torch.tensor(x.transpose(1, 0, 2, 3).reshape(L, D), device=DEV) for x in R.cache_values(small, D))
    q = torch.randn(B, 1, D, device=DEV, generator=torch.Generator(DEV).manual_seed(1)).to(dtype)
    out = torch.empty_like(q)
    pages = torch.arange(L // page, dtype=torch.int32, device=DEV)[None].repeat(B, 1)
    qmm.qmm_attn_q4_0(qmm.attn_op(qmm.kv_cache(torch.tensor(small, device=DEV), page), q, pages,
                                  torch.full((B,), L, dtype=torch.int32, device=DEV), out, max_kv=L, scale=scale))
    ref = torch.softmax(scale * (q.double()[:, 0] @ K.T), -1) @ V
    rounding = (ref.to(dtype).double() - ref).norm().item()
    err = (out.double()[:, 0] - ref).norm().item()
    assert err <= ratio * rounding, err / rounding
    assert qmm.qmm_last_device_error() == 0
