"""qmm_attn_q4_0 where max_kv is a capacity far beyond what is cached: more counts than 31 bits hold."""
import numpy as np
import pytest
import torch

import attn_reference as R
from parity import lib

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_many_sequences_of_a_large_capacity(dtype):
    """1100 sequences of up to 70 tokens that share one page of 2^20, each allowed to grow to 2^28."""
    qmm = lib()
    B, D, page, max_kv = 1100, 32, 1 << 20, 1 << 28
    rng = np.random.default_rng(4)
    small = R.random_cache(1, 1, 96, D, rng)
    data = torch.zeros(1, 1, page // 32, 36 * D, dtype=torch.uint8, device=DEV)
    data[:, :, :3] = torch.tensor(small, device=DEV)
    lens = rng.integers(0, 71, B)
    q = torch.randn(B, 2, D, device=DEV, dtype=torch.float32, generator=torch.Generator(DEV).manual_seed(1)).to(dtype)
    out = torch.full_like(q, float("nan"))
    pages = torch.full((B, max_kv // page), -9, dtype=torch.int32, device=DEV)
    pages[:, 0] = 0
    op = qmm.attn_op(qmm.kv_cache(data, page), q, pages, torch.tensor(lens, dtype=torch.int32, device=DEV), out, max_kv=max_kv)
    assert qmm.qmm_debug_attn_plan(op)[1] == qmm.ATTN_WHOLE
    qmm.qmm_attn_q4_0(op)
    assert qmm.qmm_last_device_error() == 0
    K, V = (x[0] for x in R.cache_values(small, D))
    got, qn = out.double().cpu().numpy(), q.double().cpu().numpy()
    ref = np.concatenate([R.attention(qn[b:b + 1], K, V, int(L), D ** -0.5, True, 0)[0] for b, L in enumerate(lens)])
    assert (got[lens == 0] == 0).all()
    half = torch.finfo(dtype).eps / 2 if dtype != torch.float32 else 0.0
    err = np.linalg.norm(got - ref) / np.linalg.norm(ref)
    assert err <= half + (2.0 ** -18 if dtype == torch.float32 else 2.0 ** -11), err
