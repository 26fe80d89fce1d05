"""qmm_lora's fp32 outputs against 64 bits on average (bounds and what they tell apart: lora_precision and
test_lora_precision_bounds)."""
import itertools

import pytest
import torch

import lora_precision as P
from parity import lib

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"f32": P.F32, "f16": P.F16, "bf16": P.BF16}


@pytest.mark.parametrize("x,w", list(itertools.product(TYPES, TYPES)))
@pytest.mark.parametrize("rank", [16, 64, 256])
@pytest.mark.parametrize("T,K,N", [(70, 512, 256), (3, 2048, 520), (200, 512, 131)])
def test_fp32_outputs_on_average(x, w, rank, T, K, N):
    qmm = lib()
    xs, a, b = P.inputs(T, N, K, rank, TYPES[x], TYPES[w], rank + T)
    y = torch.zeros(T, N, device=DEV)
    start = torch.tensor([0, T], dtype=torch.int32, device=DEV)
    qmm.qmm_lora(qmm.lora_op(xs.to(DEV), a.to(DEV), b.to(DEV), y, torch.zeros(1, dtype=torch.int32, device=DEV),
                             seg_start=start))
    got, bound = P.rms(y.cpu(), P.exact(xs, a, b)), P.bound(TYPES[x], TYPES[w], K, rank)
    assert got <= bound, (got, bound, got / bound)
    assert qmm.qmm_last_device_error() == 0
