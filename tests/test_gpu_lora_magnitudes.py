"""qmm_lora with very small and very large values: cut operands lose up to 2^-133 of a value where that is more than
2^-23 of it, and nothing else changes."""
import pytest
import torch

import lora_reference as R
from parity import lib

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# log2 of the magnitudes of x, A and B
@pytest.mark.parametrize("x,w,xs,ws,bs", [
    ("f32", "f32", -118, 60, 40), ("f32", "f32", -128, 60, 40), ("f32", "f32", 60, -118, 40), ("f32", "f32", 0, -130, 100),
    ("f32", "f32", 90, -100, 20), ("f32", "f32", 118, -100, -30), ("f32", "f32", 0, 30, -120),
    ("f32", "bf16", -118, 60, 40), ("f32", "bf16", -128, 60, 40), ("f32", "bf16", 60, -128, 40), ("f32", "bf16", 118, -100, -30),
    ("f32", "f16", -122, 10, 8), ("f32", "f16", 100, -20, -5), ("bf16", "bf16", -128, 60, 40), ("bf16", "bf16", 0, -130, 100),
    ("bf16", "f32", 60, -128, 40), ("bf16", "f16", -128, 10, 8), ("f16", "f16", -20, -10, 5), ("f16", "f16", 10, 3, -18)])
@pytest.mark.parametrize("rank", [5, 64])
def test_magnitudes(x, w, xs, ws, bs, rank):
    qmm = lib()
    T, N, K = 19, 72, 160
    g = torch.Generator().manual_seed(rank)
    rand = lambda s, *shape: torch.randn(*shape, generator=g, dtype=torch.float64) * 2.0 ** s  # noqa: E731
    X, A, B = rand(xs, T, K).to(TYPES[x]), rand(ws, 1, rank, K).to(TYPES[w]), rand(bs, 1, N, rank).to(TYPES[w])
    y = torch.zeros(T, N, device=DEV)
    start = torch.tensor([0, T], dtype=torch.int32, device=DEV)
    qmm.qmm_lora(qmm.lora_op(X.to(DEV), A.to(DEV), B.to(DEV), y, torch.zeros(1, dtype=torch.int32, device=DEV),
                             seg_start=start))
    want, err = R.lora(X, A, B, [(0, T, 0)], y_dtype=torch.float32)
    step = 2.0 ** -133
    one = lambda t: torch.ones_like(t.double())  # noqa: E731
    a, b, xd = A[0].double().abs(), B[0].double().abs(), X.double().abs()
    h = xd @ a.T
    if x == "f32":
        err = err + step * one(X) @ a.T @ b.T
    if w == "f32":
        err = err + step * (xd @ one(A[0]).T @ b.T + h @ one(B[0]).T)
    err = err + step * (one(h) @ b.T)
    R.check(y, want, err)
    assert qmm.qmm_last_device_error() == 0
