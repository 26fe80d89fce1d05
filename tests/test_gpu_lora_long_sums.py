"""qmm_lora's first product over many columns: sums of terms of one sign, which a truncating sum makes smaller."""
import pytest
import torch

from parity import lib

pytestmark = pytest.mark.gpu
DEV = "cuda"
HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("y_dtype", ["same", torch.float32])
@pytest.mark.parametrize("rows", [1, 40])
def test_sums_of_one_sign(dtype, y_dtype, rows):
    """What the sum may be off by, relative: a chunk's 64 products leave the tensor core after four steps, each of
    which truncates below 2^-23 of the chunk's sum; the K / 64 additions in fp32 round to nearest, independently:
    2^-24 times the root of their number, and eight times that for all values of the test.  A x is then cut to 2^-18
    (bf16 adapters and 16-bit y) or 2^-23, its two or three parts truncate twice (2^-23 each), and y is rounded."""
    y_dtype = dtype if y_dtype == "same" else y_dtype
    K, N = 1 << 23, 8
    g = torch.Generator(device=DEV).manual_seed(rows)
    x = (0.5 + torch.rand(rows, K, generator=g, device=DEV)).to(dtype)
    a = ((0.5 + torch.rand(1, 1, K, generator=g, device=DEV)) * 2.0 ** -11).to(dtype)
    b = torch.ones(1, N, 1, dtype=dtype, device=DEV)
    y = torch.zeros(rows, N, dtype=y_dtype, device=DEV)
    start = torch.tensor([0, rows], dtype=torch.int32, device=DEV)
    qmm = lib()
    qmm.qmm_lora(qmm.lora_op(x, a, b, y, torch.zeros(1, dtype=torch.int32, device=DEV), seg_start=start))
    want = torch.stack([(x[i].double() * a[0, 0].double()).sum() for i in range(rows)])[:, None]
    rel = 4 * 2.0 ** -23 + 8 * (K / 64) ** 0.5 * 2.0 ** -24 + 3 * 2.0 ** -23
    rel += 2.0 ** -18 if dtype == torch.bfloat16 and y_dtype == dtype else 2.0 ** -23
    rel += HALF_STEP[y_dtype]
    off = ((y.double() - want).abs() / want).max().item()
    assert off <= rel, (off, rel)
    assert qmm.qmm_last_device_error() == 0
