"""qmm_lora with the longest rows that it takes, N = 2^28: a tile's 16-byte parts pass 31 bits."""
import pytest
import torch

from parity import lib

pytestmark = pytest.mark.gpu
DEV = "cuda"


def test_rows_of_no_adapter_and_of_one():
    qmm = lib()
    T, N, K, rank = 116, 1 << 28, 64, 4
    if torch.cuda.mem_get_info()[0] + torch.cuda.memory_reserved() - torch.cuda.memory_allocated() < 140 << 30:
        pytest.skip("needs 140 GB")
    torch.cuda.empty_cache()
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn(T, K, generator=g, device=DEV)
    a = torch.randn(1, rank, K, generator=g, device=DEV).half()
    b = torch.empty(1, N, rank, dtype=torch.float16, device=DEV)
    b.normal_(generator=g)
    y = torch.full((T, N), 7.0, device=DEV)
    # empty segments make the launch's estimate of its tiles, and with it each CTA's columns, the largest
    cuts = [0, 64, 115] + [115] * 123
    start = torch.tensor(cuts, dtype=torch.int32, device=DEV)
    adapter = torch.tensor([-1, 0] + [0] * (len(cuts) - 3), dtype=torch.int32, device=DEV)
    qmm.qmm_lora(qmm.lora_op(x, a, b, y, adapter, seg_start=start))
    assert qmm.qmm_last_device_error() == 0
    for t in range(64):
        assert not y[t].any(), t
    assert (y[115] == 7).all()  # in no segment
    h = x.double() @ a[0].double().T
    for at in (0, N // 2 - 2048, N - 4096):  # fp32 sums of 64 and of 4 terms of magnitudes up to 50
        want = h[64:115] @ b[0, at:at + 4096].double().T
        mag = (x[64:115].double().abs() @ a[0].double().abs().T) @ b[0, at:at + 4096].double().abs().T
        assert ((y[64:115, at:at + 4096].double() - want).abs() <= 2.0 ** -19 * mag).all()
    del x, a, b, y
    torch.cuda.empty_cache()
