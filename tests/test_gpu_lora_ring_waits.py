"""qmm_lora when waits run out long before the end of its ring, without a GPU fault: no copy from the middle one on is
told of, so that slots are passed many times after the first wait has run out.  The call returns, the error word reads
QMM_ERR_TIMEOUT once, and the next call gives the bits of the one before."""
import time

import pytest
import torch

from parity import lib
from test_gpu_lora import Case

pytestmark = pytest.mark.gpu
TIMEOUT = 6  # QMM_ERR_TIMEOUT


# (few columns and a small K: the whole ring is filled by the warps that multiply, and waited for by none)
@pytest.mark.parametrize("T,N,K,rank,x,w", [
    (1, 64, 16384, 16, "f32", "f16"), (64, 64, 8192, 64, "bf16", "bf16"), (200, 40, 8192, 256, "f32", "f32"),  # in K
    (64, 20000, 64, 64, "bf16", "bf16"), (300, 8191, 32, 16, "f16", "f16"), (1, 28672, 96, 100, "f32", "bf16"),  # in N
    (300, 5000, 4096, 24, "bf16", "f16"), (3, 8, 32, 8, "f32", "f32"), (40, 64, 256, 33, "f16", "f16"),
    (60, 32, 64, 64, "f32", "bf16"), (64, 8, 32, 128, "f32", "f32"), (1, 16, 128, 16, "bf16", "bf16"), (17, 33, 64, 7, "f16", "f32")])
def test_waits_that_run_out_early(T, N, K, rank, x, w):
    qmm = lib()
    assert qmm.qmm_last_device_error() == 0
    c = Case(T, N, K, rank, [(0, T // 3, 0), (T // 3, T, 1)], x, w)
    want = c.check()
    op = c.op()
    previous = qmm.qmm_debug_stream_wait(1_000_000, True)
    try:
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        qmm.qmm_lora(op)
        assert qmm.qmm_last_device_error() == TIMEOUT
        assert time.perf_counter() - t0 < 1.0
        assert qmm.qmm_last_device_error() == 0
    finally:
        qmm.qmm_debug_stream_wait(previous, False)
    c.y.fill_(-7)
    qmm.qmm_lora(op)
    assert qmm.qmm_last_device_error() == 0
    assert torch.equal(c.y, want)
