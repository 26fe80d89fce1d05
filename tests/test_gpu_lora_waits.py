"""Every wait of qmm_lora's kernels is bounded: one that runs out sets the
error word, the launch ends, and the context stays usable."""
import pytest
import torch

from parity import lib
from test_gpu_lora import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("x,w,rank,rows", [("f32", "f16", 8, 1), ("bf16", "bf16", 64, 70), ("f32", "f32", 200, 33)])
def test_a_wait_that_runs_out(x, w, rank, rows):
    qmm = lib()
    assert qmm.qmm_last_device_error() == 0
    c = Case(2 * rows, 2000, 1024, rank, [(0, rows, 0), (rows, 2 * rows, 1)], x, w)
    previous = qmm.qmm_debug_stream_wait(2_000_000, True)
    try:
        c.qmm.qmm_lora(c.op())
        assert qmm.qmm_last_device_error() == 6
    finally:
        qmm.qmm_debug_stream_wait(previous, False)
    c.buf.fill_(-7)
    c.check()
    torch.cuda.synchronize()
