"""The bounded waits of the attention kernels, without a GPU fault: with
qmm_debug_stream_wait the bound is 1 ms and every warp that copies holds back
its last copy, so that waits run out.  The call returns, the device error word
reads QMM_ERR_TIMEOUT once, and the next call gives the bits of the one before."""
import time

import pytest
import torch

from parity import lib
from test_gpu_attn import DEV, MAY_GROW, Case

pytestmark = pytest.mark.gpu
TIMEOUT = 6  # QMM_ERR_TIMEOUT


def _run_out_and_recover(c, **kw):
    qmm = c.qmm
    want = c.run(**kw)
    c.check(want)
    prev = qmm.qmm_debug_stream_wait(1_000_000, withhold_last_copy=True)
    try:
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        c.run(**kw)
        assert qmm.qmm_last_device_error() == TIMEOUT
        assert time.perf_counter() - t0 < 1.0
        assert qmm.qmm_last_device_error() == 0  # read once, then clear
    finally:
        qmm.qmm_debug_stream_wait(prev, withhold_last_copy=False)
    out = c.run(**kw)
    assert qmm.qmm_last_device_error() == 0
    assert torch.equal(out, want)


@pytest.mark.parametrize("lens,n,Hq,Hkv,D,dtype", [
    ([100, 33], 1, 4, 2, 64, "f32"),                 # whole items: a record a warp, some warps with none
    ([1000] * 3, 2, 4, 1, 128, "bf16"),              # on clusters
    ([4096], 1, 8, 1, 96, "f32"), ([30000], 1, 8, 1, 64, "f16"),
    ([20000, 9001, 1, 0], 1, 4, 2, 64, "f32"),       # cut over the CTAs
    ([3000, 2500], 17, 8, 2, 256, "f32"),
    ([700] * 300, 2, 2, 1, 32, "f32"),
])
def test_warp_mma_kernel(lens, n, Hq, Hkv, D, dtype):
    qmm = lib()
    assert qmm.qmm_last_device_error() == 0
    _run_out_and_recover(Case(qmm, lens, [n] * len(lens), Hq, Hkv, D, 64, dtype, seed=D))


@pytest.mark.parametrize("D", [32, 128])
@pytest.mark.parametrize("many", [13, 14])
def test_tensor_memory_kernel(D, many):
    """Whole items, one or two a CTA, of 0 to 3 steps; two tiles and one."""
    qmm = lib()
    assert qmm.qmm_last_device_error() == 0
    c = Case(qmm, [0, 3, 129, 300, 70] * many, [130, 64, 128, 40, 70] * many, 4, 2, D, 96, "bf16", seed=D, q_start=True)
    _run_out_and_recover(c)


@pytest.mark.parametrize("lens,nqs,D", [([200], [64], 64), ([2000, 40, 1500], [64] * 3, 128), ([3, 700, 0, 257], [130, 40, 64, 1], 32)])
@pytest.mark.parametrize("left", [(0, 2 ** 31 - 1), (-2 ** 31, 2 ** 31 - 1), (1 << 20, 1 << 21), (2, 40)])
def test_cut_items_of_the_tensor_memory_kernel(lens, nqs, D, left):
    """An aborted CTA leaves the places unwritten that say which parts make an item; whatever was in the workspace,
    nothing outside it is read."""
    qmm = lib()
    assert qmm.qmm_last_device_error() == 0
    c = Case(qmm, lens, nqs, 4, 2, D, 96, "bf16", seed=D, q_start=True, extra_kv=MAY_GROW // 96)
    want = c.run(max_kv=MAY_GROW)
    c.check(want)
    out = torch.empty_like(want)
    op = c.op(out, max_kv=MAY_GROW)
    words = op._keep[-1].view(torch.int32)
    words.copy_(torch.tensor([left[0], left[1], 1, 0], dtype=torch.int32, device=DEV).repeat(words.numel() // 4))
    prev = qmm.qmm_debug_stream_wait(1_000_000, withhold_last_copy=True)
    try:
        qmm.qmm_attn_q4_0(op)
        assert qmm.qmm_last_device_error() == TIMEOUT
    finally:
        qmm.qmm_debug_stream_wait(prev, withhold_last_copy=False)
    qmm.qmm_attn_q4_0(op)
    assert qmm.qmm_last_device_error() == 0
    assert torch.equal(out, want)
