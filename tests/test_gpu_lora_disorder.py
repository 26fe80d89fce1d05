"""qmm_lora with segment starts that are out of order or range: each counts as the largest of those up to it, brought
into [0, T].  No row is in two segments, rows in none and behind the last stay, and the error word is set."""
import itertools
import random

import pytest
import torch

from parity import lib
import lora_reference as R
from test_gpu_lora import Case

pytestmark = pytest.mark.gpu
DEV = "cuda"
BAD_INDEX = 10


def _run(T, N, K, rank, starts, x="f32", w="f16", adapters=3, seed=1, ypad=0):
    qmm = lib()
    assert qmm.qmm_last_device_error() == 0
    top = list(itertools.accumulate((min(max(s, 0), T) for s in starts), max))
    n = len(starts) - 1
    segs = [(top[i], top[i + 1], (i * 7 + i // 3) % (adapters + 1) - 1) for i in range(n)]
    c = Case(T, N, K, rank, segs, x, w, adapters=adapters, seed=seed, ypad=ypad)
    i32 = dict(dtype=torch.int32, device=DEV)
    start, adapter = torch.tensor(starts, **i32), torch.tensor([s[2] for s in segs], **i32)
    want, err = c.want()
    none = want.isnan().to(DEV)
    for in_place in (False, True):
        # rows of the same storage behind the last
        buf = torch.full((T + 70, N + ypad), -7.0, dtype=c.y.dtype, device=DEV)
        y = buf[:T, :N]
        if in_place:
            y.copy_(c.base)
        op = qmm.lora_op(c.x, c.a, c.b, y, adapter, base=y if in_place else c.base, seg_start=start, scales=c.scales)
        qmm.qmm_lora(op)
        assert qmm.qmm_last_device_error() == BAD_INDEX
        R.check(y, want, err)
        assert torch.equal(y[none], c.base[none]) if in_place else (y[none] == -7).all()
        assert (buf[T:] == -7).all() and (buf[:, N:] == -7).all()


@pytest.mark.parametrize("starts", [[0, 10, 5, 20], [5, 0, 20, 20], [0, 20, 0, 20], [20, 0, 10, 15], [3, 25, -4, 12],
                                    [-5, -1, 30, 2 ** 31 - 1], [-2 ** 31, 7, 6, 5, 4, 19]])
@pytest.mark.parametrize("x,w", [("f32", "f16"), ("bf16", "bf16")])
def test_few_segments(starts, x, w):
    _run(20, 70, 128, 16, starts, x, w, ypad=2)


@pytest.mark.parametrize("n", [6, 255, 256, 257, 300, 700, 1500])
def test_many_segments(n):
    """Starts to and fro, in one look and in several: more tiles than rows, if each segment were taken by itself."""
    T = 900
    _run(T, 40, 64, 8, [T * (i & 1) for i in range(n + 1)])
    r = random.Random(n)
    _run(T, 40, 64, 24, [r.randrange(-3, T + 3) for _ in range(n + 1)], "bf16", "bf16")
    rise = sorted(r.randrange(T + 1) for _ in range(n + 1))  # one early, one late start out of order
    for at in {1, n // 2, n - 1}:
        s = list(rise)
        s[at] = rise[min(n, at + n // 4 + 1)] + 1
        s[n] = max(s[n], 1) - 1
        _run(T, 40, 64, 8, s)


def test_tiles_that_pass_23_bits():
    """200 segments of all of five million rows."""
    T = 5_000_000 + 13
    _run(T, 8, 32, 4, [T * (i & 1) for i in range(201)], "f16", "f16")
