"""qmm_moe_route with biases as large as fp32 holds (a program may switch experts off by its lowest value): sums of two
pass fp32, but not the 64 bits that decide."""
import pytest
import torch

from test_gpu_route import DEV, _bias, _check, _logits, lib

pytestmark = pytest.mark.gpu
LOWEST = torch.finfo(torch.float32).min


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("top2", [False, True])
def test_lowest_values(score, dtype, top2):
    qmm = lib()
    E, G, k = 64, 8, 6
    for T, masked in ((70, 0.0), (70, 0.6)):
        l = _logits(T, E, dtype, T, masked=masked)
        # whole groups switched off by -inf logits before groups switched off by biases
        l[::3, 0:16] = float("-inf")
        l[1::3, 24:31] = float("-inf")  # one is left of its group
        for off in (range(16, 64), range(8, 64), range(0, 64), range(0, 64, 2)):
            b = _bias(E, 3)
            b[list(off)] = LOWEST
            for top in (1, 2, 3, 5, 8):
                if k <= top * E // G:
                    _check(qmm, l, k, score, b, n_groups=G, top_groups=top, top2=top2)
        # different ones, whose sums pass fp32, and large positive ones
        b = _bias(E, 4)
        b[8:16], b[16:24], b[24:32] = LOWEST, 0.75 * LOWEST, 0.9 * LOWEST
        b[32:40], b[40:48], b[48:56] = -LOWEST, -0.75 * LOWEST, -0.9 * LOWEST
        for top in (1, 2, 4, 6, 7):
            _check(qmm, l, k, score, b, n_groups=G, top_groups=top, top2=top2)
        _check(qmm, l, k, score, b)
        # all of them large
        b = (0.6 + 0.4 * torch.rand(E, generator=torch.Generator().manual_seed(5))).to(DEV) * LOWEST
        for top in (1, 3, 7):
            _check(qmm, l, k, score, b, n_groups=G, top_groups=top, top2=top2)
            _check(qmm, l, k, score, -b, n_groups=G, top_groups=top, top2=top2)
