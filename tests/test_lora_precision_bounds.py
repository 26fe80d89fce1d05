"""The bounds of lora_precision tell a kernel that leaves out a part of its operands, or leaves its sums in the tensor
core, from one that does not: both emulated in 64 bits."""
import pytest
import torch

import lora_precision as P

F32, F16, BF16 = P.F32, P.F16, P.BF16


def _parts(v, n, bits):
    """The first n parts of 64-bit values, each of `bits` bits."""
    out, rest = torch.zeros_like(v), v.clone()
    for _ in range(n):
        m, e = torch.frexp(rest)
        p = torch.ldexp(torch.round(torch.ldexp(m, torch.tensor(bits))), e - bits)
        out, rest = out + p, rest - p
    return out


def _truncated(v):
    """To 24 bits, towards zero."""
    m, e = torch.frexp(v)
    return torch.ldexp(torch.trunc(torch.ldexp(m, torch.tensor(24))), e - 24)


def _sum(x, w, k, leave):
    """x [T][K] times w [N][K], k products a step; sums leave after `leave` products for exact additions."""
    total = torch.zeros(x.shape[0], w.shape[0], dtype=torch.float64)
    for at in range(0, x.shape[1], leave):
        acc = torch.zeros_like(total)
        end = min(at + leave, x.shape[1])
        for s in range(at, end, k):
            e = min(s + k, end)
            acc = _truncated(acc + x[:, s:e] @ w[:, s:e].T)
        total += acc
    return total


CASES = [(x, w, rank) for x in (F32, F16, BF16) for w in (F32, F16, BF16) for rank in (16, 64, 256)]


def _emulate(x, w, rank, x_parts=None, h_parts=None, w_parts=None, leave=16):
    K, (first, second) = 512, P.steps(x, w, rank)
    xs, a, b = P.inputs(24, 48, K, rank, x, w, rank)
    bits = 8 if w == BF16 else 11
    full = 3 if w == BF16 else 2
    cut = lambda v, n: _parts(v, n or full, bits)  # noqa: E731
    xd = cut(xs.double(), x_parts) if x == F32 else xs.double()
    ad, bd = (cut(v[0].double(), w_parts) if w == F32 else v[0].double() for v in (a, b))
    # as many steps as the kernel has: a step for each part
    h = _sum(xd, ad, max(1, 64 // first), 64).float().double()
    h = cut(h, h_parts)
    y = _sum(h, bd, max(1, 16 // (second // (min(16, rank) // 16))), leave)
    return P.rms(y.float(), P.exact(xs, a, b)), P.bound(x, w, K, rank)


@pytest.mark.parametrize("x,w,rank", CASES)
def test_whole_operands_are_within_the_bounds(x, w, rank):
    got, bound = _emulate(x, w, rank)
    assert got <= bound, (got, bound)


@pytest.mark.parametrize("x,w,rank", CASES)
def test_a_part_fewer_is_not(x, w, rank):
    fewer = 2 if w == BF16 else 1
    for kw in ({"h_parts": fewer}, {"x_parts": fewer} if x == F32 else {}, {"w_parts": 1} if w == F32 else {}):
        if kw:
            got, bound = _emulate(x, w, rank, **kw)
            assert got > bound, (kw, got, bound)


@pytest.mark.parametrize("x,w", [(x, w) for x in (F32, F16, BF16) for w in (F32, F16, BF16)])
def test_sums_of_256_ranks_left_in_the_tensor_core_are_not(x, w):
    got, bound = _emulate(x, w, 256, leave=256)
    assert got > bound, (got, bound)
