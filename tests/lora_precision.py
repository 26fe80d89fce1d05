"""How far qmm_lora's fp32 outputs are from 64 bits on average: root mean squares over all values of a call, where the
sums of magnitudes of lora_reference allow a single value many times as much."""
import torch

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def steps(x, w, rank, leave=16):
    """MMAs whose sums follow one another in the tensor core: over 64 columns of the first product (k 16 a step of one
    16-bit type, three parts of fp32 x with bf16 A; else k 8, an MMA for each product of parts but the lower ones'), and
    over `leave` ranks of the second."""
    if x == w and x != F32:
        first = 4
    elif x == F32 and w == BF16:
        first = 4 * 3
    else:
        first = 8 * (1 + (x == F32) + (w == F32))
    ranks = min(leave, -(-rank // 16) * 16)
    return first, ranks // 16 * (3 if w == BF16 else 6 if w == F32 else 4)


def bound(x, w, K, rank):
    """RMS of the error over the RMS of the result, no base, fp32 outputs.

    A step truncates the running sum: by half a unit of its last place on average, 0.72 * 2^-24 of it (mantissas
    evenly spread in their logarithm), and running sums of terms of any sign are 2/3 of the last one on average.  All
    of a sum's steps lose in the same direction, so they add up; half as much again for sums that are not average.
    Cut operands lose up to 2^-23 (fp32 x; fp32 A and B, each in its product; A x) or with two fp32 operands another
    2^-22, an even spread being 1 / sqrt(3) of that; three parts of bf16 lose 2^-24.  K / 64 chunks and up to 32 parts
    are added in fp32, and the result is rounded, 2^-25 each, independently."""
    first, second = steps(x, w, rank)
    lost = 1.5 * (first + second) * (2 / 3) * 0.72 * 2.0 ** -24
    part = 2.0 ** -24 if w == BF16 else 2.0 ** -23
    cut = ((x == F32) * part + (w == F32) * 2 * 2.0 ** -23 + (x == F32 and w == F32) * 2.0 ** -22 + part) / 3 ** 0.5
    return lost + cut + (K / 64 + 32 + 1) ** 0.5 * 2.0 ** -25


def rms(got, want):
    return ((got.double() - want).square().mean() / want.square().mean()).sqrt().item()


def inputs(T, N, K, rank, x, w, seed):
    g = torch.Generator().manual_seed(seed)
    xs = torch.randn(T, K, generator=g)
    xs[torch.rand(T, K, generator=g) < 0.01] *= 20
    a = torch.randn(1, rank, K, generator=g) * K ** -0.5
    b = torch.randn(1, N, rank, generator=g) * 0.05
    return xs.to(x), a.to(w), b.to(w)


def exact(xs, a, b):
    return (xs.double() @ a[0].double().T) @ b[0].double().T
