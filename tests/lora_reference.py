"""Low-rank adapters in 64 bits, from their definition, and how far the kernel's results may be from it."""
import torch

HALF_STEP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
SMALLEST = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -133}


def lora(x, a, b, segments, base=None, ranks=None, scales=None, y_dtype=torch.float32):
    """(y, what its roundings may add up to before the last), 64 bits [T][N]; segments [(first, last + 1, adapter)].
    Rows in no segment are NaN.

    In units of the sums of magnitudes.  First product, of sum |x a|: what is lost of fp32 operands, 2^-23 each, and
    with two of them the lower parts' product 2^-22; a chunk's MMAs, up to 12, each truncating the sum of its terms
    and of what came before (2^-22 of it, taken generously), with x and A of one 16-bit type all K / 16 of them; K /
    32 chunks and at most 8 parts of 16 CTAs added in fp32, 2^-24 each.  Then h as the second product reads it: 2^-23,
    or 2^-18 with bf16 adapters and 16-bit y; its scaling 2^-24.  Second product, of sum |h b|: 2^-23 and 2^-22 for
    fp32 adapters, its MMAs (up to three for 8 ranks) 2^-22 each; the base's addition 2^-24 of the result."""
    T, K = x.shape
    n, R, _ = a.shape
    N = b.shape[1]
    x64, a64, b64 = x.double().cpu(), a.double().cpu(), b.double().cpu()
    y = torch.full((T, N), float("nan"), dtype=torch.float64)
    err = torch.zeros(T, N, dtype=torch.float64)
    f32 = (x.dtype == torch.float32) + (a.dtype == torch.float32)
    first = f32 * 2.0 ** -23 + (f32 == 2) * 2.0 ** -22 + 12 * 2.0 ** -22 + (K / 32 + 128) * 2.0 ** -24
    if f32 == 0 and x.dtype == a.dtype:
        first += K / 16 * 2.0 ** -22
    bf16 = a.dtype == torch.bfloat16 and y_dtype != torch.float32
    second = ((a.dtype == torch.float32) * 1.5 * 2.0 ** -22 + (3 * (R // 8 + 4)) * 2.0 ** -22 + 2.0 ** -24
              + (2.0 ** -18 if bf16 else 2.0 ** -23))
    for lo, hi, i in segments:
        if hi <= lo:
            continue
        r = 0 if i < 0 else R if ranks is None else ranks[i]
        s = 1.0 if scales is None or i < 0 else float(scales[i])
        A, B = a64[max(i, 0), :r], b64[max(i, 0), :, :r]
        h = x64[lo:hi] @ A.T
        y[lo:hi] = s * (h @ B.T)
        err[lo:hi] = abs(s) * (first * (x64[lo:hi].abs() @ A.abs().T) + second * h.abs()) @ B.abs().T
        if base is not None:
            y[lo:hi] += base[lo:hi].double().cpu()
    return y, err + 2.0 ** -24 * y.abs().nan_to_num(0.0)


def check(got, want, err, where=None):
    """got within the error and one rounding to its type (or to its smallest step)."""
    h = HALF_STEP[got.dtype]
    tol = err + h * (want.abs() + err) + SMALLEST[got.dtype]
    off = (got.double().cpu() - want).abs()
    keep = ~want.isnan()
    assert torch.isfinite(got.cpu()[keep]).all()
    bad = keep & ~(off <= tol)
    assert not bad.any(), (bad.nonzero()[:5].tolist(), (off / tol)[keep].max().item())
