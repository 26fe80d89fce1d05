"""The ramp of the rotary table against the turns that its ends are defined by."""
import math

import numpy as np
import pytest

from parity import lib

pytestmark = pytest.mark.gpu


def _ends(n_rot, base, orig, fast, slow):
    """The ramp's ends: the pair index (a real number) whose frequency makes `fast` and `slow` turns over orig
    positions, found by bisection, then the whole numbers around them within the head's values 0 .. n_rot - 1."""
    def at(turns):
        lo, hi = -1e6, 1e6
        for _ in range(200):
            mid = (lo + hi) / 2
            if math.log(orig / (2 * math.pi)) - 2 * mid / n_rot * math.log(base) > math.log(turns):
                lo = mid
            else:
                hi = mid
        return lo
    return max(math.floor(at(fast)), 0), min(math.ceil(at(slow)), n_rot - 1)


@pytest.mark.parametrize("n_rot,base,orig,factor", [
    (128, 1e4, 131072.0, 4.0),   # the slow end is past the last pair: 70 of 64 pairs
    (64, 1e4, 65536.0, 8.0),     # and here
    (128, 1e4, 4096.0, 16.0), (32, 1e4, 32768.0, 2.0), (8, 1e4, 1e6, 4.0), (64, 1e6, 8192.0, 4.0), (2, 1e4, 4096.0, 4.0)])
def test_ramp(n_rot, base, orig, factor):
    qmm = lib()
    n_pos = 5000
    got = qmm.rope_table(n_pos, n_rot, base, qmm.ROPE_RAMP, factor, orig).cpu().numpy().astype(np.float64)
    lo, hi = _ends(n_rot, base, orig, 32.0, 1.0)
    m = 0.1 * math.log(factor) + 1
    for i in range(n_rot // 2):
        f = base ** (-2.0 * i / n_rot)
        share = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))  # of the slowed frequency
        f = (1 - share) * f + share * f / factor
        p = np.arange(n_pos)
        ref = m * np.stack([np.cos(p * f), np.sin(p * f)], -1)
        assert (np.abs(got[:, i] - ref) <= 2.0 ** -24 * np.abs(ref) + 1e-9).all(), (i, lo, hi)
    if (n_rot, orig) == (128, 131072.0):
        assert (lo, hi) == (45, 70)
        slowest = np.arctan2(got[1, -1, 1], got[1, -1, 0]) / base ** (-126 / 128)
        assert abs(slowest - 0.46) < 1e-3  # 1 - 18/25 of it as it was, 18/25 at a quarter
