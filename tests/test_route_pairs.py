"""The pair arithmetic of routing (scores as sums of two fp32 numbers), compiled for the host, against exact fractions
and 60-digit decimals."""
import ctypes
import os
import random
import shutil
import subprocess
from decimal import Decimal, getcontext
from fractions import Fraction

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_quantized_int4_gb300", "csrc")
SOURCE = r"""
#include "qmm_route_pair.cuh"
using namespace qmm::route;
extern "C" {
void t_sum(float a, float b, float* o) { Pair p = two_sum(a, b); o[0] = p.hi, o[1] = p.lo; }
void t_add(const float* a, const float* b, float* o) { Pair p = add(Pair{a[0], a[1]}, Pair{b[0], b[1]}); o[0] = p.hi, o[1] = p.lo; }
void t_mul(const float* a, const float* b, float* o) { Pair p = mul(Pair{a[0], a[1]}, Pair{b[0], b[1]}); o[0] = p.hi, o[1] = p.lo; }
void t_exp(const float* a, float* o) { Pair p = exp_pair(Pair{a[0], a[1]}); o[0] = p.hi, o[1] = p.lo; }
void t_inv(const float* a, float* o) { Pair p = reciprocal(Pair{a[0], a[1]}); o[0] = p.hi, o[1] = p.lo; }
void t_sigmoid(float a, float* o) { Pair p = sigmoid_pair(a); o[0] = p.hi, o[1] = p.lo; }
int t_unsure(const float* a, const float* b, float t) { return unsure(Pair{a[0], a[1]}, Pair{b[0], b[1]}, t); }
int t_before(const float* a, const float* b) { return before(Pair{a[0], a[1]}, Pair{b[0], b[1]}); }
}
"""


@pytest.fixture(scope="module")
def pairs(tmp_path_factory):
    cxx = shutil.which("g++")
    if not cxx:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("pairs")
    (d / "pairs.cpp").write_text(SOURCE)
    # a product and a sum stay two roundings, as on the device
    subprocess.run([cxx, "-O2", "-std=c++17", "-ffp-contract=off", "-shared", "-fPIC", "-x", "c++", "-I" + CSRC,
                    str(d / "pairs.cpp"), "-o", str(d / "pairs.so")], check=True)
    getcontext().prec = 60
    return ctypes.CDLL(str(d / "pairs.so"))


def _pair(*v):
    return (ctypes.c_float * 2)(*v)


def _of(lib, name, *args):
    o = _pair(0, 0)
    getattr(lib, name)(*[ctypes.c_float(a) if isinstance(a, float) else a for a in args], o)
    return o


def _exact(p):
    return Fraction(p[0]) + Fraction(p[1])


def _decimal(f):
    return Decimal(f.numerator) / Decimal(f.denominator)


def _value(r, lo=-20, hi=20):
    return float(np.float32(r.choice([-1, 1]) * r.uniform(1, 2) * 2.0 ** r.randint(lo, hi)))


def _random_pair(r, lo=-20, hi=20):
    v = _value(r, lo, hi)
    return _pair(v, float(np.float32(v * r.uniform(-1, 1) * 2.0 ** -25)))


def test_sums_and_products(pairs):
    """A sum of two numbers is exact.  Sums of pairs lose less than 2^-44 of the operands' magnitudes (the bounds of
    the method are 3 * 2^-48 of them), products 2^-44 of the result (7 * 2^-48)."""
    r = random.Random(1)
    for _ in range(4000):
        a, b = _value(r), _value(r)
        assert _exact(_of(pairs, "t_sum", a, b)) == Fraction(a) + Fraction(b)
        p, q = _random_pair(r), _random_pair(r)
        s, m = _exact(_of(pairs, "t_add", p, q)), _exact(_of(pairs, "t_mul", p, q))
        x, y = _exact(p), _exact(q)
        assert abs(s - (x + y)) <= Fraction(1, 2 ** 44) * (abs(x) + abs(y))
        assert abs(m - x * y) <= Fraction(1, 2 ** 44) * abs(x * y)


def test_scores(pairs):
    """Exponentials and reciprocals to 2^-42 of the result, sigmoids to 2^-42; the lowest parts of results below
    2^-100 may be lost."""
    r = random.Random(2)
    for i in range(4000):
        x = r.uniform(-87, 87) if i % 2 else r.uniform(-2, 2)
        p = _pair(float(np.float32(x)), float(np.float32(x * r.uniform(-1, 1) * 2.0 ** -25)))
        want = _decimal(_exact(p)).exp()
        got = _decimal(_exact(_of(pairs, "t_exp", p)))
        assert abs(got - want) <= want * Decimal(2) ** -42 + Decimal(2) ** -149, x
        p = _random_pair(r, -60, 60)
        want = 1 / _decimal(_exact(p))
        assert abs(_decimal(_exact(_of(pairs, "t_inv", p))) - want) <= abs(want) * Decimal(2) ** -42
        l = float(np.float32(r.uniform(-120, 120) if i % 2 else r.uniform(-20, 20)))
        want = 1 / (1 + Decimal(-l).exp())
        assert abs(_decimal(_exact(_of(pairs, "t_sigmoid", l))) - want) <= Decimal(2) ** -42, l


def test_order(pairs):
    """Values within the tolerance are in doubt; one that takes no part never is, though its tolerance is infinite."""
    inf = float("inf")
    one, near, off = _pair(1.0, 0.0), _pair(1.0, 2.0 ** -45), _pair(-inf, 0.0)
    assert pairs.t_unsure(one, near, ctypes.c_float(2.0 ** -39)) == 1
    assert pairs.t_unsure(one, near, ctypes.c_float(2.0 ** -46)) == 0
    assert pairs.t_before(near, one) == 1 and pairs.t_before(one, near) == 0
    for t in (2.0 ** -39, inf):
        for a, b in ((one, off), (off, one), (off, off)):
            assert pairs.t_unsure(a, b, ctypes.c_float(t)) == 0
    assert pairs.t_before(one, off) == 1 and pairs.t_before(off, off) == 0
