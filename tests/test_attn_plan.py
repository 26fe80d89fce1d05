"""Which kernel qmm_attn_q4_0 takes, and how items meet CTAs, for the calls of
tests/test_gpu_attn.py and for calls on both sides of each rule (no GPU needed:
the plan is made on the host, for 152 SMs)."""
import ctypes

import pytest

import test_gpu_attn as G

TYPES = {"f32": 0, "f16": 1, "bf16": 2}
ROWS_8, ROWS_16, TMEM = range(3)
WHOLE, CLUSTER, CUT = range(3)


@pytest.fixture(scope="module")
def plan():
    from block_quantized_int4_gb300 import _build
    _build.build()
    from block_quantized_int4_gb300 import qmm

    def plan(dtype, B, n, Hq, Hkv, D, kv, page=64, window=0):
        op = qmm.AttnOp(qmm.KvCache(None, 8, page, Hkv, D), qmm.Heads(None, Hq * D, D, Hq, TYPES[dtype]), qmm.Heads(), None,
                        None, None, None, None, -(-kv // page), B * n, B, n, kv, 1, window, D ** -0.5, None, 0)
        return qmm.qmm_debug_attn_plan(op)
    return plan


def _params(f):
    """The arguments of every call of a parametrised test, as dicts."""
    cases = [{}]
    for mark in f.pytestmark:
        if mark.name == "parametrize":
            names = [x.strip() for x in mark.args[0].split(",")]
            cases = [{**c, **dict(zip(names, v if len(names) > 1 else (v,)))} for c in cases for v in mark.args[1]]
    return cases


def test_refusals(plan):
    from block_quantized_int4_gb300 import qmm
    f = qmm.library_handle().qmm_debug_attn_plan
    k = ctypes.c_int()
    assert f(None, ctypes.byref(k), ctypes.byref(k)) == 1
    op = qmm.AttnOp()
    assert f(ctypes.byref(op), None, ctypes.byref(k)) == 1 and f(ctypes.byref(op), ctypes.byref(k), ctypes.byref(k)) == 1


def test_the_gpu_tests_reach_the_kernels_they_are_meant_for(plan):
    modes = set()
    for c in _params(G.test_many_rows_that_may_see_many_keys):
        kernel, mode = plan("bf16", len(c["lens"]), max(c["nqs"]), c["Hq"], c["Hkv"], c["D"], G.MAY_GROW, c["page"])
        assert kernel == TMEM, c
        modes.add(mode)
    for D in (32, 64, 96, 128):
        kernel, mode = plan("bf16", 70, 130, 4, 2, D, 300, 96)  # test_many_rows_of_many_items
        assert kernel == TMEM
        modes.add(mode)
    assert modes == {WHOLE, CUT}
    for c in _params(G.test_many_rows):
        assert plan("bf16", len(c["lens"]), max(c["nqs"]), c["Hq"], c["Hkv"], c["D"], max(c["lens"]), c["page"])[0] != TMEM, c
    for c in _params(G.test_wide_blocks):
        assert plan(c["dtype"], 5, c["n"], c["Hq"], c["Hkv"], c["D"], 4 * G.MAY_GROW, c["page"])[0] == (
            TMEM if c["dtype"] == "bf16" and c["n"] * c["Hq"] // c["Hkv"] >= 64 and c["D"] <= 128 else ROWS_16), c
    modes = set()
    for c in _params(G.test_clusters):
        kernel, mode = plan(c["dtype"], len(c["lens"]), c["n"], 8, 1, c["D"], max(c["lens"]), 64, c["window"])
        assert mode != WHOLE, c
        modes.add(mode)
    assert CLUSTER in modes
    for c in _params(G.test_wide_blocks_on_clusters):  # the shorter one is on the other side of both rules
        assert plan(c["dtype"], 57, 4, 16, 4, 64, c["longest"]) == ((ROWS_16, CLUSTER) if c["longest"] == 2048 else (ROWS_8, CUT))
    for c in _params(G.test_wide_blocks_of_many_items):
        kernel, mode = plan(c["dtype"], 200, 9, 12, 4, c["D"], 300, 96)
        assert kernel == ROWS_16 and mode == WHOLE, c
    assert plan("f32", 3, 1, 4, 1, 64, 20000, 256)[1] == CUT   # test_long_context


@pytest.mark.parametrize("call,kernel,mode", [
    (("f32", 1, 1, 32, 4, 64, 301), ROWS_8, CLUSTER),
    (("f32", 1, 1, 64, 8, 128, 131000), ROWS_8, CUT),
    (("bf16", 16, 1, 64, 8, 128, 32000), ROWS_8, CUT),
    (("f16", 8, 1, 24, 8, 96, 16000, 128, 1000), ROWS_8, CUT),    # by max_kv, whatever the window
    (("f32", 2, 128, 32, 4, 64, 2048), ROWS_16, CUT),
    (("bf16", 1, 509, 64, 8, 128, 8190), TMEM, WHOLE),
    (("f16", 1, 509, 64, 8, 128, 8190), ROWS_16, CUT),
    (("bf16", 1, 509, 64, 8, 160, 8190), ROWS_16, CUT),
    (("bf16", 1, 8, 64, 8, 128, 20000), TMEM, CUT),               # 64 rows a key/value head
    (("bf16", 1, 7, 64, 8, 128, 20000), ROWS_16, CUT),            # 56
    (("f32", 1000, 1, 8, 8, 64, 100), ROWS_8, WHOLE),
])
def test_calls_of_each_kind(plan, call, kernel, mode):
    assert plan(*call) == (kernel, mode)
