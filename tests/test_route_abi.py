"""Refusals of qmm_moe_route (no GPU needed: addresses are never read)."""
import ctypes

import pytest
import torch

A16 = 0x10000  # a fake, aligned address


@pytest.fixture(scope="module")
def qmm():
    from block_quantized_int4_gb300 import _build
    _build.build()
    from block_quantized_int4_gb300 import qmm as m
    return m


def _call(qmm, **kw):
    f = {"logits": A16, "ld": 64, "bias": None, "ids": A16, "gates": A16, "dtype": 0, "T": 3, "E": 64, "k": 6,
         "score": 1, "n_groups": 1, "top_groups": 1, "group_score": 0, "renormalize": 1, "scale": 1.0,
         "workspace": None, "workspace_bytes": 0, **kw}
    return qmm.library_handle().qmm_moe_route(ctypes.byref(qmm.MoeRouteOp(*f.values())), None)


def test_refusals(qmm):
    assert qmm.library_handle().qmm_moe_route(None, None) == 1
    assert _call(qmm, T=0) == 0 and _call(qmm, T=0, logits=None, ids=None, gates=None) == 0
    for bad in ({"T": -1}, {"E": 0}, {"k": 0}, {"ld": 63}, {"n_groups": 0}, {"top_groups": 0}, {"dtype": 3},
                {"dtype": -1}, {"score": 2}, {"group_score": 2}, {"logits": None}, {"ids": None}, {"gates": None},
                {"scale": float("inf")}, {"scale": float("nan")}):
        assert _call(qmm, **bad) == 1, bad
    for bad in ({"E": 1025, "ld": 1025}, {"k": 65}, {"n_groups": 3}, {"n_groups": 64}, {"n_groups": 6, "E": 60},
                {"n_groups": 8, "E": 60}, {"n_groups": 8, "top_groups": 9}, {"n_groups": 16, "k": 5},
                {"workspace": A16, "workspace_bytes": 1 << 40, "T": 1 << 23}):
        assert _call(qmm, **bad) == 2, bad
    for bad in ({"logits": A16 + 2}, {"logits": A16 + 1, "dtype": 1}, {"bias": A16 + 2}, {"ids": A16 + 1},
                {"gates": A16 + 2}, {"workspace": A16 + 8, "workspace_bytes": 1 << 20}):
        assert _call(qmm, **bad) == 3, bad
    assert _call(qmm, workspace=A16, workspace_bytes=qmm.qmm_moe_workspace_size(64, 3, 6) - 1) == 8
    if not torch.cuda.is_available():
        assert _call(qmm) == 4 and _call(qmm, logits=A16 + 2, dtype=2) == 4
        assert _call(qmm, workspace=A16, workspace_bytes=qmm.qmm_moe_workspace_size(64, 3, 6)) == 4


def test_binding_checks(qmm):
    l, i, g = torch.zeros(3, 64), torch.zeros(3, 6, dtype=torch.int32), torch.zeros(3, 6)
    op = qmm.moe_route_op(l[:, :60], i, g, bias=torch.zeros(60))
    assert (op.ld, op.T, op.E, op.k) == (64, 3, 60, 6)
    assert qmm.moe_route_op(l.as_strided((1, 64), (0, 1)), i[:1], g[:1]).ld == 64  # one row: its stride means nothing
    for bad in ({"logits": l.double()}, {"logits": l.t()}, {"logits": l[0]}, {"ids": i.long()}, {"ids": i[:2]},
                {"gates": g[:, :5]}, {"gates": g.t().contiguous().t()}, {"bias": torch.zeros(63)},
                {"bias": torch.zeros(64, dtype=torch.float16)}):
        with pytest.raises(ValueError):
            a = {"logits": l, "ids": i, "gates": g, **bad}
            qmm.moe_route_op(a.pop("logits"), a.pop("ids"), a.pop("gates"), **a)
