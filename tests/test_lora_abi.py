"""Refusals of qmm_lora (no GPU needed: addresses are never read)."""
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
    f = {"x": A16, "a": A16, "b": A16, "base": A16, "y": A16, "ldx": 64, "lda": 64, "a_stride": 512, "ldb": 8,
         "b_stride": 320, "ld_base": 40, "ldy": 40, "ranks": None, "scales": None, "seg_start": None,
         "seg_adapter": A16, "T": 6, "N": 40, "K": 64, "n_segs": 3, "n_adapters": 2, "max_rank": 8, "x_dtype": 0,
         "w_dtype": 1, "y_dtype": 0}
    assert set(kw) <= set(f)
    f.update(kw)
    return qmm.library_handle().qmm_lora(ctypes.byref(qmm.LoraOp(*f.values())), None)


def test_refusals(qmm):
    assert qmm.library_handle().qmm_lora(None, None) == 1
    assert _call(qmm, T=0) == 0 and _call(qmm, n_segs=0) == 0
    assert _call(qmm, T=0, x=None, a=None, b=None, y=None, base=None, seg_adapter=None) == 0
    for bad in ({"T": -1}, {"N": 0}, {"n_segs": -1}, {"n_adapters": 0}, {"max_rank": 0}, {"x_dtype": 3},
                {"w_dtype": -1}, {"y_dtype": 3}, {"y_dtype": 1}, {"y_dtype": 2, "x_dtype": 1}, {"ldx": 63}, {"lda": 32}, {"ldb": 7}, {"ldy": 39}, {"ld_base": 39},
                {"a_stride": -8}, {"b_stride": -8}, {"x": None}, {"a": None}, {"b": None}, {"y": None},
                {"seg_adapter": None}):
        assert _call(qmm, **bad) == 1, bad
    for bad in ({"K": 0}, {"K": 48}, {"K": 1 << 25, "ldx": 1 << 25, "lda": 1 << 25}, {"max_rank": 257, "ldb": 257},
                {"T": 7}, {"n_segs": 65537, "T": 65537}, {"T": (1 << 28) + 1, "n_segs": 1}, {"N": 1 << 29, "ldy": 1 << 29, "ld_base": 1 << 29},
                {"ldx": 1 << 41}, {"lda": 1 << 41}, {"b_stride": 1 << 41}, {"ld_base": 48}):
        assert _call(qmm, **bad) == 2, bad
    for bad in ({"x": A16 + 8}, {"ldx": 66}, {"a": A16 + 8}, {"lda": 68}, {"a_stride": 516}, {"b": A16 + 1},
                {"y": A16 + 2, "base": None}, {"base": A16 + 2}, {"ranks": A16 + 2}, {"scales": A16 + 2},
                {"seg_start": A16 + 2}, {"seg_adapter": A16 + 2}):
        assert _call(qmm, **bad) == 3, bad
    if not torch.cuda.is_available():
        assert _call(qmm) == 4 and _call(qmm, base=None, ld_base=0) == 4
        assert _call(qmm, seg_start=A16, T=7) == 4 and _call(qmm, b=A16 + 2, ldb=9) == 4
        assert _call(qmm, T=1, n_segs=1, ldx=66) == 4  # the stride of one row means nothing


def test_binding_checks(qmm):
    x, a, b = torch.zeros(6, 64), torch.zeros(2, 8, 64), torch.zeros(2, 40, 8)
    y, s = torch.zeros(6, 40), torch.zeros(3, dtype=torch.int32)
    op = qmm.lora_op(x, a[:, :4], b[:, :, :4], y, s, base=y)
    assert (op.T, op.N, op.K, op.n_segs, op.n_adapters, op.max_rank) == (6, 40, 64, 3, 2, 4)
    assert (op.ldx, op.lda, op.a_stride, op.ldb, op.b_stride, op.ldy, op.ld_base) == (64, 64, 512, 8, 320, 40, 40)
    args = dict(x=x, a=a, b=b, y=y, seg_adapter=s)
    for bad in ({"x": x.double()}, {"x": x.t()}, {"x": x[0]}, {"y": y[:5]}, {"a": a[0]}, {"a": a.half()},
                {"a": a[:1]}, {"b": b.transpose(1, 2)}, {"b": b[:, :39]}, {"seg_adapter": s.long()},
                {"seg_adapter": s[:, None]}, {"base": y.half()}, {"base": y[:, :39]},
                {"seg_start": torch.zeros(3, dtype=torch.int32)}, {"ranks": torch.zeros(3, dtype=torch.int32)},
                {"scales": torch.zeros(2, dtype=torch.float64)}):
        with pytest.raises(ValueError):
            qmm.lora_op(**{**args, **bad})
