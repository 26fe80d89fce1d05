"""The descriptors that the binding makes for the attention entries (no GPU
needed: nothing is launched)."""
import pytest
import torch


@pytest.fixture(scope="module")
def qmm():
    from block_quantized_int4_gb300 import _build
    _build.build()
    from block_quantized_int4_gb300 import qmm as m
    return m


def _attn(qmm, pages, B, **kw):
    cache = qmm.kv_cache(torch.zeros(3, 4, 2, 36 * 64, dtype=torch.uint8), 64)
    x = torch.zeros(B, 4, 64)
    return qmm.attn_op(cache, x, pages, torch.zeros(B, dtype=torch.int32), x, **kw)


def test_page_tables_stay_inside_their_storage(qmm):
    """The kernels read pages[b * pages_stride + i], i < ceil(max_kv / page_size): with the op's stride every such
    place is the tensor's own element [b][i].  Rows that share storage (a table expanded over the samples of one
    prompt, overlapping windows of one list) have no such stride and are turned down."""
    one = torch.arange(2, dtype=torch.int32)[None]
    with pytest.raises(ValueError):
        _attn(qmm, one.expand(3, -1), 3)
    flat = torch.arange(8, dtype=torch.int32)
    for step in (0, 1, 2, 3):
        with pytest.raises(ValueError):
            _attn(qmm, flat.as_strided((2, 4), (step, 1)), 2)
    whole = torch.arange(24, dtype=torch.int32).view(3, 8)
    for pages in (whole, whole[:, :2], whole[:, 3:5], whole[1:], whole[::2], whole[:1], one.expand(1, -1), flat.as_strided(
            (1, 4), (0, 1)), flat.as_strided((2, 4), (4, 1)), one.expand(3, -1).contiguous(), whole[:, 2:3]):
        B, n = pages.shape
        op = _attn(qmm, pages, B)
        assert op.pages == pages.data_ptr() and op.pages_stride >= n
        for b in range(B):
            at = pages.data_ptr() + 4 * b * op.pages_stride
            assert at == pages[b].data_ptr(), (tuple(pages.shape), pages.stride())


def _status(qmm, T, H, ts, hs, D=64):
    """qmm_rope_heads into heads of these strides (addresses are never read: no device, or turned down before)."""
    import ctypes
    x = qmm.Heads(0x10000, H * D, D, H, 0)
    op = qmm.RopeOp(x, qmm.Heads(0x10000, ts, hs, H, 0), qmm.Rope(), None, None, T, D, 1e-5)
    return qmm.library_handle().qmm_rope_heads(ctypes.byref(op), None)


def test_rows_of_an_output_that_overlap_are_turned_down(qmm):
    """Against all pairs of rows, each D values long."""
    D = 64
    seen = set()
    for T in (1, 2, 3, 4, 7):
        for H in (1, 2, 3, 5):
            for ts in (0, 32, 64, 96, 128, 192, 320, 448):
                for hs in (0, 32, 64, 80, 128, 192, 256, 64 * 7):
                    at = sorted(t * ts + h * hs for t in range(T) for h in range(H))
                    overlap = any(b - a < D for a, b in zip(at, at[1:]))
                    seen.add(overlap)
                    if overlap:
                        assert _status(qmm, T, H, ts, hs) == 2, (T, H, ts, hs)
                    elif not torch.cuda.is_available():
                        assert _status(qmm, T, H, ts, hs) == 4, (T, H, ts, hs)
    assert seen == {True, False}
    if not torch.cuda.is_available():
        assert _status(qmm, 5, 3, 1 << 62, 64) == 4 and _status(qmm, 5, 3, 64, 1 << 62) == 4  # no product overflows
    assert _status(qmm, 40, 1 << 20, 64, 64) == 2
