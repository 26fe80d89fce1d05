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


def test_sizes_beyond_the_kernels_indexes_are_turned_down(qmm):
    """Records are counted in 31 bits on the device and bytes in size_t; products of the sizes must not wrap."""
    import ctypes
    lib = qmm.library_handle()
    out = ctypes.c_size_t(7)
    for n_pages, page, heads, ok in ((1 << 20, 256, 8, True), ((1 << 31) - 1, 32, 1, True), ((1 << 31) - 1, 32, 2, False),
                                     (1 << 16, 1 << 20, 1, False), ((1 << 31) - 1, 1 << 20, 1 << 16, False), (0, 1 << 20, 1 << 16, True),
                                     (1 << 30, 64, 1, False)):
        c = qmm.KvCache(0x10000, n_pages, page, heads, 256)
        st = lib.qmm_kv_cache_bytes(ctypes.byref(c), ctypes.byref(out))
        assert st == (0 if ok else 2), (n_pages, page, heads)
        if ok:
            assert out.value == n_pages * heads * (page // 32) * 36 * 256
    h = lambda n=4: qmm.Heads(0x10000, 1 << 10, 1 << 6, n, 0)  # noqa: E731
    cache = qmm.KvCache(0x10000, 8, 64, 4, 64)
    for T in (1 << 33, 1 << 60, 1 << 61, 1 << 62, (1 << 63) - 1):  # T times the warps of a token wraps for most
        op = qmm.RopeOp(h(), h(), qmm.Rope(), None, None, T, 64, 1e-5)
        assert lib.qmm_rope_heads(ctypes.byref(op), None) == 2, T
        op = qmm.KvAppendOp(cache, h(), h(), qmm.Heads(), qmm.Heads(), qmm.Rope(), 0x10000, 0x10000, None, None, T, 1e-5, 0)
        assert lib.qmm_kv_append_q4_0(ctypes.byref(op), None) == 2, T
        op = qmm.KvReadOp(cache, h(), h(), 0x10000, T)
        assert lib.qmm_kv_read_q4_0(ctypes.byref(op), None) == 2, T
