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
