"""Refusals of the attention entries: what an argument check turns down
before anything is launched (no GPU needed: addresses are never read)."""
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


def _heads(qmm, n=4, D=64, dtype=0, data=A16, ts=None, hs=None):
    return qmm.Heads(data, n * D if ts is None else ts, D if hs is None else hs, n, dtype)


def _call(qmm, name, op):
    return getattr(qmm.library_handle(), name)(ctypes.byref(op) if op is not None else None, None)


def _no_device():
    return not torch.cuda.is_available()


def _rope(qmm, **kw):
    return qmm.Rope(*{"table": A16, "n_pos": 10, "n_rot": 64, "pairs": 0, **kw}.values())


def _rope_op(qmm, D=64, **kw):
    f = {"x": _heads(qmm), "y": _heads(qmm), "rope": _rope(qmm), "pos": A16, "norm_w": None, "T": 2, "head_dim": D,
         "norm_eps": 1e-5, **kw}
    return qmm.RopeOp(*f.values())


def test_rope_heads_refusals(qmm):
    call = lambda **kw: _call(qmm, "qmm_rope_heads", _rope_op(qmm, **kw))  # noqa: E731
    assert _call(qmm, "qmm_rope_heads", None) == 1
    assert call(T=-1) == 1
    assert call(T=0) == 0
    assert call(D=48) == 2 and call(D=0) == 2 and call(D=288) == 2
    assert call(x=_heads(qmm, data=None)) == 1
    assert call(x=_heads(qmm, dtype=3)) == 1
    assert call(y=_heads(qmm, n=5)) == 2
    assert call(y=_heads(qmm, hs=32)) == 2 and call(y=_heads(qmm, ts=32)) == 2  # rows of y overlap
    assert call(x=_heads(qmm, data=A16 + 2)) == 3 and call(x=_heads(qmm, data=A16 + 1, dtype=2)) == 3
    assert call(rope=_rope(qmm, n_rot=63)) == 2 and call(rope=_rope(qmm, n_rot=66)) == 2
    assert call(rope=_rope(qmm, n_rot=-2)) == 1 and call(rope=_rope(qmm, n_pos=-1)) == 1
    assert call(rope=_rope(qmm, table=None)) == 1 and call(pos=None) == 1
    assert call(rope=_rope(qmm, table=A16 + 4)) == 3 and call(pos=A16 + 2) == 3 and call(norm_w=A16 + 2) == 3
    if _no_device():
        assert call() == 4 and call(rope=_rope(qmm, n_rot=0, table=None), pos=None) == 4


def test_rope_table_refusals(qmm):
    f = qmm.library_handle().qmm_rope_table
    ok = dict(table=A16, n_pos=4, n_rot=64, base=1e4, scaling=2, factor=8.0, orig=4096.0, fast=32.0, slow=1.0)
    call = lambda **kw: f(*{**ok, **kw}.values(), None)  # noqa: E731
    assert call(n_pos=-1) == 1 and call(n_pos=0) == 0 and call(table=None) == 1 and call(table=A16 + 4) == 3
    assert call(n_rot=0) == 2 and call(n_rot=7) == 2 and call(n_rot=258) == 2 and call(n_pos=1 << 40) == 2
    assert call(scaling=3) == 1 and call(scaling=-1) == 1
    assert call(base=1.0) == 1 and call(base=float("nan")) == 1 and call(base=float("inf")) == 1
    assert call(factor=0.5) == 1 and call(factor=float("nan")) == 1 and call(scaling=1, factor=0.0) == 1
    assert call(orig=0.0) == 1 and call(slow=0.0) == 1 and call(fast=0.5) == 1
    if _no_device():
        assert call() == 4 and call(scaling=0, factor=0.0, orig=0.0, fast=0.0, slow=0.0) == 4


def _cache(qmm, **kw):
    return qmm.KvCache(*{"data": A16, "n_pages": 8, "page_size": 64, "n_heads": 4, "head_dim": 64, **kw}.values())


def test_cache_bytes_and_refusals(qmm):
    assert qmm.qmm_kv_cache_bytes(_cache(qmm)) == 8 * 4 * 64 * 72
    assert qmm.qmm_kv_cache_bytes(_cache(qmm, data=None, n_pages=1 << 20, page_size=256, n_heads=8, head_dim=256)) == (
        (1 << 20) * 8 * 8 * 36 * 256)
    out = ctypes.c_size_t()
    f = qmm.library_handle().qmm_kv_cache_bytes
    for bad, st in (({"n_pages": -1}, 1), ({"page_size": 0}, 1), ({"n_heads": 0}, 1), ({"page_size": 48}, 2),
                    ({"head_dim": 80}, 2), ({"head_dim": 512}, 2), ({"head_dim": 0}, 2)):
        assert f(ctypes.byref(_cache(qmm, **bad)), ctypes.byref(out)) == st, bad
    assert f(None, ctypes.byref(out)) == 1 and f(ctypes.byref(_cache(qmm)), None) == 1


def _append_op(qmm, **kw):
    f = {"cache": _cache(qmm), "k": _heads(qmm), "v": _heads(qmm), "q": _heads(qmm, n=8), "q_out": _heads(qmm, n=8),
         "rope": _rope(qmm), "slots": A16, "pos": A16, "k_norm": None, "q_norm": None, "T": 2, "norm_eps": 1e-5,
         "reserved": 0, **kw}
    return qmm.KvAppendOp(*f.values())


def test_append_and_read_refusals(qmm):
    call = lambda **kw: _call(qmm, "qmm_kv_append_q4_0", _append_op(qmm, **kw))  # noqa: E731
    assert _call(qmm, "qmm_kv_append_q4_0", None) == 1
    assert call(T=-1) == 1 and call(T=0) == 0
    assert call(cache=_cache(qmm, data=None)) == 1 and call(cache=_cache(qmm, data=A16 + 8)) == 3
    assert call(cache=_cache(qmm, page_size=40)) == 2
    assert call(k=_heads(qmm, n=3)) == 2 and call(v=_heads(qmm, n=8)) == 2 and call(k=_heads(qmm, data=None)) == 1
    assert call(q_out=_heads(qmm, n=4)) == 2 and call(q_out=_heads(qmm, data=None, n=8)) == 1
    assert call(q_out=_heads(qmm, n=8, hs=8)) == 2
    assert call(slots=None) == 1 and call(slots=A16 + 4) == 3 and call(pos=None) == 1
    assert call(rope=_rope(qmm, n_rot=128)) == 2
    assert call(k_norm=A16 + 1) == 3 and call(q_norm=A16 + 1) == 3
    read = lambda **kw: _call(qmm, "qmm_kv_read_q4_0", qmm.KvReadOp(*{  # noqa: E731
        "cache": _cache(qmm), "k": _heads(qmm), "v": _heads(qmm), "slots": A16, "T": 2, **kw}.values()))
    assert _call(qmm, "qmm_kv_read_q4_0", None) == 1
    assert read(T=-1) == 1 and read(T=0) == 0 and read(k=qmm.Heads(), v=qmm.Heads()) == 0
    assert read(k=_heads(qmm, n=2)) == 2 and read(v=_heads(qmm, dtype=7)) == 1 and read(slots=None) == 1
    assert read(slots=A16 + 2) == 3 and read(k=_heads(qmm, hs=1)) == 2
    if _no_device():
        assert call() == 4 and call(q=qmm.Heads(), q_out=qmm.Heads()) == 4 and read() == 4


def _attn_op(qmm, **kw):
    f = {"cache": _cache(qmm), "q": _heads(qmm, n=8), "out": _heads(qmm, n=8), "yq": None, "yd": None,
         "q_start": None, "kv_len": A16, "pages": A16, "pages_stride": 8, "T": 2, "n_seqs": 2, "max_q": 1,
         "max_kv": 100, "causal": 1, "window": 0, "scale": 0.125, "workspace": A16, "workspace_bytes": 1 << 30, **kw}
    return qmm.AttnOp(*f.values())


def test_attention_refusals(qmm):
    call = lambda **kw: _call(qmm, "qmm_attn_q4_0", _attn_op(qmm, **kw))  # noqa: E731
    assert _call(qmm, "qmm_attn_q4_0", None) == 1
    for name in ("n_seqs", "T", "max_q", "max_kv", "window"):
        assert call(**{name: -1}) == 1, name
    assert call(n_seqs=0, T=0) == 0 and call(T=0, q_start=A16) == 0 and call(max_q=0, T=0) == 0
    assert call(scale=float("nan")) == 1 and call(scale=float("inf")) == 1
    assert call(T=3) == 2                                  # no q_start: T == n_seqs * max_q
    assert call(q=_heads(qmm, n=6)) == 2                   # not a multiple of the cache's heads
    assert call(pages_stride=1) == 2                       # 100 tokens need two pages of 64
    assert call(max_kv=1 << 30, pages_stride=1 << 30) == 2
    assert call(out=_heads(qmm, n=8, dtype=1)) == 1 and call(out=_heads(qmm, n=4)) == 2
    assert call(out=qmm.Heads()) == 1                      # nowhere to write
    assert call(yq=A16) == 1 and call(yd=A16) == 1         # one without the other
    assert call(yq=A16, yd=A16 + 1) == 3
    assert call(kv_len=None) == 1 and call(pages=None) == 1 and call(q=_heads(qmm, n=8, data=None)) == 1
    assert call(kv_len=A16 + 1) == 3 and call(pages=A16 + 2) == 3 and call(q_start=A16 + 2) == 3
    assert call(cache=_cache(qmm, data=A16 + 4)) == 3 and call(cache=_cache(qmm, head_dim=33)) == 2
    long = dict(max_kv=100000, pages_stride=2000)
    need = qmm.qmm_attn_workspace_size(_attn_op(qmm, **long))
    assert need > 0 and need % 16 == 0
    assert call(**long, workspace=None) == 8 and call(**long, workspace_bytes=need - 1) == 8
    assert call(**long, workspace=A16 + 8) == 8
    assert qmm.qmm_attn_workspace_size(_attn_op(qmm, n_seqs=0, T=0)) == 0
    if _no_device():
        assert call() == 4 and call(**long) == 4 and call(out=qmm.Heads(), yq=A16, yd=A16) == 4


def test_binding_refusals(qmm):
    x = torch.zeros(2, 4, 64)
    slots, pos = torch.zeros(2, dtype=torch.int64), torch.zeros(2, dtype=torch.int32)
    cache = qmm.kv_cache(torch.zeros(3, 4, 2, 36 * 64, dtype=torch.uint8), 64)
    assert (cache.n_pages, cache.page_size, cache.n_heads, cache.head_dim) == (3, 64, 4, 64)
    rope = qmm.rope(torch.zeros(5, 32, 2))
    assert (rope.n_pos, rope.n_rot) == (5, 64)
    with pytest.raises(ValueError):
        qmm.kv_cache(torch.zeros(3, 4, 2, 36 * 64, dtype=torch.uint8), 32)
    with pytest.raises(ValueError):
        qmm.heads(x.transpose(1, 2))
    with pytest.raises(ValueError):
        qmm.heads(x.double())
    with pytest.raises(ValueError):
        qmm.rope(torch.zeros(5, 32))
    with pytest.raises(ValueError):
        qmm.rope_op(x, x[:1], pos, rope)
    with pytest.raises(ValueError):
        qmm.rope_op(x, x, slots, rope)  # int64 positions
    with pytest.raises(ValueError):
        qmm.kv_append_op(cache, x, x, pos)  # int32 slots
    with pytest.raises(ValueError):
        qmm.kv_append_op(cache, x, x, slots, q=x)
    with pytest.raises(ValueError):
        qmm.kv_append_op(cache, x[..., :32], x[..., :32], slots)
    with pytest.raises(ValueError):
        qmm.kv_read_op(cache, slots, k=x[:1])
    with pytest.raises(ValueError):
        qmm.attn_op(cache, x, torch.zeros(2, 2, dtype=torch.int64), pos, x)
    with pytest.raises(ValueError):
        qmm.attn_op(cache, x, torch.zeros(2, 2, dtype=torch.int32), pos, x, max_kv=129)
    with pytest.raises(ValueError):
        qmm.attn_op(cache, x, torch.zeros(2, 2, dtype=torch.int32), pos, x[:1])
