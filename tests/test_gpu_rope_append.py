"""Rotary heads, the rotary table, and the paged Q4_0 cache append and read
against plain 64-bit forms.  Tolerance of a rotated head: at most 16 fp32
roundings (2^-24 each) of |a c| + |b s| (13 of the norm's sum over two, its
square root and division, two products, the rotation's three), then half a
step of the output's type.  Cached codes and scales are compared bit for bit:
the key's values are carried in pairs of fp32, so they round as the 64-bit
ones do."""
import numpy as np
import pytest
import torch

import attn_reference as R
import workloads
from parity import lib

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def _np(t):
    return t.detach().double().cpu().numpy()


def _table(n_pos, n_rot, seed=0):
    rng = np.random.default_rng(seed)
    a = rng.uniform(0, 2 * np.pi, (n_pos, n_rot // 2))
    return torch.tensor(np.stack([np.cos(a), np.sin(a)], -1), dtype=torch.float32, device=DEV)


def _heads(T, H, D, dtype, seed, strided):
    """Heads as they lie in a fused projection's output (strided) or alone."""
    x = workloads.activations(T * (H + 2), D, seed=seed).view(T, H + 2, D)
    if strided == "odd":  # nothing is 16-byte aligned
        base = torch.zeros(T, H + 2, D + 1, dtype=dtype, device=DEV)
        base[..., 1:] = x.to(dtype).to(DEV)
        return base[:, 1:H + 1, 1:]
    x = x.to(dtype).to(DEV)
    return x[:, 1:H + 1] if strided else x[:, :H].contiguous()


def _rope_bound(x, gamma, table, pos, n_rot, pairs, y, dtype):
    n = R.rotate(x, gamma, 1e-5, None, None, 0, pairs)
    t = np.abs(np.asarray(table, np.float64)) if n_rot else None
    if n_rot:  # |a c| + |b s|: rotate magnitudes with a negative sine
        t = t * np.array([1.0, -1.0])
        lo = R.rotate(np.abs(n), None, 0, t, pos, n_rot, pairs)
        t = t * np.array([1.0, -1.0])
        hi = R.rotate(np.abs(n), None, 0, t, pos, n_rot, pairs)
        n = np.maximum(np.abs(lo), np.abs(hi))
    eps = torch.finfo(dtype).eps / 2 if dtype != torch.float32 else 0.0
    tiny = 2.0 ** -25 if dtype == torch.float16 else 1e-38
    return 16 * 2.0 ** -24 * np.abs(n) * (1 + eps) + eps * np.abs(y) + tiny


ROPE_CASES = [
    # T, H, D, n_rot, pairs, norm, dtype, strided
    (1, 1, 32, 32, False, True, "f32", False),
    (1, 32, 64, 64, False, False, "f32", True),
    (3, 5, 64, 32, True, True, "f32", True),
    (7, 3, 96, 96, False, True, "bf16", True),
    (5, 9, 96, 22, False, True, "f16", True),
    (2, 8, 128, 128, True, True, "f16", False),
    (33, 7, 128, 64, False, True, "bf16", True),
    (4, 3, 160, 160, False, True, "f32", "odd"),
    (4, 3, 160, 10, True, False, "bf16", "odd"),
    (2, 2, 224, 50, False, True, "f32", False),
    (6, 4, 256, 256, False, True, "f32", True),
    (6, 4, 256, 0, False, True, "f32", True),
]


@pytest.mark.parametrize("T,H,D,n_rot,pairs,norm,dtype,strided", ROPE_CASES)
def test_rope_heads(T, H, D, n_rot, pairs, norm, dtype, strided):
    qmm = lib()
    dt = TYPES[dtype]
    x = _heads(T, H, D, dt, 3, strided)
    gamma = workloads.norm_weights(D, seed=4).to(DEV) if norm else None
    table = _table(50, n_rot) if n_rot else None
    pos = torch.arange(T, dtype=torch.int32, device=DEV) * 7 % 50
    pos[0] = 49
    y = torch.full((T, H, D), float("nan"), dtype=dt, device=DEV)
    qmm.qmm_rope_heads(qmm.rope_op(x, y, pos, qmm.rope(table, pairs), norm_w=gamma))
    ref = R.rotate(_np(x), None if gamma is None else _np(gamma), 1e-5, None if table is None else _np(table),
                   pos.cpu().numpy(), n_rot, pairs)
    bound = _rope_bound(_np(x), None if gamma is None else _np(gamma), None if table is None else table.cpu().numpy(),
                        pos.cpu().numpy(), n_rot, pairs, ref, dt)
    err = np.abs(_np(y) - ref)
    assert (err <= bound).all(), (err / bound).max()
    z = x.clone() if strided != "odd" else x
    qmm.qmm_rope_heads(qmm.rope_op(z, z, pos, qmm.rope(table, pairs), norm_w=gamma))  # in place
    assert torch.equal(z, y)
    assert qmm.qmm_last_device_error() == 0


def test_rope_heads_passes_what_it_does_not_rotate():
    qmm = lib()
    x = torch.randn(2, 3, 64, device=DEV)
    x[0, 0, 40], x[1, 2, 41] = float("inf"), -0.0
    y = torch.empty_like(x)
    qmm.qmm_rope_heads(qmm.rope_op(x, y, torch.zeros(2, dtype=torch.int32, device=DEV), qmm.rope(_table(4, 20))))
    assert torch.equal(x[..., 20:].view(torch.int32), y[..., 20:].view(torch.int32))


@pytest.mark.parametrize("scaling,factor,n_rot", [(0, 1.0, 64), (1, 8.0, 64), (2, 8.0, 64), (2, 40.0, 128),
                                                  (2, 4.0, 2), (0, 1.0, 256)])
def test_rope_table(scaling, factor, n_rot):
    """Angles of far positions against numpy's in 64 bits: a position of 2^17 at a frequency of 1 has
    an angle error of 2^17 * 2^-53 there and here, far below half a step of the fp32 value."""
    qmm = lib()
    n_pos, base, orig = 131072 if n_rot == 64 else 1000, 10000.0, 4096.0
    t = qmm.rope_table(n_pos, n_rot, base, scaling, factor, orig)
    i = np.arange(n_rot // 2)
    f = base ** (-2.0 * i / n_rot)
    m = 1.0
    if scaling == 1:
        f = f / factor
    if scaling == 2:
        x = lambda turns: n_rot * np.log(orig / (2 * np.pi * turns)) / (2 * np.log(base))  # noqa: E731
        lo, hi = max(0.0, np.floor(x(32.0))), min(n_rot / 2 - 1.0, np.ceil(x(1.0)))
        r = np.clip((i - lo) / max(hi - lo, 0.001), 0, 1)
        f, m = f * (1 - r) + f / factor * r, 0.1 * np.log(factor) + 1
    pos = np.r_[0, 1, 2, 777, n_pos - 1]
    a = pos[:, None] * f
    ref = m * np.stack([np.cos(a), np.sin(a)], -1)
    got = t.cpu().numpy().astype(np.float64)[pos]
    assert (np.abs(got - ref) <= 2.0 ** -24 * np.abs(ref) + 1e-9).all()


def _append(qmm, T, Hq, Hkv, D, n_rot, pairs, norm, dtype, page, n_pages, slots, strided=True, seed=1):
    dt = TYPES[dtype]
    q = _heads(T, Hq, D, dt, seed, strided) if Hq else None
    k, v = (_heads(T, Hkv, D, dt, seed + s, strided) for s in (1, 2))
    gk = workloads.norm_weights(D, seed=5).to(DEV) if norm else None
    gq = workloads.norm_weights(D, seed=6).to(DEV) if norm else None
    table = _table(60, n_rot) if n_rot else None
    pos = (torch.arange(T, dtype=torch.int32, device=DEV) * 11 + 5) % 60
    data = qmm.kv_cache_data(n_pages, page, Hkv, D)
    data.copy_(torch.randint(0, 256, data.shape, dtype=torch.uint8, generator=torch.Generator().manual_seed(seed)))
    before = data.clone()
    cache = qmm.kv_cache(data, page)
    q_out = torch.full((T, Hq, D), float("nan"), dtype=dt, device=DEV) if Hq else None
    op = qmm.kv_append_op(cache, k, v, slots, pos=pos, rope=qmm.rope(table, pairs), q=q, q_out=q_out, k_norm=gk,
                          q_norm=gq)
    qmm.qmm_kv_append_q4_0(op)
    n = lambda t: None if t is None else _np(t)  # noqa: E731
    kr = R.rotate(n(k), n(gk), np.float32(1e-5), n(table), pos.cpu().numpy(), n_rot, pairs).astype(np.float32)
    want = R.q4_0_values(kr), R.q4_0_values(_np(v))
    if Hq:
        ref = R.rotate(n(q), n(gq), 1e-5, n(table), pos.cpu().numpy(), n_rot, pairs)
        bound = _rope_bound(n(q), n(gq), n(table), pos.cpu().numpy(), n_rot, pairs, ref, dt)
        assert (np.abs(_np(q_out) - ref) <= bound).all()
    return cache, data, before, want


def _check_cache(data, before, slots, want, page, D):
    slots = slots.cpu().numpy()
    got = R.cache_values(data.cpu().numpy(), D)
    live = slots >= 0
    for g, w, name in zip(got, want, "kv"):
        at = g[slots[live] // page, :, slots[live] % page]
        assert np.array_equal(at, w[live]), f"{name}: {(at != w[live]).sum()} of {at.size} values differ"
    # every other token's bytes are as they were
    (kb, _), (vb, _), ks, vs = R.places(D)
    mine = np.zeros(data.shape, bool)
    for s in slots[live]:
        p, place = s // page, s % page
        t, rec = place % 32, place // 32
        for at in (kb[t], vb[t], ks[t], ks[t] + 1, vs[t], vs[t] + 1):
            mine[p, :, rec, np.unique(at)] = True
    assert np.array_equal(data.cpu().numpy()[~mine], before.cpu().numpy()[~mine])


@pytest.mark.parametrize("T,Hq,Hkv,D,n_rot,pairs,norm,dtype,page,strided", [
    (1, 32, 4, 64, 64, False, False, "f32", 64, True),
    (1, 1, 1, 32, 32, True, True, "bf16", 32, False),
    (16, 8, 2, 128, 128, False, True, "f32", 64, True),
    (70, 0, 3, 96, 96, False, True, "f16", 32, True),
    (130, 4, 4, 128, 64, True, True, "bf16", 128, True),
    (5, 6, 2, 160, 22, False, True, "f32", 96, "odd"),
    (33, 2, 2, 256, 256, False, True, "f32", 256, True),
    (9, 2, 1, 224, 0, False, False, "f16", 32, True),
    (600, 8, 8, 128, 128, False, True, "f32", 64, True),
])
def test_append(T, Hq, Hkv, D, n_rot, pairs, norm, dtype, page, strided):
    qmm = lib()
    n_pages = -(-T // page) + 2
    g = torch.Generator().manual_seed(T + D)
    slots = torch.randperm(n_pages * page, generator=g)[:T].to(DEV)
    cache, data, before, want = _append(qmm, T, Hq, Hkv, D, n_rot, pairs, norm, dtype, page, n_pages, slots, strided)
    _check_cache(data, before, slots, want, page, D)
    for dt in TYPES.values():
        k, v = (torch.full((T, Hkv, D), float("nan"), dtype=dt, device=DEV) for _ in range(2))
        qmm.qmm_kv_read_q4_0(qmm.kv_read_op(cache, slots, k, v))
        for got, w in zip((k, v), want):
            assert torch.equal(got.cpu(), torch.tensor(w, dtype=torch.float64).float().to(dt))
    assert qmm.qmm_last_device_error() == 0


def test_append_padding_and_bad_slots_and_positions():
    qmm = lib()
    qmm.qmm_last_device_error()
    T, Hkv, D, page, n_pages = 6, 2, 64, 32, 2
    slots = torch.tensor([3, -1, 40, -(1 << 40), 63, 0], device=DEV)
    cache, data, before, want = _append(qmm, T, 3, Hkv, D, 64, False, True, "f32", page, n_pages, slots)
    _check_cache(data, before, slots, want, page, D)
    assert qmm.qmm_last_device_error() == 0
    out = torch.full((T, Hkv, D), 7.0, device=DEV)
    qmm.qmm_kv_read_q4_0(qmm.kv_read_op(cache, slots, k=out))
    assert (out[[1, 3]] == 0).all() and not (out[0] == 0).all()
    # a slot past the cache: skipped and reported; the others are written
    bad = torch.tensor([3, n_pages * page, 1 << 40], device=DEV)
    again = data.clone()
    k, v = torch.randn(3, Hkv, D, device=DEV), torch.randn(3, Hkv, D, device=DEV)
    qmm.qmm_kv_append_q4_0(qmm.kv_append_op(cache, k, v, bad))
    assert qmm.qmm_last_device_error() == 10
    _check_cache(data, again, torch.tensor([3]), (R.q4_0_values(_np(k[:1])), R.q4_0_values(_np(v[:1]))), page, D)
    out = torch.full((3, Hkv, D), 7.0, device=DEV)
    qmm.qmm_kv_read_q4_0(qmm.kv_read_op(cache, bad, v=out))
    assert qmm.qmm_last_device_error() == 10
    assert (out[1:] == 7.0).all() and torch.equal(out[0].cpu().double(), torch.tensor(R.q4_0_values(_np(v[0]))))
    # positions outside the table
    table, y = _table(10, 64), torch.full((4, Hkv, D), 7.0, device=DEV)
    x = torch.randn(4, Hkv, D, device=DEV)
    pos = torch.tensor([0, 10, -1, 9], dtype=torch.int32, device=DEV)
    qmm.qmm_rope_heads(qmm.rope_op(x, y, pos, qmm.rope(table)))
    assert qmm.qmm_last_device_error() == 10
    assert (y[1:3] == 7.0).all() and not (y[[0, 3]] == 7.0).any()
    again = data.clone()
    qmm.qmm_kv_append_q4_0(qmm.kv_append_op(cache, x, x, torch.tensor([1, 2, 4, 5], device=DEV), pos=pos,
                                            rope=qmm.rope(table)))
    assert qmm.qmm_last_device_error() == 10
    kept = R.cache_values(data.cpu().numpy(), D)[1][0, :, [2, 4]]
    assert np.array_equal(kept, R.cache_values(again.cpu().numpy(), D)[1][0, :, [2, 4]], equal_nan=True)


def test_append_of_zeros_and_small_blocks():
    qmm = lib()
    T, D = 3, 64
    k = torch.zeros(T, 1, D, device=DEV)
    k[1, 0, 5], k[2, 0, :] = 1e-30, 3e-9  # scales that round to fp16 zero
    data = qmm.kv_cache_data(1, 32, 1, D).fill_(255)
    cache = qmm.kv_cache(data, 32)
    qmm.qmm_kv_append_q4_0(qmm.kv_append_op(cache, k, k, torch.arange(T, device=DEV)))
    out = torch.full((T, 1, D), float("nan"), device=DEV)
    qmm.qmm_kv_read_q4_0(qmm.kv_read_op(cache, torch.arange(T, device=DEV), v=out))
    assert (out == 0).all()


@pytest.mark.parametrize("top", [7.0, 7 * 2.0 ** -20, 7 * 3.0, 5.3, 1.7e-37, 3e4])
def test_append_of_values_halfway_between_codes(top):
    """Quotients at a half, a step of fp32 beside it, and over the whole range: codes as the division's."""
    qmm = lib()
    T, D = 64, 64
    rng = np.random.default_rng(3)
    d = np.float32(np.float32(top) / np.float32(7))
    x = (rng.integers(-7, 7, (T, 2, D)) + 0.5).astype(np.float32) * d
    for _ in range(2):  # none, one or two steps up or down
        x = np.where(rng.random(x.shape) < 0.4, np.nextafter(x, np.float32(rng.choice([-1e38, 1e38]))), x)
    x[rng.random(x.shape) < 0.1] = 0
    x[..., ::32] = np.float32(top)
    x = np.clip(x, -np.float32(top), np.float32(top))
    kv = torch.tensor(x, dtype=torch.float32, device=DEV)
    data = qmm.kv_cache_data(2, 32, 2, D).fill_(255)
    before = data.clone()
    slots = torch.arange(T, device=DEV)
    qmm.qmm_kv_append_q4_0(qmm.kv_append_op(qmm.kv_cache(data, 32), kv, kv, slots))
    want = R.q4_0_values(x.astype(np.float64))
    _check_cache(data, before, slots, (want, want), 32, D)
    assert qmm.qmm_last_device_error() == 0


def test_empty_calls_and_another_stream():
    qmm = lib()
    data = qmm.kv_cache_data(2, 32, 1, 64).fill_(1)
    cache = qmm.kv_cache(data, 32)
    none = torch.empty(0, 1, 64, device=DEV)
    qmm.qmm_kv_append_q4_0(qmm.kv_append_op(cache, none, none, torch.empty(0, dtype=torch.int64, device=DEV)))
    qmm.qmm_rope_heads(qmm.rope_op(none, none, torch.empty(0, dtype=torch.int32, device=DEV), qmm.rope(_table(4, 64))))
    x = torch.randn(300, 4, 64, device=DEV)
    pos = torch.zeros(300, dtype=torch.int32, device=DEV)
    table = _table(4, 64)
    y, z = torch.empty_like(x), torch.empty_like(x)
    qmm.qmm_rope_heads(qmm.rope_op(x, y, pos, qmm.rope(table)))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        qmm.qmm_rope_heads(qmm.rope_op(x, z, pos, qmm.rope(table)))
    s.synchronize()
    assert torch.equal(y, z)
