"""qmm_moe_route against routing in 64 bits: choices equal, gates within the
roundings counted in route_reference."""
import numpy as np
import pytest
import torch

from parity import lib
import route_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def _run(qmm, logits, k, score, bias=None, n_groups=1, top_groups=1, top2=False, renorm=True, scale=1.0, ws=None):
    T = logits.shape[0]
    ids = torch.full((T, k), -7, dtype=torch.int32, device=DEV)
    gates = torch.full((T, k), float("nan"), device=DEV)
    op = qmm.moe_route_op(logits, ids, gates, bias=bias,
                          score=qmm.ROUTE_SOFTMAX if score == "softmax" else qmm.ROUTE_SIGMOID, n_groups=n_groups,
                          top_groups=top_groups, group_score=qmm.ROUTE_GROUP_TOP2 if top2 else qmm.ROUTE_GROUP_MAX,
                          renormalize=renorm, scale=scale, workspace=ws)
    qmm.qmm_moe_route(op)
    return ids, gates


def _check(qmm, logits, k, score, bias=None, **kw):
    ids, gates = _run(qmm, logits, k, score, bias=bias, **kw)
    kw.pop("ws", None)
    host = logits.float().cpu().numpy()
    rid, rg = R.route(host, k, score, None if bias is None else bias.cpu().numpy(), **kw)
    np.testing.assert_array_equal(ids.cpu().numpy(), rid)
    got = gates.cpu().numpy().astype(np.float64)
    assert np.isfinite(got).all()
    assert (np.abs(got - rg) <= R.gate_tolerance(host, rid, rg)).all(), np.abs(got - rg).max()
    assert qmm.qmm_last_device_error() == 0
    return ids, gates


def _logits(T, E, dtype, seed, spread=1.0, masked=0.0, pad=0, at=0):
    """Rows with foreign values between them, `at` elements behind an aligned address."""
    g = torch.Generator().manual_seed(seed)
    l = spread * (torch.randn(T, E, generator=g) + 0.5 * torch.randn(E, generator=g))
    if masked:
        l[torch.rand(T, E, generator=g) < masked] = float("-inf")
    buf = torch.full((T * (E + pad) + at,), 1e4, dtype=TYPES[dtype], device=DEV)
    out = buf[at:].view(T, E + pad)[:, :E]
    out.copy_(l)
    return out


def _bias(E, seed, scale=0.1):
    return (scale * torch.randn(E, generator=torch.Generator().manual_seed(1000 + seed))).to(DEV)


# T, E, k, groups, top groups: sizes around what a lane holds and where groups do not divide it
SHAPES = [(1, 1, 1, 1, 1), (3, 2, 2, 1, 1), (5, 31, 4, 1, 1), (7, 33, 8, 1, 1), (9, 60, 4, 1, 1), (33, 64, 6, 1, 1),
          (4, 65, 32, 1, 1), (5, 128, 33, 1, 1), (17, 256, 8, 1, 1), (2, 1024, 64, 1, 1), (9, 1023, 10, 1, 1),
          (13, 256, 8, 8, 4), (13, 160, 6, 8, 3), (6, 64, 8, 8, 1), (11, 72, 5, 2, 1), (3, 96, 7, 32, 5),
          (3, 1024, 9, 32, 31), (8, 32, 3, 32, 3), (5, 40, 5, 4, 4), (4, 512, 31, 16, 2), (4, 512, 32, 16, 2)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,E,k,G,top", SHAPES)
def test_shapes(T, E, k, G, top, dtype):
    qmm = lib()
    n = 0
    for score in ("sigmoid", "softmax"):
        for bias in (False, True):
            for top2 in (False, True) if G > 1 else (False,):
                n += 1
                _check(qmm, _logits(T, E, dtype, n, pad=n % 3, at=n % 4 == 3), k, score,
                       _bias(E, n) if bias else None, n_groups=G, top_groups=top, top2=top2, renorm=n % 2 == 0,
                       scale=[1.0, 2.5][n % 2])


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_many_tokens(score):
    """More tokens than warps; about one in three hundred has neighbours that 32 bits do not tell apart."""
    qmm = lib()
    _check(qmm, _logits(12001, 64, "f32", 1), 6, score, _bias(64, 1), scale=2.5)
    _check(qmm, _logits(3001, 256, "bf16", 2), 8, score, _bias(256, 2), n_groups=8, top_groups=4, top2=True)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,G", [(64, 1), (64, 8), (256, 4), (40, 4)])
def test_scores_that_32_bits_do_not_order(E, G, score):
    """Biases that bring every c of a token to about 0.7: what is left of them is the rounding of the bias."""
    qmm = lib()
    for seed in range(4):
        l = _logits(1, E, "f32", seed)
        p = torch.sigmoid(l[0].double()) if score == "sigmoid" else torch.softmax(l[0].double(), -1)
        bias = (0.7 - p).float()
        for top2 in (False, True) if G > 1 else (False,):
            _check(qmm, l, 6, score, bias, n_groups=G, top_groups=max(1, G // 2), top2=top2)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("G,top2", [(1, False), (8, False), (8, True)])
def test_equal_scores_go_to_the_lower_index(dtype, bias, G, top2):
    qmm = lib()
    for E in (64, 256, 80):
        g = torch.Generator().manual_seed(E)
        l = torch.randint(-3, 4, (29, E), generator=g).to(TYPES[dtype]).to(DEV) * 0.25
        l[0] = 0.5       # all equal
        l[1] = -0.0
        l[1, ::3] = 0.0  # both zeros are one value
        b = torch.zeros(E, device=DEV) if bias else None
        for score in ("sigmoid", "softmax"):
            _check(qmm, l, 7, score, b, n_groups=G, top_groups=max(1, G // 2), top2=top2)
        if bias:  # equal logits, biases that differ in the last bit
            b = 1 + torch.randint(0, 2, (E,), generator=g).to(DEV) * 2.0 ** -23
            _check(qmm, l, 7, "sigmoid", b, n_groups=G, top_groups=max(1, G // 2), top2=top2)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [False, True])
def test_experts_that_take_no_part(dtype, score, renorm):
    """-inf and NaN logits: rows with none, few and all of them, with and without biases and groups."""
    qmm = lib()
    for E, G in ((48, 1), (64, 4), (256, 8)):
        l = _logits(23, E, dtype, E, masked=0.7)
        l[0] = float("-inf")
        l[1] = float("nan")
        l[2, :E // 2] = float("nan")
        l[3] = float("-inf")
        l[3, E - 1] = -2.0  # one expert is left
        l[4, : E - E // G] = float("-inf")  # one group is left
        for bias in (None, _bias(E, 3), _bias(E, 4, 5.0)):
            for top2 in (False, True) if G > 1 else (False,):
                _check(qmm, l, 9, score, bias, n_groups=G, top_groups=max(1, G // 2), top2=top2, renorm=renorm)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [False, True])
def test_far_logits(score, renorm):
    """Scores next to 1, next to 0, and below what fp32 and 64 bits hold."""
    qmm = lib()
    for lo, hi in ((15, 40), (-40, -15), (-95, -70), (-300, -120), (-3000, -1000), (-200, 200)):
        g = torch.Generator().manual_seed(lo + 5000)
        l = (lo + (hi - lo) * torch.rand(9, 128, generator=g)).to(DEV)
        for bias in (None, _bias(128, 5), _bias(128, 6, 1e-8)):
            _check(qmm, l, 8, score, bias, renorm=renorm)
            _check(qmm, l, 8, score, bias, renorm=renorm, n_groups=4, top_groups=2, top2=True)
    l = _logits(3, 64, "f32", 9)
    if score == "sigmoid":
        l[:, 5] = float("inf")
        _check(qmm, l, 4, score, None, renorm=renorm)
        _check(qmm, l, 4, score, _bias(64, 7), renorm=renorm)


def test_large_biases_that_cancel_in_a_group():
    """Sums of two whose terms are a thousand times larger."""
    qmm = lib()
    l = _logits(200, 64, "f32", 11)
    b = _bias(64, 11, 0.01).view(8, 8)
    b[:, 0] += 40.0
    b[:, 1:] -= 40.0
    _check(qmm, l, 6, "sigmoid", b.reshape(-1).contiguous(), n_groups=8, top_groups=3, top2=True)


def _tables(ws, E, n):
    w = ws.cpu().numpy().view(np.int32)
    counts, offsets = w[:E], w[E:2 * E + 1]
    cursor, active, n_active = w[2 * E + 1:3 * E + 1], w[3 * E + 1:4 * E + 1], int(w[4 * E + 1])
    slots = w[4 * E + 2:4 * E + 2 + n]
    return (counts.tolist(), offsets.tolist(), cursor[:n_active].tolist(), active[:n_active].tolist(),
            [sorted(slots[offsets[e]:offsets[e + 1]].tolist()) for e in range(E)])


@pytest.mark.parametrize("T,E,k", [(1, 256, 8), (3, 60, 4), (5, 256, 8), (16, 256, 8), (64, 160, 6), (65, 64, 6),
                                   (700, 32, 2)])
def test_grouping(T, E, k):
    """With a workspace the slots are grouped as by qmm_moe_group_ids, and ids and gates are the same."""
    qmm = lib()
    l = _logits(T, E, "f32", T)
    plain = _check(qmm, l, k, "sigmoid", _bias(E, 1))
    n = qmm.qmm_moe_workspace_size(E, T, k)
    ws, want = (torch.full((n,), 0x5A, dtype=torch.uint8, device=DEV) for _ in range(2))
    ids, gates = _check(qmm, l, k, "sigmoid", _bias(E, 1), ws=ws)
    assert torch.equal(ids, plain[0]) and torch.equal(gates, plain[1])
    qmm.qmm_moe_group_ids(ids, T, k, E, want, n)
    assert _tables(ws, E, T * k) == _tables(want, E, T * k)


def test_captured_and_on_another_stream():
    qmm = lib()
    T, E, k = 70, 256, 8
    l, b = _logits(T, E, "bf16", 1), _bias(E, 1)
    ids = torch.zeros(T, k, dtype=torch.int32, device=DEV)
    gates = torch.zeros(T, k, device=DEV)
    ws = torch.empty(qmm.qmm_moe_workspace_size(E, T, k), dtype=torch.uint8, device=DEV)
    op = qmm.moe_route_op(l, ids, gates, bias=b, n_groups=8, top_groups=4, group_score=qmm.ROUTE_GROUP_TOP2,
                          workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        qmm.qmm_moe_route(op)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            qmm.qmm_moe_route(op)
    torch.cuda.current_stream().wait_stream(side)
    for seed in (2, 3):
        l.copy_(_logits(T, E, "bf16", seed))
        graph.replay()
        rid, _ = R.route(l.float().cpu().numpy(), k, "sigmoid", b.cpu().numpy(), 8, 4, True)
        np.testing.assert_array_equal(ids.cpu().numpy(), rid)


def test_rows_behind_the_last_token_stay():
    qmm = lib()
    l = _logits(9, 64, "f32", 1)
    ids = torch.full((16, 6), -3, dtype=torch.int32, device=DEV)
    gates = torch.full((16, 6), -3.0, device=DEV)
    qmm.qmm_moe_route(qmm.moe_route_op(l, ids[:9], gates[:9]))
    assert (ids[9:] == -3).all() and (gates[9:] == -3).all() and (ids[:9] >= 0).all()


@pytest.mark.parametrize("G,top2", [(1, False), (8, False), (8, True)])
def test_outside_the_domain(G, top2):
    """Infinite logits with softmax and biases that are not finite: some experts of the range, all others as ever."""
    qmm, E, k = lib(), 128, 8
    l = _logits(300, E, "f32", 9)
    l[5::7, 3] = float("inf")
    l[6::7, 40:50] = float("inf")
    for value in (float("inf"), float("-inf"), float("nan")):
        b = _bias(E, 9)
        b[[1, 17, 90]] = value
        for bias in (None, b):
            for score in ("softmax", "sigmoid"):
                ids, _ = _run(qmm, l, k, score, bias=bias, n_groups=G, top_groups=max(1, G // 2), top2=top2)
                assert ((ids >= 0) & (ids < E)).all()
    whole = torch.ones(300, dtype=torch.bool)
    whole[5::7] = whole[6::7] = False
    keep = l[whole.to(DEV)]
    ids, gates = _run(qmm, l, k, "softmax", bias=_bias(E, 9), n_groups=G, top_groups=max(1, G // 2), top2=top2)
    rids, rgates = _run(qmm, keep, k, "softmax", bias=_bias(E, 9), n_groups=G, top_groups=max(1, G // 2), top2=top2)
    assert torch.equal(ids[whole.to(DEV)], rids) and torch.equal(gates[whole.to(DEV)], rgates)
    assert qmm.qmm_last_device_error() == 0


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_more_candidates_than_lanes(score):
    """Few experts left, or few lanes with all of them: chosen in rounds, the switched off ones last and by index."""
    for E, k, G, top in [(56, 13, 8, 6), (384, 14, 8, 1), (128, 16, 2, 1), (512, 33, 1, 1), (1024, 64, 32, 2), (72, 15, 1, 1)]:
        for dtype, masked in [("f32", 0.0), ("bf16", 0.0), ("f16", 0.9)]:
            l = _logits(211, E, dtype, E + k, masked=masked)
            for bias in (None, _bias(E, k)):
                for top2 in ((False, True) if G > 1 else (False,)):
                    _check(lib(), l, k, score, bias, n_groups=G, top_groups=top, top2=top2, renorm=k % 2 == 0)
