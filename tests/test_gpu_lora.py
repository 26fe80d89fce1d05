"""qmm_lora against adapters in 64 bits."""
import itertools

import pytest
import torch

from parity import lib
import lora_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def _mat(shape, dtype, g, scale=1.0, pad=0, at=0, fill=float("nan")):
    """A tensor whose last dimension's rows are `pad` values apart, `at` values behind an aligned address; NaN between."""
    lead, n = shape[:-1], shape[-1]
    m = 1
    for v in lead:
        m *= v
    buf = torch.full((m * (n + pad) + at,), fill, dtype=TYPES[dtype], device=DEV)
    t = buf[at:].view(*lead, n + pad)[..., :n]
    t.copy_(scale * torch.randn(shape, generator=g))
    return t


class Case:
    def __init__(self, T, N, K, rank, segs, x="f32", w="bf16", y=None, adapters=3, base=True, ranks=None, scales=True,
                 xpad=0, apad=0, bpad=0, ypad=0, bat=0, yat=0, seed=1, uniform=False):
        g = torch.Generator().manual_seed(seed)
        self.qmm, self.segs, self.uniform = lib(), segs, uniform
        y = y or x
        self.x = _mat((T, K), x, g, pad=xpad)
        self.x[torch.rand(T, K, generator=g).to(DEV) < 0.01] *= 20
        self.a = _mat((adapters, rank, K), w, g, K ** -0.5, pad=apad)
        self.b = _mat((adapters, N, rank), w, g, 0.05, pad=bpad, at=bat)
        self.base = _mat((T, N), y, g, pad=ypad, at=yat) if base else None
        buf = torch.full((T * (N + ypad) + yat,), -7.0, dtype=TYPES[y], device=DEV)
        self.buf, self.y = buf, buf[yat:].view(T, N + ypad)[:, :N]
        self.ranks = ranks
        if ranks is not None:  # what lies behind a rank is never used
            for i, r in enumerate(ranks):
                self.a[i, r:] = float("nan")
                self.b[i, :, r:] = float("inf")
        self.scales = (0.5 + 2 * torch.rand(adapters, generator=g)).to(DEV) if scales else None

    def op(self, in_place=False):
        i32 = dict(dtype=torch.int32, device=DEV)
        start = None if self.uniform else torch.tensor([s[0] for s in self.segs] + [self.segs[-1][1]], **i32)
        return self.qmm.lora_op(self.x, self.a, self.b, self.y,
                                torch.tensor([s[2] for s in self.segs], **i32), base=self.y if in_place else self.base,
                                seg_start=start, scales=self.scales,
                                ranks=None if self.ranks is None else torch.tensor(self.ranks, **i32))

    def want(self):
        return R.lora(self.x, self.a, self.b, self.segs, self.base, self.ranks, self.scales, self.y.dtype)

    def check(self):
        self.qmm.qmm_lora(self.op())
        want, err = self.want()
        R.check(self.y, want, err)
        outside = want.isnan().to(DEV)
        assert (self.y[outside] == -7).all()  # rows in no segment
        pad = self.buf[self.buf.numel() - self.y.shape[0] * self.y.stride(0):].view(self.y.shape[0], -1)
        assert (pad[:, self.y.shape[1]:] == -7).all()
        assert self.qmm.qmm_last_device_error() == 0
        return self.y.clone()


@pytest.mark.parametrize("x,w", list(itertools.product(TYPES, TYPES)))
@pytest.mark.parametrize("rank", [1, 8, 16, 17, 64, 100])
def test_types_and_ranks(x, w, rank):
    for y in {x, "f32"}:
        Case(37, 200, 320, rank, [(0, 1, 0), (1, 20, 2), (20, 37, 1)], x, w, y, seed=rank).check()
        Case(3, 64, 96, rank, [(0, 3, 1)], x, w, y, base=False, scales=False, seed=rank).check()


@pytest.mark.parametrize("x,w", [("f32", "f32"), ("f32", "f16"), ("f16", "f16"), ("bf16", "bf16")])
@pytest.mark.parametrize("rows", [1, 2, 8, 15, 16, 17, 33, 48, 49, 63, 64, 65, 130])
def test_rows_of_a_segment(x, w, rows):
    Case(2 * rows, 130, 512, 24, [(0, rows, 0), (rows, 2 * rows, 1)], x, w, uniform=True, seed=rows).check()
    Case(rows + 1, 130, 512, 40, [(0, 1, 0), (1, rows + 1, 1)], x, w, seed=rows).check()


@pytest.mark.parametrize("x,w", [("f32", "f32"), ("f32", "bf16"), ("f16", "f16"), ("bf16", "bf16")])
@pytest.mark.parametrize("rank", [128, 200, 256])
@pytest.mark.parametrize("rows", [1, 20, 40, 64])
def test_large_ranks(x, w, rank, rows):
    Case(rows, 96, 256, rank, [(0, rows, 0)], x, w, adapters=1, seed=rank).check()


@pytest.mark.parametrize("K", [32, 64, 96, 224, 256, 800, 2048, 5632, 8192])
@pytest.mark.parametrize("N", [1, 7, 31, 33, 2051])
def test_sizes(K, N):
    Case(5, N, K, 16, [(0, 1, 0), (1, 2, 1), (2, 5, 2)], "f32", "f16", seed=K + N).check()
    Case(21, N, K, 24, [(0, 4, 2), (4, 21, 1)], "bf16", "bf16", seed=K + N).check()


@pytest.mark.parametrize("x,w", [("f32", "f32"), ("f32", "bf16"), ("f16", "f16"), ("bf16", "bf16")])
def test_strides_and_alignment(x, w):
    """Rows of x and A a multiple of 16 bytes apart; B and y at any element."""
    for rank, bpad, bat, ypad, yat in [(16, 0, 0, 0, 0), (16, 1, 0, 3, 0), (16, 0, 1, 0, 1), (24, 8, 0, 8, 0),
                                       (24, 3, 2, 5, 3), (13, 0, 0, 0, 2), (40, 4, 0, 4, 4), (12, 4, 4, 8, 8)]:
        for N in (64, 71):
            Case(19, N, 128, rank, [(0, 2, 1), (2, 19, 0)], x, w, bpad=bpad, bat=bat, ypad=ypad, yat=yat, xpad=8, apad=16,
                 seed=rank).check()


@pytest.mark.parametrize("x,w,y", [("f32", "f32", "f32"), ("f32", "bf16", "f32"), ("f16", "f16", "f16"),
                                   ("bf16", "bf16", "bf16"), ("bf16", "bf16", "f32"), ("f16", "f32", "f16")])
@pytest.mark.parametrize("rank", [40, 64, 100, 128])
def test_prompts(x, w, y, rank):
    """Enough rows for tiles of 128: whole ones, and 1 to 127 rows left of a segment."""
    lens = [1, 300, 128, 0, 17, 250, 33, 511, 90, 64, 200, 127]
    segs, at = [], 2
    for i, n in enumerate(lens):
        segs.append((at, at + n, i % 4 - 1))
        at += n
    Case(at + 5, 200, 192, rank, segs, x, w, y, seed=rank).check()
    Case(at + 5, 71, 2048, rank, segs, x, w, y, ranks=[rank, 7, 33], base=False, ypad=1, seed=rank).check()
    if rank == 64:
        Case(4 * 400, 100, 128, rank, [(400 * i, 400 * i + 400, i % 3) for i in range(4)], x, w, y, uniform=True).check()


def test_ranks_of_their_own():
    """Smaller adapters in the same storage: NaN and infinity behind their ranks; a rank of 0 is none."""
    for x, w in (("f32", "f16"), ("f32", "f32"), ("bf16", "bf16"), ("f16", "f16")):
        segs = [(0, 1, 0), (1, 3, 1), (3, 30, 2), (30, 31, 3), (31, 60, 4), (60, 62, 5)]
        Case(62, 100, 256, 64, segs, x, w, adapters=6, ranks=[64, 1, 8, 0, 33, 7]).check()
        Case(62, 100, 256, 16, segs, x, w, adapters=6, ranks=[16, 1, 8, 0, 5, 7]).check()
        Case(62, 100, 256, 160, segs, x, w, adapters=6, ranks=[160, 1, 65, 0, 129, 64]).check()


def test_segments():
    """None, empty ones, one adapter many times, rows before the first and behind the last."""
    segs = [(3, 3, 0), (3, 10, -1), (10, 10, 1), (10, 80, 2), (80, 81, 2), (81, 81, -1), (81, 100, 2), (100, 101, -1)]
    for base in (False, True):
        Case(110, 70, 160, 8, segs, "f32", "f16", base=base).check()
        Case(110, 70, 160, 8, segs, "bf16", "bf16", base=base, ypad=3).check()
    many = [(i, i + 1, i % 5 - 1) for i in range(700)]
    Case(700, 40, 64, 8, many, "f32", "f16", adapters=4, uniform=True).check()
    Case(700, 40, 64, 8, many, "f32", "f16", adapters=4).check()
    Case(710, 40, 64, 8, [(0, 0, 0)] * 600 + [(0, 710, 1)], "f32", "f16").check()


def test_same_bits_on_every_call():
    c = Case(40, 128, 512, 32, [(0, 40, 1)], "f32", "bf16")
    whole = c.check()
    assert torch.equal(whole, c.check())
    c.segs = [(0, 40, 1), (40, 40, 0)]
    assert torch.equal(whole, c.check())


def test_in_place():
    for x, y in (("f32", "f32"), ("f16", "f16"), ("bf16", "bf16"), ("bf16", "f32")):
        c = Case(50, 133, 256, 24, [(0, 1, 0), (1, 30, 1), (30, 32, -1), (32, 50, 2)], x, "f16", y, ypad=3)
        apart = c.check()
        c.y.copy_(c.base)
        c.qmm.qmm_lora(c.op(in_place=True))
        assert torch.equal(c.y, apart)


def test_rows_that_are_not_finite_stay_by_themselves():
    for x, w in (("f32", "f32"), ("f32", "f16"), ("f16", "f16"), ("bf16", "bf16")):
        c = Case(20, 64, 128, 16, [(0, 20, 0)], x, w)
        want, err = c.want()
        c.x[3, 5] = float("nan")
        c.x[11, 7] = float("inf")
        c.qmm.qmm_lora(c.op())
        bad = torch.tensor([3, 11])
        assert not torch.isfinite(c.y[bad.to(DEV)]).any()
        keep = torch.tensor([i for i in range(20) if i not in (3, 11)])
        R.check(c.y[keep.to(DEV)], want[keep], err[keep])


def test_values_out_of_range():
    """Starts, adapters and ranks outside their ranges set the error word and nothing is read out of range."""
    qmm = lib()
    i32 = dict(dtype=torch.int32, device=DEV)
    c = Case(20, 64, 128, 16, [(0, 10, 0), (10, 20, 1)], "f32", "f16")
    base, ok = torch.tensor([0, 10, 20], **i32), torch.tensor([0, 1], **i32)
    ranks = torch.tensor([16, 16, 16], **i32)
    assert qmm.qmm_last_device_error() == 0
    for start, adapter, r in [([-1, 10, 20], ok, ranks), ([0, 10, 21], ok, ranks), ([0, 30, 20], ok, ranks),
                              ([0, -5, 20], ok, ranks), (base, [3, 1], ranks), (base, [0, -2], ranks),
                              (base, ok, [16, 17, 16]), (base, ok, [-1, 16, 16])]:
        t = lambda v: torch.tensor(v, **i32) if isinstance(v, list) else v  # noqa: E731
        qmm.qmm_lora(qmm.lora_op(c.x, c.a, c.b, c.y, t(adapter), base=c.base, seg_start=t(start), ranks=t(r)))
        assert qmm.qmm_last_device_error() == 10
    # an adapter outside its range counts as none; the other segment is done
    c.y.fill_(-7)
    qmm.qmm_lora(qmm.lora_op(c.x, c.a, c.b, c.y, torch.tensor([3, 1], **i32), base=c.base, seg_start=base,
                             scales=c.scales))
    assert qmm.qmm_last_device_error() == 10
    want, err = R.lora(c.x, c.a, c.b, [(0, 10, -1), (10, 20, 1)], c.base, None, c.scales, c.y.dtype)
    R.check(c.y, want, err)


def test_captured_on_another_stream():
    c = Case(70, 200, 512, 16, [(0, 1, 0), (1, 70, 1)], "bf16", "bf16")
    op = c.op()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.qmm.qmm_lora(op)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            c.qmm.qmm_lora(op)
            c.qmm.qmm_lora(op)
    torch.cuda.current_stream().wait_stream(side)
    for seed in (3, 4):
        c.x.copy_(torch.randn(c.x.shape, generator=torch.Generator().manual_seed(seed)))
        c.y.fill_(-7)
        graph.replay()
        R.check(c.y, *c.want())


@pytest.mark.parametrize("x,w", [("f32", "bf16"), ("bf16", "bf16"), ("f16", "f32")])
def test_no_adapter(x, w):
    """Segments of none take base as it is, or zeros: whole rows, odd ones, base at any element; in place nothing."""
    for N, ypad, yat in [(1, 0, 0), (9, 0, 0), (64, 0, 0), (71, 1, 0), (2051, 0, 1), (4104, 8, 8), (5000, 4, 2)]:
        for base in (True, False):
            c = Case(80, N, 64, 8, [(0, 64, -1), (64, 67, 0), (67, 80, -1)], x, w, ypad=ypad, yat=yat, base=base, seed=N)
            c.check()
            none = torch.tensor([*range(64), *range(67, 80)], device=DEV)
            assert torch.equal(c.y[none], c.base[none] if base else torch.zeros_like(c.y[none]))


@pytest.mark.parametrize("x,w", [("f32", "bf16"), ("bf16", "bf16"), ("f32", "f32")])
def test_offsets_that_pass_32_bits(x, w):
    """Rows of A, adapters in storage, rows of x, base and y more than 2^31 values from their first."""
    rank, K, N, far = 9, 64, 40, (1 << 28) + 64
    c = Case(9, N, K, rank, [(0, 4, 1), (4, 9, 0)], x, w, adapters=2, seed=3)

    def spread(t, stride):  # the same values, `stride` apart in the second last dimension
        gap = torch.empty((t.shape[-2] - 1) * stride + t.shape[-1], dtype=t.dtype, device=DEV)
        out = torch.as_strided(gap, t.shape[-2:], (stride, 1))
        out.copy_(t)
        return out

    want, err = c.want()
    a, b = c.a, c.b
    for i in range(2):  # one adapter at a time: rows of A far apart
        c.a = spread(a[i], far)[None]
        c.b = b[i:i + 1]
        scales, c.scales = c.scales, c.scales[i:i + 1]
        lo, hi = (0, 4) if i else (4, 9)
        start = torch.tensor([lo, hi], dtype=torch.int32, device=DEV)
        c.y.fill_(-7)
        c.qmm.qmm_lora(c.qmm.lora_op(c.x, c.a, c.b, c.y, torch.zeros(1, dtype=torch.int32, device=DEV), base=c.base,
                                     seg_start=start, scales=c.scales))
        R.check(c.y[lo:hi], want[lo:hi], err[lo:hi])
        c.scales = scales
    c.a, c.b = a, b
    del a, b
    c.x, c.base, y = spread(c.x, far), spread(c.base, far), c.y
    c.y = spread(c.y, far)
    c.qmm.qmm_lora(c.op())
    R.check(c.y, want, err)
    c.x, c.base, c.y = c.x.contiguous(), c.base.contiguous(), y
    for name in ("a", "b"):  # whole adapters far apart
        t = getattr(c, name)
        buf = torch.empty((1 << 31) + 64 + t[0].numel(), dtype=t.dtype, device=DEV)
        v = torch.as_strided(buf, t.shape, ((1 << 31) + 64, t.shape[-1], 1))
        v.copy_(t)
        setattr(c, name, v)
    c.y.fill_(-7)
    c.qmm.qmm_lora(c.op())
    R.check(c.y, want, err)
    assert c.qmm.qmm_last_device_error() == 0


@pytest.mark.parametrize("x,w", [("f32", "f32"), ("f32", "bf16"), ("f16", "f16"), ("bf16", "bf16")])
def test_few_rows_with_many_columns(x, w):
    """A tile's columns shared by several clusters: even and odd numbers of them, a cut of one CTA, no adapter."""
    for N in (2048, 6000, 8191, 28672):
        Case(3, N, 256, 16, [(0, 1, 0), (1, 1, 2), (1, 3, 1)], x, w, seed=N).check()
        Case(70, N, 64, 40, [(0, 64, 0), (64, 70, -1)], x, w, seed=N).check()
    c = Case(1, 20000, 2048, 8, [(0, 1, 0)], x, w)
    whole = c.check()
    c.y.copy_(c.base)
    c.qmm.qmm_lora(c.op(in_place=True))
    assert torch.equal(c.y, whole)


@pytest.mark.parametrize("w", ["f32", "f16", "bf16"])
def test_rows_of_b_on_4_bytes(w):
    """Ranks and strides that are no multiple of 16 bytes: 4-byte copies, plain ones, and the last columns of either."""
    for rank, bpad, bat in [(6, 0, 0), (44, 0, 0), (42, 4, 2), (7, 0, 0), (67, 0, 1), (66, 0, 4), (130, 0, 0)]:
        for N in (64, 75, 515):
            Case(18, N, 128, rank, [(0, 1, 1), (1, 18, 0)], "f32", w, bpad=bpad, bat=bat, seed=rank).check()
            Case(18, N, 128, rank, [(0, 1, 1), (1, 18, 0)], "f32", w, bpad=bpad, bat=bat, ranks=[rank, 1, rank - 1]).check()
