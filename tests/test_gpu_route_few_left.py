"""qmm_moe_route where fewer experts are left than are asked for and 32 bits do not order those that are: the others
follow by index, and such tokens cost what close tokens cost, not the 64-bit choice of all."""
import pytest
import torch

from test_gpu_route import DEV, TYPES, _check, lib

pytestmark = pytest.mark.gpu


def _few(T, E, live, dtype, seed):
    """Logits of 17 to 25: sigmoids within 5e-8 of 1, equal or neighbours in fp32."""
    g = torch.Generator().manual_seed(seed)
    l = torch.full((T, E), float("-inf"))
    at = torch.rand(T, E, generator=g).argsort(1)[:, :live]
    l.scatter_(1, at, 17 + 8 * torch.rand(T, live, generator=g))
    return l.to(TYPES[dtype]).to(DEV)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("E,k,G,top", [(256, 8, 1, 1), (24, 12, 1, 1), (64, 8, 8, 3), (512, 40, 1, 1), (32, 32, 2, 2)])
def test_choices(dtype, E, k, G, top):
    qmm = lib()
    for live in (1, 2, k - 1, k, k + 1):
        l = _few(61, E, min(live, E), dtype, live)
        for b in (torch.zeros(E, device=DEV), 0.1 * (torch.arange(E, device=DEV) % 3).float()):
            for top2 in (False, True) if G > 1 else (False,):
                _check(qmm, l, k, "sigmoid", b, n_groups=G, top_groups=top, top2=top2)


def test_what_they_cost():
    """Against tokens whose closest experts are as many as they ask for, which pairs settle: 182 us for 32,003 of them,
    and 119 us with five left (612 us where those took the 64-bit choice).  The bound is twice the former."""
    E, k = 256, 8
    qmm = lib()
    T, b = 32003, torch.zeros(E, device=DEV)
    took = []
    for live in (k + 2, k - 3):
        l = _few(T, E, live, "f32", 3)
        ids, gates = torch.zeros(T, k, dtype=torch.int32, device=DEV), torch.zeros(T, k, device=DEV)
        op = qmm.moe_route_op(l, ids, gates, bias=b)
        best = float("inf")
        for _ in range(5):
            start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            qmm.qmm_moe_route(op)
            start.record()
            for _ in range(4):
                qmm.qmm_moe_route(op)
            end.record()
            torch.cuda.synchronize()
            best = min(best, start.elapsed_time(end))
        took.append(best / 4 * 1e3)
    assert took[1] <= 2 * took[0], took
