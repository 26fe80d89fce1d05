"""The forms that rotary heads and the cache append take for prompts (four
groups of heads a warp, adjacent and halved pairs, three types)."""
import numpy as np
import pytest
import torch

import attn_reference as R
import workloads
from parity import lib
from test_gpu_rope_append import DEV, TYPES, _append, _check_cache, _heads, _np, _rope_bound, _table

pytestmark = pytest.mark.gpu


PROMPTS = [  # T, H, D, n_rot, norm
    (5000, 5, 32, 32, True), (5000, 9, 96, 48, False), (2500, 7, 256, 256, True), (5000, 1, 128, 128, True),
    (3000, 9, 128, 64, True), (3000, 33, 64, 64, False)]


@pytest.mark.parametrize("T,H,D,n_rot,norm", PROMPTS)
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_prompt_heads(T, H, D, n_rot, norm, pairs, dtype):
    """Heads that are not a multiple of what a warp takes, from a fused projection's output, and in place."""
    qmm = lib()
    dt = TYPES[dtype]
    x = _heads(T, H, D, dt, 7, True)
    gamma = workloads.norm_weights(D, seed=4).to(DEV) if norm else None
    table = _table(50, n_rot)
    pos = torch.arange(T, dtype=torch.int32, device=DEV) * 7 % 50
    base = torch.full((T, H + 1, D), 7.0, dtype=dt, device=DEV)
    y = base[:, :H]
    qmm.qmm_rope_heads(qmm.rope_op(x, y, pos, qmm.rope(table, pairs), norm_w=gamma))
    n = lambda t: None if t is None else _np(t)  # noqa: E731
    ref = R.rotate(_np(x), n(gamma), 1e-5, n(table), pos.cpu().numpy(), n_rot, pairs)
    bound = _rope_bound(_np(x), n(gamma), n(table), pos.cpu().numpy(), n_rot, pairs, ref, dt)
    err = np.abs(_np(y) - ref)
    assert (err <= bound).all(), (err / bound).max()
    assert (base[:, H] == 7.0).all()
    z = _heads(T, H + 2, D, dt, 8, False)
    z[:, 1:H + 1] = x
    around = z[:, [0, H + 1]].clone()
    qmm.qmm_rope_heads(qmm.rope_op(z[:, 1:H + 1], z[:, 1:H + 1], pos, qmm.rope(table, pairs), norm_w=gamma))
    assert torch.equal(z[:, 1:H + 1], y) and torch.equal(z[:, [0, H + 1]], around)
    assert qmm.qmm_last_device_error() == 0


@pytest.mark.parametrize("T,Hq,Hkv,D,n_rot,norm", [(1200, 9, 3, 96, 96, True), (2000, 7, 1, 32, 16, False),
                                                  (1500, 5, 2, 256, 128, True), (1500, 33, 1, 128, 128, False)])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_prompt_append(T, Hq, Hkv, D, n_rot, norm, pairs, dtype):
    qmm = lib()
    page = 64
    n_pages = -(-T // page) + 2
    slots = torch.randperm(n_pages * page, generator=torch.Generator().manual_seed(T))[:T].to(DEV)
    slots[::97] = -1
    _, data, before, want = _append(qmm, T, Hq, Hkv, D, n_rot, pairs, norm, dtype, page, n_pages, slots)
    _check_cache(data, before, slots, want, page, D)
    assert qmm.qmm_last_device_error() == 0
