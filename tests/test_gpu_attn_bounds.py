"""bf16 calls of many rows on the warp-MMA kernel, under the bound of that
kernel: test_gpu_attn.py allows for keys and values rounded to fp16 from 32 rows a
key/value head on, but only the tensor-memory kernel rounds them."""
import pytest

import test_gpu_attn as G
from parity import lib
from test_attn_plan import TMEM, _params

pytestmark = pytest.mark.gpu


def _check(c, tmem, **kw):
    kernel, _ = c.qmm.qmm_debug_attn_plan(c.op(c.run(**kw), **kw))
    assert (kernel == TMEM) == tmem
    out = c.run(**kw)
    if not tmem:
        c.max_q = 0  # read by the check alone from here on: fewer than 32 rows
    c.check(out)


@pytest.mark.parametrize("case", _params(G.test_many_rows), ids=str)
def test_warp_mma(case):
    c = case
    _check(G.Case(lib(), c["lens"], c["nqs"], c["Hq"], c["Hkv"], c["D"], c["page"], "bf16", c["causal"], c["window"],
                  seed=c["D"] + len(c["lens"]), q_start=True), False)


@pytest.mark.parametrize("n,L,Hq,Hkv,D", [(17, 400, 8, 2, 128), (40, 700, 8, 1, 96), (9, 5000, 16, 2, 128)])
def test_warp_mma_chunks(n, L, Hq, Hkv, D):
    _check(G.Case(lib(), [L, L // 2, n], [n] * 3, Hq, Hkv, D, 96, "bf16", seed=n), False)


@pytest.mark.parametrize("lens,nqs,Hq,Hkv,D", [([300, 128], [64, 64], 4, 1, 64), ([3, 700, 0, 257], [130, 40, 64, 1], 4, 2, 128)])
def test_tensor_memory(lens, nqs, Hq, Hkv, D):
    c = G.Case(lib(), lens, nqs, Hq, Hkv, D, 64, "bf16", seed=D, q_start=True, extra_kv=G.MAY_GROW // 64)
    _check(c, True, max_kv=G.MAY_GROW)
