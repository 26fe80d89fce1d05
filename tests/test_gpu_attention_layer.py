"""The attention half of a decode layer (examples/attention_layer.py), stage by
stage: each stage against its plain form on the library's own output of the
stage before, and a captured step against the plain calls."""
import os
import sys

import numpy as np
import pytest
import torch

import attn_reference as R
import workloads
from oracle import oracle as O
from parity import assert_close, lib, u16

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_layer_steps():
    qmm = lib()
    from attention_layer import AttentionLayer
    T, steps = 77, 3
    layer = AttentionLayer(qmm, T + steps + 1)
    H, D, Hq, Hkv = workloads.TINYLLAMA["hidden"], layer.HEAD_DIM, layer.HEADS, layer.KV_HEADS
    x = workloads.activations(T, H, seed=3).cuda()
    layer.prefill(x)
    table = layer.table.cpu().numpy()
    o_w = workloads.weights(H, H, workloads.TINYLLAMA["sigma"], 0, 1, "cuda").cpu().numpy()
    oq, od = O.quantize_q4_0(o_w)
    for s in range(steps):
        layer.h.copy_(workloads.activations(1, H, seed=10 + s)[0])
        layer.step()
        torch.cuda.synchronize()
        assert int(layer.pos) == T + s and int(layer.kv_len) == T + s + 1
        qkv = layer.qkv[0].double().cpu().numpy()
        # the token's key and value in the cache, and its rotated queries
        k = R.rotate(qkv[None, Hq:Hq + Hkv], None, 0, table, [T + s], D, False).astype(np.float32)
        K, V = R.cache_values(layer.cache_data.cpu().numpy(), D)
        slot = int(layer.slot)
        page, place = slot // layer.PAGE, slot % layer.PAGE
        assert np.array_equal(K[page, :, place], R.q4_0_values(k)[0])
        assert np.array_equal(V[page, :, place], R.q4_0_values(qkv[Hq + Hkv:]))
        q = R.rotate(qkv[None, :Hq], None, 0, table, [T + s], D, False)
        err = np.abs(layer.q.double().cpu().numpy() - q)
        assert (err <= 4 * 2.0 ** -24 * np.abs(qkv[:Hq]).max(-1)[None, :, None] * 2).all()  # two products, one sum
        # attention of the library's queries: Q8_0, half a code step (and half an fp16 step of d) off the reference
        n = T + s + 1
        at = np.arange(n)
        pg = layer.pages[0].cpu().numpy()[at // layer.PAGE]
        k_all, v_all = (c[pg, :, at % layer.PAGE].transpose(1, 0, 2) for c in (K, V))
        ref, mag, _, _ = R.attention(layer.q.double().cpu().numpy(), k_all, v_all, n, D ** -0.5, True, 0)
        d = layer.attn_d.cpu().numpy().view(np.float16).astype(np.float64)
        got = (layer.attn_q8.cpu().numpy().astype(np.float64).reshape(-1, 32) * d.reshape(-1, 1)).reshape(ref.shape)
        half = np.repeat(d.reshape(-1), 32).reshape(ref.shape) * 0.5
        assert (np.abs(got - ref) <= half * (1 + 2.0 ** -10) + np.abs(ref) * 2.0 ** -10 + 1e-4 * mag).all()
        # O and the residual, from the library's Q8_0
        y, S = O.matmul_int(oq, od, layer.attn_q8.cpu().numpy(), u16(layer.attn_d))
        h = layer.h.double().cpu().numpy()
        assert_close(layer.out[None], y + h, S + np.abs(h), "O product")
        layer.advance()
    assert qmm.qmm_last_device_error() == 0


def test_captured_steps_give_the_same_bits():
    qmm = lib()
    from attention_layer import AttentionLayer
    outs = []
    for graphed in (False, True):
        layer = AttentionLayer(qmm, 400)
        H = workloads.TINYLLAMA["hidden"]
        layer.cache_data.zero_()
        layer.prefill(workloads.activations(300, H, seed=4).cuda())
        layer.h.copy_(workloads.activations(1, H, seed=5)[0])
        layer.step()
        layer.advance()
        torch.cuda.synchronize()
        if graphed:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                layer.step()
                layer.advance()
            run = graph.replay
        else:
            def run():
                layer.step()
                layer.advance()
        got = []
        for _ in range(5):
            run()
            torch.cuda.synchronize()
            got.append(layer.out.clone())
        outs.append((torch.stack(got), layer.cache_data.clone()))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
