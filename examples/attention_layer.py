"""The attention half of a decoder layer over a 4-bit paged cache, with the
library's entries from end to end, at the TinyLLaMA shape of workloads.py
(hidden 2048, 32 query and 4 key/value heads of 64):

    RMSNorm + QKV product      qmm_gemv_fused_op
    rotate q and k, append     qmm_kv_append_q4_0
    attention, Q8_0 output     qmm_attn_q4_0
    O product + residual       qmm_gemv_fused_op

A decode step is four calls on one stream, captured once in a CUDA graph; the
position, slot and length live in device memory and advance by themselves, so
every replay is the next token.

    python examples/attention_layer.py [--context 2048] [--steps 64]
"""
from __future__ import annotations

import argparse
import os
import sys
import time

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch  # noqa: E402

import workloads  # noqa: E402


class AttentionLayer:
    """One layer's attention for one sequence of up to max_len tokens."""

    HEADS, KV_HEADS, HEAD_DIM, PAGE = 32, 4, 64, 64

    def __init__(self, qmm, max_len, seed=0, device="cuda"):
        self.qmm = qmm
        c = workloads.TINYLLAMA
        H, N = c["hidden"], c["qkv"]
        D = self.HEAD_DIM
        self.qkv_w = qmm.quantize_q4_0(workloads.weights(N, H, c["sigma"], seed, 0, device))
        self.o_w = qmm.quantize_q4_0(workloads.weights(H, H, c["sigma"], seed, 1, device))
        self.gamma = workloads.norm_weights(H, seed, device=device)
        pages = -(-max_len // self.PAGE)
        self.max_len = pages * self.PAGE
        self.cache_data = qmm.kv_cache_data(pages, self.PAGE, self.KV_HEADS, D, device)
        self.cache = qmm.kv_cache(self.cache_data, self.PAGE)
        # any order of pages will do: token j of the sequence is in page table[j / page]
        g = torch.Generator().manual_seed(seed)
        self.pages = torch.randperm(pages, generator=g).to(torch.int32)[None].contiguous().to(device)
        self.table = qmm.rope_table(self.max_len, D, device=device)
        self.rope = qmm.rope(self.table)
        i32 = dict(dtype=torch.int32, device=device)
        self.pos = torch.zeros(1, **i32)        # of the token that a step decodes
        self.kv_len = torch.ones(1, **i32)      # cached tokens, that one included
        self.slot = torch.zeros(1, dtype=torch.int64, device=device)
        self.h = torch.zeros(H, device=device)  # residual stream in
        self.out = torch.zeros(H, device=device)
        self.qkv = torch.zeros(1, N // D, D, device=device)
        self.q = torch.zeros(1, self.HEADS, D, device=device)
        self.attn_q8 = torch.zeros(1, H, dtype=torch.int8, device=device)
        self.attn_d = torch.zeros(1, H // 32, dtype=torch.int16, device=device)
        heads = self.qkv.split([self.HEADS, self.KV_HEADS, self.KV_HEADS], 1)
        self.ops = (
            qmm.gemv_op(*self.qkv_w, N, H, x=self.h, y=self.qkv, norm_w=self.gamma),
            qmm.kv_append_op(self.cache, heads[1], heads[2], self.slot, pos=self.pos, rope=self.rope, q=heads[0],
                             q_out=self.q),
            qmm.attn_op(self.cache, self.q, self.pages, self.kv_len, yq=self.attn_q8, yd=self.attn_d,
                        max_kv=self.max_len),
            qmm.gemv_op(*self.o_w, H, H, xq=self.attn_q8, xd=self.attn_d, residual=self.h, y=self.out),
        )

    def prefill(self, x):
        """Cache the keys and values of x [T][hidden] (fp32), the tokens from position 0, and attend over them:
        the attention's output [T][heads][head_dim]."""
        qmm, T = self.qmm, x.shape[0]
        if T > self.max_len:
            raise ValueError(f"prefill: {T} tokens, and the cache holds {self.max_len}")
        z = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-5) * self.gamma
        xq, xd = qmm.quantize_q8_0(z.contiguous())
        qkv = torch.cat([qmm.gemm(*self.qkv_w, xq[i:i + 64], xd[i:i + 64]) for i in range(0, T, 64)])
        heads = qkv.view(T, -1, self.HEAD_DIM).split([self.HEADS, self.KV_HEADS, self.KV_HEADS], 1)
        at = torch.arange(T, device=x.device)
        slots = self.pages[0].long()[at // self.PAGE] * self.PAGE + at % self.PAGE
        q = torch.empty(T, self.HEADS, self.HEAD_DIM, device=x.device)
        qmm.qmm_kv_append_q4_0(qmm.kv_append_op(self.cache, heads[1], heads[2], slots, pos=at.to(torch.int32),
                                                rope=self.rope, q=heads[0], q_out=q))
        out = torch.empty_like(q)
        n = torch.full((1,), T, dtype=torch.int32, device=x.device)
        qmm.qmm_attn_q4_0(qmm.attn_op(self.cache, q, self.pages, n, out, max_q=T, max_kv=T))
        self.seek(T)
        return out

    def seek(self, position):
        """The next step decodes the token at this position."""
        self.pos.fill_(position)
        self.kv_len.fill_(position + 1)
        self._place()

    def _place(self):
        page = self.pages[0].gather(0, (self.pos // self.PAGE).clamp_max(self.pages.shape[1] - 1).long())
        self.slot.copy_(page.long() * self.PAGE + self.pos % self.PAGE)

    def step(self):
        """One token: out = h + O(attention(norm(h)))."""
        qkv, append, attend, o = self.ops
        self.qmm.qmm_gemv_fused_op(qkv)
        self.qmm.qmm_kv_append_q4_0(append)
        self.qmm.qmm_attn_q4_0(attend)
        self.qmm.qmm_gemv_fused_op(o)

    def advance(self):
        self.pos.add_(1)
        self.kv_len.add_(1)
        self._place()


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--context", type=int, default=2048)
    ap.add_argument("--steps", type=int, default=64)
    a = ap.parse_args()
    from block_quantized_int4_gb300 import _build
    _build.build()
    from block_quantized_int4_gb300 import qmm

    layer = AttentionLayer(qmm, a.context + a.steps + 2)
    layer.prefill(workloads.activations(a.context, workloads.TINYLLAMA["hidden"], seed=1, device="cuda"))
    layer.h.copy_(workloads.activations(1, workloads.TINYLLAMA["hidden"], seed=2, device="cuda")[0])
    layer.step()
    layer.advance()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.step()
        layer.advance()
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    for _ in range(a.steps):
        graph.replay()
    torch.cuda.synchronize()
    us = (time.perf_counter() - t0) / a.steps * 1e6
    status = qmm.qmm_last_device_error()
    print(f"{a.steps} steps behind {a.context} tokens: {us:.1f} us a step (QKV, append, attention, O; positions "
          f"advanced on the device), status {qmm.status_string(status)}")
    return status


if __name__ == "__main__":
    sys.exit(main())
