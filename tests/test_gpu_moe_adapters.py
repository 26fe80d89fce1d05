"""The MoE half of a decoder layer for a batch of requests: routing with a
bias and groups, the experts' products, and beside them a shared projection
with the requests' adapters; captured in one graph, each stage against 64 bits."""
import pytest
import torch

from parity import lib
import lora_reference
import route_reference
import workloads

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _planes(qmm, E, N, K, seed):
    qs = torch.zeros(E, N, K // 2, dtype=torch.uint8, device=DEV)
    d = torch.zeros(E, N, K // 32, dtype=torch.int16, device=DEV)
    for e in range(E):
        q, s = qmm.quantize_q4_0(workloads.weights(N, K, 0.05, seed, e, DEV))
        qs[e], d[e] = q, s
    return qs, d


def _values(qs, d):
    """What Q4_0 planes stand for, 64 bits [..., N, K]."""
    b = qs.unflatten(-1, (-1, 16))
    codes = torch.cat([b & 15, b >> 4], -1).double() - 8
    return (codes * d.view(torch.float16).double()[..., None]).flatten(-2)


def _q8(qmm, x):
    q, d = qmm.quantize_q8_0(x)
    return (q.double().unflatten(-1, (-1, 32)) * d.view(torch.float16).double()[..., None]).flatten(-2)


@pytest.mark.parametrize("T", [1, 5, 70])
def test_layer(T):
    qmm = lib()
    H, F, E, k, N, rank, n = 512, 256, 16, 4, 1000, 16, 3
    g = torch.Generator().manual_seed(T)
    gu, down = _planes(qmm, E, 2 * F, H, 1), _planes(qmm, E, H, F, 2)
    proj = qmm.quantize_q4_0(workloads.weights(N, H, 0.05, 3, 0, DEV))
    gate_w = (0.1 * torch.randn(E, H, generator=g)).to(DEV)
    bias = (0.05 * torch.randn(E, generator=g)).to(DEV)
    a = (torch.randn(n, rank, H, generator=g) * H ** -0.5).half().to(DEV)
    b = (0.1 * torch.randn(n, N, rank, generator=g)).half().to(DEV)
    adapter = torch.randint(-1, n, (T,), generator=g).to(torch.int32).to(DEV)
    scales = torch.tensor([0.5, 1.0, 2.0], device=DEV)

    x, logits = torch.zeros(T, H, device=DEV), torch.zeros(T, E, device=DEV)
    ids, gates = torch.zeros(T, k, dtype=torch.int32, device=DEV), torch.zeros(T, k, device=DEV)
    ws_bytes = qmm.qmm_moe_workspace_size(E, T, k)
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=DEV)
    h, z, y = torch.zeros(T * k, F, device=DEV), torch.zeros(T * k, H, device=DEV), torch.zeros(T, H, device=DEV)
    xq, xd = torch.zeros(T, H, dtype=torch.int8, device=DEV), torch.zeros(T, H // 32, dtype=torch.int16, device=DEV)
    out = torch.zeros(T, N, device=DEV)
    route = qmm.moe_route_op(logits, ids, gates, bias=bias, n_groups=4, top_groups=2,
                             group_score=qmm.ROUTE_GROUP_TOP2, scale=2.5, workspace=ws)
    lora = qmm.lora_op(x, a, b, out, adapter, base=out, scales=scales)

    def layer():
        qmm.qmm_moe_route(route)
        qmm.qmm_moe_gemv_gate_up(*gu, E, 2 * F, H, T, k, x, None, None, 0, h, ws, ws_bytes)
        qmm.qmm_moe_gemv_pregrouped_f32(*down, E, H, F, T, k, h, 1, z, ws, ws_bytes)
        qmm.qmm_moe_combine(z, gates, T, k, H, y)
        qmm.qmm_quantize_q8_0(x, T, H, H, xq, xd)
        for t in range(0, T, 64):  # the product's largest batch
            m = min(64, T - t)
            qmm.qmm_gemm_q4_0_q8_0(*proj, N, H, m, xq[t:], xd[t:], out[t:], N)
        qmm.qmm_lora(lora)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            layer()
    torch.cuda.current_stream().wait_stream(side)
    w_gu, w_down, w_proj = _values(*gu), _values(*down), _values(*proj)
    for seed in (11, 12):
        x.copy_(workloads.activations(T, H, seed))
        logits.copy_(x @ gate_w.T)
        graph.replay()
        torch.cuda.synchronize()
        rid, rg = route_reference.route(logits.cpu().numpy(), k, "sigmoid", bias.cpu().numpy(), 4, 2, True, True, 2.5)
        assert (ids.cpu().numpy() == rid).all()
        assert (abs(gates.cpu().numpy() - rg) <= route_reference.gate_tolerance(logits.cpu().numpy(), rid, rg)).all()
        # the experts' products on Q8_0 rows, 1e-5 of the sum of magnitudes as everywhere
        e = ids.long().flatten()
        row = _q8(qmm, x).repeat_interleave(k, 0)
        p = torch.einsum("sk,snk->sn", row, w_gu[e])
        mag = torch.einsum("sk,snk->sn", row.abs(), w_gu[e].abs())
        gate, up = p[:, 0::2], p[:, 1::2]
        slack = 1e-5 * (mag[:, 0::2] * (up.abs() + 1) + mag[:, 1::2] * gate.abs()) * 2 + 1e-6
        assert ((h.double() - gate * torch.sigmoid(gate) * up).abs() <= slack).all()
        row = _q8(qmm, h)
        want = torch.einsum("sk,snk->sn", row, w_down[e])
        mag = torch.einsum("sk,snk->sn", row.abs(), w_down[e].abs())
        assert ((z.double() - want).abs() <= 1e-5 * mag + 1e-6).all()
        want = (gates.double()[..., None] * z.double().view(T, k, H)).sum(1)
        assert ((y.double() - want).abs() <= 1e-6 * (gates[..., None] * z.view(T, k, H).abs()).sum(1) + 1e-6).all()
        # the projection and the adapters' part
        base = _q8(qmm, x) @ w_proj.T
        segs = [(t, t + 1, int(adapter[t])) for t in range(T)]
        want, err = lora_reference.lora(x, a, b, segs, base, None, scales)
        err = err + 1e-5 * (_q8(qmm, x).abs() @ w_proj.abs().T).cpu() + 1e-6
        lora_reference.check(out, want, err)
    assert qmm.qmm_last_device_error() == 0
