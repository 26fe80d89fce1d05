// qmm_moe_route.cu -- qmm_moe_route on the host: argument checks and launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "qmm.h"
#include "qmm_internal.h"
#include "qmm_route.h"

namespace qmm {
namespace {

// Tokens up to which one block routes them all and groups their slots, too:
// beyond that the grouping is a launch of its own.
constexpr int ONE_BLOCK_TOKENS = 64;

bool off(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

size_t size_of(int dtype) { return dtype == QMM_F32 ? 4 : 2; }

qmm_status check(const qmm_moe_route_op& op) {
    if (op.T < 0 || op.E <= 0 || op.k <= 0 || op.n_groups <= 0 || op.top_groups <= 0 || op.ld < op.E ||
        !std::isfinite(op.scale))
        return QMM_ERR_ARG;
    if (op.dtype != QMM_F32 && op.dtype != QMM_F16 && op.dtype != QMM_BF16) return QMM_ERR_ARG;
    if (op.score != QMM_ROUTE_SOFTMAX && op.score != QMM_ROUTE_SIGMOID) return QMM_ERR_ARG;
    if (op.group_score != QMM_ROUTE_GROUP_MAX && op.group_score != QMM_ROUTE_GROUP_TOP2) return QMM_ERR_ARG;
    if (op.E > QMM_ROUTER_MAX_EXPERTS || op.k > QMM_ROUTER_MAX_K || op.n_groups > 32 ||
        (op.n_groups & (op.n_groups - 1)) || op.E % op.n_groups || op.top_groups > op.n_groups ||
        op.k > op.E / op.n_groups * op.top_groups || op.ld > int64_t(1) << 40)
        return QMM_ERR_SHAPE;
    if (op.workspace && (int64_t)op.T * op.k > 1 << 24) return QMM_ERR_SHAPE;
    if (op.T == 0) return QMM_OK;
    if (!op.logits || !op.ids || !op.gates) return QMM_ERR_ARG;
    if (op.workspace && op.workspace_bytes < moe_ws_bytes(op.E, (int64_t)op.T * op.k)) return QMM_ERR_WORKSPACE;
    if (off(op.logits, size_of(op.dtype)) || off(op.bias, 4) || off(op.ids, 4) || off(op.gates, 4) ||
        off(op.workspace, 16))
        return QMM_ERR_ALIGN;
    return QMM_OK;
}

}  // namespace
}  // namespace qmm

using namespace qmm;

extern "C" qmm_status qmm_moe_route(const qmm_moe_route_op* op, void* stream) {
    if (!op) return QMM_ERR_ARG;
    if (qmm_status s = check(*op)) return s;
    if (op->T == 0) return QMM_OK;
    int sms = 0, optin = 0;
    if (!device_facts(&sms, &optin)) return QMM_ERR_DEVICE;
    RouteArgs a = {};
    a.logits = op->logits;
    a.ld = op->ld;
    a.bias = op->bias;
    a.ids = op->ids;
    a.gates = op->gates;
    a.T = op->T;
    a.k = op->k;
    a.n_groups = op->n_groups;
    a.group_size = op->E / op->n_groups;
    a.top_groups = op->top_groups;
    a.softmax = op->score == QMM_ROUTE_SOFTMAX;
    a.top2 = op->group_score == QMM_ROUTE_GROUP_TOP2;
    a.renorm = op->renormalize != 0;
    a.scale = op->scale;
    // Lanes hold 1, 2, 4, .. 32 experts of one group, up to four side by side.
    const int lanes = 32 / a.n_groups;
    int slot = 0;
    while ((lanes << slot) < a.group_size) ++slot;
    const int beside = std::min(4, 1 << slot);
    a.vec = a.group_size % beside == 0 && !off(op->logits, beside * size_of(op->dtype)) &&
            (op->T == 1 || op->ld % beside == 0);
    if (a.vec && lanes << slot == a.group_size) a.vec = 2;
    const bool scores = op->bias || (a.n_groups > 1 && a.top2);
    const bool group = op->workspace && op->T <= ONE_BLOCK_TOKENS;
    const RouteKernel kernel = op->dtype == QMM_F32   ? route_kernel_f32(slot, scores, group)
                               : op->dtype == QMM_F16 ? route_kernel_f16(slot, scores, group)
                                                      : route_kernel_bf16(slot, scores, group);
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(32 * (group ? route_group_warps(1 << slot) : ROUTE_WARPS));
    cfg.gridDim = dim3(
        group ? 1 : (unsigned)std::min<int64_t>(((int64_t)op->T + ROUTE_WARPS - 1) / ROUTE_WARPS, 8 * (int64_t)sms));
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const MoeWs ws = op->workspace ? moe_ws(op->workspace, op->E) : MoeWs{};
    if (cudaLaunchKernelEx(&cfg, kernel, a, ws, device_error_word()) != cudaSuccess) {
        cudaGetLastError();
        return QMM_ERR_CUDA;
    }
    if (op->workspace && !group)
        return qmm_moe_group_ids(op->ids, op->T, op->k, op->E, op->workspace, op->workspace_bytes, stream);
    return QMM_OK;
}
