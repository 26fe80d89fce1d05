// qmm_route.h -- what the host and the kernels of qmm_moe_route share.
#pragma once

#include <stdint.h>

#include "qmm_moe_group.cuh"

namespace qmm {

struct RouteArgs {
    const void* logits;
    int64_t ld;
    const float* bias;
    int32_t* ids;
    float* gates;
    int T, k;
    int n_groups, group_size, top_groups;  // n_groups a power of two up to 32
    int per;                               // experts of a lane
    int vec;                               // rows and lanes start on vector loads' boundaries
    int softmax, top2, renorm;
    float scale;
};

using RouteKernel = void (*)(RouteArgs, MoeWs, int*);

// The kernel for lanes of up to 1 << slot experts; group: one block, which
// builds the tables of the workspace, too.
RouteKernel route_kernel_f32(int slot, bool group);
RouteKernel route_kernel_f16(int slot, bool group);
RouteKernel route_kernel_bf16(int slot, bool group);

}  // namespace qmm
