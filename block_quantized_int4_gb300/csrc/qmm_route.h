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
    int vec;                               // rows and lanes start on vector loads' boundaries; 2: all lanes are full
    int softmax, top2, renorm;
    float scale;
};

constexpr int ROUTE_WARPS = 8;  // of a block
// Of the one block that also groups the slots, by the experts of a lane: as many
// as their shared memory allows.
__host__ __device__ constexpr int route_group_warps(int per) { return per <= 8 ? 16 : per <= 16 ? 8 : 4; }

using RouteKernel = void (*)(RouteArgs, MoeWs, int*);

// The kernel for lanes of up to 1 << slot experts; scores: the choice takes
// scores, not logits alone; group: one block, which builds the tables of the
// workspace, too.
RouteKernel route_kernel_f32(int slot, bool scores, bool group);
RouteKernel route_kernel_f16(int slot, bool scores, bool group);
RouteKernel route_kernel_bf16(int slot, bool scores, bool group);

}  // namespace qmm
