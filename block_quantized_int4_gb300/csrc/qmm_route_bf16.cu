// qmm_route_bf16.cu -- routing to experts, bf16 logits.
#include "qmm_route.cuh"

namespace qmm {

RouteKernel route_kernel_bf16(int slot, bool scores, bool group) { return route::kernel_of<__nv_bfloat16>(slot, scores, group); }

}  // namespace qmm
