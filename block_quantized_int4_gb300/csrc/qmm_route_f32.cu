// qmm_route_f32.cu -- routing to experts, f32 logits.
#include "qmm_route.cuh"

namespace qmm {

RouteKernel route_kernel_f32(int slot, bool scores, bool group) { return route::kernel_of<float>(slot, scores, group); }

}  // namespace qmm
