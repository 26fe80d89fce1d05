// qmm_route_f16.cu -- routing to experts, f16 logits.
#include "qmm_route.cuh"

namespace qmm {

RouteKernel route_kernel_f16(int slot, bool scores, bool group) { return route::kernel_of<__half>(slot, scores, group); }

}  // namespace qmm
