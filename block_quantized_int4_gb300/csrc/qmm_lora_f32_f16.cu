// qmm_lora_f32_f16.cu -- low-rank adapters, f32 rows and f16 adapters.
#include "qmm_lora.cuh"

namespace qmm {

LoraKernel lora_kernel_f32_f16(bool low) {
    return low ? lora::lora_kernel<float, __half, true> : lora::lora_kernel<float, __half, false>;
}

}  // namespace qmm
