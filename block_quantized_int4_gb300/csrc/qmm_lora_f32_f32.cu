// qmm_lora_f32_f32.cu -- low-rank adapters, f32 rows and f32 adapters.
#include "qmm_lora.cuh"

namespace qmm {

LoraKernel lora_kernel_f32_f32(bool low) {
    return low ? lora::lora_kernel<float, float, true> : lora::lora_kernel<float, float, false>;
}

}  // namespace qmm
