// qmm_lora_f16_f32.cu -- low-rank adapters, f16 rows and f32 adapters.
#include "qmm_lora.cuh"

namespace qmm {

LoraKernel lora_kernel_f16_f32(bool low) {
    return low ? lora::lora_kernel<__half, float, true> : lora::lora_kernel<__half, float, false>;
}

}  // namespace qmm
