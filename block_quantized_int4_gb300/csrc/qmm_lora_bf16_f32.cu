// qmm_lora_bf16_f32.cu -- low-rank adapters, bf16 rows and f32 adapters.
#include "qmm_lora.cuh"

namespace qmm {

LoraKernel lora_kernel_bf16_f32(bool low) {
    return low ? lora::lora_kernel<__nv_bfloat16, float, true> : lora::lora_kernel<__nv_bfloat16, float, false>;
}

}  // namespace qmm
