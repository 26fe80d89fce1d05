// qmm_lora_bf16_f16.cu -- low-rank adapters, bf16 rows and f16 adapters.
#include "qmm_lora.cuh"

namespace qmm {

LoraKernel lora_kernel_bf16_f16(bool low) {
    return low ? lora::lora_kernel<__nv_bfloat16, __half, true> : lora::lora_kernel<__nv_bfloat16, __half, false>;
}

}  // namespace qmm
