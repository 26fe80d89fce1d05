// qmm_lora_f16_bf16.cu -- low-rank adapters, f16 rows and bf16 adapters.
#include "qmm_lora.cuh"

namespace qmm {

LoraKernel lora_kernel_f16_bf16(bool low) {
    return low ? lora::lora_kernel<__half, __nv_bfloat16, true> : lora::lora_kernel<__half, __nv_bfloat16, false>;
}

}  // namespace qmm
