// qmm_lora_f16_f16.cu -- low-rank adapters, f16 rows and f16 adapters.
#include "qmm_lora.cuh"

namespace qmm {

LoraKernel lora_kernel_f16_f16(bool low) {
    return low ? lora::lora_kernel<__half, __half, true> : lora::lora_kernel<__half, __half, false>;
}

}  // namespace qmm
