// qmm_lora_bf16_f16.cu -- low-rank adapters, bf16 rows and f16 adapters.
#include "qmm_lora.cuh"

namespace qmm {

LoraKernel lora_kernel_bf16_f16(bool f32, bool whole, int tile) {
    return lora::kernel_of<__nv_bfloat16, __half>(f32, whole, tile);
}

}  // namespace qmm
