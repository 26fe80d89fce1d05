// qmm_lora_f16_bf16.cu -- low-rank adapters, f16 rows and bf16 adapters.
#include "qmm_lora.cuh"

namespace qmm {

LoraKernel lora_kernel_f16_bf16(bool f32, bool whole, int tile) {
    return lora::kernel_of<__half, __nv_bfloat16>(f32, whole, tile);
}

}  // namespace qmm
