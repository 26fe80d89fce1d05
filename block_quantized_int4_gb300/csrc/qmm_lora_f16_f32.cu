// qmm_lora_f16_f32.cu -- low-rank adapters, f16 rows and f32 adapters.
#include "qmm_lora.cuh"

namespace qmm {

LoraKernel lora_kernel_f16_f32(bool f32, bool whole, int tile) {
    return lora::kernel_of<__half, float>(f32, whole, tile);
}

}  // namespace qmm
