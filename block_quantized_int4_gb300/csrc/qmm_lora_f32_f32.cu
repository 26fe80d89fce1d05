// qmm_lora_f32_f32.cu -- low-rank adapters, f32 rows and f32 adapters.
#include "qmm_lora.cuh"

namespace qmm {

LoraKernel lora_kernel_f32_f32(bool f32, bool whole, int tile) {
    return lora::kernel_of<float, float>(f32, whole, tile);
}

}  // namespace qmm
