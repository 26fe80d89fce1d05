// qmm_lora_f32_f16.cu -- low-rank adapters, f32 rows and f16 adapters.
#include "qmm_lora.cuh"

namespace qmm {

LoraKernel lora_kernel_f32_f16(bool f32, bool whole, int tile) {
    return lora::kernel_of<float, __half>(f32, whole, tile);
}

}  // namespace qmm
