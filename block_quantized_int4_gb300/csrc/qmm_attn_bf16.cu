// qmm_attn_bf16.cu -- the attention kernels for bf16 activations, one a head size
// (a translation unit a type, so that they compile side by side).
#include "qmm_attn.cuh"

namespace qmm {

AttnKernel attn_kernel_bf16(int NB) {
    static constexpr AttnKernel kernels[8] = {attn::attn_kernel<1, QMM_BF16>, attn::attn_kernel<2, QMM_BF16>,
                                              attn::attn_kernel<3, QMM_BF16>, attn::attn_kernel<4, QMM_BF16>,
                                              attn::attn_kernel<5, QMM_BF16>, attn::attn_kernel<6, QMM_BF16>,
                                              attn::attn_kernel<7, QMM_BF16>, attn::attn_kernel<8, QMM_BF16>};
    return kernels[NB - 1];
}

}  // namespace qmm
