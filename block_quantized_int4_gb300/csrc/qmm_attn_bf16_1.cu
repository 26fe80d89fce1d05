// qmm_attn_bf16_1.cu -- the attention kernels for bf16 activations and one tile of 8 rows
// a warp, one a head size (translation units side by side, so that they
// compile side by side).
#include "qmm_attn.cuh"

namespace qmm {

AttnKernel attn_kernel_bf16_1(int NB) {
    static constexpr AttnKernel kernels[8] = {attn::attn_kernel<1, QMM_BF16, 1>, attn::attn_kernel<2, QMM_BF16, 1>,
                                              attn::attn_kernel<3, QMM_BF16, 1>, attn::attn_kernel<4, QMM_BF16, 1>,
                                              attn::attn_kernel<5, QMM_BF16, 1>, attn::attn_kernel<6, QMM_BF16, 1>,
                                              attn::attn_kernel<7, QMM_BF16, 1>, attn::attn_kernel<8, QMM_BF16, 1>};
    return kernels[NB - 1];
}

}  // namespace qmm
