// qmm_attn_f16_2.cu -- the attention kernels for f16 activations and two tiles of 8 rows
// a warp, one a head size (translation units side by side, so that they
// compile side by side).
#include "qmm_attn.cuh"

namespace qmm {

AttnKernel attn_kernel_f16_2(int NB) {
    static constexpr AttnKernel kernels[8] = {attn::attn_kernel<1, QMM_F16, 2>, attn::attn_kernel<2, QMM_F16, 2>,
                                              attn::attn_kernel<3, QMM_F16, 2>, attn::attn_kernel<4, QMM_F16, 2>,
                                              attn::attn_kernel<5, QMM_F16, 2>, attn::attn_kernel<6, QMM_F16, 2>,
                                              attn::attn_kernel<7, QMM_F16, 2>, attn::attn_kernel<8, QMM_F16, 2>};
    return kernels[NB - 1];
}

}  // namespace qmm
