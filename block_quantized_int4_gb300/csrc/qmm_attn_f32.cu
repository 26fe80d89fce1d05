// qmm_attn_f32.cu -- the attention kernels for fp32 activations (two fp16 parts),
// one a head size.
#include "qmm_attn.cuh"

namespace qmm {
namespace {

template <int NB>
bool prepare(int optin) {
    const auto k = attn::attn_kernel<NB, true>;
    return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, optin - 4096) == cudaSuccess &&
           cudaFuncSetAttribute(k, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared) ==
               cudaSuccess;
}

using Kernel = void (*)(AttnArgs);
constexpr Kernel KERNELS[8] = {attn::attn_kernel<1, true>, attn::attn_kernel<2, true>, attn::attn_kernel<3, true>,
                               attn::attn_kernel<4, true>, attn::attn_kernel<5, true>, attn::attn_kernel<6, true>,
                               attn::attn_kernel<7, true>, attn::attn_kernel<8, true>};
constexpr bool (*PREPARE[8])(int) = {prepare<1>, prepare<2>, prepare<3>, prepare<4>,
                                     prepare<5>, prepare<6>, prepare<7>, prepare<8>};

}  // namespace

bool attn_prepare_f32(int NB, int smem_optin) {
    if (PREPARE[NB - 1](smem_optin)) return true;
    cudaGetLastError();
    return false;
}

cudaError_t attn_launch_f32(int NB, const AttnArgs& a, unsigned grid, int smem, cudaStream_t st) {
    KERNELS[NB - 1]<<<grid, ATTN_THREADS, smem, st>>>(a);
    return cudaGetLastError();
}

}  // namespace qmm
