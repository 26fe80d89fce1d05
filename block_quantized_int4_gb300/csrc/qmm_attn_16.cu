// qmm_attn_16.cu -- the attention kernels for 16-bit activations (one fp16 part),
// one a head size.
#include "qmm_attn.cuh"

namespace qmm {
namespace {

template <int NB>
bool prepare(int optin) {
    const auto k = attn::attn_kernel<NB, false>;
    return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, optin - 4096) == cudaSuccess &&
           cudaFuncSetAttribute(k, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared) ==
               cudaSuccess;
}

using Kernel = void (*)(AttnArgs);
constexpr Kernel KERNELS[8] = {attn::attn_kernel<1, false>, attn::attn_kernel<2, false>, attn::attn_kernel<3, false>,
                               attn::attn_kernel<4, false>, attn::attn_kernel<5, false>, attn::attn_kernel<6, false>,
                               attn::attn_kernel<7, false>, attn::attn_kernel<8, false>};
constexpr bool (*PREPARE[8])(int) = {prepare<1>, prepare<2>, prepare<3>, prepare<4>,
                                     prepare<5>, prepare<6>, prepare<7>, prepare<8>};

}  // namespace

bool attn_prepare_16(int NB, int smem_optin) {
    if (PREPARE[NB - 1](smem_optin)) return true;
    cudaGetLastError();
    return false;
}

cudaError_t attn_launch_16(int NB, const AttnArgs& a, unsigned grid, int smem, cudaStream_t st) {
    KERNELS[NB - 1]<<<grid, ATTN_THREADS, smem, st>>>(a);
    return cudaGetLastError();
}

}  // namespace qmm
