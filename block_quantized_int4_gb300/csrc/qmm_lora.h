// qmm_lora.h -- what the host and the kernels of qmm_lora share.
#pragma once

#include <stdint.h>

namespace qmm {

constexpr int LORA_THREADS = 256;
constexpr int LORA_GROUP_RANKS = 64;  // that a warp sums at a time
constexpr int LORA_MAX_RANK = 256;
constexpr int LORA_CHUNK = 32;      // columns of x that a warp multiplies at a time

struct LoraArgs {
    const void *x, *a, *b, *base;
    void* y;
    int64_t ldx, lda, a_stride, ldb, b_stride, ld_base, ldy;
    const int32_t* ranks;
    const float* scales;
    const int32_t* seg_start;
    const int32_t* seg_adapter;
    int64_t T;
    int N, K, n_segs, seg_rows, n_adapters, max_rank;
    int tile_rows;      // at most
    int cluster_shift;  // of the CTAs of a tile, a power of two
    int vec_b, vec_base, vec_out;  // rows on 16-byte boundaries: of B, of base, of y and base (if any)
    int frag_at, ring_at, ring_bytes;  // shared memory: parts of h, its fragments, the columns' ring
    int* err;
};

using LoraKernel = void (*)(LoraArgs);

// Ranks in shared memory: whole chunks of the expanding products.
inline int lora_rank_room(int max_rank) { return max_rank <= 16 ? 16 : (max_rank + 31) / 32 * 32; }

// Kernels by the types of x and of the adapters; f32: fp32 base and y, else
// x's type; low: max_rank <= 16.
LoraKernel lora_kernel_f32_f32(bool f32, bool low);
LoraKernel lora_kernel_f32_f16(bool f32, bool low);
LoraKernel lora_kernel_f32_bf16(bool f32, bool low);
LoraKernel lora_kernel_f16_f32(bool f32, bool low);
LoraKernel lora_kernel_f16_f16(bool f32, bool low);
LoraKernel lora_kernel_f16_bf16(bool f32, bool low);
LoraKernel lora_kernel_bf16_f32(bool f32, bool low);
LoraKernel lora_kernel_bf16_f16(bool f32, bool low);
LoraKernel lora_kernel_bf16_bf16(bool f32, bool low);

// Bytes of a value of h in the fragments: three bf16 where the adapters are
// bf16, else two fp32 that hold 11 bits each.
inline int lora_frag_bytes(int w_type) { return w_type == 2 ? 6 : 8; }

}  // namespace qmm
