// qmm_lora.h -- what the host and the kernels of qmm_lora share.
#pragma once

#include <stdint.h>

namespace qmm {

// Warps of a CTA that copy, by the ranks of its kernel (16: three CTAs an SM and
// 72 registers a thread with one; 32 and 64: two CTAs either way, as far as
// registers go).
template <int RANKS>
constexpr int LORA_COPIERS = RANKS == 16 ? 1 : 2;
constexpr int LORA_MAX_CLUSTER = 8;  // CTAs of a tile
constexpr int LORA_CHUNK = 64;  // columns of x that are multiplied at a time

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
    int tile_rows;                 // at most
    int cluster_shift;             // of the CTAs of a tile, a power of two
    int parts_shift;               // of the clusters of a tile, which share its columns
    int vec_b;                     // rows of B on 16-byte boundaries, on 4-byte ones, or 0
    int vec_out;                   // rows of y and base (if any) on 16-byte boundaries
    // shared memory: parts of h, its fragments, the ring's slots
    int frag_at, ring_at, slot_bytes, depth;
    int* err;
    unsigned long long wait_ns;  // bound of a wait, and whether the last copy's arrival is held back (qmm_debug_stream_wait)
    int withhold;
};

using LoraKernel = void (*)(LoraArgs);

// Kernels by the types of x and of the adapters; f32: fp32 base and y, else
// x's type; whole: rows of y and base on 16-byte boundaries and of a multiple of
// eight columns; tile: 16, 32 or 64 ranks at a time.
LoraKernel lora_kernel_f32_f32(bool f32, bool whole, int tile);
LoraKernel lora_kernel_f32_f16(bool f32, bool whole, int tile);
LoraKernel lora_kernel_f32_bf16(bool f32, bool whole, int tile);
LoraKernel lora_kernel_f16_f32(bool f32, bool whole, int tile);
LoraKernel lora_kernel_f16_f16(bool f32, bool whole, int tile);
LoraKernel lora_kernel_f16_bf16(bool f32, bool whole, int tile);
LoraKernel lora_kernel_bf16_f32(bool f32, bool whole, int tile);
LoraKernel lora_kernel_bf16_f16(bool f32, bool whole, int tile);
LoraKernel lora_kernel_bf16_bf16(bool f32, bool whole, int tile);

}  // namespace qmm
