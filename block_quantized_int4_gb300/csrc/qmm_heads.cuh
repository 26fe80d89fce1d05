// qmm_heads.cuh -- what the attention entries share: strided heads of three
// element types, loaded and stored eight values at a time, and the places of
// a token's codes in a cache record (include/qmm.h, qmm_kv_cache).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "qmm.h"
#include "qmm_device.cuh"

namespace qmm {

constexpr int MAX_HEAD = 256;  // largest head size
constexpr int GROUP = 32;      // tokens of a cache record
constexpr int MAX_HEADS = 1 << 24;                // heads of an argument, tokens of a call and
constexpr int64_t MAX_TOKENS = int64_t(1) << 31;  // records of a cache, so that no product of
constexpr int64_t MAX_RECORDS = INT32_MAX;        // sizes leaves the kernels' indexes

inline int dtype_size(int dtype) { return dtype == QMM_F32 ? 4 : 2; }

// Bytes of a record of head size D: codes of K and V, and their scales.
__host__ __device__ constexpr int record_bytes(int D) { return 36 * D; }

// Places of token `tok` of a record, in bytes from the block's codes or
// scales (see qmm_kv_cache).
__device__ __forceinline__ int k_word_at(int tok, int m) { return (((tok & 7) * 4 + m) * 4 + (tok >> 3)) * 4; }
__device__ __forceinline__ int v_unit_at(int tok, int e) {
    return (((e * 4 + ((tok >> 1) & 3)) * 4 + (tok >> 3)) * 2 + (tok & 1)) * 2;
}
__device__ __forceinline__ int scale_at(int tok) { return ((((tok >> 1) & 3) * 4 + (tok >> 3)) * 2 + (tok & 1)) * 2; }

// Heads as the kernels see them: the C struct and whether runs of 8 (and of
// 4) values starting at multiples of 8 (4) sit on 16-byte (8-byte)
// boundaries, decided on the host.
struct Heads {
    char* data;
    int64_t ts, hs;  // strides in elements
    int dtype;
    int wide;
};

__device__ __forceinline__ float bits_to_f32(unsigned short u, int dtype) {
    return dtype == QMM_F16 ? __half2float(__ushort_as_half(u)) : __uint_as_float((unsigned)u << 16);
}
__device__ __forceinline__ unsigned short f32_to_bits(float f, int dtype) {
    return dtype == QMM_F16 ? __half_as_ushort(__float2half_rn(f)) : __bfloat16_as_ushort(__float2bfloat16_rn(f));
}
__device__ __forceinline__ unsigned pack2(float a, float b, int dtype) {
    if (dtype == QMM_F16) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const unsigned*>(&h);
    }
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const unsigned*>(&h);
}
__device__ __forceinline__ void unpack2(unsigned w, int dtype, float* v) {
    v[0] = bits_to_f32((unsigned short)(w & 0xffff), dtype);
    v[1] = bits_to_f32((unsigned short)(w >> 16), dtype);
}

__device__ __forceinline__ float load1(const char* p, int64_t i, int dtype) {
    return dtype == QMM_F32 ? reinterpret_cast<const float*>(p)[i]
                            : bits_to_f32(reinterpret_cast<const unsigned short*>(p)[i], dtype);
}
__device__ __forceinline__ void store1(char* p, int64_t i, float v, int dtype) {
    if (dtype == QMM_F32)
        reinterpret_cast<float*>(p)[i] = v;
    else
        reinterpret_cast<unsigned short*>(p)[i] = f32_to_bits(v, dtype);
}

// N = 4 or 8 consecutive values from element i (a multiple of N past an
// aligned head).
template <int N>
__device__ __forceinline__ void loadn(const char* p, int64_t i, int dtype, int wide, float* v) {
    if (!wide) {
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = load1(p, i + j, dtype);
    } else if (dtype == QMM_F32) {
#pragma unroll
        for (int j = 0; j < N; j += 4) {
            const float4 f = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p) + i + j);
            v[j] = f.x, v[j + 1] = f.y, v[j + 2] = f.z, v[j + 3] = f.w;
        }
    } else {
        const unsigned short* s = reinterpret_cast<const unsigned short*>(p) + i;
        if constexpr (N == 8) {
            const uint4 u = *reinterpret_cast<const uint4*>(s);
            unpack2(u.x, dtype, v), unpack2(u.y, dtype, v + 2), unpack2(u.z, dtype, v + 4), unpack2(u.w, dtype, v + 6);
        } else {
            const uint2 u = *reinterpret_cast<const uint2*>(s);
            unpack2(u.x, dtype, v), unpack2(u.y, dtype, v + 2);
        }
    }
}

template <int N>
__device__ __forceinline__ void storen(char* p, int64_t i, int dtype, int wide, const float* v) {
    if (!wide) {
#pragma unroll
        for (int j = 0; j < N; ++j) store1(p, i + j, v[j], dtype);
    } else if (dtype == QMM_F32) {
#pragma unroll
        for (int j = 0; j < N; j += 4)
            *reinterpret_cast<float4*>(reinterpret_cast<float*>(p) + i + j) =
                make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
    } else {
        unsigned short* s = reinterpret_cast<unsigned short*>(p) + i;
        if constexpr (N == 8)
            *reinterpret_cast<uint4*>(s) = make_uint4(pack2(v[0], v[1], dtype), pack2(v[2], v[3], dtype),
                                                      pack2(v[4], v[5], dtype), pack2(v[6], v[7], dtype));
        else
            *reinterpret_cast<uint2*>(s) = make_uint2(pack2(v[0], v[1], dtype), pack2(v[2], v[3], dtype));
    }
}

// ---------------------------------------------------------------- host checks
// Pointers and shapes of a heads argument; D values a head.
inline qmm_status check_heads(const qmm_heads& h, int n_heads) {
    if (h.dtype != QMM_F32 && h.dtype != QMM_F16 && h.dtype != QMM_BF16) return QMM_ERR_ARG;
    if (!h.data || h.n_heads <= 0 || h.token_stride < 0 || h.head_stride < 0) return QMM_ERR_ARG;
    if ((n_heads && h.n_heads != n_heads) || h.n_heads > MAX_HEADS) return QMM_ERR_SHAPE;
    if (reinterpret_cast<uintptr_t>(h.data) % dtype_size(h.dtype)) return QMM_ERR_ALIGN;
    return QMM_OK;
}

// Whether two of the T * n_heads rows of D values share places.  Nested layouts
// (all heads of a token before the next token's, or the other way round) are seen
// at once; else j steps of one stride are compared with the steps of the other on
// both sides of them.
inline bool rows_overlap(const qmm_heads& h, int64_t T, int D) {
    using wide = __int128;
    const wide n[2] = {T, h.n_heads}, s[2] = {h.token_stride, h.head_stride};
    for (int i = 0; i < 2; ++i)
        if (n[i] > 1 && s[i] < D) return true;
    const int few = n[0] < n[1] ? 0 : 1, many = 1 - few;
    if (n[few] <= 1 || (n[few] - 1) * s[few] + D <= s[many] || (n[many] - 1) * s[many] + D <= s[few]) return false;
    if (n[few] > 1 << 17) return true;  // more rows than a launch takes
    for (wide j = 1; j < n[few]; ++j) {
        const wide at = j * s[few], k = at / s[many];
        if (k >= 1 && k < n[many] && at - k * s[many] < D) return true;
        if (k + 1 < n[many] && (k + 1) * s[many] - at < D) return true;
    }
    return false;
}

// The same for heads that are written: rows of D values that do not overlap.
inline qmm_status check_output(const qmm_heads& h, int n_heads, int64_t T, int D) {
    if (qmm_status s = check_heads(h, n_heads)) return s;
    return rows_overlap(h, T, D) ? QMM_ERR_SHAPE : QMM_OK;
}

inline Heads kernel_heads(const qmm_heads& h) {
    const int size = dtype_size(h.dtype);
    const int wide = h.data && reinterpret_cast<uintptr_t>(h.data) % 16 == 0 && h.token_stride * size % 16 == 0 &&
                     h.head_stride * size % 16 == 0;
    return Heads{static_cast<char*>(h.data), h.token_stride, h.head_stride, h.dtype, wide};
}

inline bool valid_head_dim(int D) { return D > 0 && D % QK == 0 && D <= MAX_HEAD; }

inline qmm_status check_cache(const qmm_kv_cache& c, bool data) {
    if (c.n_pages < 0 || c.page_size <= 0 || c.n_heads <= 0) return QMM_ERR_ARG;
    if (c.page_size % GROUP || c.page_size > 1 << 20 || c.n_heads > 1 << 16 || !valid_head_dim(c.head_dim))
        return QMM_ERR_SHAPE;
    if ((int64_t)c.n_pages * c.n_heads * (c.page_size / GROUP) > MAX_RECORDS) return QMM_ERR_SHAPE;
    if (data && !c.data) return QMM_ERR_ARG;
    if (data && reinterpret_cast<uintptr_t>(c.data) % 16) return QMM_ERR_ALIGN;
    return QMM_OK;
}

}  // namespace qmm
