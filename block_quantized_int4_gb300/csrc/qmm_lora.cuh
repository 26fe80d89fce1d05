// qmm_lora.cuh -- low-rank adapters of many requests beside a shared
// projection: y = base + scale_a B_a (A_a x) for the rows of each segment,
// which share an adapter a.
//
// One launch.  A cluster of CTAs takes a tile of up to 64 rows of a segment:
//   1. h = A x: each CTA sums over its part of K; its 8 warps share out
//      16-row blocks, 64 ranks at a time, and what is left of K;
//   2. the parts of h meet through distributed shared memory: each CTA adds up
//      a share of them in a fixed order, scales it and hands it to all;
//   3. y = base + h B^T: each CTA has its part of the N columns.
// x, base and y pass once; A and B are read once a tile (from L2 where tiles
// share an adapter).  So the bound is memory for the ranks in use: 2 r flops
// against the 2 or 4 bytes of a value of x.
//
// Products are warp MMAs whose fragments come straight from global memory:
// sums over k go in any order, so a lane takes 8 consecutive k of its row
// (16 bytes, or 32 of fp32) where the instruction's layout would give it pairs,
// and B's columns are dealt out so that a lane ends up with 8 consecutive
// outputs of a row.  x and A of one 16-bit type multiply as they are, fp32 x
// with bf16 A in three parts of 8 bits; all others as tf32, which holds either
// 16-bit type exactly, with fp32 values in two parts of 11 bits (2^-23 of a value
// is lost, and with fp32 on both sides the product of the lower parts, 2^-22 of
// a term).  h is fp32.  The second product reads it in two such parts, or, of
// bf16 B, in two parts of bf16 for 16-bit outputs (2^-18 is lost, against their
// rounding of 2^-12 or 2^-9) and three for fp32 outputs.  With fp32 x or A, sums
// of 32 products leave the tensor core, which truncates, for fp32 additions.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "qmm.h"
#include "qmm_device.cuh"
#include "qmm_lora.h"

namespace qmm {
namespace lora {

constexpr int WARPS = LORA_THREADS / 32;

// ---------------------------------------------------------------- clusters
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t peer(uint32_t addr, uint32_t cta) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(cta));
    return r;
}
__device__ __forceinline__ float4 ld_peer(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr));
    return v;
}
__device__ __forceinline__ void st_peer(uint32_t addr, uint32_t x, uint32_t y) {
    asm volatile("st.shared::cluster.b32 [%0], %1;\n\tst.shared::cluster.b32 [%0 + 8], %2;" ::"r"(addr), "r"(x), "r"(y)
                 : "memory");
}

// ---------------------------------------------------------------- copies
// 16 bytes global -> shared, the last 16 - n of them zeros.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int n) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits until at most n groups are on their way.
__device__ __forceinline__ void copies_wait(int n) {
    if (n >= 2)
        asm volatile("cp.async.wait_group 2;" ::: "memory");
    else if (n == 1)
        asm volatile("cp.async.wait_group 1;" ::: "memory");
    else
        asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// ---------------------------------------------------------------- products
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_tf32(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The parts of an fp32 value that tf32 holds: its upper 11 bits rounded to
// nearest, and what is left, of which the instruction reads 11 bits: 2^-23 of
// the value is lost.  (The upper part of a NaN may lose it; the lower never
// does.)
__device__ __forceinline__ uint32_t tf_high(float v) { return (__float_as_uint(v) + 0x1000u) & 0xFFFFE000u; }
__device__ __forceinline__ uint32_t tf_low(float v) { return __float_as_uint(v - __uint_as_float(tf_high(v))); }
// A value that came from 16 bits is its own upper part.
template <typename T>
__device__ __forceinline__ uint32_t tf_main(float v) {
    return std::is_same<T, float>::value ? tf_high(v) : __float_as_uint(v);
}

// Eight consecutive values of a row as they lie in memory.
template <typename T>
struct Raw {
    uint4 q[sizeof(T) / 2];
};

template <typename T>
__device__ __forceinline__ Raw<T> zero_raw() {
    Raw<T> r;
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.q[i] = make_uint4(0, 0, 0, 0);
    return r;
}
// x and base: every value is read once.
template <typename T>
__device__ __forceinline__ Raw<T> stream_raw(const T* p) {
    Raw<T> r;
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
        uint4& q = r.q[i];
        asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w)
                     : "l"(reinterpret_cast<const uint4*>(p) + i));
    }
    return r;
}

// The same where `in` is true.
template <typename T>
__device__ __forceinline__ void load_raw_if(Raw<T>& r, const T* p, bool in) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
        uint4& q = r.q[i];
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\t@p ld.global.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
            : "+r"(q.x), "+r"(q.y), "+r"(q.z), "+r"(q.w)
            : "l"(reinterpret_cast<const uint4*>(p) + i), "r"((int)in));
    }
}

__device__ __forceinline__ uint32_t word(const uint4& q, int i) {
    return i == 0 ? q.x : i == 1 ? q.y : i == 2 ? q.z : q.w;
}

// Value i (of 8) as fp32.
template <typename T>
__device__ __forceinline__ float value(const Raw<T>& r, int i) {
    if constexpr (std::is_same<T, float>::value) {
        return __uint_as_float(word(r.q[i >> 2], i & 3));
    } else {
        const uint32_t w = word(r.q[0], i >> 1);
        if constexpr (std::is_same<T, __nv_bfloat16>::value) return __uint_as_float((i & 1) ? w & 0xFFFF0000u : w << 16);
        return __half2float(__ushort_as_half((unsigned short)((i & 1) ? w >> 16 : w & 0xFFFFu)));
    }
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// A pair's next 8 bits as bf16; what is left of it stays.
__device__ __forceinline__ uint32_t bf16_part(float& lo, float& hi) {
    const uint32_t p = pack_bf16(lo, hi);
    lo -= __uint_as_float(p << 16);
    hi -= __uint_as_float(p & 0xFFFF0000u);
    return p;
}

// How x and A multiply.
template <typename X, typename W>
struct Types {
    static constexpr bool wide_x = std::is_same<X, float>::value, wide_w = std::is_same<W, float>::value;
    static constexpr bool w_bf16 = std::is_same<W, __nv_bfloat16>::value;
    static constexpr bool same = std::is_same<X, W>::value && !wide_x;  // as they are
    static constexpr bool thirds = wide_x && w_bf16;                    // x in three parts of bf16
    // registers of a chunk of a row of x as an operand: words of its 8 values
    static constexpr int words = same ? 4 : thirds ? 12 : wide_x ? 16 : 8;
};

// Eight values of x as the operands of mma_chunk.
template <typename X, typename W>
__device__ __forceinline__ void operand(const Raw<X>& r, uint32_t (&o)[Types<X, W>::words]) {
    using T = Types<X, W>;
    if constexpr (T::same) {
        o[0] = r.q[0].x, o[1] = r.q[0].y, o[2] = r.q[0].z, o[3] = r.q[0].w;
    } else if constexpr (T::thirds) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float lo = value(r, 2 * i), hi = value(r, 2 * i + 1);
            o[i] = bf16_part(lo, hi);
            o[4 + i] = bf16_part(lo, hi);
            o[8 + i] = pack_bf16(lo, hi);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float v = value(r, i);
            o[i] = tf_main<X>(v);
            if constexpr (T::wide_x) o[8 + i] = tf_low(v);
        }
    }
}

// d += rows g and g + 8 of x times column g of w, over the 32 k of a chunk (a
// lane's eight, and its three neighbours').
template <typename X, typename W, int N>
__device__ __forceinline__ void mma_chunk(float (&d)[4], const uint32_t (&x0)[N], const uint32_t (&x1)[N],
                                          const Raw<W>& w) {
    using T = Types<X, W>;
    if constexpr (T::same && T::w_bf16) {
        mma_bf16(d, x0[0], x1[0], x0[1], x1[1], w.q[0].x, w.q[0].y);
        mma_bf16(d, x0[2], x1[2], x0[3], x1[3], w.q[0].z, w.q[0].w);
    } else if constexpr (T::same) {
        mma_f16(d, x0[0], x1[0], x0[1], x1[1], w.q[0].x, w.q[0].y);
        mma_f16(d, x0[2], x1[2], x0[3], x1[3], w.q[0].z, w.q[0].w);
    } else if constexpr (T::thirds) {
#pragma unroll
        for (int p = 8; p >= 0; p -= 4) {
            mma_bf16(d, x0[p], x1[p], x0[p + 1], x1[p + 1], w.q[0].x, w.q[0].y);
            mma_bf16(d, x0[p + 2], x1[p + 2], x0[p + 3], x1[p + 3], w.q[0].z, w.q[0].w);
        }
    } else {
#pragma unroll
        for (int q = 0; q < 8; q += 2) {
            const float u = value(w, q), v = value(w, q + 1);
            const uint32_t b0 = tf_main<W>(u), b1 = tf_main<W>(v);
            if constexpr (T::wide_x) mma_tf32(d, x0[8 + q], x1[8 + q], x0[9 + q], x1[9 + q], b0, b1);
            if constexpr (T::wide_w) mma_tf32(d, x0[q], x1[q], x0[q + 1], x1[q + 1], tf_low(u), tf_low(v));
            mma_tf32(d, x0[q], x1[q], x0[q + 1], x1[q + 1], b0, b1);
        }
    }
}

// ---------------------------------------------------------------- tiles
struct Tile {
    int64_t row;
    int rows, adapter;  // rows == 0: none; adapter < 0: none
};

// The tile of this number, counting 64 rows at a time through the segments.
// Every thread of the block; starts that are out of order or out of range are
// brought into it (the first block looks at all of them).
__device__ __forceinline__ Tile find_tile(const LoraArgs& a, int tile) {
    __shared__ int s_sum[WARPS], s_tile[3];
    Tile t = {0, 0, -1};
    int seg = -1;
    if (!a.seg_start) {
        const int per = (a.seg_rows + a.tile_rows - 1) / a.tile_rows;
        seg = tile / per;
        const int at = (tile - seg * per) * a.tile_rows;
        if (seg >= a.n_segs) return t;
        t.row = (int64_t)seg * a.seg_rows + at;
        t.rows = min(a.tile_rows, a.seg_rows - at);
    } else {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        if (threadIdx.x == 0) s_tile[2] = 0;
        int before = 0;
        for (int s0 = 0; s0 < a.n_segs; s0 += LORA_THREADS) {
            const int s = s0 + threadIdx.x;
            int n = 0, first = 0, last = 0;
            if (s < a.n_segs) {
                const int f = a.seg_start[s], l = a.seg_start[s + 1];
                first = max(0, min(f, (int)a.T));
                last = max(first, min(l, (int)a.T));
                if (blockIdx.x == 0 && (first != f || last != l)) atomicOr(a.err, ERR_BAD_INDEX);
                n = (last - first + a.tile_rows - 1) / a.tile_rows;
            }
            int end = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(FULL, end, o);
                if (lane >= o) end += v;
            }
            if (lane == 31) s_sum[warp] = end;
            __syncthreads();
            int all = 0;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) {
                if (w < warp) end += s_sum[w];
                all += s_sum[w];
            }
            const int at = tile - (before + end - n);
            if (at >= 0 && at < n) {
                s_tile[0] = s;
                s_tile[1] = first + at * a.tile_rows;
                s_tile[2] = min(a.tile_rows, last - first - at * a.tile_rows);
            }
            __syncthreads();
            before += all;
            if (before > tile && blockIdx.x != 0) break;
        }
        seg = s_tile[0];
        t.row = s_tile[1];
        t.rows = s_tile[2];
        if (t.rows == 0) return t;
    }
    const int id = a.seg_adapter[seg];
    t.adapter = id >= 0 && id < a.n_adapters ? id : -1;
    if ((id < -1 || id >= a.n_adapters) && threadIdx.x == 0) atomicOr(a.err, ERR_BAD_INDEX);
    return t;
}

// ---------------------------------------------------------------- outputs
__device__ __forceinline__ float as_float(float v) { return v; }
__device__ __forceinline__ float as_float(__half v) { return __half2float(v); }
__device__ __forceinline__ float as_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__half* p, float v) { *p = __float2half_rn(v); }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// Eight consecutive values of a row of base or y, as fp32.
struct Eight {
    float v[8];
};

// The end of a row, or what does not lie on 16-byte boundaries: y = e (+ base).
template <typename Y>
__device__ __noinline__ void finish_plain(Y* p, const Y* base, int n, Eight e) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (j < n) put(p + j, base ? as_float(base[j]) + e.v[j] : e.v[j]);
}

template <typename Y>
__device__ __forceinline__ void store_eight(Y* p, const Eight& e) {
    if constexpr (sizeof(Y) == 4) {
        reinterpret_cast<float4*>(p)[0] = make_float4(e.v[0], e.v[1], e.v[2], e.v[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(e.v[4], e.v[5], e.v[6], e.v[7]);
    } else if constexpr (std::is_same<Y, __half>::value) {
        *reinterpret_cast<uint4*>(p) = make_uint4(pack_f16(e.v[0], e.v[1]), pack_f16(e.v[2], e.v[3]),
                                                  pack_f16(e.v[4], e.v[5]), pack_f16(e.v[6], e.v[7]));
    } else {
        *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(e.v[0], e.v[1]), pack_bf16(e.v[2], e.v[3]),
                                                  pack_bf16(e.v[4], e.v[5]), pack_bf16(e.v[6], e.v[7]));
    }
}

// ---------------------------------------------------------------- columns
__device__ __forceinline__ uint4 lds(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
    return v;
}

// What a thread copies into a stage of the ring: 32-column blocks of B,
// [column][ranks] as in memory with zeros behind the rank, then of base,
// [row][column].  Where rows are whole multiples of 128 bytes, 16-byte units of
// odd rows change places, so that the two rows that eight lanes read lie in
// different banks.
__device__ __forceinline__ int swizzle(int row, int units, bool wide) {
    return (units & 7) ? 0 : wide ? row & 1 : (row & 1) << 2;
}

// Values that are kept, not worked out again where they are used.
__device__ __forceinline__ void keep(int& v) { asm volatile("" : "+r"(v)); }
__device__ __forceinline__ void keep(uint32_t& v) { asm volatile("" : "+r"(v)); }
template <typename P>
__device__ __forceinline__ void keep(P*& v) {
    asm volatile("" : "+l"(v));
}

template <typename W, typename Y>
struct Fill {
    const W* b;            // this thread's unit of its first column of the next stage
    const Y* base;         // and of its first row
    uint32_t b_dst, base_dst;  // where they go, from a stage's start
    int col, b_bytes;      // b_bytes < 0: this thread copies none of B
    int row, at;           // at: the unit's column in a stage; row past the rows: none of base
};

// Units of a row of B: threads side by side on a column (a power of two).
__device__ __forceinline__ int across_shift(int units) { return units > 1 ? 32 - __clz(units - 1) : 0; }

// n: the first stage's first column; per: columns of a stage, bshift + 5 its binary logarithm.
template <typename W, typename Y>
__device__ __forceinline__ Fill<W, Y> fill_init(const LoraArgs& a, const W* b, int rank, int units, int n, int bshift,
                                                uint32_t base_at, int64_t row, int rows) {
    constexpr int E = 16 / (int)sizeof(W), YE = 16 / (int)sizeof(Y), YL = sizeof(Y) == 4 ? 3 : 2;
    int tid = threadIdx.x;
    keep(tid);
    Fill<W, Y> f;
    const int shift = across_shift(units), unit = tid & ((1 << shift) - 1);
    f.col = tid >> shift;
    f.b_bytes = unit < units ? max(0, min(16, (rank - unit * E) * (int)sizeof(W))) : -1;
    f.b = b + (int64_t)(n + f.col) * a.ldb + unit * E;
    f.b_dst = (f.col * units + (unit ^ swizzle(f.col, units, sizeof(W) == 4))) * 16;
    const int s2 = bshift + YL, u2 = tid & ((1 << s2) - 1);
    f.row = a.vec_base ? tid >> s2 : rows;
    f.at = u2 * YE;
    f.base = static_cast<const Y*>(a.base) + (row + (tid >> s2)) * a.ld_base + n + f.at;
    f.base_dst = base_at + (((tid >> s2) << s2) + (u2 ^ swizzle(tid >> s2, 1 << s2, sizeof(Y) == 4))) * 16;
    return f;
}

// B's units where they do not lie on 16-byte boundaries.
template <typename W>
__device__ __noinline__ void copy_plain(uint32_t dst, const W* src, int bytes) {
    uint32_t v[4] = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < 16 / (int)sizeof(W); ++e)
        if (e * (int)sizeof(W) < bytes) {
            if constexpr (sizeof(W) == 4)
                v[e] = reinterpret_cast<const uint32_t*>(src)[e];
            else
                v[e >> 1] |= (uint32_t) reinterpret_cast<const unsigned short*>(src)[e] << (16 * (e & 1));
        }
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3])
                 : "memory");
}

// The next stage, columns [n, n + cols), to `slot`; `per` columns on to the one after.
template <typename W, typename Y>
__device__ __forceinline__ void fill_stage(Fill<W, Y>& f, const LoraArgs& a, int units, int bshift, int n, int cols,
                                           int rows, uint32_t slot) {
    constexpr int YL = sizeof(Y) == 4 ? 3 : 2;
    const int shift = across_shift(units), step = LORA_THREADS >> shift;
    if (f.b_bytes >= 0) {
        const W* src = f.b;
        uint32_t dst = slot + f.b_dst;
        const int in = min(cols, a.N - n);
        if (a.vec_b && in == cols) {
            for (int col = f.col; col < cols; col += step) {
                copy16(dst, src, f.b_bytes);
                src += step * a.ldb;
                dst += step * units * 16;
            }
        } else {
            for (int col = f.col; col < cols; col += step) {
                copy_plain(dst, src, col < in ? f.b_bytes : 0);
                src += step * a.ldb;
                dst += step * units * 16;
            }
        }
        f.b += (32 << bshift) * a.ldb;
    }
    if (f.at < cols && f.row < rows) {
        const int s2 = bshift + YL, step = LORA_THREADS >> s2;
        const int bytes = max(0, min(16, (a.N - n - f.at) * (int)sizeof(Y)));
        const Y* src = bytes ? f.base : static_cast<const Y*>(a.base);
        uint32_t dst = slot + f.base_dst;
        for (int r = f.row; r < rows; r += step) {
            copy16(dst, src, bytes);
            src += bytes ? step * a.ld_base : 0;
            dst += step << s2 << 4;
        }
    }
    f.base += 32 << bshift;
}

// ---------------------------------------------------------------- the kernel
// LOW: max_rank <= 16, chunks of 16 ranks in the second product.
template <typename X, typename W, typename Y, bool LOW>
__global__ void __launch_bounds__(LORA_THREADS, LOW ? 3 : 2) lora_kernel(const __grid_constant__ LoraArgs a) {
    using T = Types<X, W>;
    constexpr bool BF = T::w_bf16;               // fragments of h: parts of bf16, else of tf32
    constexpr int NT = LOW ? 2 : 8;              // blocks of 8 ranks that a warp sums at a time
    constexpr int RC = LOW ? 16 : 32;            // ranks of a chunk
    constexpr int MPC = BF ? RC / 16 : RC / 8;   // MMAs of a chunk
    constexpr int PARTS = BF ? 3 : 2;            // of a value of h (the third of bf16 for fp32 outputs alone)
    constexpr int AHEAD = T::wide_x ? 1 : 2;     // chunks of x that are loaded before the ones in use
    constexpr int ys = sizeof(Y);
    const Y* base = static_cast<const Y*>(a.base);
    Y* y = static_cast<Y*>(a.y);
    extern __shared__ __align__(128) uint8_t smem[];
    // launched after the kernels that write x and base, possibly early
    // (programmatic dependent launch): nothing is read before they complete
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // numbers of CTAs, of warps on rows and of parts of K are powers of two, as
    // shifts: a division costs more than most of what follows
    const int cs = a.cluster_shift;
    const uint32_t C = 1u << cs, cta = cs ? cluster_rank() : 0;
    const Tile t = find_tile(a, blockIdx.x >> cs);
    if (t.rows == 0) return;  // of all CTAs of the cluster
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
    const int mtiles = (t.rows + 15) >> 4;
    const int N = a.N, blocks = (N + 31) / 32;  // of 32 columns
    const int nb0 = (int)(blocks * cta >> cs), nb1 = (int)(blocks * (cta + 1) >> cs);  // N <= 2^28, C <= 16: 32 bits do
    const bool vec_base = a.vec_base;

    int rank = 0;
    if (t.adapter >= 0) {
        const int r = a.ranks ? a.ranks[t.adapter] : a.max_rank;
        rank = max(0, min(r, a.max_rank));
        if (r != rank && threadIdx.x == 0) atomicOr(a.err, ERR_BAD_INDEX);
    }
    const float scale = a.scales && t.adapter >= 0 ? a.scales[t.adapter] : 1.f;
    if (rank == 0) {  // y = base
        if (a.y == a.base) return;
        for (int r = 0; r < t.rows; ++r)
            for (int n = nb0 * 32 + threadIdx.x * 8; n < min(N, nb1 * 32); n += LORA_THREADS * 8) {
                Y* to = y + (t.row + r) * a.ldy + n;
                const Y* from = base ? base + (t.row + r) * a.ld_base + n : nullptr;
                const Eight e = {};
                if (!a.vec_out || n + 8 > N) {
                    finish_plain(to, from, N - n, e);
                } else {
                    const Raw<Y> v = from ? stream_raw(from) : zero_raw<Y>();
#pragma unroll
                    for (int i = 0; i < (int)sizeof(Y) / 2; ++i) reinterpret_cast<uint4*>(to)[i] = v.q[i];
                }
            }
        return;
    }

    // The columns' copies start now: a stage has two 32-column blocks for each
    // of the warps beside each other on 16 rows, or fewer where three stages of
    // them do not fit.
    const int room = (rank + RC - 1) / RC * RC;      // ranks of h, the last of them zeros
    const int mshift = mtiles > 2 ? 2 : mtiles - 1;  // 1, 2 or 4 warps take the rows of a block
    const int b_units = room * (int)sizeof(W) / 16;
    int bshift = 4 - mshift, depth, base_at, stage_bytes;
    for (;; --bshift) {
        base_at = (32 * b_units * 16) << bshift;
        stage_bytes = base_at + (vec_base ? (mtiles * 16 * 32 * ys) << bshift : 0);
        depth = a.ring_bytes >= 4 * stage_bytes ? 4 : a.ring_bytes >= 3 * stage_bytes ? 3 : 2;
        if (depth >= 3 || bshift == 0) break;
    }
    const int nblk = 1 << bshift, per = nblk * 32, first_n = nb0 * 32, stages = (nb1 - nb0 + nblk - 1) >> bshift;
    const uint32_t ring = smem_u32(smem) + a.ring_at;
    const W* b = static_cast<const W*>(a.b) + (int64_t)t.adapter * a.b_stride;
    {
        Fill<W, Y> fill = fill_init<W, Y>(a, b, rank, b_units, first_n, bshift, base_at, t.row, t.rows);
        for (int i = 0; i < depth - 1; ++i) {
            const int n = first_n + i * per;
            if (i < stages)
                fill_stage(fill, a, b_units, bshift, n, min(per, nb1 * 32 - n), t.rows, ring + i * stage_bytes);
            copies_commit();
        }
    }

    // 1. parts of h: [part of K][16 * mtiles][room + 8] fp32.  Rows and ranks
    // that are not there repeat others; what becomes of them is not used (rows)
    // or set to zero (ranks).
    float* part = reinterpret_cast<float*>(smem);
    const int ps = room + 8;
    // a warp takes (part of K, 64 ranks, 16 rows), the last of these in the lowest bits
    const int rshift = room <= 64 ? 0 : room <= 128 ? 1 : 2, kshift = max(0, 3 - mshift - rshift), kways = 1 << kshift;
    {
        const W* wa = static_cast<const W*>(a.a) + (int64_t)t.adapter * a.a_stride;
        const int chunks = a.K / LORA_CHUNK;
        const int cc0 = (int)(chunks * cta >> cs), ccn = (int)(chunks * (cta + 1) >> cs) - cc0;
        for (int u = warp; u < 1 << (kshift + rshift + mshift); u += WARPS) {
            const int mt = u & ((1 << mshift) - 1), rr = ((u >> mshift) & ((1 << rshift) - 1)) * LORA_GROUP_RANKS;
            const int kp = u >> (mshift + rshift);
            if (mt >= mtiles || rr >= rank) continue;
            const int c0 = cc0 + (ccn * kp >> kshift), c1 = cc0 + (ccn * (kp + 1) >> kshift);
            const int r0 = mt * 16 + g;
            const int nt = min(NT, (rank - rr + 7) >> 3);
            const bool two = t.rows > mt * 16 + 8;
            const X* x0 = static_cast<const X*>(a.x) + (t.row + min(r0, t.rows - 1)) * a.ldx + 8 * c;
            const X* x1 = static_cast<const X*>(a.x) + (t.row + min(r0 + 8, t.rows - 1)) * a.ldx + 8 * c;
            const W* w0 = wa + (int64_t)(rr + g) * a.lda + 8 * c;
            // rows of A up to a multiple of 8, as far as there are any, are read
            const int w_rows = min((rank + 7) & ~7, a.max_rank) - rr - g;
            float acc[NT][4] = {};
            Raw<W> w[NT];
#pragma unroll
            for (int j = 0; j < NT; ++j) w[j] = zero_raw<W>();
            Raw<X> v0[AHEAD], v1[AHEAD], n0[AHEAD], n1[AHEAD];
            const int last = max(0, c1 - 1) * LORA_CHUNK;
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                const int at = min((c0 + i) * LORA_CHUNK, last);
                n0[i] = stream_raw(x0 + at);
                n1[i] = two ? stream_raw(x1 + at) : n0[i];
            }
            for (int ch = c0; ch < c1; ch += AHEAD) {
#pragma unroll
                for (int i = 0; i < AHEAD; ++i) {
                    v0[i] = n0[i];
                    v1[i] = n1[i];
                    const int at = min((ch + AHEAD + i) * LORA_CHUNK, last);
                    n0[i] = stream_raw(x0 + at);
                    n1[i] = two ? stream_raw(x1 + at) : n0[i];
                }
#pragma unroll
                for (int i = 0; i < AHEAD; ++i) {
                    if (ch + i >= c1) break;
                    const W* wc = w0 + (ch + i) * LORA_CHUNK;
#pragma unroll
                    for (int j = 0; j < NT; ++j) load_raw_if(w[j], wc + 8 * j * a.lda, 8 * j < w_rows);
                    uint32_t o0[T::words], o1[T::words];
                    operand<X, W>(v0[i], o0);
                    operand<X, W>(v1[i], o1);
#pragma unroll
                    for (int j = 0; j < NT; ++j)
                        if (j < nt) {
                            if constexpr (T::same) {
                                mma_chunk<X, W>(acc[j], o0, o1, w[j]);
                            } else {
                                float d[4] = {};
                                mma_chunk<X, W>(d, o0, o1, w[j]);
#pragma unroll
                                for (int e = 0; e < 4; ++e) acc[j][e] += d[e];
                            }
                        }
                }
            }
            float* to = part + (kp * mtiles * 16 + r0) * ps + rr + 2 * c;
#pragma unroll
            for (int j = 0; j < NT; ++j)
                if (rr + 8 * j < room) {
                    const int r = rr + 8 * j + 2 * c;
                    *reinterpret_cast<float2*>(to + 8 * j) =
                        make_float2(r < rank ? acc[j][0] : 0.f, r + 1 < rank ? acc[j][1] : 0.f);
                    *reinterpret_cast<float2*>(to + 8 * ps + 8 * j) =
                        make_float2(r < rank ? acc[j][2] : 0.f, r + 1 < rank ? acc[j][3] : 0.f);
                }
        }
    }
    if (cs)
        cluster_barrier();
    else
        __syncthreads();

    // 2. this CTA's share of h, four ranks of a row at a time on C lanes: each
    // adds up the parts of one CTA, a butterfly adds these (in one order for
    // all), and each hands the sum, scaled and cut, to one CTA.  A fragment
    // holds [16-row block][MMA][part][lane][registers]: of rows g and g + 8 one k,
    // of both the other.
    const int chunks = room / RC;
    {
        const int per_row = room / 4, quads = t.rows * per_row;
        const int q0 = (int)(quads * cta >> cs), q1 = (int)(quads * (cta + 1) >> cs);
        const uint32_t other = threadIdx.x & (C - 1);
        const uint32_t from = cs ? peer(smem_u32(part), other) : smem_u32(part);
        const uint32_t frag_at = smem_u32(smem) + a.frag_at, to = cs ? peer(frag_at, other) : frag_at;
        for (int qb = q0; qb < q1; qb += LORA_THREADS >> cs) {
            const int q = qb + (threadIdx.x >> cs);
            const bool mine = q < q1;
            const int row = mine ? q / per_row : 0, j = mine ? (q - row * per_row) * 4 : 0;
            float4 v[8];
#pragma unroll
            for (int kp = 0; kp < 8; ++kp)
                if (kp < kways) v[kp] = ld_peer(from + ((kp * mtiles * 16 + row) * ps + j) * 4);
            float4 h = v[0];
#pragma unroll
            for (int kp = 1; kp < 8; ++kp)
                if (kp < kways) h.x += v[kp].x, h.y += v[kp].y, h.z += v[kp].z, h.w += v[kp].w;
            for (uint32_t o = 1; o < C; o <<= 1) {
                h.x += __shfl_xor_sync(FULL, h.x, o);
                h.y += __shfl_xor_sync(FULL, h.y, o);
                h.z += __shfl_xor_sync(FULL, h.z, o);
                h.w += __shfl_xor_sync(FULL, h.w, o);
            }
            if (!mine) continue;
            h.x *= scale, h.y *= scale, h.z *= scale, h.w *= scale;
            // ranks j .. j + 3 are half of a lane's eight (RC 32) or all four (RC 16)
            const int in = j % RC, cc = LOW ? in / 4 : in / 8, half = LOW ? 0 : (in / 4) & 1;
            const int to_lane = (row & 7) * 4 + cc, reg = ((row >> 3) & 1) * 4;
            const int first = ((row >> 4) * chunks + j / RC) * MPC;
            if constexpr (BF) {
                const uint32_t at = to + (first + half) * PARTS * 512 + to_lane * 16 + reg;
#pragma unroll
                for (int p = 0; p < PARTS; ++p) {
                    const uint32_t lo = bf16_part(h.x, h.y), hi = bf16_part(h.z, h.w);
                    st_peer(at + p * 512, lo, hi);
                }
            } else {
                const uint32_t at = to + (first + half * 2) * PARTS * 512 + to_lane * 16 + reg;
                st_peer(at, tf_high(h.x), tf_high(h.y));
                st_peer(at + 512, tf_low(h.x), tf_low(h.y));
                st_peer(at + 1024, tf_high(h.z), tf_high(h.w));
                st_peer(at + 1536, tf_low(h.z), tf_low(h.w));
            }
        }
    }
    if (cs)
        cluster_barrier();
    else
        __syncthreads();

    // 3. the columns, stage by stage; a warp takes 16 rows of a 32-column block.
    // Column q of MMA block i is column 8 (q / 2) + 2 i + q % 2 of the 32, so
    // that lane c of a row gets columns 8 c .. 8 c + 7.
    const int mt = warp & ((1 << mshift) - 1), wb = warp >> mshift, r0 = mt * 16 + g, beside = WARPS >> mshift;
    const bool in0 = r0 < t.rows, in1 = r0 + 8 < t.rows;
    uint32_t frag = smem_u32(smem) + a.frag_at + (mt * chunks * MPC * PARTS * 32 + lane) * 16;
    const uint32_t b_swz = swizzle(g, b_units, sizeof(W) == 4) * 16, b_two = 2 * b_units * 16;
    uint32_t b_lane = (wb * 32 + 8 * (g >> 1) + (g & 1)) * b_units * 16;
    const int across = per * ys / 16;
    const uint32_t base_swz = swizzle(g, across, ys == 4) * 16;
    uint32_t base_lane = base_at + r0 * across * 16 + (wb * 4 + c) * (ys / 2) * 16;
    int n = first_n + wb * 32 + 8 * c;
    Y* y0 = y + (t.row + r0) * a.ldy + n;
    Y* y1 = y0 + 8 * a.ldy;
    keep(frag), keep(b_lane), keep(base_lane), keep(y0), keep(y1), keep(n);
    const int ahead = depth - 1;
    Fill<W, Y> fill = fill_init<W, Y>(a, b, rank, b_units, first_n + ahead * per, bshift, base_at, t.row, t.rows);
    keep(fill.b), keep(fill.base), keep(fill.b_dst), keep(fill.base_dst), keep(fill.col), keep(fill.b_bytes);
    keep(fill.row), keep(fill.at);
    int slot = 0;
    for (int st = 0; st < stages; ++st) {
        copies_wait(depth - 2);
        __syncthreads();
        if (st + ahead < stages) {
            const int at = first_n + (st + ahead) * per;
            fill_stage(fill, a, b_units, bshift, at, min(per, nb1 * 32 - at), t.rows,
                       ring + (slot ? slot - 1 : ahead) * stage_bytes);
        }
        copies_commit();
        const int nb = min(nblk, nb1 - nb0 - (st << bshift));  // blocks of this stage
        for (int blk = mt < mtiles ? wb : nblk; blk < nb; blk += beside) {
            const uint32_t stage = ring + slot * stage_bytes;
            uint32_t src = stage + b_lane + (blk - wb) * 32 * b_units * 16, f = frag;
            float d[4][4] = {};
            for (int ch = 0; ch < chunks; ++ch, f += MPC * PARTS * 512) {
                Raw<W> w[4];  // LOW: the first half of each
                if constexpr (!LOW && sizeof(W) == 4) {
                    const uint32_t u0 = src + ((ch * 128 + c * 32) ^ b_swz), u1 = src + ((ch * 128 + c * 32 + 16) ^ b_swz);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        w[i].q[0] = lds(u0 + i * b_two);
                        w[i].q[1] = lds(u1 + i * b_two);
                    }
                } else if constexpr (!LOW) {
                    const uint32_t u = src + ((ch * 64 + c * 16) ^ b_swz);
#pragma unroll
                    for (int i = 0; i < 4; ++i) w[i].q[0] = lds(u + i * b_two);
                } else if constexpr (sizeof(W) == 4) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) w[i].q[0] = lds(src + c * 16 + i * b_two);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint2 v = lds64(src + c * 8 + i * b_two);
                        w[i].q[0] = make_uint4(v.x, v.y, 0, 0);
                    }
                }
#pragma unroll
                for (int m = 0; m < MPC; ++m) {
                    const uint4 hi = lds(f + m * PARTS * 512), lo = lds(f + m * PARTS * 512 + 512);
                    if constexpr (BF) {
                        if constexpr (ys == 4) {
                            const uint4 least = lds(f + m * PARTS * 512 + 1024);
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                mma_bf16(d[i], least.x, least.y, least.z, least.w, m ? w[i].q[0].z : w[i].q[0].x,
                                         m ? w[i].q[0].w : w[i].q[0].y);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if constexpr (BF) {
                            const uint32_t b0 = m ? w[i].q[0].z : w[i].q[0].x, b1 = m ? w[i].q[0].w : w[i].q[0].y;
                            mma_bf16(d[i], lo.x, lo.y, lo.z, lo.w, b0, b1);
                            mma_bf16(d[i], hi.x, hi.y, hi.z, hi.w, b0, b1);
                        } else {
                            const float u = value(w[i], 2 * m), v = value(w[i], 2 * m + 1);
                            const uint32_t b0 = tf_main<W>(u), b1 = tf_main<W>(v);
                            mma_tf32(d[i], lo.x, lo.y, lo.z, lo.w, b0, b1);
                            if constexpr (T::wide_w) mma_tf32(d[i], hi.x, hi.y, hi.z, hi.w, tf_low(u), tf_low(v));
                            mma_tf32(d[i], hi.x, hi.y, hi.z, hi.w, b0, b1);
                        }
                    }
                }
            }
            Eight e0, e1;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                e0.v[2 * i] = d[i][0], e0.v[2 * i + 1] = d[i][1];
                e1.v[2 * i] = d[i][2], e1.v[2 * i + 1] = d[i][3];
            }
            if (vec_base) {  // of rows that are not there, too: what the stage holds
                const uint32_t at = stage + base_lane + (blk - wb) * (32 * ys);
                Raw<Y> v0, v1;
                v0.q[0] = lds(at ^ base_swz);
                v1.q[0] = lds((at + 8 * across * 16) ^ base_swz);
                if constexpr (ys == 4) {
                    v0.q[1] = lds((at + 16) ^ base_swz);
                    v1.q[1] = lds((at + 8 * across * 16 + 16) ^ base_swz);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) e0.v[e] += value(v0, e), e1.v[e] += value(v1, e);
            }
            const int off = (blk - wb) * 32, left = N - n - off;
            if (a.vec_out && (nb0 + (st << bshift) + blk) * 32 + 32 <= N) {
                if (in0) store_eight(y0 + off, e0);
                if (in1) store_eight(y1 + off, e1);
            } else {
                const Y* b0 = base && !vec_base ? base + (t.row + r0) * a.ld_base + n + off : nullptr;
                if (in0) finish_plain(y0 + off, b0, left, e0);
                if (in1) finish_plain(y1 + off, b0 ? b0 + 8 * a.ld_base : nullptr, left, e1);
            }
        }
        n += per;
        y0 += per;
        y1 += per;
        slot = slot + 1 == depth ? 0 : slot + 1;
    }
}

template <typename X, typename W>
LoraKernel kernel_of(bool f32, bool low) {
    if (f32) return low ? lora_kernel<X, W, float, true> : lora_kernel<X, W, float, false>;
    return low ? lora_kernel<X, W, X, true> : lora_kernel<X, W, X, false>;
}

}  // namespace lora
}  // namespace qmm
