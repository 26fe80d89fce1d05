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
// outputs of a row.  bf16 with bf16 and fp16 with fp16 multiply as they are;
// all others as tf32, which holds either 16-bit type exactly, with fp32 values
// cut in two parts of 11 bits (2^-23 of a value is lost, and with fp32 on both
// sides the product of the lower parts, 2^-22 of a term).  h is fp32, and the
// second product carries it in two parts, too (2^-23 is lost), or in two of bf16
// for bf16 outputs (2^-18, against their rounding of 2^-9) and three of bf16 for
// fp32 outputs (2^-27).  Sums of 32 products leave the tensor core, which
// truncates, for fp32 additions.
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
constexpr int GROUP_RANKS = 64;  // that a warp sums at a time

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
                 : "r"(addr)
                 : "memory");
    return v;
}
__device__ __forceinline__ void st_peer(uint32_t addr, uint32_t x, uint32_t y) {
    asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(x), "r"(y) : "memory");
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

// The parts of an fp32 value that tf32 holds, each rounded to nearest: 11 bits,
// and 11 bits of what is left, 2^-23 of it together.  (The conversion keeps NaN,
// which adding to the bits would turn into a zero.)
__device__ __forceinline__ uint32_t tf_high(float v) {
    uint32_t r;
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ uint32_t tf_low(float v) { return tf_high(v - __uint_as_float(tf_high(v))); }
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
template <typename T>
__device__ __forceinline__ Raw<T> load_raw(const T* p) {
    Raw<T> r;
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.q[i] = reinterpret_cast<const uint4*>(p)[i];
    return r;
}
// Of these, x's: every value is read once.
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

template <typename X, typename W>
struct Types {
    static constexpr bool bf16 = std::is_same<X, __nv_bfloat16>::value && std::is_same<W, __nv_bfloat16>::value;
    static constexpr bool f16 = std::is_same<X, __half>::value && std::is_same<W, __half>::value;
};

// d += rows g and g + 8 of x (x0, x1) times column g of w, over the 32 k of a
// chunk (a lane's eight, and its three neighbours').
template <typename X, typename W>
__device__ __forceinline__ void mma_chunk(float (&d)[4], const Raw<X>& x0, const Raw<X>& x1, const Raw<W>& w) {
    if constexpr (Types<X, W>::bf16) {
        mma_bf16(d, x0.q[0].x, x1.q[0].x, x0.q[0].y, x1.q[0].y, w.q[0].x, w.q[0].y);
        mma_bf16(d, x0.q[0].z, x1.q[0].z, x0.q[0].w, x1.q[0].w, w.q[0].z, w.q[0].w);
    } else if constexpr (Types<X, W>::f16) {
        mma_f16(d, x0.q[0].x, x1.q[0].x, x0.q[0].y, x1.q[0].y, w.q[0].x, w.q[0].y);
        mma_f16(d, x0.q[0].z, x1.q[0].z, x0.q[0].w, x1.q[0].w, w.q[0].z, w.q[0].w);
    } else {
        constexpr bool xs = std::is_same<X, float>::value, ws = std::is_same<W, float>::value;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float a0 = value(x0, 2 * q), a1 = value(x1, 2 * q), a2 = value(x0, 2 * q + 1),
                        a3 = value(x1, 2 * q + 1), b0 = value(w, 2 * q), b1 = value(w, 2 * q + 1);
            if constexpr (xs)
                mma_tf32(d, tf_low(a0), tf_low(a1), tf_low(a2), tf_low(a3), tf_main<W>(b0), tf_main<W>(b1));
            if constexpr (ws)
                mma_tf32(d, tf_main<X>(a0), tf_main<X>(a1), tf_main<X>(a2), tf_main<X>(a3), tf_low(b0), tf_low(b1));
            mma_tf32(d, tf_main<X>(a0), tf_main<X>(a1), tf_main<X>(a2), tf_main<X>(a3), tf_main<W>(b0),
                     tf_main<W>(b1));
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
        const int per = (a.seg_rows + LORA_ROWS - 1) / LORA_ROWS;
        seg = tile / per;
        const int at = (tile - seg * per) * LORA_ROWS;
        if (seg >= a.n_segs) return t;
        t.row = (int64_t)seg * a.seg_rows + at;
        t.rows = min(LORA_ROWS, a.seg_rows - at);
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
                n = (last - first + LORA_ROWS - 1) / LORA_ROWS;
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
                s_tile[1] = first + at * LORA_ROWS;
                s_tile[2] = min(LORA_ROWS, last - first - at * LORA_ROWS);
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
// Eight consecutive values of a row of base or y.
struct Eight {
    float v[8];
};

__device__ __forceinline__ float to_float(const void* p, int64_t i, int type) {
    if (type == QMM_F32) return static_cast<const float*>(p)[i];
    if (type == QMM_F16) return __half2float(static_cast<const __half*>(p)[i]);
    return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}
__device__ __forceinline__ void from_float(void* p, int64_t i, int type, float v) {
    if (type == QMM_F32)
        static_cast<float*>(p)[i] = v;
    else if (type == QMM_F16)
        static_cast<__half*>(p)[i] = __float2half_rn(v);
    else
        static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}

__device__ __forceinline__ Eight load_eight(const void* p, int64_t i, int n, int type, bool vec) {
    Eight e;
    if (vec && n >= 8) {
        if (type == QMM_F32) {
            const Raw<float> r = stream_raw(static_cast<const float*>(p) + i);
#pragma unroll
            for (int j = 0; j < 8; ++j) e.v[j] = value(r, j);
        } else if (type == QMM_F16) {
            const Raw<__half> r = stream_raw(static_cast<const __half*>(p) + i);
#pragma unroll
            for (int j = 0; j < 8; ++j) e.v[j] = value(r, j);
        } else {
            const Raw<__nv_bfloat16> r = stream_raw(static_cast<const __nv_bfloat16*>(p) + i);
#pragma unroll
            for (int j = 0; j < 8; ++j) e.v[j] = value(r, j);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) e.v[j] = j < n ? to_float(p, i + j, type) : 0.f;
    }
    return e;
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

__device__ __forceinline__ void store_eight(void* p, int64_t i, int n, int type, bool vec, const Eight& e) {
    if (vec && n >= 8) {
        if (type == QMM_F32) {
            float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
            q[0] = make_float4(e.v[0], e.v[1], e.v[2], e.v[3]);
            q[1] = make_float4(e.v[4], e.v[5], e.v[6], e.v[7]);
        } else if (type == QMM_F16) {
            *reinterpret_cast<uint4*>(static_cast<__half*>(p) + i) =
                make_uint4(pack_f16(e.v[0], e.v[1]), pack_f16(e.v[2], e.v[3]), pack_f16(e.v[4], e.v[5]),
                           pack_f16(e.v[6], e.v[7]));
        } else {
            *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p) + i) =
                make_uint4(pack_bf16(e.v[0], e.v[1]), pack_bf16(e.v[2], e.v[3]), pack_bf16(e.v[4], e.v[5]),
                           pack_bf16(e.v[6], e.v[7]));
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < n) from_float(p, i + j, type, e.v[j]);
    }
}

// ---------------------------------------------------------------- the kernel
// LOW: max_rank <= 16, chunks of 16 ranks in the second product.
template <typename X, typename W, bool LOW>
__global__ void __launch_bounds__(LORA_THREADS, 2) lora_kernel(const __grid_constant__ LoraArgs a) {
    constexpr bool BF = Types<X, W>::bf16;       // fragments of h: bf16 pairs, else tf32
    constexpr int NT = LOW ? 2 : 8;              // blocks of 8 ranks that a warp sums at a time
    constexpr int RC = LOW ? 16 : 32;            // ranks of a chunk
    constexpr int MPC = BF ? RC / 16 : RC / 8;   // MMAs of a chunk
    constexpr int PARTS = BF ? 3 : 2;            // of a value of h (the third of bf16 for fp32 outputs alone)
    constexpr int AHEAD = sizeof(X) == 4 ? 2 : 4;  // chunks of x that are loaded at a time
    extern __shared__ __align__(16) uint8_t smem[];
    // launched after the kernels that write x and base, possibly early
    // (programmatic dependent launch): nothing is read before they complete
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const uint32_t C = a.cluster, cta = C > 1 ? cluster_rank() : 0;
    const Tile t = find_tile(a, blockIdx.x / C);
    if (t.rows == 0) return;  // of all CTAs of the cluster
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
    const int mtiles = (t.rows + 15) >> 4;
    const int N = a.N, blocks = (N + 31) / 32;  // of 32 columns
    const int nb0 = (int)((int64_t)blocks * cta / C), nb1 = (int)((int64_t)blocks * (cta + 1) / C);
    const bool vec_y = a.vec_y, vec_base = a.vec_base;

    int rank = 0;
    if (t.adapter >= 0) {
        const int r = a.ranks ? a.ranks[t.adapter] : a.max_rank;
        rank = max(0, min(r, a.max_rank));
        if (r != rank && threadIdx.x == 0) atomicOr(a.err, ERR_BAD_INDEX);
    }
    if (rank == 0) {  // y = base
        if (a.y == a.base) return;
        for (int r = 0; r < t.rows; ++r)
            for (int n = nb0 * 32 + threadIdx.x * 8; n < min(N, nb1 * 32); n += LORA_THREADS * 8) {
                Eight e = {};
                if (a.base) e = load_eight(a.base, (t.row + r) * a.ld_base + n, N - n, a.y_type, vec_base);
                store_eight(a.y, (t.row + r) * a.ldy + n, N - n, a.y_type, vec_y, e);
            }
        return;
    }

    const int room = (rank + RC - 1) / RC * RC;  // ranks of h, the last of them zeros
    const W* wa = static_cast<const W*>(a.a) + (int64_t)t.adapter * a.a_stride;
    const W* wb = static_cast<const W*>(a.b) + (int64_t)t.adapter * a.b_stride;

    // 1. parts of h: [part of K][16 * mtiles][room + 8] fp32
    float* part = reinterpret_cast<float*>(smem);
    const int ps = room + 8;
    const int rgroups = (room + GROUP_RANKS - 1) / GROUP_RANKS, units = mtiles * rgroups;
    int kways = 1;
    while (2 * kways * units <= WARPS) kways *= 2;
    {
        const int64_t chunks = a.K / LORA_CHUNK;
        const int64_t cc0 = chunks * cta / C, ccn = chunks * (cta + 1) / C - cc0;
        for (int u = warp; u < units * kways; u += WARPS) {
            const int kp = u / units, mt = u % units % mtiles, rg = u % units / mtiles;
            const int c0 = (int)(cc0 + ccn * kp / kways), c1 = (int)(cc0 + ccn * (kp + 1) / kways);
            const int r0 = mt * 16 + g, rr = rg * GROUP_RANKS;
            const int nt = min(NT, (rank - rr + 7) >> 3);
            const bool in0 = r0 < t.rows, in1 = r0 + 8 < t.rows;
            const X* x0 = static_cast<const X*>(a.x) + (t.row + (in0 ? r0 : 0)) * a.ldx + 8 * c;
            const X* x1 = static_cast<const X*>(a.x) + (t.row + (in1 ? r0 + 8 : 0)) * a.ldx + 8 * c;
            const W* w0 = wa + (int64_t)(rr + g) * a.lda + 8 * c;
            float acc[NT][4] = {};
            for (int ch = c0; ch < c1; ch += AHEAD) {
                Raw<X> v0[AHEAD], v1[AHEAD];
#pragma unroll
                for (int i = 0; i < AHEAD; ++i) {
                    v0[i] = v1[i] = zero_raw<X>();
                    if (ch + i < c1 && in0) v0[i] = stream_raw(x0 + (ch + i) * LORA_CHUNK);
                    if (ch + i < c1 && in1) v1[i] = stream_raw(x1 + (ch + i) * LORA_CHUNK);
                }
#pragma unroll
                for (int i = 0; i < AHEAD; ++i) {
                    if (ch + i >= c1) break;
                    Raw<W> w[NT];
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        w[j] = zero_raw<W>();
                        if (rr + 8 * j + g < rank) w[j] = load_raw(w0 + (int64_t)(8 * j) * a.lda + (ch + i) * LORA_CHUNK);
                    }
#pragma unroll
                    for (int j = 0; j < NT; ++j)
                        if (j < nt) {
                            float d[4] = {};
                            mma_chunk<X, W>(d, v0[i], v1[i], w[j]);
#pragma unroll
                            for (int e = 0; e < 4; ++e) acc[j][e] += d[e];
                        }
                }
            }
            float* to = part + (kp * mtiles * 16 + r0) * ps + rr + 2 * c;
#pragma unroll
            for (int j = 0; j < NT; ++j)
                if (rr + 8 * j < room) {
                    *reinterpret_cast<float2*>(to + 8 * j) = make_float2(acc[j][0], acc[j][1]);
                    *reinterpret_cast<float2*>(to + 8 * ps + 8 * j) = make_float2(acc[j][2], acc[j][3]);
                }
        }
    }
    if (C > 1)
        cluster_barrier();
    else
        __syncthreads();

    // 2. this CTA's share of h: summed over CTAs and parts of K, scaled, cut in
    // two, to every CTA.  A fragment holds [16-row block][MMA][part][lane][16
    // bytes] with a lane's registers of row g before those of row g + 8.
    {
        const float scale = a.scales ? a.scales[t.adapter] : 1.f;
        const int per_row = room / 4, quads = mtiles * 16 * per_row, chunks = room / RC;
        const uint32_t part_at = smem_u32(part), frag_at = smem_u32(smem) + a.frag_at;
        for (int q = (int)((int64_t)quads * cta / C) + threadIdx.x; q < (int)((int64_t)quads * (cta + 1) / C);
             q += LORA_THREADS) {
            const int row = q / per_row, j = (q - row * per_row) * 4;
            float4 h = make_float4(0.f, 0.f, 0.f, 0.f);
            for (uint32_t s = 0; s < C; ++s) {
                const uint32_t from = C > 1 ? peer(part_at, s) : part_at;
                for (int kp = 0; kp < kways; ++kp) {
                    const float4 v = ld_peer(from + ((kp * mtiles * 16 + row) * ps + j) * 4);
                    h.x += v.x, h.y += v.y, h.z += v.z, h.w += v.w;
                }
            }
            h.x *= scale, h.y *= scale, h.z *= scale, h.w *= scale;
            // ranks j .. j + 3 are half of a lane's eight (RC 32) or all four (RC 16)
            const int in = j % RC, cc = LOW ? in / 4 : in / 8, half = LOW ? 0 : (in / 4) & 1;
            const int to_lane = (row & 7) * 4 + cc, reg = ((row >> 3) & 1) * 8;
            const int first = ((row >> 4) * chunks + j / RC) * MPC;
            for (uint32_t s = 0; s < C; ++s) {
                const uint32_t dst = (s + cta) % C, to = C > 1 ? peer(frag_at, dst) : frag_at;
                if constexpr (BF) {
                    const uint32_t at = to + (first + half) * PARTS * 512 + to_lane * 16 + reg;
                    float4 rest = h;
#pragma unroll
                    for (int p = 0; p < PARTS; ++p) {
                        const uint32_t u = pack_bf16(rest.x, rest.y), v = pack_bf16(rest.z, rest.w);
                        st_peer(at + p * 512, u, v);
                        rest.x -= __uint_as_float(u << 16), rest.y -= __uint_as_float(u & 0xFFFF0000u);
                        rest.z -= __uint_as_float(v << 16), rest.w -= __uint_as_float(v & 0xFFFF0000u);
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
    }
    if (C > 1)
        cluster_barrier();
    else
        __syncthreads();

    // 3. columns nb0 * 32 .. nb1 * 32: a warp takes 32 columns of 16 rows.
    // Column q of MMA block i is column 8 (q / 2) + 2 i + q % 2 of the 32, so
    // that lane c of a row gets columns 8 c .. 8 c + 7.
    const int chunks = room / RC;
    const uint8_t* frag = smem + a.frag_at;
    for (int item = warp; item < (nb1 - nb0) * mtiles; item += WARPS) {
        const int mt = item % mtiles, n0 = (nb0 + item / mtiles) * 32, r0 = mt * 16 + g, n = n0 + 8 * c;
        const int left = min(8, N - n);
        const int64_t row0 = t.row + r0;
        const bool in0 = r0 < t.rows && left > 0, in1 = r0 + 8 < t.rows && left > 0;
        Eight y0 = {}, y1 = {};
        if (a.base && in0) y0 = load_eight(a.base, row0 * a.ld_base + n, left, a.y_type, vec_base);
        if (a.base && in1) y1 = load_eight(a.base, (row0 + 8) * a.ld_base + n, left, a.y_type, vec_base);
        float d[4][4] = {};
        for (int ch = 0; ch < chunks; ++ch) {
            Raw<W> w[4];  // LOW: the first half of each
            const int k = ch * RC + (LOW ? 4 : 8) * c;  // this lane's ranks
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int col = n0 + 8 * (g >> 1) + 2 * i + (g & 1);
                const W* src = wb + col * a.ldb + k;
                w[i] = zero_raw<W>();
                if (col >= N) continue;
                constexpr int LANE = LOW ? 4 : 8;
                if (a.vec_b && k + LANE <= rank) {
                    if constexpr (!LOW) {
                        w[i] = load_raw(src);
                    } else if constexpr (sizeof(W) == 4) {
                        w[i].q[0] = *reinterpret_cast<const uint4*>(src);
                    } else {
                        const uint2 v = *reinterpret_cast<const uint2*>(src);
                        w[i].q[0].x = v.x;
                        w[i].q[0].y = v.y;
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < LANE; ++e)
                        if (k + e < rank) {
                            if constexpr (sizeof(W) == 4) {
                                reinterpret_cast<uint32_t*>(w[i].q)[e] = reinterpret_cast<const uint32_t*>(src)[e];
                            } else {
                                const uint32_t v = reinterpret_cast<const unsigned short*>(src)[e];
                                reinterpret_cast<uint32_t*>(w[i].q)[e >> 1] |= v << (16 * (e & 1));
                            }
                        }
                }
            }
            const uint4* f = reinterpret_cast<const uint4*>(frag) + (mt * chunks + ch) * MPC * PARTS * 32 + lane;
#pragma unroll
            for (int m = 0; m < MPC; ++m) {
                const uint4 hi = f[m * PARTS * 32], lo = f[m * PARTS * 32 + 32];  // (row g: two, row g + 8: two)
                uint4 least;
                if (BF && a.y_type == QMM_F32) least = f[m * PARTS * 32 + 64];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if constexpr (BF) {
                        const uint32_t b0 = m ? w[i].q[0].z : w[i].q[0].x, b1 = m ? w[i].q[0].w : w[i].q[0].y;
                        if (a.y_type == QMM_F32) mma_bf16(d[i], least.x, least.z, least.y, least.w, b0, b1);
                        mma_bf16(d[i], lo.x, lo.z, lo.y, lo.w, b0, b1);
                        mma_bf16(d[i], hi.x, hi.z, hi.y, hi.w, b0, b1);
                    } else {
                        const float b0 = value(w[i], 2 * m), b1 = value(w[i], 2 * m + 1);
                        mma_tf32(d[i], lo.x, lo.z, lo.y, lo.w, tf_main<W>(b0), tf_main<W>(b1));
                        if constexpr (sizeof(W) == 4)
                            mma_tf32(d[i], hi.x, hi.z, hi.y, hi.w, tf_low(b0), tf_low(b1));
                        mma_tf32(d[i], hi.x, hi.z, hi.y, hi.w, tf_main<W>(b0), tf_main<W>(b1));
                    }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            y0.v[2 * i] += d[i][0];
            y0.v[2 * i + 1] += d[i][1];
            y1.v[2 * i] += d[i][2];
            y1.v[2 * i + 1] += d[i][3];
        }
        if (in0) store_eight(a.y, row0 * a.ldy + n, left, a.y_type, vec_y, y0);
        if (in1) store_eight(a.y, (row0 + 8) * a.ldy + n, left, a.y_type, vec_y, y1);
    }
}

}  // namespace lora
}  // namespace qmm
