// qmm_lora.cuh -- low-rank adapters of many requests beside a shared
// projection: y = base + scale_a B_a (A_a x) for the rows of each segment,
// which share an adapter a.
//
// One launch.  A cluster of CTAs takes a tile of up to 64 rows of a segment:
//   1. h = A x: each CTA sums over its part of K;
//   2. the parts of h meet through distributed shared memory: each CTA adds all
//      of them up;
//   3. y = base + h B^T: each CTA has its part of the N columns.
// Few tiles with many columns have several clusters each, which find h each and
// share the columns.
// x, base and y pass once; A and B are read once a tile (from L2 where tiles
// share an adapter).  So the bound is memory for the ranks in use: 2 r flops
// against the 2 or 4 bytes of a value of x.  Measured: 4093 rows of 8192 -> 28672,
// rank 64, bf16, 166 us, 3.4 TB/s (the columns take 111 of a CTA's 143 us, the
// last 171; shared memory's data path is at 72% of its peak in the cycles that an
// SM is busy, the tensor pipe at 42%, at 18 warps an SM: two CTAs fill the shared
// memory); one row of 2048 -> 2048 6.3 us, the chain of its phases, of which h's way
// through the cluster 2.6.
//
// x and A (64 columns of K at a time), then B and base (32-column blocks of N)
// come through one ring of asynchronous copies: the first columns are on their
// way while the last of K is multiplied.  Shapes of tiles are constants of the
// kernel, so that an operand costs one load at a constant offset: products of a
// few ranks are short, and what stands around them decides (with shapes from
// registers, 4093 rows of 8192 -> 28672, rank 64, bf16 ran 98 million
// instructions in 230 us).
//
// Products are warp MMAs.  x and A of one 16-bit type multiply as they are, fp32
// x with bf16 A in three parts of 8 bits; all others as tf32, which holds either
// 16-bit type exactly, with fp32 values in two parts of 11 bits (2^-23 of a value
// is lost, and with fp32 on both sides the product of the lower parts, 2^-22 of
// a term).  h is fp32.  The second product reads it in two such parts, or, of
// bf16 B, in two parts of bf16 for 16-bit outputs (2^-18 is lost, against their
// rounding of 2^-12 or 2^-9) and three for fp32 outputs.  The tensor core
// truncates its sums, so those of 64 columns leave it for fp32 additions (left
// there, fp16 sums of 2^23 positive terms came out 1.7e-3 low; 4093 rows of 8192 ->
// 28672, rank 64, bf16, took 168 us instead of 163); with fp32 outputs those of 16
// ranks, too (rank 256, all fp32: error 2.0e-6 of the result without).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "qmm.h"
#include "qmm_device.cuh"
#include "qmm_lora.h"

namespace qmm {
namespace lora {

constexpr int WARPS = 8;             // that multiply
constexpr int THREADS = WARPS * 32;  // of these

__device__ __forceinline__ void bar_sync(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
constexpr int BAR_MULTIPLY = 1;

// ---------------------------------------------------------------- clusters
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
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

// ---------------------------------------------------------------- copies, loads
// 16 bytes global -> shared, the last 16 - n of them zeros.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int n) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
// The same of 4 bytes.
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, int n) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
// All of this thread's copies have landed.
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// An arrival of this thread when its copies until now have landed.
__device__ __forceinline__ void arrive_with_copies(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// Between the warps that copy and those that multiply: a slot is full when the
// copies into it have landed, and empty when all eight warps have read it, by
// mbarriers that count threads.  (A named barrier for the latter is 2 to 4% faster
// for prompts, but takes the arrivals of warps that no longer wait for others', and
// closes without the warps that copy, which then never leave it.)
//
// A wait gives up, for all lanes of its warp, when its time has run out or that of
// another of the CTA: the error word says so, the warp leaves the ring, and what
// follows has no meaning but ends as ever.
struct Ring {
    uint64_t full[4], empty[4];
    int dead;      // a wait has run out
    int disorder;  // of the segments' starts
};
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, const LoraArgs& a, volatile int* dead) {
    if (__all_sync(FULL, mbar_try_wait(bar, parity))) return true;
    const uint64_t t0 = global_ns();
    while (!__all_sync(FULL, mbar_try_wait_sleep(bar, parity, 20000))) {
        const bool late = global_ns() - t0 > a.wait_ns;
        if (late) {
            atomicOr(a.err, ERR_TIMEOUT);
            *dead = 1;
        }
        if (__any_sync(FULL, *dead)) return false;
    }
    return true;
}
__device__ __forceinline__ uint4 lds(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}
__device__ __forceinline__ void sts(uint32_t addr, uint32_t x) {
    asm volatile("st.shared.b32 [%0], %1;" ::"r"(addr), "r"(x) : "memory");
}
__device__ __forceinline__ float2 lds_pair(uint32_t addr) {
    float2 v;
    asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr));
    return v;
}
// Four (two) 8 x 16-byte matrices: register j of lane (g, c) is word c of row g
// of matrix j, whose rows' addresses lanes 8 j .. 8 j + 7 give.
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(a), "=r"(b), "=r"(c), "=r"(d)
                 : "r"(addr));
}
__device__ __forceinline__ void ldsm2(uint32_t addr, uint32_t& a, uint32_t& b) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x2.shared.b16 {%0, %1}, [%2];" : "=r"(a), "=r"(b) : "r"(addr));
}

// ---------------------------------------------------------------- products
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The parts of an fp32 value that tf32 holds: its upper 11 bits rounded to
// nearest, and what is left, of which the instruction reads 11 bits: 2^-23 of
// the value is lost.  (The upper part of a NaN may lose it; the lower never
// does.)
__device__ __forceinline__ uint32_t tf_high(float v) { return (__float_as_uint(v) + 0x1000u) & 0xFFFFE000u; }
__device__ __forceinline__ uint32_t tf_low(float v) { return __float_as_uint(v - __uint_as_float(tf_high(v))); }

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
__device__ __forceinline__ uint32_t bf16_part(float2& v) {
    const uint32_t p = pack_bf16(v.x, v.y);
    v.x -= __uint_as_float(p << 16);
    v.y -= __uint_as_float(p & 0xFFFF0000u);
    return p;
}
// A pair of 16-bit values as fp32.
template <typename T>
__device__ __forceinline__ float2 unpack(uint32_t w) {
    if constexpr (std::is_same<T, __nv_bfloat16>::value)
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    const __half2 h = *reinterpret_cast<const __half2*>(&w);
    return __half22float2(h);
}

// ---------------------------------------------------------------- operands
// A tile in shared memory: rows of UNITS 16-byte units, moved about within a
// row (or a group of short ones) so that what one load reads lies in different
// banks: of 16-bit types eight rows' unit u (ldmatrix), of fp32 four rows'
// units u and u + 1 (pairs, a half warp at a time).
template <typename T, int UNITS>
struct Tile {
    static constexpr bool wide = sizeof(T) == 4;
    static constexpr int pitch = UNITS * 16;
    __device__ static __forceinline__ int key(int row) {
        if constexpr (wide) return UNITS >= 8 ? (row & 3) << 1 : ((row >> 1) & 1) << 1;
        return UNITS >= 8 ? row & 7 : UNITS == 4 ? (row >> 1) & 3 : (row >> 2) & 1;
    }
    __device__ static __forceinline__ uint32_t at(int row, int unit) { return row * pitch + (unit ^ key(row)) * 16; }
};

// Fragments over 16 k, [k 0..7 and 8..15]: as 16-bit pairs or as fp32 pairs,
// lane (g, c) holding values 2 c and 2 c + 1 of each eight of row g.
template <typename T>
struct Frag {
    uint32_t w[sizeof(T) / 2][2];  // fp32: [value of the pair][eight]

    __device__ __forceinline__ float value(int eight, int i) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[i][eight]);
        const float2 p = unpack<T>(w[0][eight]);
        return i ? p.y : p.x;
    }
    __device__ __forceinline__ float2 pair(int eight) const { return make_float2(value(eight, 0), value(eight, 1)); }
};

// Rows row .. row + 15 over k16 step `step` of a tile, as two fragments (rows g, rows g + 8).
template <typename T, int UNITS>
__device__ __forceinline__ void load16(uint32_t tile, int row, int step, Frag<T> (&f)[2]) {
    const int lane = threadIdx.x & 31;
    using L = Tile<T, UNITS>;
    if constexpr (sizeof(T) == 4) {
        const int r = row + (lane >> 2), u = step * 4 + ((lane & 3) >> 1);
        const uint32_t low = tile + (lane & 1) * 8;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float2 v = lds_pair(low + L::at(r, u + 2 * e) + h * 8 * L::pitch);  // the key of rows 8 apart is the same
                f[h].w[0][e] = __float_as_uint(v.x);
                f[h].w[1][e] = __float_as_uint(v.y);
            }
    } else {
        const int r = row + (lane & 15);
        ldsm4(tile + L::at(r, step * 2 + (lane >> 4)), f[0].w[0][0], f[1].w[0][0], f[0].w[0][1], f[1].w[0][1]);
    }
}

// The other operand: N blocks of 8 rows from `row` on.  A lane's place for it ..
template <typename T, int UNITS, int N>
__device__ __forceinline__ uint32_t place8(int row, int step) {
    const int lane = threadIdx.x & 31;
    using L = Tile<T, UNITS>;
    if constexpr (sizeof(T) == 4) return L::at(row + (lane >> 2), step * 4 + ((lane & 3) >> 1)) + (lane & 1) * 8;
    return L::at(row + (lane & 7) + (N == 1 ? 0 : lane >> 4) * 8, step * 2 + ((lane >> 3) & 1));
}
// .. and the loads from there on (of fp32 the second eight k are two units on: a
// bit that the places of rows and steps leave to the key).
template <typename T, int UNITS, int N>
__device__ __forceinline__ void load8(uint32_t at, Frag<T> (&f)[N]) {
    using L = Tile<T, UNITS>;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float2 v = lds_pair((at ^ (32 * e)) + n * 8 * L::pitch);
                f[n].w[0][e] = __float_as_uint(v.x);
                f[n].w[1][e] = __float_as_uint(v.y);
            }
    } else if constexpr (N == 1) {
        ldsm2(at, f[0].w[0][0], f[0].w[0][1]);
    } else {
#pragma unroll
        for (int n = 0; n < N; n += 2)
            ldsm4(at + n * 8 * L::pitch, f[n].w[0][0], f[n].w[0][1], f[n + 1].w[0][0], f[n + 1].w[0][1]);
    }
}

// d[n] += x (16 rows) times w[n] (8 columns each), over 16 k.
template <typename X, typename W, int N>
__device__ __forceinline__ void multiply(float (&d)[N][4], const Frag<X> (&x)[2], const Frag<W> (&w)[N]) {
    constexpr bool wide_x = sizeof(X) == 4, wide_w = sizeof(W) == 4;
    if constexpr (std::is_same<X, W>::value && !wide_x) {
        const uint32_t a[4] = {x[0].w[0][0], x[1].w[0][0], x[0].w[0][1], x[1].w[0][1]};
#pragma unroll
        for (int n = 0; n < N; ++n) {
            if constexpr (std::is_same<X, __half>::value)
                mma_f16(d[n], a, w[n].w[0][0], w[n].w[0][1]);
            else
                mma_bf16(d[n], a, w[n].w[0][0], w[n].w[0][1]);
        }
    } else if constexpr (wide_x && std::is_same<W, __nv_bfloat16>::value) {
        float2 v[4] = {x[0].pair(0), x[1].pair(0), x[0].pair(1), x[1].pair(1)};
#pragma unroll
        for (int p = 0; p < 3; ++p) {
            const uint32_t a[4] = {bf16_part(v[0]), bf16_part(v[1]), bf16_part(v[2]), bf16_part(v[3])};
#pragma unroll
            for (int n = 0; n < N; ++n) mma_bf16(d[n], a, w[n].w[0][0], w[n].w[0][1]);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float v[4] = {x[0].value(e, 0), x[1].value(e, 0), x[0].value(e, 1), x[1].value(e, 1)};
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                hi[i] = wide_x ? tf_high(v[i]) : __float_as_uint(v[i]);
                lo[i] = wide_x ? tf_low(v[i]) : 0u;
            }
#pragma unroll
            for (int n = 0; n < N; ++n) {
                const float b0 = w[n].value(e, 0), b1 = w[n].value(e, 1);
                const uint32_t h0 = wide_w ? tf_high(b0) : __float_as_uint(b0), h1 = wide_w ? tf_high(b1) : __float_as_uint(b1);
                if constexpr (wide_x) mma_tf32(d[n], lo, h0, h1);
                if constexpr (wide_w) mma_tf32(d[n], hi, tf_low(b0), tf_low(b1));
                mma_tf32(d[n], hi, h0, h1);
            }
        }
    }
}

// h as an operand of the second product, [16 rows][16 k][MMA][part][lane][4
// registers]: parts of bf16 where B is bf16 (one MMA), else of tf32 (an MMA for
// each eight k; a lane's registers: value 2 c of rows g and g + 8, value 2 c + 1).
template <typename W, typename Y>
struct Hidden {
    static constexpr bool bf16 = std::is_same<W, __nv_bfloat16>::value;
    static constexpr int parts = bf16 && sizeof(Y) == 4 ? 3 : 2, mmas = bf16 ? 1 : 2, bytes = mmas * parts * 512;

    // Values k .. k + 3 of a row, k a multiple of 4, to `to`, where the tile's fragments are; k16s: of a row.
    __device__ static __forceinline__ void put(uint32_t to, int row, int k, int k16s, const float4& h) {
        const uint32_t at = to + ((row >> 4) * k16s + (k >> 4)) * bytes + (row & 7) * 64 + ((row >> 3) & 1) * 4;
        if constexpr (bf16) {
            const uint32_t b = at + ((k >> 3) & 1) * 8 + ((k >> 1) & 3) * 16;
            float2 v0 = make_float2(h.x, h.y), v1 = make_float2(h.z, h.w);
#pragma unroll
            for (int p = 0; p < parts; ++p) {
                sts(b + p * 512, bf16_part(v0));
                sts(b + p * 512 + 16, bf16_part(v1));
            }
        } else {
            const uint32_t b = at + ((k >> 3) & 1) * parts * 512 + ((k >> 1) & 3) * 16;
            const float v[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                sts(b + (i >> 1) * 16 + (i & 1) * 8, tf_high(v[i]));
                sts(b + (i >> 1) * 16 + (i & 1) * 8 + 512, tf_low(v[i]));
            }
        }
    }

    // d[n] += h times w[n]; f: this lane's registers of the 16 rows and 16 k.
    template <int N>
    __device__ static __forceinline__ void multiply(float (&d)[N][4], uint32_t f, const Frag<W> (&w)[N]) {
#pragma unroll
        for (int m = 0; m < mmas; ++m)
#pragma unroll
            for (int p = parts - 1; p >= 0; --p) {
                const uint4 q = lds(f + (m * parts + p) * 512);
                const uint32_t a[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    if constexpr (bf16) {
                        mma_bf16(d[n], a, w[n].w[0][0], w[n].w[0][1]);
                    } else {
                        const float b0 = w[n].value(m, 0), b1 = w[n].value(m, 1);
                        if constexpr (sizeof(W) == 4) {
                            if (p == 0) mma_tf32(d[n], a, tf_low(b0), tf_low(b1));
                            mma_tf32(d[n], a, tf_high(b0), tf_high(b1));
                        } else {
                            mma_tf32(d[n], a, __float_as_uint(b0), __float_as_uint(b1));
                        }
                    }
                }
            }
    }
};

// ---------------------------------------------------------------- tiles
struct RowTile {
    int64_t row;
    int rows, adapter;  // rows == 0: none; adapter < 0: none
};

// The segment of a tile and the tile's place in it, to s_tile (segment, first row,
// rows), counting tile_rows at a time through the segments; tiles of up to 16 rows
// come last, where one look sees all segments: they are done soon, and 64 rows that
// started behind 40 rows of one made a mix of 1013, 6144 -> 2051, rank 24, fp16 take
// 52 us instead of 43.
// Every thread of the block.  A start counts as the largest of those up to it,
// brought into [0, T], so that segments never share rows (which tiles of two CTAs
// would write) and their tiles are never more than were launched.  An order that
// is not kept is seen between neighbours, and all is counted again, ORDERED: with
// the largest start until now carried along.  (The first block looks at all of
// them.)
template <bool ORDERED>
__device__ __forceinline__ void find_segment(const LoraArgs& a, int tile, volatile int* disorder, int (&s_tile)[3]) {
    __shared__ uint32_t s_sum[WARPS];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) s_tile[2] = 0;
    // counts of both kinds in one number: below 2^23, and up to 256
    const bool split = a.n_segs <= THREADS && a.T <= 1 << 27;
    const uint32_t counts = split ? 0x7FFFFFu : 0xFFFFFFFFu;
    const int shift = __ffs(a.tile_rows) - 1;
    int before = 0, top = 0;  // top: the largest start until now
    for (int s0 = 0; s0 < a.n_segs; s0 += THREADS) {
        const int s = s0 + threadIdx.x;
        int n = 0, few = 0, first = 0, last = 0;
        if (s < a.n_segs && threadIdx.x < THREADS) {
            const int f = a.seg_start[s], l = a.seg_start[s + 1];
            first = max(0, min(f, (int)a.T));
            last = max(first, min(l, (int)a.T));
            if (!ORDERED && (first != f || last != l)) {
                *disorder = 1;
                if (blockIdx.x == 0) atomicOr(a.err, ERR_BAD_INDEX);
            }
        }
        if constexpr (ORDERED) {
            int most = first;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(FULL, most, o);
                if (lane >= o) most = max(most, v);
            }
            if (lane == 31 && warp < WARPS) s_sum[warp] = most;
            __syncthreads();
            most = max(most, top);
            for (int w = 0; w < WARPS; ++w) {
                const int v = (int)s_sum[w];
                if (w < warp) most = max(most, v);
                top = max(top, v);
            }
            __syncthreads();
            if (s < a.n_segs && threadIdx.x < THREADS) {
                first = most;
                last = max(most, last);
            }
        }
        n = (last - first + a.tile_rows - 1) >> shift;
        const int left = (last - first) & (a.tile_rows - 1);
        few = split && left > 0 && left <= 16;
        n -= few;
        uint32_t end = n | (uint32_t)few << 23;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t v = __shfl_up_sync(FULL, end, o);
            if (lane >= o) end += v;
        }
        if (lane == 31 && warp < WARPS) s_sum[warp] = end;
        __syncthreads();
        uint32_t all = 0;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            if (w < warp) end += s_sum[w];
            all += s_sum[w];
        }
        int at = tile - (before + (int)(end & counts) - n), tiles = n;
        if (few && tile - (int)(all & counts) == (int)(end >> 23) - 1) at = n, tiles = n + 1;
        if (at >= 0 && at < tiles) {
            s_tile[0] = s;
            s_tile[1] = first + at * a.tile_rows;
            s_tile[2] = min(a.tile_rows, last - first - at * a.tile_rows);
        }
        __syncthreads();
        before += (int)(all & counts);
        if (before > tile && blockIdx.x != 0) break;
    }
}

__device__ __forceinline__ RowTile find_tile(const LoraArgs& a, int tile, volatile int* disorder) {
    __shared__ int s_tile[3];
    RowTile t = {0, 0, -1};
    int seg = -1;
    if (!a.seg_start) {
        const int per = (a.seg_rows + a.tile_rows - 1) / a.tile_rows;
        seg = tile / per;
        const int at = (tile - seg * per) * a.tile_rows;
        if (seg >= a.n_segs) return t;
        t.row = (int64_t)seg * a.seg_rows + at;
        t.rows = min(a.tile_rows, a.seg_rows - at);
    } else {
        find_segment<false>(a, tile, disorder, s_tile);
        if (*disorder) {
            __syncthreads();  // s_tile is read by none
            find_segment<true>(a, tile, disorder, s_tile);
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

// Eight consecutive values of a row, as fp32.
struct Eight {
    float v[8];
};

// A row's part of rows that start anywhere: y = e (+ base) at two of every eight
// columns, so that four lanes store eight side by side.  (y may be base: all loads
// first, and of its own values.)
template <typename Y>
__device__ __noinline__ void finish_plain(Y* p, const Y* base, int n, Eight e) {
    Y b[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int at = (j >> 1) * 8 + (j & 1);
        b[j] = base && at < n ? base[at] : Y(0.f);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int at = (j >> 1) * 8 + (j & 1);
        if (at < n) put(p + at, as_float(b[j]) + e.v[j]);
    }
}

__device__ __forceinline__ void store16(void* p, uint4 v, bool in) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\t@p st.global.v4.b32 [%0], {%1, %2, %3, %4};\n\t}" ::"l"(p),
                 "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w), "r"((int)in)
                 : "memory");
}

template <typename Y>
__device__ __forceinline__ void store_eight(Y* p, const Eight& e, bool in) {
    if constexpr (sizeof(Y) == 4) {
        const uint32_t* v = reinterpret_cast<const uint32_t*>(e.v);
        store16(p, make_uint4(v[0], v[1], v[2], v[3]), in);
        store16(p + 4, make_uint4(v[4], v[5], v[6], v[7]), in);
    } else if constexpr (std::is_same<Y, __half>::value) {
        store16(p, make_uint4(pack_f16(e.v[0], e.v[1]), pack_f16(e.v[2], e.v[3]), pack_f16(e.v[4], e.v[5]),
                              pack_f16(e.v[6], e.v[7])), in);
    } else {
        store16(p, make_uint4(pack_bf16(e.v[0], e.v[1]), pack_bf16(e.v[2], e.v[3]), pack_bf16(e.v[4], e.v[5]),
                              pack_bf16(e.v[6], e.v[7])), in);
    }
}

// A unit of B whose rows lie on 16-byte boundaries (the last block's), on 4-byte
// ones, or on neither: a plain store then.  Nothing is read for no bytes.
template <typename W>
__device__ __noinline__ void copy_uneven(uint32_t dst, const W* src, int bytes, int vec, const void* safe) {
    if (vec == 16) {
        copy16(dst, bytes ? src : safe, bytes);
    } else if (vec == 4) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int n = max(0, min(4, bytes - 4 * q));
            copy4(dst + 4 * q, n ? reinterpret_cast<const uint32_t*>(src) + q : safe, n);
        }
    } else {
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
}

// ---------------------------------------------------------------- the kernel
// RT: ranks that are multiplied at a time (of more, groups one after another).
template <typename X, typename W, typename Y, int RT, bool WHOLE>
struct Work {
    static constexpr int XU = LORA_CHUNK * sizeof(X) / 16, AU = LORA_CHUNK * sizeof(W) / 16, BU = RT * sizeof(W) / 16;
    static constexpr int XE = 16 / sizeof(X), WE = 16 / sizeof(W), YE = 16 / sizeof(Y);
    static constexpr int YU = 32 / YE;  // units of a row of base in a 32-column block
    static constexpr int COPIERS = LORA_COPIERS<RT>;  // warps that copy, a part of each stage each
    using XT = Tile<X, XU>;
    using AT = Tile<W, AU>;
    using BT = Tile<W, BU>;

    const LoraArgs& a;
    RowTile t;
    int rank, groups, copier;
    // 1: chunks of K of this CTA, chunks of a stage, and where this thread's units come from
    int chunk0, chunks, km, a_at;  // a_at: bytes of x's rows in a chunk
    const X* x;
    const W* wa;
    // 2: columns
    const W* wb;
    const Y* base;
    int n_begin, n_end, per, blk_shift, base_at;

    // Column `col` of a 32-column block lies in row 8 i + q for column q of its
    // MMA i, q / 2 * 8 + 2 i + q % 2 = col: a lane's outputs are then eight
    // consecutive columns.
    __device__ static __forceinline__ int place(int col) {
        return !WHOLE ? col : (col & ~31) | (((col >> 1) & 3) * 8 + ((col >> 3) & 3) * 2 + (col & 1));
    }

    // The warp that copies.  Counts are constants where whole tiles are there;
    // rows that are not are left out (x, base) or zeros (A, B).
    __device__ __forceinline__ void fill_chunks(uint32_t slot, int group, int first) {
        constexpr int XS = 32 / XU, AS = 32 / AU;  // rows that are copied at a time
        const int lane = threadIdx.x & 31, n = min(km, chunks - first);
        int k0 = (chunk0 + first) * LORA_CHUNK;
        const W* wg = wa + (int64_t)group * RT * a.lda;
        const int x_row = lane / XU, w_row = lane / AU, w_left = rank - group * RT - w_row;
#pragma unroll 1
        for (int j = 0; j < n; ++j, k0 += LORA_CHUNK, slot += a_at + RT * AT::pitch) {
            // the last chunk may be half of one
            const bool xin = k0 + LORA_CHUNK <= a.K || (lane % XU) * 2 < XU;
            const bool win = k0 + LORA_CHUNK <= a.K || (lane % AU) * 2 < AU;
            const X* xs = x + (xin ? k0 : 0);
            const int xb = xin ? 16 : 0;
            xs += 16 * copier * a.ldx;
#pragma unroll 1
            for (int r = 16 * copier; r < t.rows; r += 16 * COPIERS) {
#pragma unroll
                for (int i = 0; i < 16 / XS; ++i)
                    if (r + i * XS + x_row < t.rows)
                        copy16(slot + r * XT::pitch + XT::at(i * XS + x_row, lane % XU), xs + i * XS * a.ldx, xb);
                xs += 16 * COPIERS * a.ldx;
            }
            const int first_row = copier * (RT / COPIERS), left = w_left - first_row;
            const W* ws = wg + (win ? k0 : 0) + first_row * a.lda;
            const uint32_t to = slot + a_at + first_row * AT::pitch;
#pragma unroll
            for (int i = 0; i < RT / COPIERS / AS; ++i) {
                const bool in = win && i * AS < left;
                copy16(to + AT::at(i * AS + w_row, lane % AU), in ? ws + i * AS * a.lda : wa, in ? 16 : 0);
            }
        }
    }

    // Whether plain stores were among the copies.
    __device__ __forceinline__ bool fill_columns(uint32_t slot, int n) {
        constexpr int BS = 32 / BU;  // 32 columns are BU copies of a lane
        const int lane = threadIdx.x & 31, cols = min(per, n_end - n), col = lane / BU, unit = lane % BU;
        const W* src = wb + (n - n_begin) * a.ldb;
        const bool whole = a.vec_b == 16 && n + cols <= a.N;
#pragma unroll 1
        for (int g = 0; g < groups; ++g, src += RT) {
            const int bytes = max(0, min(16, (rank - g * RT - unit * WE) * (int)sizeof(W)));
            const int64_t ld = bytes ? a.ldb : 0;
            // half a block of columns (a quarter, ..) of each copier
            constexpr int PART = BU / COPIERS;
            const int c1 = col + copier * PART * BS;
            const W* from = (bytes ? src : static_cast<const W*>(a.b)) + copier * PART * BS * ld;
            uint32_t to = slot + g * per * BT::pitch;
#pragma unroll 1
            for (int c0 = 0; c0 < cols; c0 += 32, to += 32 * BT::pitch, from += 32 * ld) {
                if (whole) {
#pragma unroll
                    for (int i = 0; i < PART; ++i) copy16(to + BT::at(place(c1 + i * BS), unit), from + i * BS * ld, bytes);
                } else {
#pragma unroll 1
                    for (int i = 0; i < PART; ++i)
                        copy_uneven(to + BT::at(place(c1 + i * BS), unit), from + i * BS * ld,
                                    n + c0 + c1 + i * BS < a.N ? bytes : 0, a.vec_b, a.b);
                }
            }
        }
        if (WHOLE && a.base) {
            // a row is 4 to 64 units: whole ones, or 32 units at a time
            const int shift = blk_shift + (YU == 8 ? 3 : 2), wide = max(0, shift - 5), s = min(shift, 5);
            const int row = (lane >> s) + copier * (32 >> s), step = COPIERS * 32 >> s;
#pragma unroll 1
            for (int h = 0; h < 1 << wide; ++h) {
                const int u = (lane & ((1 << s) - 1)) + h * 32, at = u * YE;
                const int left = at < cols ? max(0, min(16, (a.N - n - at) * (int)sizeof(Y))) : 0;
                const Y* from = left ? base + row * a.ld_base + n + at : static_cast<const Y*>(a.base);
                const int64_t ld = left ? step * a.ld_base : 0;
#pragma unroll 8
                for (int r = row; r < t.rows; r += step, from += ld)
                    copy16(slot + base_at + ((r << shift) + (u ^ base_key(r, shift))) * 16, from, left);
            }
        }
        return !a.vec_b;
    }
    // Eight lanes read a unit (two, of fp32) of four column groups of two rows.
    __device__ static __forceinline__ int base_key(int row, int shift) {
        return YU == 8 ? row & 1 : shift > 2 ? (row & 1) << 2 : 0;
    }
};

template <typename X, typename W, typename Y, int RT, bool WHOLE>
__global__ void __launch_bounds__(THREADS + 32 * LORA_COPIERS<RT>, RT == 16 ? 3 : 2)
    lora_kernel(const __grid_constant__ LoraArgs a) {
    constexpr int ALL = THREADS + 32 * LORA_COPIERS<RT>;
    using K = Work<X, W, Y, RT, WHOLE>;
    using H = Hidden<W, Y>;
    constexpr int NT = RT / 16;  // blocks of 8 ranks of a warp: half of RT
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ Ring sync;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 4; ++i) mbar_init(&sync.full[i], 32 * K::COPIERS), mbar_init(&sync.empty[i], THREADS);
        sync.dead = sync.disorder = 0;
    }
    __syncthreads();  // sync is there
    // launched after the kernels that write x and base, possibly early
    // (programmatic dependent launch): nothing is read before they complete.  What
    // follows is not let in early: its CTAs would take places as they become free,
    // unevenly, and wait there (one call after another: 2039 rows of 5632 -> 8192,
    // rank 32, 48 us instead of 42, with base 62 instead of 49; one row equal)
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // numbers of CTAs and of warps beside each other are powers of two, as
    // shifts: a division costs more than most of what follows
    const int cs = a.cluster_shift;
    const uint32_t cta = cs ? cluster_rank() : 0;
    const int parts = a.parts_shift, part = (blockIdx.x >> cs) & ((1 << parts) - 1);
    const RowTile t = find_tile(a, blockIdx.x >> (cs + parts), &sync.disorder);
    if (t.rows == 0) return;  // of all CTAs of the cluster
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
    const int N = a.N, blocks = (N + 31) / 32;
    const int64_t share = (part << cs) + (int)cta;  // of the columns
    const int nb0 = (int)(blocks * share >> (cs + parts)), nb1 = (int)(blocks * (share + 1) >> (cs + parts));
    const Y* base = static_cast<const Y*>(a.base);
    Y* y = static_cast<Y*>(a.y);

    int rank = 0;
    float scale = 1.f;
    if (t.adapter >= 0) {
        const int r = a.ranks ? a.ranks[t.adapter] : a.max_rank;
        if (a.scales) scale = a.scales[t.adapter];
        rank = max(0, min(r, a.max_rank));
        if (r != rank && threadIdx.x == 0) atomicOr(a.err, ERR_BAD_INDEX);
    }
    if (rank == 0) {
        // y = base, several loads at a time of each thread: with one, 4093 rows of 8192
        // bf16 took 47 us and 2051 fp16, which start anywhere, 93, and now 30 and 17
        // (4.5 and 2.0 TB/s)
        if (a.y == a.base) return;
        const int first = nb0 * 32, cols = min(N, nb1 * 32) - first;
        if (a.vec_out) {
            constexpr int YE = 16 / (int)sizeof(Y);
            // all rows as one list, or of long rows (whose list would pass 31 bits) one at a time
            const int units = cols / YE, at_once = units <= 1 << 24 ? t.rows : 1, all = units * at_once;
            for (int r0 = 0; r0 < t.rows; r0 += at_once)
                for (int i = threadIdx.x; i < all; i += 4 * ALL) {
                    uint4 v[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int q = i + j * ALL, r = q / units;
                        v[j] = make_uint4(0, 0, 0, 0);
                        if (q < all && base)
                            v[j] = *reinterpret_cast<const uint4*>(base + (t.row + r0 + r) * a.ld_base + first +
                                                                   (q - r * units) * YE);
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int q = i + j * ALL, r = q / units;
                        if (q < all)
                            *reinterpret_cast<uint4*>(y + (t.row + r0 + r) * a.ldy + first + (q - r * units) * YE) = v[j];
                    }
                }
        }
        const int done = a.vec_out ? cols - cols % (16 / (int)sizeof(Y)) : 0, left = cols - done;
        for (int n = threadIdx.x; n < left; n += ALL)
            for (int r0 = 0; r0 < t.rows; r0 += 8) {
                Y v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    v[j] = base && r0 + j < t.rows ? base[(t.row + r0 + j) * a.ld_base + first + done + n] : Y(0.f);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (r0 + j < t.rows) y[(t.row + r0 + j) * a.ldy + first + done + n] = v[j];
            }
        return;
    }

    // what there is to do, and the ring's first stages
    const int mtiles = (t.rows + 15) >> 4, mshift = mtiles > 2 ? 2 : mtiles - 1;  // 1, 2 or 4 warps on 16 rows each
    const int groups = (rank + RT - 1) / RT, room = groups * RT, depth = a.depth, slot_bytes = a.slot_bytes;
    const uint32_t ring = smem_u32(smem) + a.ring_at;
    K k = {a, t, rank, groups, warp - WARPS};
    {
        const int all = (a.K + LORA_CHUNK - 1) / LORA_CHUNK, tid = lane;  // (of the warp that copies)
        k.chunk0 = (int)((int64_t)all * cta >> cs);
        k.chunks = (int)((int64_t)all * (cta + 1) >> cs) - k.chunk0;
        k.a_at = mtiles * 16 * K::XT::pitch;
        k.km = 4;
        while (k.km > 1 && k.km * (k.a_at + RT * K::AT::pitch) > slot_bytes) --k.km;
        k.x = static_cast<const X*>(a.x) + (t.row + tid / K::XU) * a.ldx + tid % K::XU * K::XE;
        k.wa = static_cast<const W*>(a.a) + t.adapter * a.a_stride;
        k.wa += (tid / K::AU < rank ? tid / K::AU : 0) * a.lda + tid % K::AU * K::WE;
        k.n_begin = nb0 * 32;
        k.n_end = nb1 * 32;
        k.wb = static_cast<const W*>(a.b) + t.adapter * a.b_stride + (k.n_begin + tid / K::BU) * a.ldb + tid % K::BU * K::WE;
        k.blk_shift = 3 - mshift;
        const int block = 32 * (groups * K::BT::pitch + (WHOLE && base ? t.rows * (int)sizeof(Y) : 0));
        while (k.blk_shift && (block << k.blk_shift) > slot_bytes) --k.blk_shift;
        k.per = 32 << k.blk_shift;
        k.base_at = k.per * groups * K::BT::pitch;
        k.base = base + t.row * a.ld_base;
    }
    const int stage_k = k.km == 4   ? (k.chunks + 3) >> 2
                        : k.km == 2 ? (k.chunks + 1) >> 1
                        : k.km == 1 ? k.chunks
                                    : (k.chunks + 2) / 3,
              stages_k = stage_k * groups;  // of a group of ranks, of all
    const int stages_n = (nb1 - nb0 + (1 << k.blk_shift) - 1) >> k.blk_shift;
    const int stages = stages_k + stages_n;

    // stage s, by COPIERS warps; arrivals from the middle on may be withheld (a test's)
    const auto fill = [&](int s, int slot, int group, int chunk) {
        const uint32_t to = ring + slot * slot_bytes;
        bool plain = false;
        if (s < stages_k)
            k.fill_chunks(to, group, chunk);
        else
            plain = k.fill_columns(to, k.n_begin + (s - stages_k) * k.per);
        if (a.withhold && s >= stages / 2) return;
        if (plain) {
            copies_wait();
            mbar_arrive(&sync.full[slot]);
        } else {
            arrive_with_copies(&sync.full[slot]);
        }
    };
    // the warps that multiply fill the ring for the first time, all at once
    {
        const int s = warp / K::COPIERS;
        if (s < min(depth, stages)) {
            int group = 0, chunk = s * k.km;
            while (chunk >= k.chunks && s < stages_k) chunk -= stage_k * k.km, ++group;
            k.copier = warp % K::COPIERS;
            fill(s, s, group, chunk);
        }
    }
    if (warp >= WARPS) {
        int slot = 0, group = 0, chunk = 0;
        uint32_t parity = 0;
        asm volatile("" : "+r"(k.a_at));  // kept, not worked out again for each stage (2039 rows, fp32, rank 64: 105 -> 95 us)
        const auto step = [&] {
            chunk += k.km;
            if (chunk >= k.chunks) chunk = 0, ++group;
        };
        for (int s = 0; s < depth; ++s) step();
        const auto run = [&](int from, int until) {
            for (int s = from; s < until; ++s) {
                if (!wait(&sync.empty[slot], parity, a, &sync.dead)) return;
                fill(s, slot, group, chunk);
                step();
                slot = slot + 1 == depth ? 0 : slot + 1;
                parity ^= slot == 0;
            }
        };
        // no slot is free for more before the third step
        const int before = max(depth, min(stages, stages_k + depth));
        run(depth, before);
        if (cs) cluster_arrive(), cluster_wait(), cluster_arrive();
        run(before, stages);
        copies_wait();
        if (cs) cluster_wait();
        return;
    }

    // 1. parts of h: [part of a stage's K][16 * mtiles][room + 8] fp32.  A warp
    // has 16 rows, half of the ranks, and all of K, a half or a quarter.
    const int mt = warp & ((1 << mshift) - 1), kways = 4 >> mshift;
    const int ps = room + 8;
    int slot = 0;
    uint32_t parity = 0;
    const auto release = [&](int s, int at) {  // stage s has been read
        if (s + depth < stages) mbar_arrive(&sync.empty[at]);
    };
    {
        const int half = (warp >> mshift) & 1, kq = warp >> (mshift + 1);
        float* part = reinterpret_cast<float*>(smem) + (kq * mtiles * 16 + mt * 16 + g) * ps + half * (RT / 2) + 2 * c;
        float acc[NT][4] = {};
        int chunk = 0;
        // of a stage's chunks, or of a chunk's steps, those of this part of K
        const bool by_chunk = k.km >= kways;
        for (int s = 0; s < stages_k; ++s) {
            if (!wait(&sync.full[slot], parity, a, &sync.dead)) break;
            if (mt < mtiles) {
                const int n = min(k.km, k.chunks - chunk);
                const int chunk_bytes = k.a_at + RT * K::AT::pitch, step = by_chunk ? kways : 1;
                uint32_t xt = ring + slot * slot_bytes + (by_chunk ? kq * chunk_bytes : 0);
                for (int j = by_chunk ? kq : 0; j < n; j += step, xt += step * chunk_bytes) {
                    float d[NT][4] = {};
#pragma unroll
                    for (int st = 0; st < 4; ++st)
                        if (by_chunk || (st & (kways - 1)) == kq) {
                            Frag<X> xf[2];
                            Frag<W> wf[NT];
                            load16<X, K::XU>(xt, mt * 16, st, xf);
                            load8<W, K::AU, NT>(xt + k.a_at + place8<W, K::AU, NT>(half * (RT / 2), st), wf);
                            multiply<X, W, NT>(d, xf, wf);
                        }
#pragma unroll
                    for (int i = 0; i < NT; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[i][e] += d[i][e];
                }
            }
            release(s, slot);
            chunk += k.km;
            slot = slot + 1 == depth ? 0 : slot + 1;
            parity ^= slot == 0;
            if (chunk >= k.chunks) {  // the group's sums are done
                chunk = 0;
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    if (mt < mtiles) {
                        *reinterpret_cast<float2*>(part + 8 * i) = make_float2(acc[i][0], acc[i][1]);
                        *reinterpret_cast<float2*>(part + 8 * i + 8 * ps) = make_float2(acc[i][2], acc[i][3]);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;
                }
                part += RT;
            }
        }
    }
    if (cs)
        cluster_arrive(), cluster_wait();
    else
        bar_sync(BAR_MULTIPLY, THREADS);

    // 2. h, four ranks of a row at a time: every CTA adds up the parts of all,
    // in one order, scales the sums and cuts them up for itself.  The cluster
    // waits for one another's reads at the end alone.  (Shares of h that each CTA
    // summed for all, over a second barrier, took 7 us at 64 rows of 32 ranks and
    // 8 CTAs, scattered stores to the others most of it.)
    {
        const int per_row = room / 4, quads = t.rows * per_row;
        const uint32_t part = smem_u32(smem), frag = part + a.frag_at;
        int row = threadIdx.x / per_row, j = threadIdx.x - row * per_row;
        const int rows_on = THREADS / per_row, j_on = THREADS - rows_on * per_row;
        for (int q = threadIdx.x; q < quads; q += THREADS) {
            float4 h = make_float4(0.f, 0.f, 0.f, 0.f);
            uint32_t at = part + (row * ps + 4 * j) * 4;
            for (int kp = 0; kp < kways; ++kp, at += mtiles * 16 * ps * 4) {
                float4 v[LORA_MAX_CLUSTER];  // all on their way at once
#pragma unroll
                for (int s = 0; s < LORA_MAX_CLUSTER; ++s)
                    if (s < 1 << cs) v[s] = ld_peer(cs ? peer(at, s) : at);
#pragma unroll
                for (int s = 0; s < LORA_MAX_CLUSTER; ++s)
                    if (s < 1 << cs) h.x += v[s].x, h.y += v[s].y, h.z += v[s].z, h.w += v[s].w;
            }
            h.x *= scale, h.y *= scale, h.z *= scale, h.w *= scale;
            H::put(frag, row, 4 * j, room / 16, h);
            row += rows_on;
            j += j_on;
            if (j >= per_row) j -= per_row, ++row;
        }
    }
    if (cs) cluster_arrive();
    bar_sync(BAR_MULTIPLY, THREADS);

    // 3. the columns; a warp takes 16 rows of a 32-column block
    const int blk = warp >> mshift, r0 = mt * 16 + g;
    const bool in0 = r0 < t.rows, in1 = r0 + 8 < t.rows;
    const uint32_t frag = smem_u32(smem) + a.frag_at + mt * (room / 16) * H::bytes + lane * 16;
    // base of rows g and g + 8; rows that are not there read the last one's
    uint32_t base_of[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int shift = k.blk_shift + (K::YU == 8 ? 3 : 2), r = min(r0 + 8 * h, t.rows - 1);
        base_of[h] = k.base_at + ((r << shift) + ((blk * K::YU + c * (K::YU / 4)) ^ K::base_key(r, shift))) * 16;
        asm volatile("" : "+r"(base_of[h]));
    }
    uint32_t b_at[RT / 16];  // kept, not worked out again for each stage
#pragma unroll
    for (int st = 0; st < RT / 16; ++st) {
        b_at[st] = place8<W, K::BU, 4>(blk * 32, st);
        asm volatile("" : "+r"(b_at[st]));
    }
    constexpr int FIRST = WHOLE ? 8 : 2;  // a lane's columns in a block start at c times this
    int n = k.n_begin + blk * 32 + FIRST * c;
    Y* y0 = y + (t.row + r0) * a.ldy + n;
    for (int s = stages_k; s < stages; ++s, n += k.per, y0 += k.per) {
        if (!wait(&sync.full[slot], parity, a, &sync.dead)) break;
        const uint32_t stage = ring + slot * slot_bytes;
        const int at_slot = slot;
        slot = slot + 1 == depth ? 0 : slot + 1;
        parity ^= slot == 0;
        if (mt >= mtiles || blk >= 1 << k.blk_shift || n - FIRST * c >= k.n_end) {
            release(s, at_slot);
            continue;
        }
        float d[4][4] = {};
        uint32_t group_at = stage, h_at = frag;
#pragma unroll 1
        for (int gr = 0; gr < groups; ++gr, group_at += k.per * K::BT::pitch, h_at += RT / 16 * H::bytes) {
#pragma unroll
            for (int st = 0; st < RT / 16; ++st) {
                Frag<W> wf[4];
                load8<W, K::BU, 4>(group_at + b_at[st], wf);
                if constexpr (sizeof(Y) == 4) {
                    // sums of 16 ranks leave the tensor core, which truncates
                    float part[4][4] = {};
                    H::template multiply<4>(part, h_at + st * H::bytes, wf);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e) d[i][e] += part[i][e];
                } else {
                    H::template multiply<4>(d, h_at + st * H::bytes, wf);
                }
            }
        }
        Eight e0, e1;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            e0.v[2 * i] = d[i][0], e0.v[2 * i + 1] = d[i][1];
            e1.v[2 * i] = d[i][2], e1.v[2 * i + 1] = d[i][3];
        }
        if (WHOLE && base) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                Eight& e = h ? e1 : e0;
                const uint32_t at = stage + base_of[h];
                const uint4 q = lds(at);
                if constexpr (sizeof(Y) == 4) {
                    const uint4 r = lds(at ^ 16);  // of fp32 two units, next to one another
                    e.v[0] += __uint_as_float(q.x), e.v[1] += __uint_as_float(q.y);
                    e.v[2] += __uint_as_float(q.z), e.v[3] += __uint_as_float(q.w);
                    e.v[4] += __uint_as_float(r.x), e.v[5] += __uint_as_float(r.y);
                    e.v[6] += __uint_as_float(r.z), e.v[7] += __uint_as_float(r.w);
                } else {
                    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 p = unpack<std::conditional_t<sizeof(Y) == 4, __half, Y>>(w[i]);
                        e.v[2 * i] += p.x;
                        e.v[2 * i + 1] += p.y;
                    }
                }
            }
        }
        release(s, at_slot);
        if constexpr (WHOLE) {
            store_eight(y0, e0, in0 && n < N);
            store_eight(y0 + 8 * a.ldy, e1, in1 && n < N);
        } else {
            const Y* b = base ? base + (t.row + r0) * a.ld_base + n : nullptr;
            if (in0) finish_plain(y0, b, N - n, e0);
            if (in1) finish_plain(y0 + 8 * a.ldy, b ? b + 8 * a.ld_base : nullptr, N - n, e1);
        }
    }
    // these warps' own copies, of the first stages; unless a wait gave up they have been waited for
    if (*static_cast<volatile int*>(&sync.dead)) copies_wait();
    if (cs) cluster_wait();
}

template <typename X, typename W, typename Y, bool WHOLE>
LoraKernel kernel_of_rank(int tile) {
    return tile == 0   ? lora_kernel<X, W, Y, 16, WHOLE>
           : tile == 1 ? lora_kernel<X, W, Y, 32, WHOLE>
                       : lora_kernel<X, W, Y, 64, WHOLE>;
}

template <typename X, typename W>
LoraKernel kernel_of(bool f32, bool whole, int tile) {
    return f32 ? whole ? kernel_of_rank<X, W, float, true>(tile) : kernel_of_rank<X, W, float, false>(tile)
               : whole ? kernel_of_rank<X, W, X, true>(tile)
                       : kernel_of_rank<X, W, X, false>(tile);
}

}  // namespace lora
}  // namespace qmm
