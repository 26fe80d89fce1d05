// qmm_rope_append.cu -- what happens to q, k and v between the QKV product
// and the attention: RMSNorm of each head, rotary positions, and the write
// of k and v into the paged Q4_0 cache (qmm_rope_heads, qmm_kv_append_q4_0),
// the set-up of a rotary table (qmm_rope_table) and the values of cached
// tokens (qmm_kv_read_q4_0).
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "qmm.h"
#include "qmm_heads.cuh"
#include "qmm_internal.h"

namespace qmm {
namespace {

// ---------------------------------------------------------------- rotary table
struct Freqs {
    double f[MAX_HEAD / 2];
    double mag;
};

// Set-up: one thread an angle, in 64 bits (an angle of 131072 is good to
// 2^-36).  Bound by the 64-bit rate, once a model.
__global__ void rope_table_kernel(float2* table, int64_t n, int half, const __grid_constant__ Freqs fr) {
    for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t p = i / half;
        double s, c;
        sincos((double)p * fr.f[i - p * half], &s, &c);
        table[i] = make_float2((float)(fr.mag * c), (float)(fr.mag * s));
    }
}

// ---------------------------------------------------------------- pairs of fp32
// A value as an unevaluated sum h + l of two fp32 (|l| <= half a step of h):
// about 47 bits from error-free sums and products (Dekker 1971, Knuth's
// two-sum), in a few fp32 operations where GB300's fp64 rate is 1/64 of fp32.
// The _rn intrinsics keep the compiler from contracting them.
struct Two {
    float h, l;
};
__device__ __forceinline__ Two two_sum(float a, float b) {
    const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
    return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Two fast_two_sum(float a, float b) {  // |a| >= |b|
    const float s = __fadd_rn(a, b);
    return {s, __fsub_rn(b, __fsub_rn(s, a))};
}
__device__ __forceinline__ Two two_prod(float a, float b) {
    const float p = __fmul_rn(a, b);
    return {p, __fmaf_rn(a, b, -p)};
}
__device__ __forceinline__ Two add(Two a, Two b) {
    const Two s = two_sum(a.h, b.h);
    return fast_two_sum(s.h, __fadd_rn(s.l, __fadd_rn(a.l, b.l)));
}
__device__ __forceinline__ Two mul(Two a, Two b) {
    const Two p = two_prod(a.h, b.h);
    return fast_two_sum(p.h, __fmaf_rn(a.h, b.l, __fmaf_rn(a.l, b.h, p.l)));
}
__device__ __forceinline__ Two mul(Two a, float b) {
    const Two p = two_prod(a.h, b);
    return fast_two_sum(p.h, __fmaf_rn(a.l, b, p.l));
}

__device__ __forceinline__ float sum_of(Two a, Two b) {  // rounded once
    const Two s = two_sum(a.h, b.h);
    return __fadd_rn(s.h, __fadd_rn(s.l, __fadd_rn(a.l, b.l)));
}

// 1 / sqrt(sum / D + eps): rsqrtf's 22 bits and one step of the series
// (1 - e)^(-1/2) = 1 + e/2 + 3 e^2 / 8, e = 1 - m r^2 (about 2^-22).
__device__ __forceinline__ Two rms_inverse(Two sum, int D, float eps) {
    const float d = (float)D, q0 = __fdiv_rn(sum.h, d);
    const float rest = __fadd_rn(__fmaf_rn(-q0, d, sum.h), sum.l);
    const Two m = add(fast_two_sum(q0, __fdiv_rn(rest, d)), Two{eps, 0.f});
    const float r = rsqrtf(m.h);
    const Two p = mul(m, two_prod(r, r));
    const float e = __fsub_rn(__fsub_rn(1.f, p.h), p.l);
    return fast_two_sum(r, __fmul_rn(r, __fmul_rn(e, __fmaf_rn(0.375f, e, 0.5f))));
}

// ---------------------------------------------------------------- the kernel
enum { GROUP_Q = 0, GROUP_K = 1, GROUP_V = 2 };

// Quotients of numbers below 2^31 by one divisor d (Granlund and Montgomery):
// m = (2^(31 + s) + e) / d with 2^s >= d and 0 < e <= d, so n m / 2^(31 + s) is
// above n / d by less than 1 / d.
struct Divide {
    unsigned m, d;
    int shift;
    __host__ __device__ unsigned operator()(unsigned n) const { return (unsigned)((unsigned long long)n * m >> shift); }
};
Divide divide_by(unsigned d) {  // d in [1, 2^31)
    int s = 0;
    while ((1u << s) < d) ++s;
    return Divide{(unsigned)((1ull << (31 + s)) / d + 1), d, 31 + s};
}

struct HeadsArgs {
    Heads in[3];  // q, k, v
    Heads out;    // of q
    int heads[3], groups[3];  // heads, and warps a token for them (0: none)
    const float* norm[2];     // of q, k
    const float2* table;
    const int* pos;
    const int64_t* slots;
    uint8_t* cache;
    int64_t n_slots, n_pos, warps;  // warps: T * (sum of groups), below 2^31
    Divide per_token, page;  // by the groups of a token, by the page size
    int D, lanes, lanes_log2, n_rot, pairs;
    float eps, inv_D;
    int* err;
};

// A lane holds eight values of a head, the runs A[0..3] and B[0..3], in a
// power of two of `lanes` lanes a head and 32 / lanes heads a warp: norm and
// rotation stay in registers and sums cost log2(lanes) shuffles.  Adjacent
// pairs (PAIRS): A and B follow one another, pairs (A0, A1), (A2, A3), (B0, B1),
// (B2, B3).  Halves: pairs (Aj, Bj), A in the lower and B in the upper half of
// the rotated part; lanes past it hold what passes.  In the FAST kernels runs
// are whole aligned vectors, of the table and of the norm's weights too
// (n_rot % 8 == 0), and a lane's pairs are all rotated or none; else every
// value has its own place.
template <bool PAIRS, bool FAST>
struct Places {
    int s0, n_rot, a0, b0;
    __device__ Places(int first, int rot) : s0(first), n_rot(rot) {
        const bool halves = !PAIRS && first < rot;
        a0 = halves ? first >> 1 : first;
        b0 = halves ? (first >> 1) + (rot >> 1) : first + 4;
    }
    // Element of value j (A then B).
    __device__ int element(int j) const {
        if (FAST || PAIRS || n_rot == 0) return j < 4 ? a0 + j : b0 + j - 4;
        const int s = s0 + 2 * (j & 3) + (j >> 2);  // pairs side by side
        return s >= n_rot ? s : (s >> 1) + (s & 1) * (n_rot >> 1);
    }
    // Whether pair j is rotated, and the values that it is made of.
    __device__ bool rotated(int j) const { return (FAST ? s0 : s0 + 2 * j) < n_rot; }
    static __device__ int first(int j) { return PAIRS ? 2 * j : j; }
    static __device__ int second(int j) { return PAIRS ? 2 * j + 1 : j + 4; }
};

// The bits of a lane's eight values; loaded by themselves, so that several
// heads' loads are on their way before the first is used.  Plain loads: heads may
// be rotated in place, and what a launch writes must not be read as constant.
template <int DT, bool PAIRS>
struct Raw {
    using Run = typename std::conditional<DT == QMM_F32, uint4, uint2>::type;
    Run a, b;
    __device__ void load(const char* head, int a0, int b0) {
        if constexpr (DT != QMM_F32 && PAIRS) {  // one run of 16 bytes
            const uint4 v = *reinterpret_cast<const uint4*>(head + a0 * 2);
            a = make_uint2(v.x, v.y), b = make_uint2(v.z, v.w);
        } else {
            constexpr int size = DT == QMM_F32 ? 4 : 2;
            a = *reinterpret_cast<const Run*>(head + a0 * size);
            b = *reinterpret_cast<const Run*>(head + b0 * size);
        }
    }
    __device__ void values(float* x) const {
        if constexpr (DT == QMM_F32) {
            x[0] = __uint_as_float(a.x), x[1] = __uint_as_float(a.y), x[2] = __uint_as_float(a.z);
            x[3] = __uint_as_float(a.w), x[4] = __uint_as_float(b.x), x[5] = __uint_as_float(b.y);
            x[6] = __uint_as_float(b.z), x[7] = __uint_as_float(b.w);
        } else {
            unpack2(a.x, DT, x), unpack2(a.y, DT, x + 2), unpack2(b.x, DT, x + 4), unpack2(b.y, DT, x + 6);
        }
    }
};

template <int DT, bool PAIRS>
__device__ __forceinline__ void store_runs(char* head, int a0, int b0, const float* x) {
    if constexpr (DT == QMM_F32) {
        *reinterpret_cast<float4*>(head + a0 * 4) = make_float4(x[0], x[1], x[2], x[3]);
        *reinterpret_cast<float4*>(head + b0 * 4) = make_float4(x[4], x[5], x[6], x[7]);
    } else if constexpr (PAIRS) {
        *reinterpret_cast<uint4*>(head + a0 * 2) = make_uint4(pack2(x[0], x[1], DT), pack2(x[2], x[3], DT),
                                                              pack2(x[4], x[5], DT), pack2(x[6], x[7], DT));
    } else {
        *reinterpret_cast<uint2*>(head + a0 * 2) = make_uint2(pack2(x[0], x[1], DT), pack2(x[2], x[3], DT));
        *reinterpret_cast<uint2*>(head + b0 * 2) = make_uint2(pack2(x[4], x[5], DT), pack2(x[6], x[7], DT));
    }
}

// cos and sin of the lane's four pairs, where they are rotated.
template <bool FAST>
__device__ __forceinline__ void load_turns(const HeadsArgs& a, int p, int s0, float2* cs) {
    const float2* row = a.table + (int64_t)p * (a.n_rot / 2) + s0 / 2;
    if (FAST) {
        if (s0 >= a.n_rot) return;
        const float4 u = __ldg(reinterpret_cast<const float4*>(row));
        const float4 v = __ldg(reinterpret_cast<const float4*>(row + 2));
        cs[0] = make_float2(u.x, u.y), cs[1] = make_float2(u.z, u.w);
        cs[2] = make_float2(v.x, v.y), cs[3] = make_float2(v.z, v.w);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (s0 + 2 * j < a.n_rot) cs[j] = __ldg(row + j);
    }
}

// Small blocks: the warps of k, which take longest, hold back few others
// (4093 x 64 x 128 bf16 normed and rotated: 30.0 us with 8 warps, 28.4 with 4,
// 28.1 with 2; one token of 32 heads of 64, fp32: 2.30, 2.17 and 2.05).
constexpr int HEAD_WARPS = 2;
constexpr int READ_WARPS = 8;

// Q4_0 of a block of 32 on four lanes (lane r of them holds values 8r .. 8r +
// 7 in x), written to its places in the cache.
__device__ __forceinline__ void quantize_store(const HeadsArgs& a, int kind, const float* x, bool live, int blk, int r,
                                               uint8_t* rec, int tok) {
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(x[j]));
    m = fmaxf(m, __shfl_xor_sync(FULL, m, 1));
    m = fmaxf(m, __shfl_xor_sync(FULL, m, 2));
    const float d = __fdiv_rn(m, 7.0f), inv = __fdiv_rn(1.0f, d);
    // The code is the nearest integer of the rounded quotient x / d.  x inv is
    // less than 2^-19 from it (|x / d| < 7.01, three roundings), so both
    // have the same one unless x inv comes that close to a half; then, and where
    // d is subnormal, zero or not a number, the quotient itself decides.  Adding
    // 1.5 2^23 + 8 leaves the integer + 8 in the low byte.
    constexpr float MAGIC = 12582920.f, NEAR = 0.5f - 0x1p-19f;
    unsigned code[8];
    bool safe = d >= 0x1p-120f;  // (false for NaN)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float t = __fmul_rn(x[j], inv), at = __fadd_rn(t, MAGIC);
        safe &= fabsf(__fsub_rn(t, __fsub_rn(at, MAGIC))) <= NEAR;
        code[j] = __float_as_uint(at);
    }
    if (!__all_sync(FULL, safe || !live)) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float q = d > 0.f ? fminf(fmaxf(roundf(__fdiv_rn(x[j], d)), -8.f), 7.f) : 0.f;
            code[j] = (unsigned)((int)q + 8);
        }
    }
    const int NB = a.D / QK;
    if (kind == GROUP_K) {
        // low nibbles (values 0..15) on lanes 0, 1; high ones on lanes 2, 3
        const auto bytes = [&](int j) {
            return __byte_perm(__byte_perm(code[j], code[j + 1], 0x0040),
                               __byte_perm(code[j + 2], code[j + 3], 0x0040), 0x5410);
        };
        unsigned w0 = bytes(0), w1 = bytes(4);
        if (r >= 2) w0 <<= 4, w1 <<= 4;
        w0 |= __shfl_xor_sync(FULL, w0, 2);
        w1 |= __shfl_xor_sync(FULL, w1, 2);
        if (live) {
            const int word = 2 * (r & 1) + (r >> 1);
            *reinterpret_cast<unsigned*>(rec + blk * 512 + k_word_at(tok, word)) = r >> 1 ? w1 : w0;
            if (r == 0)
                *reinterpret_cast<unsigned short*>(rec + NB * 1024 + blk * 64 + scale_at(tok)) = f32_to_f16_bits(d);
        }
    } else {
        // lane r's values 8r + e are nibble r of unit e
        unsigned w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            w[j] = (__byte_perm(code[2 * j], code[2 * j + 1], 0x0400) & 0x000F000Fu) << (4 * r);
            w[j] |= __shfl_xor_sync(FULL, w[j], 1);
            w[j] |= __shfl_xor_sync(FULL, w[j], 2);
        }
        if (live) {
            const unsigned v = r == 0 ? w[0] : r == 1 ? w[1] : r == 2 ? w[2] : w[3];
            uint8_t* vb = rec + NB * 512 + blk * 512;
            *reinterpret_cast<unsigned short*>(vb + v_unit_at(tok, 2 * r)) = (unsigned short)(v & 0xffff);
            *reinterpret_cast<unsigned short*>(vb + v_unit_at(tok, 2 * r + 1)) = (unsigned short)(v >> 16);
            if (r == 0)
                *reinterpret_cast<unsigned short*>(rec + NB * 1088 + blk * 64 + scale_at(tok)) = f32_to_f16_bits(d);
        }
    }
}

// One warp: heads of one token, U times 32 / lanes of q (their loads are on
// their way before the first is used; the token's turns are read once) or 32 /
// lanes of k or v.  DT >= 0: every heads argument has this type and whole
// aligned runs; DT < 0: any types and strides, value by value.
//
// What bounds it.  fp32 rows of 4093 x 64 x 128: 42.3 us, 6.4 TB/s, 95% of a
// copy.  bf16 halves the bytes but not the work: 26.7 us normed, 23.0 without
// the norm, 5.1 and 5.9 TB/s; 140 instructions a warp's 32 x 8 values, 67% of
// the issue slots.  An append of 2039 tokens (64 + 8 + 8 heads, bf16) 22 us:
// k's pairs, and codes stored two or four bytes at a time because a record's
// order is the reader's.  Four of q's groups a warp against two: 30.0 and 38.2
// us for the bf16 case (with blocks of eight warps), eight as four; one group
// below 32 warps an SM, where the work would not fill the device.
template <int DT, bool PAIRS, int U>
__global__ void __launch_bounds__(HEAD_WARPS * 32) heads_kernel(const __grid_constant__ HeadsArgs a) {
    constexpr bool FAST = DT >= 0;
    __shared__ float stage[HEAD_WARPS][MAX_HEAD];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned id = blockIdx.x * HEAD_WARPS + warp;
    if (id >= (unsigned)a.warps) return;
    const int t = (int)a.per_token(id);
    int i = (int)(id - (unsigned)t * a.per_token.d);
    const int kind = i < a.groups[0] ? GROUP_Q : i < a.groups[0] + a.groups[1] ? GROUP_K : GROUP_V;
    if (kind != GROUP_Q) i -= kind == GROUP_K ? a.groups[0] : a.groups[0] + a.groups[1];
    const Heads& in = a.in[kind];
    const int sub = lane >> a.lanes_log2, u = lane & (a.lanes - 1), per = 32 >> a.lanes_log2;
    const int s0 = u * 8;
    const bool inside = s0 < a.D;
    const Places<PAIRS, FAST> at(s0, kind == GROUP_V ? 0 : a.n_rot);
    const int64_t row = t * in.ts;
    constexpr int SIZE = DT == QMM_F32 ? 4 : 2;

    Raw<FAST ? DT : QMM_F32, PAIRS> raw[U];
    const int head0 = (kind == GROUP_Q ? i * U : i) * per + sub;
    const int left = inside ? a.heads[kind] - head0 : 0;  // head k of this lane exists where k * per < left
    const char* src = in.data + (row + head0 * in.hs) * SIZE;
    const int64_t src_step = per * in.hs * SIZE;
#pragma unroll
    for (int k = 0; k < U; ++k) {
        raw[k] = {};
        if (FAST && (k == 0 || kind == GROUP_Q) && k * per < left) raw[k].load(src, at.a0, at.b0);
        src += src_step;
    }
    float2 cs[4];
    if (a.n_rot) {
        const int p = a.pos[t];
        if (p < 0 || p >= a.n_pos) {  // the whole warp: one token
            if (lane == 0) atomicOr(a.err, ERR_BAD_INDEX);
            return;
        }
        if (kind != GROUP_V) load_turns<FAST>(a, p, s0, cs);
    }
    float gamma[8];
    const float* norm = kind == GROUP_V ? nullptr : a.norm[kind];
    if (norm && inside) {
        if (FAST) {
            const float4 v = __ldg(reinterpret_cast<const float4*>(norm + at.a0));
            const float4 w = __ldg(reinterpret_cast<const float4*>(norm + at.b0));
            gamma[0] = v.x, gamma[1] = v.y, gamma[2] = v.z, gamma[3] = v.w;
            gamma[4] = w.x, gamma[5] = w.y, gamma[6] = w.z, gamma[7] = w.w;
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) gamma[j] = __ldg(norm + at.element(j));
        }
    }
    float x[8];
    const auto values = [&](int k, bool live) {
        if (FAST) {
            raw[k].values(x);
        } else {
            const int64_t head = row + (head0 + k * per) * in.hs;
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = live ? load1(in.data, head + at.element(j), in.dtype) : 0.f;
        }
    };

    if (kind == GROUP_Q) {  // fp32, rounded once to the output's type
        const int64_t to0 = t * a.out.ts + head0 * a.out.hs;
        char* dst = a.out.data + to0 * SIZE;
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const bool live = k * per < left;
            values(k, live);
            if (norm) {
                float s = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) s = fmaf(x[j], x[j], s);
                s += __shfl_xor_sync(FULL, s, 1);
                s += __shfl_xor_sync(FULL, s, 2);
                if (a.lanes > 4) s += __shfl_xor_sync(FULL, s, 4);
                if (a.lanes > 8) s += __shfl_xor_sync(FULL, s, 8);
                if (a.lanes > 16) s += __shfl_xor_sync(FULL, s, 16);
                const float r = rsqrtf(fmaf(s, a.inv_D, a.eps));
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = x[j] * r * gamma[j];
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (at.rotated(j)) {
                    float &f = x[at.first(j)], &g = x[at.second(j)];
                    const float p = f, q = g;
                    f = p * cs[j].x - q * cs[j].y;
                    g = q * cs[j].x + p * cs[j].y;
                }
            }
            if (live) {
                if constexpr (FAST) {
                    store_runs<DT, PAIRS>(dst, at.a0, at.b0, x);
                } else {  // U == 1
#pragma unroll
                    for (int j = 0; j < 8; ++j) store1(a.out.data, to0 + at.element(j), x[j], a.out.dtype);
                }
            }
            dst += per * a.out.hs * SIZE;
        }
        return;
    }

    const int64_t slot = a.slots[t];
    if (slot < 0) return;
    if (slot >= a.n_slots) {
        if (lane == 0) atomicOr(a.err, ERR_BAD_INDEX);
        return;
    }
    const bool live = inside && head0 < a.heads[kind];
    values(0, live);
    if (kind == GROUP_K) {  // pairs of fp32 up to the one rounding that the codes depend on
        Two r = {1.f, 0.f};
        if (norm) {
            Two s = {0.f, 0.f};
#pragma unroll
            for (int j = 0; j < 8; ++j) s = add(s, two_prod(x[j], x[j]));
            for (int o = a.lanes / 2; o; o >>= 1)
                s = add(s, Two{__shfl_xor_sync(FULL, s.h, o), __shfl_xor_sync(FULL, s.l, o)});
            r = rms_inverse(s, a.D, a.eps);
        }
        float* st = stage[warp] + sub * a.D;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int jp = at.first(j), jq = at.second(j);
            float p1 = x[jp], q1 = x[jq];
            if (norm) {
                Two p = mul(r, two_prod(p1, gamma[jp]));
                Two q = mul(r, two_prod(q1, gamma[jq]));
                if (at.rotated(j)) {
                    const Two pc = mul(p, cs[j].x), qs = mul(q, -cs[j].y), qc = mul(q, cs[j].x), ps = mul(p, cs[j].y);
                    p = add(pc, qs);
                    q = add(qc, ps);
                }
                p1 = __fadd_rn(p.h, p.l);
                q1 = __fadd_rn(q.h, q.l);
            } else if (at.rotated(j)) {  // the products are pairs as they are
                const float p = p1, q = q1;
                p1 = sum_of(two_prod(p, cs[j].x), two_prod(q, -cs[j].y));
                q1 = sum_of(two_prod(q, cs[j].x), two_prod(p, cs[j].y));
            }
            if (live) {
                st[at.element(jp)] = p1;
                st[at.element(jq)] = q1;
            }
        }
        __syncwarp();
        if (live) {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = st[s0 + j];
        }
    }
    const int page_size = (int)a.page.d;
    const int64_t page = (unsigned long long)slot >> 31 ? slot / page_size : (int64_t)a.page((unsigned)slot);
    const int in_page = (int)(slot - page * page_size);
    uint8_t* rec = a.cache + ((page * a.heads[kind] + head0) * (page_size / GROUP) + in_page / GROUP) *
                                 (int64_t)record_bytes(a.D);
    quantize_store(a, kind, x, live, u >> 2, u & 3, rec, in_page & 31);
}

struct ReadArgs {
    Heads out[2];  // k, v (data may be null)
    const uint8_t* cache;
    const int64_t* slots;
    int64_t n_slots, warps;
    Divide per_token, page;  // by the warps of a token, by the page size
    int D, lanes, lanes_log2, heads;
    int* err;
};

// The values of cached tokens, d (u - 8) rounded once: a lane holds eight values
// of a head, as above.  One chain of dependent loads a token (slot, then codes
// and scales): 2039 tokens of 8 heads of 128 take 7 us, in which an issued
// instruction waits 14 cycles for loads and 6 for their queue and the stores', at
// 31% of the issue slots and 36 of 64 warps an SM.
__global__ void __launch_bounds__(READ_WARPS * 32) kv_read_kernel(const __grid_constant__ ReadArgs a) {
    const int lane = threadIdx.x & 31;
    const unsigned id = blockIdx.x * READ_WARPS + (threadIdx.x >> 5);
    if (id >= (unsigned)a.warps) return;
    const int t = (int)a.per_token(id);
    const int sub = lane >> a.lanes_log2, u = lane & (a.lanes - 1);
    const int head = (int)(id - (unsigned)t * a.per_token.d) * (32 >> a.lanes_log2) + sub, s0 = u * 8;
    if (head >= a.heads || s0 >= a.D) return;
    const int64_t slot = a.slots[t];
    if (slot >= a.n_slots) {
        if (u == 0) atomicOr(a.err, ERR_BAD_INDEX);
        return;
    }
    float x[8] = {}, y[8] = {};
    if (slot >= 0) {
        const int NB = a.D / QK, blk = u >> 2, r = u & 3;
        const int page_size = (int)a.page.d;
        const int64_t page = (unsigned long long)slot >> 31 ? slot / page_size : (int64_t)a.page((unsigned)slot);
        const int in_page = (int)(slot - page * page_size), tok = in_page & 31;
        const uint8_t* base = a.cache + ((page * a.heads + head) * (page_size / GROUP) + in_page / GROUP) *
                                            (int64_t)record_bytes(a.D);
        if (a.out[0].data) {
            const float d = f16_bits_to_f32(
                *reinterpret_cast<const unsigned short*>(base + NB * 1024 + blk * 64 + scale_at(tok)));
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                const unsigned v =
                    *reinterpret_cast<const unsigned*>(base + blk * 512 + k_word_at(tok, 2 * (r & 1) + w));
#pragma unroll
                for (int j = 0; j < 4; ++j) x[4 * w + j] = d * (float)((int)(v >> (8 * j + 4 * (r >> 1)) & 15) - 8);
            }
        }
        if (a.out[1].data) {
            const float d = f16_bits_to_f32(
                *reinterpret_cast<const unsigned short*>(base + NB * 1088 + blk * 64 + scale_at(tok)));
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const unsigned v =
                    *reinterpret_cast<const unsigned short*>(base + NB * 512 + blk * 512 + v_unit_at(tok, e));
                y[e] = d * (float)((int)(v >> (4 * r) & 15) - 8);
            }
        }
    }
    if (a.out[0].data)
        storen<8>(a.out[0].data, t * a.out[0].ts + head * a.out[0].hs + s0, a.out[0].dtype, a.out[0].wide, x);
    if (a.out[1].data)
        storen<8>(a.out[1].data, t * a.out[1].ts + head * a.out[1].hs + s0, a.out[1].dtype, a.out[1].wide, y);
}

// ---------------------------------------------------------------- host side
qmm_status status_of_launch() { return cudaGetLastError() == cudaSuccess ? QMM_OK : QMM_ERR_CUDA; }

bool misaligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

qmm_status check_rope(const qmm_rope& r, int D, const int32_t* pos) {
    if (r.n_rot < 0 || r.n_pos < 0) return QMM_ERR_ARG;
    if (r.n_rot % 2 || r.n_rot > D) return QMM_ERR_SHAPE;
    if (r.n_rot == 0) return QMM_OK;
    if (!r.table || !pos) return QMM_ERR_ARG;
    if (misaligned(r.table, 8) || misaligned(pos, 4)) return QMM_ERR_ALIGN;
    return QMM_OK;
}

int lanes_of(int D) {
    int n = 4;
    while (n * 8 < D) n *= 2;
    return n;
}

int log2_of(int lanes) {
    int n = 0;
    while (1 << n < lanes) ++n;
    return n;
}

int groups_of(int heads, int lanes) { return (heads + 32 / lanes - 1) / (32 / lanes); }

void set_rope(HeadsArgs& a, const qmm_rope& r, const int32_t* pos) {
    a.table = reinterpret_cast<const float2*>(r.table);
    a.n_pos = r.n_pos;
    a.n_rot = r.n_rot;
    a.pairs = r.pairs != 0;
    a.pos = pos;
}

constexpr int64_t MAX_WARPS = (int64_t(1) << 31) - 64;
constexpr int MANY = 4;  // q's head groups a warp takes when there is plenty of work

// Warps of T tokens at `u` of q's head groups a warp.
int64_t set_groups(HeadsArgs& a, int64_t T, int u) {
    for (int g = 0; g < 3; ++g) a.groups[g] = groups_of(a.heads[g], a.lanes);
    a.groups[GROUP_Q] = (a.groups[GROUP_Q] + u - 1) / u;
    const int all = a.groups[0] + a.groups[1] + a.groups[2];
    a.per_token = divide_by(all);
    return T * all;
}

template <int DT, bool PAIRS>
void launch_form(const HeadsArgs& a, bool many, cudaStream_t st) {
    const unsigned blocks = (unsigned)((a.warps + HEAD_WARPS - 1) / HEAD_WARPS);
    if (DT >= 0 && many)
        heads_kernel<DT, PAIRS, DT >= 0 ? MANY : 1><<<blocks, HEAD_WARPS * 32, 0, st>>>(a);
    else
        heads_kernel<DT, PAIRS, 1><<<blocks, HEAD_WARPS * 32, 0, st>>>(a);
}

qmm_status launch_heads(HeadsArgs& a, int64_t T, int sms, void* stream) {
    int dt = -1;
    bool fast = a.n_rot % 8 == 0 && !misaligned(a.table, 16) && !misaligned(a.norm[0], 16) && !misaligned(a.norm[1], 16);
    a.lanes_log2 = log2_of(a.lanes);
    if (!a.page.d) a.page = divide_by(1);
    const Heads* all[4] = {&a.in[0], &a.in[1], &a.in[2], &a.out};
    for (const Heads* h : all) {
        if (!h->data) continue;
        fast &= h->wide && (dt < 0 || dt == h->dtype);
        dt = h->dtype;
    }
    if (!fast) dt = -1;
    a.warps = set_groups(a, T, MANY);
    const bool many = dt >= 0 && a.warps >= 32 * (int64_t)sms;
    if (!many) a.warps = set_groups(a, T, 1);
    if (a.warps > MAX_WARPS) return QMM_ERR_SHAPE;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    static constexpr void (*FORMS[4][2])(const HeadsArgs&, bool, cudaStream_t) = {
        {launch_form<-1, false>, launch_form<-1, true>},
        {launch_form<QMM_F32, false>, launch_form<QMM_F32, true>},
        {launch_form<QMM_F16, false>, launch_form<QMM_F16, true>},
        {launch_form<QMM_BF16, false>, launch_form<QMM_BF16, true>}};
    FORMS[dt + 1][a.pairs](a, many, st);
    return status_of_launch();
}

}  // namespace
}  // namespace qmm

using namespace qmm;

extern "C" {

qmm_status qmm_rope_table(float* table, int64_t n_pos, int32_t n_rot, double base, int32_t scaling, double factor,
                          double orig_len, double beta_fast, double beta_slow, void* stream) {
    if (n_pos < 0 || scaling < QMM_ROPE_PLAIN || scaling > QMM_ROPE_RAMP || !(base > 1.0) || !std::isfinite(base))
        return QMM_ERR_ARG;
    if (scaling != QMM_ROPE_PLAIN && !(factor >= 1.0 && std::isfinite(factor))) return QMM_ERR_ARG;
    if (scaling == QMM_ROPE_RAMP && !(orig_len > 0 && beta_slow > 0 && beta_fast >= beta_slow)) return QMM_ERR_ARG;
    if (n_rot < 2 || n_rot % 2 || n_rot > MAX_HEAD || n_pos > (int64_t(1) << 31)) return QMM_ERR_SHAPE;
    if (n_pos == 0) return QMM_OK;
    if (!table) return QMM_ERR_ARG;
    if (misaligned(table, 8)) return QMM_ERR_ALIGN;
    int sms = 0, optin = 0;
    if (!device_facts(&sms, &optin)) return QMM_ERR_DEVICE;
    Freqs fr = {};
    const int half = n_rot / 2;
    const double pi = 3.14159265358979323846;
    const auto place = [&](double turns) { return n_rot * std::log(orig_len / (2 * pi * turns)) / (2 * std::log(base)); };
    // the method clamps both ends to the head's values, 0 .. n_rot - 1, so the ramp may end past the last pair
    const double lo = scaling == QMM_ROPE_RAMP ? std::max(0.0, std::floor(place(beta_fast))) : 0;
    const double hi = scaling == QMM_ROPE_RAMP ? std::min(n_rot - 1.0, std::ceil(place(beta_slow))) : 0;
    for (int i = 0; i < half; ++i) {
        const double f = std::pow(base, -2.0 * i / n_rot);
        const double r = scaling == QMM_ROPE_LINEAR ? 1.0
                         : scaling == QMM_ROPE_RAMP
                             ? std::min(1.0, std::max(0.0, (i - lo) / std::max(hi - lo, 0.001)))
                             : 0.0;
        fr.f[i] = r > 0 ? f * (1 - r) + f / factor * r : f;
    }
    fr.mag = scaling == QMM_ROPE_RAMP ? 0.1 * std::log(factor) + 1.0 : 1.0;
    const int64_t n = n_pos * half;
    const unsigned grid = (unsigned)std::min<int64_t>((n + 255) / 256, 16 * (int64_t)sms);
    rope_table_kernel<<<grid, 256, 0, static_cast<cudaStream_t>(stream)>>>(reinterpret_cast<float2*>(table), n, half,
                                                                          fr);
    return status_of_launch();
}

qmm_status qmm_rope_heads(const qmm_rope_op* op, void* stream) {
    if (!op || op->T < 0) return QMM_ERR_ARG;
    if (!valid_head_dim(op->head_dim) || op->T > MAX_TOKENS) return QMM_ERR_SHAPE;
    if (op->T == 0) return QMM_OK;
    if (qmm_status s = check_heads(op->x, 0)) return s;
    if (qmm_status s = check_output(op->y, op->x.n_heads, op->T, op->head_dim)) return s;
    if (qmm_status s = check_rope(op->rope, op->head_dim, op->pos)) return s;
    if (misaligned(op->norm_w, 4)) return QMM_ERR_ALIGN;
    int sms = 0, optin = 0;
    if (!device_facts(&sms, &optin)) return QMM_ERR_DEVICE;
    HeadsArgs a = {};
    a.D = op->head_dim;
    a.lanes = lanes_of(a.D);
    a.in[GROUP_Q] = kernel_heads(op->x);
    a.out = kernel_heads(op->y);
    a.heads[GROUP_Q] = op->x.n_heads;
    a.norm[GROUP_Q] = op->norm_w;
    a.eps = op->norm_eps;
    a.inv_D = 1.f / a.D;
    a.err = device_error_word();
    set_rope(a, op->rope, op->pos);
    return launch_heads(a, op->T, sms, stream);
}

qmm_status qmm_kv_cache_bytes(const qmm_kv_cache* cache, size_t* bytes) {
    if (!cache || !bytes) return QMM_ERR_ARG;
    if (qmm_status s = check_cache(*cache, false)) return s;
    *bytes = (size_t)cache->n_pages * cache->n_heads * (cache->page_size / GROUP) * record_bytes(cache->head_dim);
    return QMM_OK;
}

qmm_status qmm_kv_append_q4_0(const qmm_kv_append_op* op, void* stream) {
    if (!op || op->T < 0) return QMM_ERR_ARG;
    if (op->T > MAX_TOKENS) return QMM_ERR_SHAPE;
    if (qmm_status s = check_cache(op->cache, op->T > 0)) return s;
    if (op->T == 0) return QMM_OK;
    const int D = op->cache.head_dim;
    if (qmm_status s = check_heads(op->k, op->cache.n_heads)) return s;
    if (qmm_status s = check_heads(op->v, op->cache.n_heads)) return s;
    if (op->q.data) {
        if (qmm_status s = check_heads(op->q, 0)) return s;
        if (qmm_status s = check_output(op->q_out, op->q.n_heads, op->T, D)) return s;
    }
    if (qmm_status s = check_rope(op->rope, D, op->pos)) return s;
    if (!op->slots) return QMM_ERR_ARG;
    if (misaligned(op->slots, 8) || misaligned(op->k_norm, 4) || misaligned(op->q_norm, 4)) return QMM_ERR_ALIGN;
    int sms = 0, optin = 0;
    if (!device_facts(&sms, &optin)) return QMM_ERR_DEVICE;
    HeadsArgs a = {};
    a.D = D;
    a.lanes = lanes_of(D);
    const qmm_heads* in[3] = {&op->q, &op->k, &op->v};
    for (int g = op->q.data ? GROUP_Q : GROUP_K; g <= GROUP_V; ++g) {
        a.in[g] = kernel_heads(*in[g]);
        a.heads[g] = in[g]->n_heads;
    }
    if (op->q.data) a.out = kernel_heads(op->q_out);
    a.norm[GROUP_Q] = op->q_norm;
    a.norm[GROUP_K] = op->k_norm;
    a.eps = op->norm_eps;
    a.inv_D = 1.f / a.D;
    a.err = device_error_word();
    set_rope(a, op->rope, op->pos);
    a.slots = op->slots;
    a.cache = op->cache.data;
    a.page = divide_by(op->cache.page_size);
    a.n_slots = (int64_t)op->cache.n_pages * op->cache.page_size;
    return launch_heads(a, op->T, sms, stream);
}

qmm_status qmm_kv_read_q4_0(const qmm_kv_read_op* op, void* stream) {
    if (!op || op->T < 0) return QMM_ERR_ARG;
    if (op->T > MAX_TOKENS) return QMM_ERR_SHAPE;
    if (qmm_status s = check_cache(op->cache, op->T > 0)) return s;
    if (op->T == 0 || (!op->k.data && !op->v.data)) return QMM_OK;
    if (op->k.data)
        if (qmm_status s = check_output(op->k, op->cache.n_heads, op->T, op->cache.head_dim)) return s;
    if (op->v.data)
        if (qmm_status s = check_output(op->v, op->cache.n_heads, op->T, op->cache.head_dim)) return s;
    if (!op->slots) return QMM_ERR_ARG;
    if (misaligned(op->slots, 8)) return QMM_ERR_ALIGN;
    int* err = device_error_word();
    if (!err) return QMM_ERR_DEVICE;
    ReadArgs a = {};
    a.D = op->cache.head_dim;
    a.lanes = lanes_of(a.D);
    a.heads = op->cache.n_heads;
    a.out[0] = kernel_heads(op->k);
    a.out[1] = kernel_heads(op->v);
    a.cache = op->cache.data;
    a.slots = op->slots;
    a.page = divide_by(op->cache.page_size);
    a.n_slots = (int64_t)op->cache.n_pages * op->cache.page_size;
    a.err = err;
    a.lanes_log2 = log2_of(a.lanes);
    a.per_token = divide_by(groups_of(a.heads, a.lanes));
    a.warps = op->T * groups_of(a.heads, a.lanes);
    if (a.warps > MAX_WARPS) return QMM_ERR_SHAPE;
    kv_read_kernel<<<(unsigned)((a.warps + READ_WARPS - 1) / READ_WARPS), READ_WARPS * 32, 0, static_cast<cudaStream_t>(stream)>>>(a);
    return status_of_launch();
}

}  // extern "C"
