// qmm_attn.cuh -- attention over the paged Q4_0 cache (qmm_attn_q4_0): the
// kernel and what its launch passes.
//
// Mathematics.  A row is one (query, query head) pair of a key/value head's
// group.  With q', the row times a power of two, u the stored nibbles and M
// the running maximum of the row,
//   s_j = f * sum_b d_k[j][b] * sum_{e in b} q'_e (u_je - 8)
//   w_j = exp2(s_j - M)
//   out = sum_j sum_b (w_j d_v[j][b]) (u_je - 8) / sum_j w_j,
// one pass over the keys.  Scales never meet the codes: k's multiplies a
// block's sum, v's the weight, once for 32 columns.  So the codes are MMA
// operands as exact fp16 integers, a few bit operations from the stored words,
// and their products with fp16 parts of q' and of the weights are exact.
//
// Precision.  fp32 activations: q' and the weights are two fp16 parts, hi +
// lo, 22 bits; a tile of m16n8k16 holds the hi parts of eight rows in its
// upper and the lo parts in its lower half, so both parts meet each code in
// one instruction.  16-bit activations: one part (exact for q, but for bf16
// values below 2^-24 of the row's largest; a half step of 2^-12 for a weight,
// next to 2^-9 or 2^-12 of the output's own), and for k the nibbles stay
// masked as they are, the fp16 subnormals u 2^-24, with -8 sum_e q'_e as the
// accumulator's start: one operation a register less, but the tensor core
// aligns its addends to the largest, and starting from that large a value
// costs 5 bits (fp32 rows: 4e-6 of the output against 2e-7 from q = u - 8).
// Sums are fp32 throughout.  Weights times d_v are scaled by the power of two
// that brings the largest d_v so far to 2^13, so they keep their bits whatever
// the magnitude of v.
#pragma once

#include <cuda_runtime.h>

#include "qmm_heads.cuh"

namespace qmm {

constexpr int ATTN_WARPS = 4;
constexpr int ATTN_THREADS = ATTN_WARPS * 32;
constexpr int ATTN_STAGES = 4;  // records in flight or in use per token group

struct AttnMeta {  // of a CTA: the item that it leaves to the CTAs after it
    int last;      // last CTA of the item, or -1
    int seq, block, head;
    int slot;      // which of this CTA's parts is the item's
};

struct AttnArgs {
    const uint8_t* cache;
    Heads q, out;
    int8_t* yq;
    uint16_t* yd;
    const int* q_start;
    const int* kv_len;
    const int* pages;
    int64_t pages_stride, T;
    int n_pages, page_groups, kv_heads, group;  // group: query heads a key/value head
    int n_seqs, max_q, max_kv, causal, window;
    float scale_log2;
    int row_warps, blocks;  // warps along the rows of a CTA, row blocks a sequence at most
    int split;              // 0: one CTA an item; 1: items cut where the CTAs' shares end
    float* part;            // [ctas][2][rows][D + 2]
    AttnMeta* meta;         // [ctas]
    int* err;
};

// Launches the kernel of head size 32 * NB (qmm_attn_f32.cu, qmm_attn_16.cu).
cudaError_t attn_launch_f32(int NB, const AttnArgs& a, unsigned grid, int smem, cudaStream_t st);
cudaError_t attn_launch_16(int NB, const AttnArgs& a, unsigned grid, int smem, cudaStream_t st);
// Opt-in of the dynamic shared memory, once a device.
bool attn_prepare_f32(int NB, int smem_optin);
bool attn_prepare_16(int NB, int smem_optin);

// Rows of a warp's tile.
__host__ __device__ constexpr int attn_tile_rows(bool split_parts) { return split_parts ? 8 : 16; }
// CTAs an SM by registers (launch bound).
constexpr int attn_ctas(int NB) { return NB <= 4 ? 3 : 2; }

#ifdef __CUDACC__
namespace attn {

__device__ __forceinline__ void mma16816(float* c, unsigned a0, unsigned a1, unsigned a2, unsigned a3, unsigned b0,
                                         unsigned b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void cp16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ float exp2_fast(float x) {  // ex2.approx: 2 ulp, results below 2^-126 are 0
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ unsigned pack_half(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const unsigned*>(&h);
}
__device__ __forceinline__ float2 unpack_half(unsigned w) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// Two codes q = u - 8 as fp16: nibbles 0 and 4 of w (HIGH: 16 q of nibbles 1
// and 5).  An OR into fp16's exponent makes 1024 + u (1024 + 16 u), minus
// 1024 + 8 (1024 + 128); exact.
template <int HIGH>
__device__ __forceinline__ unsigned signed_codes(unsigned w) {
    const unsigned bits = (w & (HIGH ? 0x00F000F0u : 0x000F000Fu)) | 0x64006400u;
    const __half2 q =
        __hsub2(*reinterpret_cast<const __half2*>(&bits), __float2half2_rn(HIGH ? 1152.f : 1032.f));
    return *reinterpret_cast<const unsigned*>(&q);
}

// One sequence as a call sees it, its numbers clamped to their ranges.
struct Seq {
    int q0, n, L;
};
__device__ __forceinline__ Seq sequence(const AttnArgs& a, int b, bool report) {
    Seq s;
    bool bad = false;
    if (a.q_start) {
        const int x = a.q_start[b], y = a.q_start[b + 1], T = (int)a.T;
        s.q0 = min(max(x, 0), T);
        const int end = min(max(y, s.q0), T);
        s.n = min(end - s.q0, a.max_q);
        bad = x != s.q0 || y != s.q0 + s.n;
    } else {
        s.q0 = b * a.max_q;
        s.n = a.max_q;
    }
    const int L = a.kv_len[b];
    s.L = min(max(L, 0), a.max_kv);
    bad |= L != s.L;
    if (bad && report) atomicOr(a.err, ERR_BAD_INDEX);
    return s;
}

// Keys [lo, hi) that any row of a row block sees, and its units (steps of
// one record a token group); a block with rows but no keys has one unit, in
// which its zeros are written.
struct Span {
    int lo, hi, units;
};
__device__ __forceinline__ Span span_of(const AttnArgs& a, const Seq& s, int block, int block_rows, int token_warps) {
    Span r = {0, 0, 0};
    const int64_t r0 = (int64_t)block * block_rows, rows = (int64_t)s.n * a.group;
    if (r0 >= rows) return r;
    const int i0 = (int)(r0 / a.group), i1 = (int)((min(r0 + block_rows, rows) - 1) / a.group);
    r.hi = a.causal ? max(0, min(s.L, s.L - s.n + i1 + 1)) : s.L;
    r.lo = a.window ? max(0, s.L - s.n + i0 - a.window + 1) : 0;
    if (r.lo >= r.hi) {
        r.lo = r.hi = 0;
        r.units = 1;
    } else {
        r.units = ((r.hi + GROUP - 1) / GROUP - r.lo / GROUP + token_warps - 1) / token_warps;
    }
    return r;
}

// A place in the list of all units, ordered by (sequence, row block, head,
// unit).
struct Place {
    int entry, head, unit;  // entry: sequence * blocks + row block
};

// The CTA's share [u0, u1) of all units and where u0 lies.
struct Scan {
    int64_t total;
    int64_t warp_sum[ATTN_WARPS];
    Place at;
};

__device__ __forceinline__ int64_t warp_sum64(int64_t v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
    return v;
}

__device__ __forceinline__ void find_share(const AttnArgs& a, int block_rows, int token_warps, Scan& sc, int64_t& u0, int64_t& u1,
                           int64_t& share) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int entries = a.n_seqs * a.blocks;
    int64_t mine = 0;
    for (int e = tid; e < entries; e += ATTN_THREADS) {
        const int b = e / a.blocks;
        mine += span_of(a, sequence(a, b, blockIdx.x == 0), e - b * a.blocks, block_rows, token_warps).units;
    }
    mine = warp_sum64(mine);
    if (lane == 0) sc.warp_sum[warp] = mine;
    __syncthreads();
    int64_t total = 0;
#pragma unroll
    for (int w = 0; w < ATTN_WARPS; ++w) total += sc.warp_sum[w];
    total *= a.kv_heads;
    share = max((total + gridDim.x - 1) / gridDim.x, (int64_t)1);
    u0 = share * blockIdx.x;
    u1 = min(u0 + share, total);
    __syncthreads();
    if (u0 >= u1) return;
    int64_t before = 0;  // units of the entries before this chunk, times the heads
    for (int base = 0; base < entries && before <= u0; base += ATTN_THREADS) {
        const int e = base + tid;
        int units = 0;
        if (e < entries) {
            const int b = e / a.blocks;
            units = span_of(a, sequence(a, b, false), e - b * a.blocks, block_rows, token_warps).units;
        }
        int64_t incl = units;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t v = __shfl_up_sync(FULL, incl, o);
            if (lane >= o) incl += v;
        }
        if (lane == 31) sc.warp_sum[warp] = incl;
        __syncthreads();
        int64_t chunk = 0, prior = 0;
#pragma unroll
        for (int w = 0; w < ATTN_WARPS; ++w) {
            prior += w < warp ? sc.warp_sum[w] : 0;
            chunk += sc.warp_sum[w];
        }
        const int64_t start = before + (prior + incl - units) * a.kv_heads;
        if (units && u0 >= start && u0 < start + (int64_t)units * a.kv_heads) {
            const int64_t off = u0 - start;
            sc.at.entry = e;
            sc.at.head = (int)(off / units);
            sc.at.unit = (int)(off % units);
        }
        before += chunk * a.kv_heads;
        __syncthreads();
    }
}

// ---------------------------------------------------------------- the kernel
template <int NB, bool SPLIT>
struct Shape {
    static constexpr int D = NB * 32;
    static constexpr int REC = record_bytes(D);
    static constexpr int ROWS = attn_tile_rows(SPLIT);
};

// Output of a finished row of fp32 values: lane holds values 32b + lane.
template <int NB>
__device__ __forceinline__ void write_row(const AttnArgs& a, int64_t token, int head, const float* o, int lane) {
    if (a.out.data) {
        const int64_t at = token * a.out.ts + head * a.out.hs;
#pragma unroll
        for (int b = 0; b < NB; ++b) store1(a.out.data, at + b * 32 + lane, o[b], a.out.dtype);
    }
    if (a.yq) {
        const int64_t at = (token * ((int64_t)a.kv_heads * a.group) + head) * NB;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            float m = fabsf(o[b]);
#pragma unroll
            for (int s = 16; s; s >>= 1) m = fmaxf(m, __shfl_xor_sync(FULL, m, s));
            const float d = __fdiv_rn(m, 127.0f);
            const float q = d > 0.f ? fminf(fmaxf(roundf(__fdiv_rn(o[b], d)), -127.f), 127.f) : 0.f;
            a.yq[(at + b) * 32 + lane] = (int8_t)(int)q;
            if (lane == 0) a.yd[at + b] = f32_to_f16_bits(d);
        }
    }
}

template <int NB, bool SPLIT>
__global__ void __launch_bounds__(ATTN_THREADS, attn_ctas(NB)) attn_kernel(const __grid_constant__ AttnArgs a) {
    using S = Shape<NB, SPLIT>;
    constexpr int D = S::D, REC = S::REC, ROWS = S::ROWS;
    constexpr int RS = SPLIT ? 1 : 2;  // rows a lane keeps statistics of
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ Scan sc;
    __shared__ float s_m[ATTN_WARPS][16], s_l[ATTN_WARPS][16];

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, c = lane & 3;
    const int RW = a.row_warps, TW = ATTN_WARPS / RW;
    const int wr = warp / TW, wt = warp - wr * TW;
    const int block_rows = RW * ROWS;
    uint8_t* ring = smem + wt * (ATTN_STAGES * REC);

    Place at;
    int64_t u0, u1, share = 0;
    if (a.split) {
        if (tid == 0) a.meta[blockIdx.x].last = -1;
        find_share(a, block_rows, TW, sc, u0, u1, share);
        if (u0 >= u1) return;
        at = sc.at;
    } else {  // one CTA an item, later row blocks (more keys) first
        const int e = blockIdx.x / a.kv_heads, b = e / a.blocks;
        at.head = blockIdx.x - e * a.kv_heads;
        at.entry = b * a.blocks + (a.blocks - 1 - (e - b * a.blocks));
        at.unit = 0;
        u0 = 0;
        u1 = 1;
    }

    for (int64_t u = u0; u < u1;) {
        const int b = at.entry / a.blocks, block = at.entry - b * a.blocks;
        const Seq seq = sequence(a, b, !a.split && tid == 0);
        const Span sp = span_of(a, seq, block, block_rows, TW);
        if (sp.units == 0) {
            if (!a.split) return;
            ++at.entry, at.head = 0, at.unit = 0;
            continue;
        }
        const int unit_end = a.split ? (int)min((int64_t)sp.units, at.unit + (u1 - u)) : sp.units;
        const int rec0 = sp.lo / GROUP + at.unit * TW;
        const int rec_end = min((sp.hi + GROUP - 1) / GROUP, sp.lo / GROUP + unit_end * TW);

        // ---- the rows of this lane, q' as MMA operands
        const int rows = seq.n * a.group;
        int lo[RS], hi[RS];
        float f[RS], seed[RS][NB];
        unsigned qa[NB][2][4];  // [block][k step][a0..a3]
#pragma unroll
        for (int r = 0; r < RS; ++r) {
            const int row = block * block_rows + wr * ROWS + g + 8 * r;
            const bool live = row < rows;
            const int i = live ? row / a.group : 0, h = live ? row - i * a.group : 0;
            const int p = seq.L - seq.n + i;
            hi[r] = live && a.causal ? min(seq.L, p + 1) : sp.hi;
            lo[r] = live && a.window ? p - a.window + 1 : sp.lo;
            const int64_t at_q = (int64_t)(seq.q0 + i) * a.q.ts + (int64_t)(at.head * a.group + h) * a.q.hs;
            float x[NB][8], top = 0.f;
#pragma unroll
            for (int k = 0; k < NB; ++k) {
                if (live) {
                    loadn<4>(a.q.data, at_q + 32 * k + 4 * c, a.q.dtype, a.q.wide, x[k]);
                    loadn<4>(a.q.data, at_q + 32 * k + 16 + 4 * c, a.q.dtype, a.q.wide, x[k] + 4);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[k][e] = 0.f;
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(x[k][e]));
            }
            top = fmaxf(top, __shfl_xor_sync(FULL, top, 1));
            top = fmaxf(top, __shfl_xor_sync(FULL, top, 2));
            // top * 2^up in [2^13, 2^14); a negative scale goes into q', a scale of 0 makes it 0
            const int up = top > 0.f ? 13 - min(max(ilogbf(top), -100), 100) : 0;
            const float mul = a.scale_log2 == 0.f ? 0.f : copysignf(exp2f((float)up), a.scale_log2);
            // a masked nibble as it is (16-bit types) is the subnormal u 2^-24
            f[r] = a.scale_log2 == 0.f ? 1.f : fabsf(a.scale_log2) * exp2f((float)((SPLIT ? 0 : 24) - up));
#pragma unroll
            for (int k = 0; k < NB; ++k) {
                float sum = 0.f;
                float y[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = x[k][e] * (e < 4 ? mul : mul * 0.0625f);  // high nibbles weigh 16
                // order of the operand's k places: values 4c, 4c+2 | 4c+1, 4c+3 of each half of the block
#pragma unroll
                for (int st = 0; st < 2; ++st) {
                    const unsigned h0 = pack_half(y[4 * st], y[4 * st + 2]);
                    const unsigned h1 = pack_half(y[4 * st + 1], y[4 * st + 3]);
                    const float2 a0 = unpack_half(h0), a1 = unpack_half(h1);
                    qa[k][st][r] = h0;
                    qa[k][st][2 + r] = h1;
                    if constexpr (SPLIT) {
                        const unsigned l0 = pack_half(y[4 * st] - a0.x, y[4 * st + 2] - a0.y);
                        const unsigned l1 = pack_half(y[4 * st + 1] - a1.x, y[4 * st + 3] - a1.y);
                        qa[k][st][1] = l0;
                        qa[k][st][3] = l1;
                    } else {
                        const float part = a0.x + a0.y + a1.x + a1.y;
                        sum += st ? 16.f * part : part;
                    }
                }
                if constexpr (!SPLIT) {
                    sum += __shfl_xor_sync(FULL, sum, 1);
                    sum += __shfl_xor_sync(FULL, sum, 2);
                    seed[r][k] = sum * (-8.f * 5.9604644775390625e-8f);  // -8 in units of 2^-24
                }
            }
        }

        float acc[NB][4][4] = {};  // [block][n tile][rows g: 2 columns, rows g + 8 (or lo parts): 2 columns]
        float top[RS], l[RS];  // running maximum of the scores (before f) and sum of the weights
        float vs = 1.f;        // power of two that acc holds the weighted v times, from the largest scale so far
        int vexp = 100;
#pragma unroll
        for (int r = 0; r < RS; ++r) top[r] = -INFINITY, l[r] = 0.f;

        // ---- the ring: one record a step and token group
        const int64_t table = (int64_t)b * a.pages_stride;
        const int n_mine = rec_end > rec0 + wt ? (rec_end - rec0 - wt + TW - 1) / TW : 0;
        unsigned bad = 0;  // stages whose page does not exist
        const auto issue = [&](int k) {
            if (k < n_mine) {
                const int rec = rec0 + wt + k * TW;
                const int pg = rec / a.page_groups, in = rec - pg * a.page_groups;
                int page = a.pages[table + pg];
                const int stage = k % ATTN_STAGES;
                if (page < 0 || page >= a.n_pages) {
                    bad |= 1u << stage;
                    if (lane == 0) atomicOr(a.err, ERR_BAD_INDEX);
                } else {
                    bad &= ~(1u << stage);
                    const uint8_t* src =
                        a.cache + (((int64_t)page * a.kv_heads + at.head) * a.page_groups + in) * (int64_t)REC;
                    uint8_t* dst = ring + stage * REC;
                    for (int i = wr * 32 + lane; i < REC / 16; i += RW * 32) cp16(dst + 16 * i, src + 16 * i);
                }
            }
            cp_commit();
        };
        const auto sync_group = [&]() {
            if (RW == 1)
                __syncwarp();
            else
                asm volatile("bar.sync %0, %1;" ::"r"(1 + wt), "r"(RW * 32) : "memory");
        };
#pragma unroll
        for (int k = 0; k < ATTN_STAGES - 1; ++k) issue(k);

        for (int k = 0; k < n_mine; ++k) {
            cp_wait<ATTN_STAGES - 2>();
            sync_group();  // everyone's copies of record k are there, and its predecessor is read
            issue(k + ATTN_STAGES - 1);
            const uint8_t* rec = ring + (k % ATTN_STAGES) * REC;
            const int tok0 = (rec0 + wt + k * TW) * GROUP;

            // scores
            float s[4][2 * RS] = {};
#pragma unroll
            for (int kb = 0; kb < NB; ++kb) {
                const uint4 w4 = lds128(rec + kb * 512 + lane * 16);
                const uint4 d4 = lds128(rec + NB * 1024 + kb * 64 + c * 16);
                const unsigned w[4] = {w4.x, w4.y, w4.z, w4.w}, d[4] = {d4.x, d4.y, d4.z, d4.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float t[4];
                    if constexpr (SPLIT) {
                        t[0] = t[1] = t[2] = t[3] = 0.f;
                        mma16816(t, qa[kb][0][0], qa[kb][0][1], qa[kb][0][2], qa[kb][0][3], signed_codes<0>(w[j]),
                                 signed_codes<0>(w[j] >> 8));
                        mma16816(t, qa[kb][1][0], qa[kb][1][1], qa[kb][1][2], qa[kb][1][3], signed_codes<1>(w[j]),
                                 signed_codes<1>(w[j] >> 8));
                    } else {
                        t[0] = t[1] = seed[0][kb], t[2] = t[3] = seed[RS - 1][kb];
                        const unsigned w8 = w[j] >> 8;
                        mma16816(t, qa[kb][0][0], qa[kb][0][1], qa[kb][0][2], qa[kb][0][3], w[j] & 0x000F000Fu,
                                 w8 & 0x000F000Fu);
                        mma16816(t, qa[kb][1][0], qa[kb][1][1], qa[kb][1][2], qa[kb][1][3], w[j] & 0x00F000F0u,
                                 w8 & 0x00F000F0u);
                    }
                    const float2 dk = unpack_half(d[j]);
                    if constexpr (SPLIT) {
                        s[j][0] = fmaf(dk.x, t[0] + t[2], s[j][0]);
                        s[j][1] = fmaf(dk.y, t[1] + t[3], s[j][1]);
                    } else {
                        s[j][0] = fmaf(dk.x, t[0], s[j][0]);
                        s[j][1] = fmaf(dk.y, t[1], s[j][1]);
                        s[j][2] = fmaf(dk.x, t[2], s[j][2]);
                        s[j][3] = fmaf(dk.y, t[3], s[j][3]);
                    }
                }
            }
            // the mask, where a row does not see all 32 keys
            const bool gone = bad >> (k % ATTN_STAGES) & 1;
            bool full = !gone;
#pragma unroll
            for (int r = 0; r < RS; ++r) full &= tok0 >= lo[r] && tok0 + GROUP <= hi[r];
            const bool masked = __any_sync(FULL, !full);
            if (masked) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int e = 0; e < 2 * RS; ++e) {
                        const int key = tok0 + 8 * j + 2 * c + (e & 1);
                        if (gone || key < lo[e >> 1] || key >= hi[e >> 1]) s[j][e] = -INFINITY;
                    }
            }

            // scales of v, and the weights' reference
            unsigned vd[NB][4];
            __half2 big = __float2half2_rn(0.f);
#pragma unroll
            for (int kb = 0; kb < NB; ++kb) {
                const uint4 d4 = lds128(rec + NB * 1088 + kb * 64 + c * 16);
                vd[kb][0] = d4.x, vd[kb][1] = d4.y, vd[kb][2] = d4.z, vd[kb][3] = d4.w;
                if (masked) {  // keys that no row of the block sees may hold anything
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int key = tok0 + 8 * j + 2 * c;
                        if (gone || key < sp.lo || key >= sp.hi) vd[kb][j] &= 0xFFFF0000u;
                        if (gone || key + 1 < sp.lo || key + 1 >= sp.hi) vd[kb][j] &= 0x0000FFFFu;
                    }
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) big = __hmax2(big, __habs2(*reinterpret_cast<const __half2*>(&vd[kb][j])));
            }
            float dmax = fmaxf(__low2float(big), __high2float(big));
            dmax = fmaxf(dmax, __shfl_xor_sync(FULL, dmax, 1));
            dmax = fmaxf(dmax, __shfl_xor_sync(FULL, dmax, 2));
            // dmax * vs < 2^14
            const int room = 13 - (int)((__float_as_uint(dmax) >> 23) - 127);
            float ratio = 1.f;
            if (room < vexp) {
                vexp = max(room, -100);
                const float now = exp2f((float)vexp);
                ratio = now / vs;
                vs = now;
            }
            float ref[RS], alpha[RS];
            bool moved = ratio != 1.f;
#pragma unroll
            for (int r = 0; r < RS; ++r) {
                float m = top[r];
#pragma unroll
                for (int j = 0; j < 4; ++j) m = fmaxf(m, fmaxf(s[j][2 * r], s[j][2 * r + 1]));
                m = fmaxf(m, __shfl_xor_sync(FULL, m, 1));
                m = fmaxf(m, __shfl_xor_sync(FULL, m, 2));
                ref[r] = m == -INFINITY ? 0.f : m * f[r];  // nothing seen yet: every weight is 0
                moved |= m != top[r];
                alpha[r] = exp2_fast(fmaf(top[r], f[r], -ref[r]));
                top[r] = m;
            }
            if (__any_sync(FULL, moved)) {
#pragma unroll
                for (int r = 0; r < RS; ++r) {
                    l[r] *= alpha[r];
                    const float by = alpha[r] * ratio;
#pragma unroll
                    for (int kb = 0; kb < NB; ++kb)
#pragma unroll
                        for (int n = 0; n < 4; ++n) {
                            acc[kb][n][2 * r] *= by, acc[kb][n][2 * r + 1] *= by;
                            if (SPLIT) acc[kb][n][2] *= by, acc[kb][n][3] *= by;
                        }
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int e = 0; e < 2 * RS; ++e) {
                    const float w = exp2_fast(fmaf(s[j][e], f[e >> 1], -ref[e >> 1]));
                    l[e >> 1] += w;
                    s[j][e] = w * vs;
                }

            // weights times v
#pragma unroll
            for (int kb = 0; kb < NB; ++kb) {
                const uint4 w4 = lds128(rec + NB * 512 + kb * 512 + lane * 16);
                const unsigned w[4] = {w4.x, w4.y, w4.z, w4.w};
                unsigned up[4], dn[4];  // the A operand's rows 0..7 and 8..15, two tokens each
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 d = unpack_half(vd[kb][j]);
                    const float x = s[j][0] * d.x, y = s[j][1] * d.y;
                    up[j] = pack_half(x, y);
                    if constexpr (SPLIT) {
                        const float2 h = unpack_half(up[j]);
                        dn[j] = pack_half(x - h.x, y - h.y);
                    } else {
                        dn[j] = pack_half(s[j][2] * d.x, s[j][3] * d.y);
                    }
                }
#pragma unroll
                for (int st = 0; st < 2; ++st) {
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        const unsigned x = n >= 2 ? w[2 * st] >> 8 : w[2 * st];
                        const unsigned y = n >= 2 ? w[2 * st + 1] >> 8 : w[2 * st + 1];
                        mma16816(acc[kb][n], up[2 * st], dn[2 * st], up[2 * st + 1], dn[2 * st + 1],
                                 n & 1 ? signed_codes<1>(x) : signed_codes<0>(x),
                                 n & 1 ? signed_codes<1>(y) : signed_codes<0>(y));
                    }
                }
            }
        }

        // ---- join the token groups: O, M and l of every row
#pragma unroll
        for (int r = 0; r < RS; ++r) {
            l[r] += __shfl_xor_sync(FULL, l[r], 1);
            l[r] += __shfl_xor_sync(FULL, l[r], 2);
            top[r] *= f[r];  // -inf stays: f > 0
            if (c == 0) s_m[warp][g + 8 * r] = top[r], s_l[warp][g + 8 * r] = l[r];
        }
        cp_wait<0>();
        __syncthreads();  // the ring is free
        float* buf = reinterpret_cast<float*>(smem);  // [warp][ROWS][D]
#pragma unroll
        for (int r = 0; r < RS; ++r) {
            float m = -INFINITY;
            for (int t = 0; t < TW; ++t) m = fmaxf(m, s_m[wr * TW + t][g + 8 * r]);
            const float w = top[r] == -INFINITY ? 0.f : exp2_fast(top[r] - m) / vs;
            float* o = buf + (warp * ROWS + g + 8 * r) * D;
#pragma unroll
            for (int kb = 0; kb < NB; ++kb)
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const float wn = n & 1 ? w * 0.0625f : w;  // high nibbles weigh 16
                    float2 v;
                    if (SPLIT)
                        v = make_float2((acc[kb][n][0] + acc[kb][n][2]) * wn, (acc[kb][n][1] + acc[kb][n][3]) * wn);
                    else
                        v = make_float2(acc[kb][n][2 * r] * wn, acc[kb][n][2 * r + 1] * wn);
                    *reinterpret_cast<float2*>(o + kb * 32 + n * 8 + 2 * c) = v;
                }
        }
        __syncthreads();
        const bool whole = at.unit == 0 && unit_end == sp.units;
        // a share's first segment keeps its part in slot 0, its last in slot 1
        float* part = nullptr;
        if (!whole) part = a.part + ((int64_t)blockIdx.x * 2 + (u != u0)) * block_rows * (D + 2);
        for (int row = warp; row < block_rows; row += ATTN_WARPS) {
            const int rw = row / ROWS, rr = row - rw * ROWS;
            float m = -INFINITY, sum = 0.f, o[NB] = {};
            for (int t = 0; t < TW; ++t) m = fmaxf(m, s_m[rw * TW + t][rr]);
            for (int t = 0; t < TW; ++t) {
                const float mt = s_m[rw * TW + t][rr];
                sum += mt == -INFINITY ? 0.f : s_l[rw * TW + t][rr] * exp2_fast(mt - m);
#pragma unroll
                for (int kb = 0; kb < NB; ++kb) o[kb] += buf[((rw * TW + t) * ROWS + rr) * D + kb * 32 + lane];
            }
            const int global_row = block * block_rows + row;
            if (global_row >= rows) break;
            if (whole) {
                const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
                for (int kb = 0; kb < NB; ++kb) o[kb] *= inv;
                const int i = global_row / a.group;
                write_row<NB>(a, seq.q0 + i, at.head * a.group + global_row - i * a.group, o, lane);
            } else {
#pragma unroll
                for (int kb = 0; kb < NB; ++kb) part[row * (D + 2) + kb * 32 + lane] = o[kb];
                if (lane == 0) part[row * (D + 2) + D] = m, part[row * (D + 2) + D + 1] = sum;
            }
        }
        if (a.split) {
            if (tid == 0 && at.unit == 0 && !whole) {
                AttnMeta& mt = a.meta[blockIdx.x];
                mt.last = (int)((u + sp.units - 1) / share);
                mt.seq = b, mt.block = block, mt.head = at.head, mt.slot = u != u0;
            }
            __syncthreads();  // buf and the statistics are read
        }
        u += unit_end - at.unit;
        at.unit = 0;
        if (++at.head == a.kv_heads) at.head = 0, ++at.entry;
        if (!a.split) return;
    }
}

// Joins the parts of the items that were cut: block (x, y) takes rows y, y +
// gridDim.y, ... of the item that CTA x left unfinished, its parts in the
// order of the CTAs.
template <int NB>
__global__ void __launch_bounds__(128) attn_join_kernel(const __grid_constant__ AttnArgs a, int block_rows) {
    constexpr int D = NB * 32;
    const AttnMeta mt = a.meta[blockIdx.x];
    if (mt.last < 0) return;
    const int lane = threadIdx.x & 31;
    const Seq seq = sequence(a, mt.seq, false);
    const int rows = seq.n * a.group;
    for (int row = blockIdx.y * 4 + (threadIdx.x >> 5); row < block_rows; row += gridDim.y * 4) {
        const int global_row = mt.block * block_rows + row;
        if (global_row >= rows) return;
        float m = -INFINITY, sum = 0.f, o[NB] = {};
        const int64_t step = (int64_t)block_rows * (D + 2);
        for (int x = blockIdx.x; x <= mt.last; ++x) {
            const float* p = a.part + ((int64_t)x * 2) * step + row * (D + 2);
            if (x == (int)blockIdx.x && mt.slot) p += step;
            const float pm = p[D], pl = p[D + 1];
            const float now = fmaxf(m, pm);
            const float use = now == -INFINITY ? 0.f : now;
            const float wo = exp2_fast(m - use), wp = exp2_fast(pm - use);
            sum = sum * wo + pl * wp;
#pragma unroll
            for (int kb = 0; kb < NB; ++kb) o[kb] = o[kb] * wo + p[kb * 32 + lane] * wp;
            m = now;
        }
        const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
        for (int kb = 0; kb < NB; ++kb) o[kb] *= inv;
        const int i = global_row / a.group;
        write_row<NB>(a, seq.q0 + i, mt.head * a.group + global_row - i * a.group, o, lane);
    }
}

}  // namespace attn
#endif  // __CUDACC__

}  // namespace qmm
