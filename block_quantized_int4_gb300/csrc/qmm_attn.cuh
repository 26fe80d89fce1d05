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
// Work.  A warp takes records of 32 keys, for all rows of the CTA (8 or 16).
// Codes are the A operand of m16n8k16 (16 keys, or 16 columns of v), rows the
// B operand, 8 a tile: so what is unpacked serves all rows, and a sum takes
// half the registers of the other order (74 us became 54 for sixteen ragged
// bf16 sequences up to 32000 tokens).  All four warps of a CTA take the same
// rows, and more rows more CTAs, for what a record costs again is small beside
// waiting for the warps of other rows (4 x 5 queries over 4001 tokens: 14.4 us
// with one row group of warps, 18 to 21 with two or four).
//
// What bounds it.  One token over 524000 tokens, 64 heads on 8 of 128: bf16 106
// us, 5.7 TB/s, 85% of a copy; fp32 146 us, 4.1 TB/s.  Memory is not waited for
// (two records a warp are enough): a 32-token tile of a record is about 520
// warp instructions in bf16 and 700 in fp32, most of them unpacking (LOP3,
// fp16 adds), 32 and 64 MMAs among them, and 12 warps an SM fill 55% of the
// issue slots between the fixed latencies of their chains.  131000 tokens take
// 34 (bf16), 40 (fp16) and 44 us (fp32): 8 us of start, look-ups, q and the second
// launch's join are not shared among more keys.
//
// Precision.  fp32 activations: q' and the weights are two fp16 parts, hi +
// lo, 22 bits, each multiplied by the codes q = u - 8.  16-bit activations: q'
// is one part (exact, but for bf16 values below 2^-24 of the row's largest),
// and for k the nibbles stay masked as they are, the fp16 subnormals u 2^-24,
// with -8 sum_e q'_e as the accumulator's start: one operation a register
// less, but the tensor core aligns its addends to the largest, and starting
// from that large a value costs 5 bits (fp32 rows: 4e-6 of the output against
// 2e-7 from q = u - 8).  A weight times d_v is two fp16 parts, as for fp32: one
// part, 2^-12, would show beside fp16 outputs, which round at 2^-12 themselves
// (2.6e-4 of the window case's output, 2.0e-4 with two and sums to nearest, which
// cost 39.6 us instead of 35.6 over 131000 tokens, 783 instead of 649 for 509
// queries over 8190).  bf16,
// whose outputs round at 2^-9, takes one, rounded twice (1.67e-3 against 1.65e-3;
// two parts: 54 us instead of 48 for the sixteen ragged sequences).
// Sums are fp32 throughout, to nearest but for what the tensor core adds up, which
// truncates: scores over the 32 values of a block, weighted v over 32 keys (fp32,
// fp16) or over all keys of a warp (bf16).  Weights times d_v are scaled by the power of two
// that brings the largest d_v so far to 2^9, so they keep their bits whatever
// the magnitude of v.
#pragma once

#include <cuda_runtime.h>

#include "qmm_heads.cuh"

namespace qmm {

// A cut launch counts an item as its units and `start` more for what starting
// and ending it costs a CTA: ATTN_START, or 0 where every unit can have a CTA.
// (Counted as 1, 2 and 4: sixteen ragged bf16 sequences up to 32000 tokens 62,
// 52 and 48 us, 128 fp32 queries over 2 sequences up to 2048 42, 32.6 and
// 33.3; as 3, 48 and 32.9.)  These
// counts come before the item's first unit: a share that ends among them
// leaves the item to the next CTA.
constexpr int ATTN_START = 3;

constexpr int ATTN_WARPS = 4;
constexpr int ATTN_THREADS = ATTN_WARPS * 32;
constexpr int ATTN_STAGES = 2;  // a warp's records: one in use, one in flight

// How the items (a row block of a sequence and key/value head) meet the CTAs:
// one CTA an item; a cluster of CTAs an item, joined through shared memory; or
// all units in equal shares, items cut where a share ends and their parts
// joined by a second kernel.
enum AttnMode { ATTN_WHOLE = QMM_ATTN_MODE_WHOLE, ATTN_CLUSTER = QMM_ATTN_MODE_CLUSTER, ATTN_CUT = QMM_ATTN_MODE_CUT };

struct AttnMeta {  // of an item: the CTAs that its units are cut over
    int first, last;  // first > last: not cut
    int slot;         // which of the first CTA's parts is the item's
    int pad;
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
    int ring_bytes, part_at;  // shared memory: the rows of q, a cluster's part
    int blocks;      // row blocks a sequence at most
    int mode;        // AttnMode
    int start;       // counts before an item's units (ATTN_CUT)
    int cluster;     // CTAs of a cluster (ATTN_CLUSTER)
    int ctas;        // CTAs of a cut launch
    float* part;     // [ctas][2][rows][attn_part_floats]
    AttnMeta* meta;  // [sequence][row block][head]
    int* err;
    unsigned long long wait_ns;  // bound of a wait
    unsigned wait_ns_tc;         // the same, as the tensor-memory kernel takes it
    int withhold;                // records whose copies a warp holds back, the last of its share (0 or 1)
};

// The kernel of head size 32 * NB for one type of activations and one or two
// tiles of 8 rows a warp.
using AttnKernel = void (*)(AttnArgs);
AttnKernel attn_kernel_f32_1(int NB);
AttnKernel attn_kernel_f32_2(int NB);
AttnKernel attn_kernel_f16_1(int NB);
AttnKernel attn_kernel_f16_2(int NB);
AttnKernel attn_kernel_bf16_1(int NB);
AttnKernel attn_kernel_bf16_2(int NB);

// Shared memory: the ring, later the joined rows, and the rows of q.
constexpr int ATTN_PAD = 4;  // floats after a joined row: rows two apart use other banks
inline int attn_ring_bytes(int D, int NT) {
    const int ring = ATTN_WARPS * ATTN_STAGES * record_bytes(D);
    const int rows = ATTN_WARPS * 8 * NT * (D + ATTN_PAD) * 4;
    return ring > rows ? ring : rows;
}
inline int attn_q_bytes(int D, int NT, int dtype) { return NT * (D / QK) * 512 * (dtype == QMM_F32 ? 2 : 1); }

// Floats of a row's part: D values, the reference and the sum; 16-byte rows.
__host__ __device__ constexpr int attn_part_floats(int D) { return D + 4; }

// CTAs an SM by registers (launch bound).  One row tile, D = 128, fp32 over
// 131000 tokens: 48.3 us with 3, 50.7 with 4, which spills.  Two row tiles, 8 x
// 8 fp16 queries over 4000 tokens, 64 heads of 128: 62.7 with 2, 68.4 with 3; 4 x 5
// fp32 of 32 heads of 64: 18.2 with 3, 21.3 with 4.
constexpr int attn_ctas(int NB, int NT) { return NT == 1 ? (NB <= 2 ? 4 : NB <= 4 ? 3 : 2) : NB <= 2 ? 3 : 2; }

#ifdef __CUDACC__
namespace attn {

// c = a b + c, and c = a b.
__device__ __forceinline__ void mma_add(float* c, const unsigned* a, unsigned b0, unsigned b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_from(float* c, const unsigned* a, unsigned b0, unsigned b1, const float* x) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%10,%11,%12,%13};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]));
}

// An 8 x 8 tile of 16-bit values (lane (g, c): row g, columns 2c, 2c + 1), transposed.
__device__ __forceinline__ unsigned transposed(unsigned x) {
    unsigned y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// Two fp32 lanes in one instruction, each rounded as its scalar form.
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 r;
    asm("{.reg .b64 x, y; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5}; add.rn.f32x2 x, x, y; mov.b64 {%0, %1}, x;}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 r;
    asm("{.reg .b64 x, y; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5}; mul.rn.f32x2 x, x, y; mov.b64 {%0, %1}, x;}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("{.reg .b64 x, y, z; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5}; mov.b64 z, {%6, %7}; fma.rn.f32x2 x, x, y, z; "
        "mov.b64 {%0, %1}, x;}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}

// Shared memory of the CTA of rank `x` in the cluster, and a barrier of all its
// threads (release and acquire).
__device__ __forceinline__ unsigned in_cluster(unsigned addr, int x) {
    unsigned r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(x));
    return r;
}
__device__ __forceinline__ float ld_cluster(unsigned addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void cluster_sync() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ __half2 as_half2(unsigned w) { return *reinterpret_cast<const __half2*>(&w); }
__device__ __forceinline__ unsigned as_bits(__half2 h) { return *reinterpret_cast<const unsigned*>(&h); }

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
// `magic` is 0x64006400 in a register: with both constants as
// immediates the compiler needs two operations where one does.
template <int HIGH>
__device__ __forceinline__ unsigned signed_codes(unsigned w, unsigned magic) {
    unsigned bits;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(bits) : "r"(w), "n"(HIGH ? 0x00F000F0u : 0x000F000Fu), "r"(magic));
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
// one record a warp); a block with rows but no keys has one unit, in
// which its zeros are written.
struct Span {
    int lo, hi, units;
};
__device__ __forceinline__ Span span_of(const AttnArgs& a, const Seq& s, int block, int block_rows, int unit_records) {
    Span r = {0, 0, 0};
    const int r0 = block * block_rows, rows = s.n * a.group;  // below 2^28 (checked on the host)
    if (r0 >= rows) return r;
    const int i0 = r0 / a.group, i1 = (min(r0 + block_rows, rows) - 1) / a.group;
    r.hi = a.causal ? max(0, min(s.L, s.L - s.n + i1 + 1)) : s.L;
    r.lo = a.window ? max(0, s.L - s.n + i0 - a.window + 1) : 0;
    if (r.lo >= r.hi) {
        r.lo = r.hi = 0;
        r.units = 1;
    } else {
        r.units = ((r.hi + GROUP - 1) / GROUP - r.lo / GROUP + unit_records - 1) / unit_records;
    }
    return r;
}

// A CTA's share [u0, u1) of all counts, ordered by (sequence, row block, head,
// unit), and where u0 lies.  entry: sequence * blocks + row block.
template <int WARPS>
struct Share {
    int warp_units[WARPS];
    int entry, start, units;  // the entry of u0, counts before it (all heads) and its own (one head)
};

// Every CTA gets `share` counts, the first `more` CTAs one more: shares rounded
// up left CTAs without any (131000 tokens, fp32: 46.2 us instead of 44.0).
struct Cut {
    int share, more;
    __device__ int cta_of(int u) const {
        const int wide = more * (share + 1);
        return u < wide ? u / (share + 1) : more + (u - wide) / share;
    }
};

__device__ __forceinline__ int entry_units(const AttnArgs& a, int e, int entries, int block_rows, int unit_records,
                                           bool report) {
    if (e >= entries) return 0;
    const int b = a.blocks == 1 ? e : e / a.blocks;
    const int units = span_of(a, sequence(a, b, report), e - b * a.blocks, block_rows, unit_records).units;
    return units ? units + a.start : 0;
}

// Inclusive sum of v over the block's threads and the block's total.
template <int WARPS>
__device__ __forceinline__ int block_scan(int v, int* warp_units, int& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(FULL, v, o);
        if (lane >= o) v += x;
    }
    if (lane == 31) warp_units[warp] = v;
    __syncthreads();
    total = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
        const int x = warp_units[w];
        if (w < warp) v += x;
        total += x;
    }
    return v;
}

// Up to THREADS entries are read once; more in two rounds (their units,
// then the place of u0).  The units of all heads fit 31 bits (checked on the
// host).
template <int THREADS>
__device__ __forceinline__ void find_share(const AttnArgs& a, int block_rows, int unit_records, Share<THREADS / 32>& sh,
                                           int& u0, int& u1, Cut& cut) {
    const int tid = threadIdx.x, entries = a.n_seqs * a.blocks;
    const bool one = entries <= THREADS;
    int units = 0, mine = 0, total;
    for (int e = tid; e < entries; e += THREADS) {
        units = entry_units(a, e, entries, block_rows, unit_records, blockIdx.x == 0);
        mine += units;
    }
    int incl = block_scan<THREADS / 32>(mine, sh.warp_units, total);
    const int all = total * a.kv_heads;
    cut.share = all / (int)gridDim.x;
    cut.more = all - cut.share * (int)gridDim.x;
    u0 = (int)blockIdx.x * cut.share + min((int)blockIdx.x, cut.more);
    u1 = u0 + cut.share + ((int)blockIdx.x < cut.more);
    if (u0 >= u1) return;
    int before = 0;
    for (int base = 0; base < entries; base += THREADS) {
        if (!one) {
            __syncthreads();
            units = entry_units(a, base + tid, entries, block_rows, unit_records, false);
            incl = block_scan<THREADS / 32>(units, sh.warp_units, total);
        }
        const int start = before + (incl - units) * a.kv_heads;
        if (units && u0 >= start && u0 - start < units * a.kv_heads)
            sh.entry = base + tid, sh.start = start, sh.units = units;
        before += total * a.kv_heads;
    }
    __syncthreads();
}

// ---------------------------------------------------------------- the kernel
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

// Exponents: 2^e <= the largest scale < 2^(e + 1); weights are at most
// 2^REF_SLACK, so 2^room times weight and scale is below 2^15 with room = 14 -
// REF_SLACK - e.  Of it the weights take 2^MIN_WEIGHT_EXP to 2^(15 - REF_SLACK):
// with less the low parts of ordinary weights would be subnormal (fp32 rows, 4096
// keys, scales of v from 0.4 to 2.2: an error of 1.4e-5 with a factor of 2^-7,
// 2.4e-7 with 2^8).  The rest goes into the scales: upwards below 2^-7, which is exact, and
// downwards from 2^5 on, which is exact for scales down to 2^-18 of the largest.
// A weight's parts end at fp16's 2^-25: at 2^-35 of the reference, 2^-30 beside
// scales of 2^5 and more.
__device__ __forceinline__ int scale_exponent(int bits) {  // exponent bits of fp16
    return (bits >> 10) - 15 + (bits == 0);                // subnormal scales count as 2^-14
}

constexpr int REF_SLACK = 5;
constexpr int MIN_WEIGHT_EXP = 5;

template <int NB, int DTYPE, int NT>
__global__ void __launch_bounds__(ATTN_THREADS, attn_ctas(NB, NT)) attn_kernel(const __grid_constant__ AttnArgs a) {
    constexpr bool SPLIT = DTYPE == QMM_F32;
    constexpr int PARTS = SPLIT ? 2 : 1;  // fp16 parts of q and of the weights
    constexpr int D = NB * 32, REC = record_bytes(D), ROWS = 8 * NT, PITCH = D + ATTN_PAD;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ Share<ATTN_WARPS> sh;
    __shared__ float s_m[ATTN_WARPS][ROWS], s_l[ATTN_WARPS][ROWS];
    __shared__ uint64_t s_full[ATTN_WARPS][ATTN_STAGES];
    __shared__ int s_gone[ATTN_WARPS][ATTN_STAGES];  // the record's page does not exist
    __shared__ int s_abort;
    __shared__ __align__(8) int s_lo[ROWS], s_hi[ROWS];  // of a row: keys it sees,
    __shared__ __align__(8) float s_f[ROWS];             // from its sums to its scores,
    __shared__ __align__(8) float s_seed[NB][ROWS];      // -8 sum q' of each block

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, c = lane & 3;
    uint8_t* ring = smem + warp * (ATTN_STAGES * REC);
    uint64_t* full = s_full[warp];
    unsigned magic;  // kept in a register (signed_codes)
    asm volatile("mov.b32 %0, 0x64006400;" : "=r"(magic));

    if (tid < ATTN_WARPS * ATTN_STAGES) mbar_init(&s_full[0][0] + tid, 1);
    if (tid == 0) s_abort = 0;
    fence_mbar_init();

    struct {
        int entry, head, unit;  // unit: in a cut launch first a count, a.start before unit 0
    } at;
    int u0, u1;
    Cut shares = {};
    const bool cut = a.mode == ATTN_CUT;
    int rank = 0;  // in the cluster
    if (cut) {
        find_share<ATTN_THREADS>(a, ROWS, ATTN_WARPS, sh, u0, u1, shares);  // synchronises the block
        // the join kernel's blocks may come in beside the last of this one's (they wait for its end)
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
        if (u0 >= u1) return;
        at.entry = sh.entry;
        at.head = (u0 - sh.start) / sh.units;
        at.unit = u0 - sh.start - at.head * sh.units;
    } else {  // later row blocks (more keys) first
        __syncthreads();
        int item = blockIdx.x;
        if (a.mode == ATTN_CLUSTER) {
            item = (int)blockIdx.x / a.cluster;
            rank = (int)blockIdx.x - item * a.cluster;
        }
        const int e = item / a.kv_heads, b = e / a.blocks;
        at.head = item - e * a.kv_heads;
        at.entry = b * a.blocks + (a.blocks - 1 - (e - b * a.blocks));
        at.unit = 0;
        u0 = 0;
        u1 = 1;
    }

    unsigned done = 0;  // records of this warp so far: stage and phase of the ring
    bool stopped = false;  // a wait of this warp ran out: it takes no more records, and the outputs are not used
    for (int u = u0; u < u1;) {
        const int b = a.blocks == 1 ? at.entry : at.entry / a.blocks, block = at.entry - b * a.blocks;
        const Seq seq = sequence(a, b, !cut && tid == 0);
        const Span sp = span_of(a, seq, block, ROWS, ATTN_WARPS);
        if (sp.units == 0) {
            if (!cut) return;  // of a cluster, all
            ++at.entry, at.head = 0, at.unit = 0;
            continue;
        }
        int counts = 0;  // of the share that this segment takes
        int unit_end = sp.units;
        if (cut) {
            counts = min(sp.units + a.start - at.unit, u1 - u);
            unit_end = at.unit + counts - a.start;
            if (unit_end <= 0) break;  // the share ends before the item's first unit
            at.unit = max(at.unit - a.start, 0);
        }
        if (a.mode == ATTN_CLUSTER) {
            at.unit = (int)((int64_t)sp.units * rank / a.cluster);
            unit_end = (int)((int64_t)sp.units * (rank + 1) / a.cluster);
        }
        const int rec0 = sp.lo / GROUP + at.unit * ATTN_WARPS + warp;
        const int rec_end = min((sp.hi + GROUP - 1) / GROUP, sp.lo / GROUP + unit_end * ATTN_WARPS);
        const int n_mine = rec_end > rec0 && !stopped ? (rec_end - rec0 + ATTN_WARPS - 1) / ATTN_WARPS : 0;

        // ---- the ring: a warp copies its records whole; its lanes look up the next
        // 32 records' places in the cache at once
        const int* table = a.pages + (int64_t)b * a.pages_stride;
        int place = -1;  // of record k = base + lane, in records; -1: its page does not exist
        const auto look_up = [&](int base) {
            const int k = base + lane;
            if (k < n_mine) {
                const int rec = rec0 + k * ATTN_WARPS, pg = rec / a.page_groups, page = table[pg];
                const bool gone = page < 0 || page >= a.n_pages;
                if (gone) atomicOr(a.err, ERR_BAD_INDEX);
                place = gone ? -1 : (page * a.kv_heads + at.head) * a.page_groups + rec - pg * a.page_groups;
            }
        };
        const int n_copy = n_mine - a.withhold;
        const auto issue = [&](int k) {
            if (k < n_copy) {
                if (k % 32 == 0) look_up(k);
                const int from = __shfl_sync(FULL, place, k % 32);
                if (lane == 0) {
                    const unsigned stage = (done + k) % ATTN_STAGES;
                    s_gone[warp][stage] = from < 0;
                    if (from < 0) {
                        mbar_arrive(&full[stage]);
                    } else {
                        mbar_arrive_expect_tx(&full[stage], REC);
                        bulk_g2s(ring + stage * REC, a.cache + (int64_t)from * REC, REC, &full[stage]);
                    }
                }
            }
        };
#pragma unroll
        for (int k = 0; k < ATTN_STAGES - 1; ++k) issue(k);

        // ---- q' as MMA operands, laid down once for the CTA: lane (g, c) takes its
        // places of rows g (+ 8), the warps take turns at the blocks
        const int rows = seq.n * a.group;
        uint4* qb = reinterpret_cast<uint4*>(smem + a.ring_bytes) + lane;
        constexpr int MINE = (NB + ATTN_WARPS - 1) / ATTN_WARPS;
        float x[NT][MINE][8];
        const auto each_block = [&](auto&& body) {
#pragma unroll
            for (int i = 0; i < MINE; ++i)
                if (ATTN_WARPS * i + warp < NB) body(i, ATTN_WARPS * i + warp);
        };
        int64_t at_q[NT];
        bool live[NT];
#pragma unroll
        for (int r = 0; r < NT; ++r) {
            const int row = block * ROWS + g + 8 * r;
            live[r] = row < rows;
            const int i = live[r] ? row / a.group : 0, h = live[r] ? row - i * a.group : 0;
            const int p = seq.L - seq.n + i;
            if (c == 0 && warp == 0) {
                s_hi[g + 8 * r] = live[r] && a.causal ? min(seq.L, p + 1) : sp.hi;
                s_lo[g + 8 * r] = live[r] && a.window ? p - a.window + 1 : sp.lo;
            }
            at_q[r] = (int64_t)(seq.q0 + i) * a.q.ts + (int64_t)(at.head * a.group + h) * a.q.hs + 4 * c;
        }
        const auto load = [&](float* y, int r, int kb) {
            if (!live[r]) {
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = 0.f;
            } else if (a.q.wide) {  // both loads on their way before either is used
                loadn<4>(a.q.data, at_q[r] + 32 * kb, DTYPE, 1, y);
                loadn<4>(a.q.data, at_q[r] + 32 * kb + 16, DTYPE, 1, y + 4);
            } else {
                loadn<4>(a.q.data, at_q[r] + 32 * kb, DTYPE, 0, y);
                loadn<4>(a.q.data, at_q[r] + 32 * kb + 16, DTYPE, 0, y + 4);
            }
        };
        float top[NT] = {};
        each_block([&](int i, int kb) {
#pragma unroll
            for (int r = 0; r < NT; ++r) {
                load(x[r][i], r, kb);
#pragma unroll
                for (int e = 0; e < 8; ++e) top[r] = fmaxf(top[r], fabsf(x[r][i][e]));
            }
        });
#pragma unroll
        for (int r = 0; r < NT; ++r) {
            top[r] = fmaxf(top[r], __shfl_xor_sync(FULL, top[r], 1));
            top[r] = fmaxf(top[r], __shfl_xor_sync(FULL, top[r], 2));
            if (c == 0) s_m[warp][g + 8 * r] = top[r];
        }
        __syncthreads();
        float mul[NT];
#pragma unroll
        for (int r = 0; r < NT; ++r) {
#pragma unroll
            for (int t = 0; t < ATTN_WARPS; ++t) top[r] = fmaxf(top[r], s_m[t][g + 8 * r]);
            // top * 2^up in [2^13, 2^14); a negative scale goes into q', a scale of 0 makes it 0
            const int up = top[r] > 0.f ? 13 - min(max(ilogbf(top[r]), -100), 100) : 0;
            mul[r] = a.scale_log2 == 0.f ? 0.f : copysignf(exp2f((float)up), a.scale_log2);
            // a masked nibble as it is (16-bit types) is the subnormal u 2^-24
            if (c == 0 && warp == 0)
                s_f[g + 8 * r] =
                    a.scale_log2 == 0.f ? 1.f : fabsf(a.scale_log2) * exp2f((float)((SPLIT ? 0 : 24) - up));
        }
        each_block([&](int i, int kb) {
#pragma unroll
            for (int r = 0; r < NT; ++r) {
                // order of the operand's k places: values 4c, 4c+2 | 4c+1, 4c+3 of each half of the block
                unsigned h[4], lo[4];
                float sum = 0.f;
#pragma unroll
                for (int st = 0; st < 2; ++st) {
                    const float by = st ? mul[r] * 0.0625f : mul[r];  // high nibbles weigh 16
                    const float* y = x[r][i] + 4 * st;
                    const float y0 = y[0] * by, y1 = y[1] * by, y2 = y[2] * by, y3 = y[3] * by;
                    h[2 * st] = pack_half(y0, y2);
                    h[2 * st + 1] = pack_half(y1, y3);
                    const float2 p0 = unpack_half(h[2 * st]), p1 = unpack_half(h[2 * st + 1]);
                    if (SPLIT) {
                        lo[2 * st] = pack_half(y0 - p0.x, y2 - p0.y);
                        lo[2 * st + 1] = pack_half(y1 - p1.x, y3 - p1.y);
                    } else {
                        const float part = p0.x + p0.y + p1.x + p1.y;
                        sum += st ? 16.f * part : part;
                    }
                }
                uint4* to = qb + (r * NB + kb) * (PARTS * 32);
                to[0] = make_uint4(h[0], h[1], h[2], h[3]);
                if (SPLIT) to[32] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                if (!SPLIT) {
                    sum += __shfl_xor_sync(FULL, sum, 1);
                    sum += __shfl_xor_sync(FULL, sum, 2);
                    if (c == 0) s_seed[kb][g + 8 * r] = sum * (-8.f * 5.9604644775390625e-8f);  // -8 2^-24
                }
            }
        });
        __syncthreads();

        // From here a lane's rows are 2c and 2c + 1 of each tile (x, y of a float2).
        float2 f[NT], ref[NT], l[NT];  // ref: reference of the weights, w = exp2(s - ref); l: their sums
        int2 lo[NT], hi[NT];
        float seed[NT][NB][4];
        int lo_all = 0, hi_all = 0x7FFFFFFF;  // keys that every row of the warp sees
#pragma unroll
        for (int r = 0; r < NT; ++r) {
            f[r] = *reinterpret_cast<const float2*>(&s_f[8 * r + 2 * c]);
            lo[r] = *reinterpret_cast<const int2*>(&s_lo[8 * r + 2 * c]);
            hi[r] = *reinterpret_cast<const int2*>(&s_hi[8 * r + 2 * c]);
            lo_all = max(lo_all, max(lo[r].x, lo[r].y));
            hi_all = min(hi_all, min(hi[r].x, hi[r].y));
            ref[r] = make_float2(-INFINITY, -INFINITY);
            l[r] = make_float2(0.f, 0.f);
#pragma unroll
            for (int kb = 0; kb < NB; ++kb) {
                float2 v = make_float2(0.f, 0.f);
                if (!SPLIT) v = *reinterpret_cast<const float2*>(&s_seed[kb][8 * r + 2 * c]);
                seed[r][kb][0] = seed[r][kb][2] = v.x, seed[r][kb][1] = seed[r][kb][3] = v.y;
            }
        }
        lo_all = __reduce_max_sync(FULL, lo_all);
        hi_all = __reduce_min_sync(FULL, hi_all);
        float acc[NT][NB][2][4] = {};  // [tile][block][16 columns of D][column g, rows 2c, 2c + 1; column g + 8]
        int top_bits = -1;             // exponent bits of the largest scale of v so far
        float vs = 1.f, ds = 1.f;      // acc holds the weighted v times vs (on the weights) * ds (on the scales)
        float unscale = 1.f;           // 1 / (vs * ds)

        for (int k = 0; k < n_mine; ++k) {
            __syncwarp();  // the record before is read
            issue(k + ATTN_STAGES - 1);
            const unsigned stage = (done + k) % ATTN_STAGES;
            // a vote: lanes that disagree about a copy that lands at the limit would part
            if (!__all_sync(FULL, mbar_wait(&full[stage], (done + k) / ATTN_STAGES & 1, &s_abort, a.wait_ns))) {
                if (lane == 0) {
                    s_abort = 1;
                    atomicOr(a.err, ERR_TIMEOUT);
                }
                // the copies on their way end before the CTA does, or their own limit passes
                int never = 0;
                for (int x = k; x < min(k + ATTN_STAGES, n_copy); ++x)
                    mbar_wait(&full[(done + x) % ATTN_STAGES], (done + x) / ATTN_STAGES & 1, &never, a.wait_ns);
                __syncwarp();
                stopped = true;
                break;
            }
            const bool gone = s_gone[warp][stage] != 0;
            const uint8_t* rec = ring + stage * REC;
            const int tok0 = (rec0 + k * ATTN_WARPS) * GROUP;

            // scores: keys 8j + g of the record
            float2 s[NT][4] = {};
#pragma unroll
            for (int kb = 0; kb < NB; ++kb) {
                const uint4 w4 = lds128(rec + kb * 512 + lane * 16);
                const uint4 d4 = lds128(rec + NB * 1024 + kb * 64 + (g >> 1) * 16);
                const unsigned w[4] = {w4.x, w4.y, w4.z, w4.w}, d[4] = {d4.x, d4.y, d4.z, d4.w};
                uint4 q[NT][PARTS];
#pragma unroll
                for (int r = 0; r < NT; ++r)
#pragma unroll
                    for (int e = 0; e < PARTS; ++e) q[r][e] = qb[((r * NB + kb) * PARTS + e) * 32];
#pragma unroll
                for (int i = 0; i < 2; ++i) {  // 16 keys: rows 16i + g and 16i + 8 + g of the operand
                    const unsigned x = w[2 * i], y = w[2 * i + 1], x8 = x >> 8, y8 = y >> 8;
                    unsigned a0[4], a1[4];
                    if (SPLIT) {
                        a0[0] = signed_codes<0>(x, magic), a0[1] = signed_codes<0>(y, magic);
                        a0[2] = signed_codes<0>(x8, magic), a0[3] = signed_codes<0>(y8, magic);
                        a1[0] = signed_codes<1>(x, magic), a1[1] = signed_codes<1>(y, magic);
                        a1[2] = signed_codes<1>(x8, magic), a1[3] = signed_codes<1>(y8, magic);
                    } else {
                        a0[0] = x & 0x000F000Fu, a0[1] = y & 0x000F000Fu, a0[2] = x8 & 0x000F000Fu;
                        a0[3] = y8 & 0x000F000Fu, a1[0] = x & 0x00F000F0u, a1[1] = y & 0x00F000F0u;
                        a1[2] = x8 & 0x00F000F0u, a1[3] = y8 & 0x00F000F0u;
                    }
                    const float dx = unpack_half(g & 1 ? d[2 * i] >> 16 : d[2 * i]).x;
                    const float dy = unpack_half(g & 1 ? d[2 * i + 1] >> 16 : d[2 * i + 1]).x;
#pragma unroll
                    for (int r = 0; r < NT; ++r) {
                        float t[4];
                        mma_from(t, a0, q[r][0].x, q[r][0].y, seed[r][kb]);
                        mma_add(t, a1, q[r][0].z, q[r][0].w);
                        if (SPLIT) {
                            mma_add(t, a0, q[r][PARTS - 1].x, q[r][PARTS - 1].y);
                            mma_add(t, a1, q[r][PARTS - 1].z, q[r][PARTS - 1].w);
                        }
                        s[r][2 * i] = fma2(make_float2(dx, dx), make_float2(t[0], t[1]), s[r][2 * i]);
                        s[r][2 * i + 1] = fma2(make_float2(dy, dy), make_float2(t[2], t[3]), s[r][2 * i + 1]);
                    }
                }
            }

            // the mask, where a row does not see all 32 keys
            const bool masked = gone || tok0 < lo_all || tok0 + GROUP > hi_all;
            if (masked) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int r = 0; r < NT; ++r) {
                        const int key = tok0 + 8 * j + g;
                        if (gone || key < lo[r].x || key >= hi[r].x) s[r][j].x = -INFINITY;
                        if (gone || key < lo[r].y || key >= hi[r].y) s[r][j].y = -INFINITY;
                    }
            }

            // Scales of v, and the power of two that they and the weights share.
            // Keys that no row of the block sees may hold anything: their
            // scales become zeros.
            uint8_t* vscale = ring + stage * REC + NB * 1088;
            if (masked) {
#pragma unroll
                for (int t = 0; t < NB; ++t) {
                    const int key = tok0 + lane;
                    if (gone || key < sp.lo || key >= sp.hi)
                        *reinterpret_cast<unsigned short*>(vscale + t * 64 + scale_at(lane)) = 0;
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // a later copy lands on them
                __syncwarp();
            }
            __half2 any = __float2half2_rn(0.f);  // the largest magnitude
#pragma unroll
            for (int kb = 0; kb < NB; ++kb) {
                const uint4 d4 = lds128(vscale + kb * 64 + c * 16);
                any = __hmax2(__hmax2(any, __habs2(as_half2(d4.x))), __habs2(as_half2(d4.y)));
                any = __hmax2(__hmax2(any, __habs2(as_half2(d4.z))), __habs2(as_half2(d4.w)));
            }
            // The reference follows the running maximum by steps of more than
            // 2^REF_SLACK, so acc is rarely rescaled; so with the scales of v.
            int exponent = max((int)(as_bits(any) & 0x7C00), (int)(as_bits(any) >> 16 & 0x7C00));
            float2 m[NT];
            bool moved = exponent > top_bits;
#pragma unroll
            for (int r = 0; r < NT; ++r) {
                m[r] = s[r][0];
#pragma unroll
                for (int j = 1; j < 4; ++j) m[r].x = fmaxf(m[r].x, s[r][j].x), m[r].y = fmaxf(m[r].y, s[r][j].y);
                m[r] = mul2(m[r], f[r]);  // f > 0
                moved |= m[r].x > ref[r].x + REF_SLACK || m[r].y > ref[r].y + REF_SLACK;
            }
            if (__any_sync(FULL, moved)) {
                exponent = __reduce_max_sync(FULL, exponent);
                float ratio = 1.f;
                if (exponent > top_bits) {
                    const int room = 14 - REF_SLACK - scale_exponent(exponent);
                    const int w = min(max(room, MIN_WEIGHT_EXP), 15 - REF_SLACK);
                    vs = exp2f((float)w);
                    ds = room > 21 - REF_SLACK || room < w ? exp2f((float)(room - w)) : 1.f;
                    ratio = top_bits < 0 ? 1.f : vs * ds * unscale;
                    unscale = 1.f / (vs * ds);
                    top_bits = exponent;
                }
#pragma unroll
                for (int r = 0; r < NT; ++r) {
#pragma unroll
                    for (int o = 4; o < 32; o *= 2) {
                        m[r].x = fmaxf(m[r].x, __shfl_xor_sync(FULL, m[r].x, o));
                        m[r].y = fmaxf(m[r].y, __shfl_xor_sync(FULL, m[r].y, o));
                    }
                    const float2 now = make_float2(fmaxf(ref[r].x, m[r].x), fmaxf(ref[r].y, m[r].y));
                    float2 by = make_float2(now.x == -INFINITY ? 0.f : exp2_fast(ref[r].x - now.x),
                                            now.y == -INFINITY ? 0.f : exp2_fast(ref[r].y - now.y));
                    ref[r] = now;
                    l[r] = mul2(l[r], by);
                    by = mul2(by, make_float2(ratio, ratio));
#pragma unroll
                    for (int kb = 0; kb < NB; ++kb)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float* v = acc[r][kb][e >> 1] + 2 * (e & 1);
                            v[0] *= by.x, v[1] *= by.y;
                        }
                }
            }
            // weights, as fp16 pairs of keys 8j + 2c, 8j + 2c + 1 of row g: the operand of v's product
            unsigned ph[NT][4], pl[NT][4];
#pragma unroll
            for (int r = 0; r < NT; ++r) {
                // nothing seen yet: every weight is exp2(-inf - 0)
                const float2 use = make_float2(ref[r].x == -INFINITY ? 0.f : -ref[r].x,
                                               ref[r].y == -INFINITY ? 0.f : -ref[r].y);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 x = fma2(s[r][j], f[r], use);
                    float2 w = make_float2(exp2_fast(x.x), exp2_fast(x.y));
                    l[r] = add2(l[r], w);
                    w = mul2(w, make_float2(vs, vs));
                    const unsigned h = pack_half(w.x, w.y);
                    ph[r][j] = transposed(h);
                    if (DTYPE != QMM_BF16) {
                        const float2 p = unpack_half(h);
                        pl[r][j] = transposed(pack_half(w.x - p.x, w.y - p.y));
                    }
                }
            }

            // weights times v: columns g + 16 e (and + 8) of the block, a row of the operand each
#pragma unroll
            for (int kb = 0; kb < NB; ++kb) {
                const uint4 w4 = lds128(rec + NB * 512 + kb * 512 + lane * 16);
                const uint4 d4 = lds128(vscale + kb * 64 + c * 16);
                const unsigned w[4] = {w4.x, w4.y, w4.z, w4.w};
                unsigned vd[4] = {d4.x, d4.y, d4.z, d4.w};
                if (ds != 1.f) {
                    const __half2 by = __float2half2_rn(ds);
#pragma unroll
                    for (int j = 0; j < 4; ++j) vd[j] = as_bits(__hmul2(as_half2(vd[j]), by));
                }
                unsigned b[NT][4], bl[NT][4];
#pragma unroll
                for (int r = 0; r < NT; ++r)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const __half2 d = as_half2(vd[j]), h = as_half2(ph[r][j]);
                        if constexpr (DTYPE != QMM_BF16) {
                            // (hi + lo) d as two parts: the product, and its exact error plus lo d
                            const __half2 pr = __hmul2(h, d);
                            b[r][j] = as_bits(pr);
                            bl[r][j] = as_bits(__hfma2(as_half2(pl[r][j]), d, __hfma2(h, d, __hneg2(pr))));
                        } else {
                            b[r][j] = as_bits(__hmul2(h, d));  // two roundings of 2^-12, next to the output's 2^-9
                        }
                    }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float t[NT][4] = {};
#pragma unroll
                    for (int st = 0; st < 2; ++st) {
                        const unsigned x = w[2 * st] >> (8 * e), y = w[2 * st + 1] >> (8 * e);
                        const unsigned v[4] = {signed_codes<0>(x, magic), signed_codes<1>(x, magic),
                                               signed_codes<0>(y, magic), signed_codes<1>(y, magic)};
#pragma unroll
                        for (int r = 0; r < NT; ++r) {
                            if constexpr (DTYPE != QMM_BF16) {
                                mma_add(t[r], v, bl[r][2 * st], bl[r][2 * st + 1]);
                                mma_add(t[r], v, b[r][2 * st], b[r][2 * st + 1]);
                            } else {
                                mma_add(acc[r][kb][e], v, b[r][2 * st], b[r][2 * st + 1]);
                            }
                        }
                    }
                    if constexpr (DTYPE != QMM_BF16) {
                        // The tensor core truncates its sums: 32 keys at a time, and
                        // the sums of those rounded to nearest.  (Over 524288 keys of
                        // a CTA fp16 outputs were 1.5e-4 low, bf16's are 7e-5.)
#pragma unroll
                        for (int r = 0; r < NT; ++r) {
                            float* o = acc[r][kb][e];
                            const float2 lo2 = add2(make_float2(o[0], o[1]), make_float2(t[r][0], t[r][1]));
                            const float2 hi2 = add2(make_float2(o[2], o[3]), make_float2(t[r][2], t[r][3]));
                            o[0] = lo2.x, o[1] = lo2.y, o[2] = hi2.x, o[3] = hi2.y;
                        }
                    }
                }
            }
        }
        done += n_mine;

        // ---- join the warps: O, reference and sum of every row
#pragma unroll
        for (int r = 0; r < NT; ++r) {
#pragma unroll
            for (int o = 4; o < 32; o *= 2) {
                l[r].x += __shfl_xor_sync(FULL, l[r].x, o);
                l[r].y += __shfl_xor_sync(FULL, l[r].y, o);
            }
            if (g == 0) {
                s_m[warp][8 * r + 2 * c] = ref[r].x, s_m[warp][8 * r + 2 * c + 1] = ref[r].y;
                s_l[warp][8 * r + 2 * c] = l[r].x, s_l[warp][8 * r + 2 * c + 1] = l[r].y;
            }
        }
        __syncthreads();  // the ring is read
        float* buf = reinterpret_cast<float*>(smem);  // [warp][ROWS][PITCH]
#pragma unroll
        for (int r = 0; r < NT; ++r)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const int row = 8 * r + 2 * c + y;
                const float mine = y ? ref[r].y : ref[r].x;
                float m = -INFINITY;
#pragma unroll
                for (int t = 0; t < ATTN_WARPS; ++t) m = fmaxf(m, s_m[t][row]);
                const float w = mine == -INFINITY ? 0.f : exp2_fast(mine - m) * unscale;
                float* o = buf + (warp * ROWS + row) * PITCH + g;
#pragma unroll
                for (int kb = 0; kb < NB; ++kb)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        o[kb * 32 + e * 16] = acc[r][kb][e][y] * w;
                        o[kb * 32 + e * 16 + 8] = acc[r][kb][e][2 + y] * (w * 0.0625f);  // high nibbles weigh 16
                    }
            }
        __syncthreads();
        const bool uncut = a.mode != ATTN_CLUSTER && at.unit == 0 && unit_end == sp.units;
        float* part = nullptr;
        if (a.mode == ATTN_CLUSTER)
            part = reinterpret_cast<float*>(smem + a.part_at);
        else if (!uncut)  // a share's first segment keeps its part in slot 0, its last in slot 1
            part = a.part + ((int64_t)blockIdx.x * 2 + (u != u0)) * ROWS * attn_part_floats(D);
        const auto write = [&](int row, const float* o) {
            const int global_row = block * ROWS + row, i = global_row / a.group;
            write_row<NB>(a, seq.q0 + i, at.head * a.group + global_row - i * a.group, o, lane);
        };
        const int live_rows = min(ROWS, rows - block * ROWS);
        for (int row = warp; row < live_rows; row += ATTN_WARPS) {
            float m = -INFINITY, sum = 0.f, o[NB] = {};
#pragma unroll
            for (int t = 0; t < ATTN_WARPS; ++t) m = fmaxf(m, s_m[t][row]);
#pragma unroll
            for (int t = 0; t < ATTN_WARPS; ++t) {
                const float mt = s_m[t][row];
                sum += mt == -INFINITY ? 0.f : s_l[t][row] * exp2_fast(mt - m);
#pragma unroll
                for (int kb = 0; kb < NB; ++kb) o[kb] += buf[(t * ROWS + row) * PITCH + kb * 32 + lane];
            }
            if (uncut) {
                const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
                for (int kb = 0; kb < NB; ++kb) o[kb] *= inv;
                write(row, o);
            } else {
#pragma unroll
                for (int kb = 0; kb < NB; ++kb) part[row * attn_part_floats(D) + kb * 32 + lane] = o[kb];
                if (lane == 0) part[row * attn_part_floats(D) + D] = m, part[row * attn_part_floats(D) + D + 1] = sum;
            }
        }
        if (a.mode == ATTN_CLUSTER) {
            // every CTA of the cluster joins some of the rows, from all parts in their order
            cluster_sync();
            for (int row = rank + warp * a.cluster; row < live_rows; row += ATTN_WARPS * a.cluster) {
                const unsigned mine = smem_u32(part + row * attn_part_floats(D));
                float m = -INFINITY, sum = 0.f, o[NB] = {};
                for (int x = 0; x < a.cluster; ++x) {
                    const unsigned p = in_cluster(mine, x);
                    const float pm = ld_cluster(p + D * 4), pl = ld_cluster(p + D * 4 + 4);
                    const float now = fmaxf(m, pm), use = now == -INFINITY ? 0.f : now;
                    const float wo = exp2_fast(m - use), wp = exp2_fast(pm - use);
                    sum = sum * wo + pl * wp;
#pragma unroll
                    for (int kb = 0; kb < NB; ++kb) o[kb] = o[kb] * wo + ld_cluster(p + (kb * 32 + lane) * 4) * wp;
                    m = now;
                }
                const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
                for (int kb = 0; kb < NB; ++kb) o[kb] *= inv;
                write(row, o);
            }
            cluster_sync();  // the others' shared memory stays until it is read
        }
        if (!cut) return;
        if (tid == 0 && at.unit == 0) {
            // the item's counts end where its last unit does
            const int first = (int)blockIdx.x, last = uncut ? first - 1 : shares.cta_of(u + counts + sp.units - unit_end - 1);
            a.meta[(int64_t)at.entry * a.kv_heads + at.head] = AttnMeta{first, last, u != u0, 0};
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // buf is used before the ring's next copies
        __syncthreads();
        u += counts;
        at.unit = 0;
        if (++at.head == a.kv_heads) at.head = 0, ++at.entry;
    }
}

// Joins the parts of an item that was cut over CTAs: with the reference m_i,
// sum l_i and weighted sum o_i of part i, out = sum_i e_i o_i / sum_i e_i l_i,
// e_i = exp2(m_i - max m).  A few kilobytes a row, so latency bounds it, 3 to 5
// us behind the first kernel; hence all loads at once, and warps side by side
// where a row has many parts (one warp adding up 57 parts in turn took 50 us).
// TEAM warps share a row:
// warp w of them takes the parts w, w + TEAM, ..., eight at a time, all of
// whose loads are on their way at once; block (item, y) takes rows from
// y * (8 / TEAM).  What each part gets depends on its place alone, so results
// do not change from call to call.
constexpr int JOIN_WARPS = 8;
constexpr int JOIN_AT_ONCE = 8;

template <int NB, int TEAM>
__global__ void __launch_bounds__(JOIN_WARPS * 32)
    attn_join_kernel(const __grid_constant__ AttnArgs a, int block_rows) {
    constexpr int D = NB * 32, ROWS = JOIN_WARPS / TEAM;  // rows a block works on at once
    __shared__ float s_o[JOIN_WARPS][TEAM > 1 ? D : 1], s_m[JOIN_WARPS], s_l[JOIN_WARPS];
    const int entry = blockIdx.x / a.kv_heads, head = blockIdx.x - entry * a.kv_heads;
    const int b = a.blocks == 1 ? entry : entry / a.blocks, block = entry - b * a.blocks;
    const Seq seq = sequence(a, b, false);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, team = warp / TEAM, member = warp - team * TEAM;
    const int rows = min(block_rows, seq.n * a.group - block * block_rows);
    if ((int)blockIdx.y * ROWS >= rows) return;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const AttnMeta mt = a.meta[blockIdx.x];
    // not cut; or never written, by a CTA of which a wait ran out, and then it may hold anything
    if (mt.first < 0 || mt.last <= mt.first || mt.last >= a.ctas) return;
    const int n = mt.last - mt.first + 1;
    const int64_t step = (int64_t)block_rows * attn_part_floats(D);
    for (int row0 = blockIdx.y * ROWS; row0 < rows; row0 += gridDim.y * ROWS) {
        const int row = row0 + team;
        const bool live = row < rows;
        const float* base = a.part + (int64_t)mt.first * 2 * step + (live ? row : row0) * attn_part_floats(D);
        float m = -INFINITY, sum = 0.f, o[NB] = {};
        for (int x0 = member; x0 < n; x0 += TEAM * JOIN_AT_ONCE) {
            float pm[JOIN_AT_ONCE], pl[JOIN_AT_ONCE], po[JOIN_AT_ONCE][NB];
#pragma unroll
            for (int i = 0; i < JOIN_AT_ONCE; ++i) {
                const int x = x0 + i * TEAM;
                const float* p = base + 2 * step * x + (x == 0 && mt.slot ? step : 0);
                const bool there = x < n;
                pm[i] = there ? p[D] : -INFINITY;
                pl[i] = there ? p[D + 1] : 0.f;
#pragma unroll
                for (int kb = 0; kb < NB; ++kb) po[i][kb] = there ? p[kb * 32 + lane] : 0.f;
            }
            float now = m;
#pragma unroll
            for (int i = 0; i < JOIN_AT_ONCE; ++i) now = fmaxf(now, pm[i]);
            const float use = now == -INFINITY ? 0.f : now, w = exp2_fast(m - use);
            sum *= w;
#pragma unroll
            for (int kb = 0; kb < NB; ++kb) o[kb] *= w;
#pragma unroll
            for (int i = 0; i < JOIN_AT_ONCE; ++i) {
                const float wi = exp2_fast(pm[i] - use);
                sum = fmaf(wi, pl[i], sum);
#pragma unroll
                for (int kb = 0; kb < NB; ++kb) o[kb] = fmaf(wi, po[i][kb], o[kb]);
            }
            m = now;
        }
        if constexpr (TEAM > 1) {
            if (lane == 0) s_m[warp] = m, s_l[warp] = sum;
#pragma unroll
            for (int kb = 0; kb < NB; ++kb) s_o[warp][kb * 32 + lane] = o[kb];
            __syncthreads();
            if (member == 0) {
                m = -INFINITY, sum = 0.f;
#pragma unroll
                for (int w = 0; w < TEAM; ++w) m = fmaxf(m, s_m[warp + w]);
                const float use = m == -INFINITY ? 0.f : m;
#pragma unroll
                for (int kb = 0; kb < NB; ++kb) o[kb] = 0.f;
#pragma unroll
                for (int w = 0; w < TEAM; ++w) {
                    const float by = exp2_fast(s_m[warp + w] - use);
                    sum = fmaf(by, s_l[warp + w], sum);
#pragma unroll
                    for (int kb = 0; kb < NB; ++kb) o[kb] = fmaf(by, s_o[warp + w][kb * 32 + lane], o[kb]);
                }
            }
            __syncthreads();
        }
        if (member == 0 && live) {
            const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
            for (int kb = 0; kb < NB; ++kb) o[kb] *= inv;
            const int global_row = block * block_rows + row, i = global_row / a.group;
            write_row<NB>(a, seq.q0 + i, head * a.group + global_row - i * a.group, o, lane);
        }
    }
}

}  // namespace attn
#endif  // __CUDACC__

}  // namespace qmm
