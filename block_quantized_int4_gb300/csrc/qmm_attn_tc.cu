// qmm_attn_tc.cu -- attention over the paged Q4_0 cache for many rows (a
// prompt's chunk) of bf16 activations, on the 5th-generation tensor cores.
//
// Why another form.  The warp-MMA kernel (qmm_attn.cuh) unpacks a record once
// for 16 rows and multiplies at the legacy rate; with hundreds of rows a
// key/value head that is compute bound.  Here a record is unpacked once for
// 256 rows, into fp16 operands in shared memory, and both products are
// tcgen05.mma with accumulators in tensor memory:
//   S = Q K^T   M = 128 rows, N = 128 keys, both operands in shared memory
//   O += P V    M = 128 rows, N = D, P from tensor memory, V^T from shared
// Scales meet the codes here (d * (u - 8) rounded to fp16, 2^-12), and weights are
// fp16, so this form serves bf16 alone, whose output rounds at 2^-9 (error 1.69e-3,
// of which the output's rounding alone is 1.66e-3).  O is added up by the tensor
// core, which truncates: outputs over 131072 keys of a CTA are 1.7e-4 low, over
// 524288 7e-4.
//
// A CTA (one an SM, 24 warps) holds two row tiles of 128 rows and walks the
// keys in steps of 128 (4 records):
//  - warps 0..3 and 4..7: the softmax of tile 0 and 1, a thread a row: S from
//    tensor memory, weights back into its place as fp16 (P), the row's sum.
//    One pass: the reference of the weights is what it was, unless a score is
//    above it by more than SLACK; then O, the sum and what is written of P are
//    rescaled first, which is rare.
//  - warps 8..15: V of a step as fp16 operand, half a record a warp, warps
//    16..19: K, a record a warp.  The cache's word order makes them as it makes
//    the warp MMA's: a word of K is eight values of one key (Q is laid down in
//    the same order of its values), a word of V two keys of four values, so
//    every store of a warp is one run of shared memory.
//  - warps 20, 21: page look-ups and bulk copies of the records' K and V parts
//    (rings of records); warp 22: issues the MMAs.
// The two tiles take turns: while one is in its softmax, the other's products
// run.  The operands of K and V are double buffered.
//
// What bounds it.  509 queries over 8190 tokens, 64 heads on 8 of 128: 161 us,
// 824 TFLOP/s, 44% of the library's best large product (the warp-MMA kernel:
// 630 us).  128 items on 128 of the 152 SMs; the longest CTA takes 318,000 cycles
// for its 64 steps of 128 keys, 4970 a step with start and end counted in, and a
// step is 11,500 warp instructions (softmax, unpacking, polling), 61% of the issue
// slots of the SMs in use.  A row's 128 scores pass one thread (read, exponential,
// packed, written back); MMAs fill 42%, of which S reads both operands from shared
// memory.
// Steps of 64 keys with S double buffered: 198 to 240 us against 172 then,
// twice the waits and commits.
//
// Keys and values are fp16 here.  Where a scale that some row sees is so large
// that d (u - 8) might not fit, the segment is done again with keys and values in
// sixteenths (exact but for scales below 2^-10): its products and sums so far are
// not used, and no output has been written.
//
// Operands lie as K-major core matrices of 8 rows x 16 bytes without swizzle.
// Every wait is bounded in time; on expiry the error word is set, copies and
// products on their way are waited for, and the CTA ends.
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "qmm_attn.cuh"
#include "qmm_attn_tc.h"

namespace qmm {
namespace attn_tc {

using attn::Seq;
using attn::Span;

constexpr int SOFTMAX_WARPS = 8, WARP_V = 8, WARP_K = 16;
constexpr int V_WARPS = 8, K_WARPS = 4;   // two warps a record of V, one a record of K
constexpr int K_SLOTS = 8, V_SLOTS = 6;   // records of the rings (what shared memory has left at D = 128)
constexpr int WARP_LOAD_K = 20, WARP_LOAD_V = 21, WARP_MMA = 22;
constexpr int THREADS = 24 * 32;  // six warpgroups; the last warp only keeps its warpgroup whole
// Registers a thread: 80 at launch (61,440 of the SM), then 144 for the two
// softmax warpgroups and 48 for the four others (61,440).
constexpr int SOFTMAX_REGS = 144, OTHER_REGS = 48;
constexpr int STEP = 128;              // keys of a step
constexpr int STEP_RECORDS = STEP / GROUP;
constexpr float SLACK = 5.f;           // weights reach 2^(SLACK + LIFT)
constexpr float LIFT = 10.f;           // weights are 2^LIFT times exp2(s - reference): fp16 keeps small ones
constexpr uint32_t TMEM_COLS = 512, S_COL = 0, O_COL = 256;  // S of tile x at 128 x, O at 256 + 128 x

template <int NB>
struct Smem {
    static constexpr int D = NB * 32;
    static constexpr int REC = record_bytes(D);
    static constexpr int Q = 0;                          // [2][128][D] fp16
    static constexpr int K = Q + 2 * 128 * D * 2;        // [2][128][D]
    static constexpr int V = K + 2 * STEP * D * 2;       // [2][D][128]
    static constexpr int PART = REC / 2;                 // a record's codes and scales of K, or of V
    static constexpr int RAW = V + 2 * STEP * D * 2;     // rings of [K_SLOTS] and [V_SLOTS] parts
    static constexpr int BYTES = RAW + (K_SLOTS + V_SLOTS) * PART;
    static_assert(SOFTMAX_WARPS * 32 * (D + 4) * 4 <= RAW, "output rows in the operands' place");
};

// Shared-memory operand: the low word of its descriptor holds the address and
// the byte distance of core matrices adjacent along K (128), the high word
// that along the rows and the version.
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr) { return ((addr >> 4) & 0x3FFFu) | ((128u >> 4) << 16); }
__host__ __device__ constexpr uint32_t desc_hi(uint32_t row_stride) { return ((row_stride >> 4) & 0x3FFFu) | (1u << 14); }

// D (+)= A B.  The operands are values that the whole warp agrees on, so that
// they live in uniform registers; with per-thread ones each instruction waits
// for several transfers (85 to 100 cycles an MMA instead of the tensor core's
// 45 to 64).
template <bool ADD>
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t a_hi, uint32_t b, uint32_t b_hi, uint32_t idesc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tmov.b64 x, {%1, %2};\n\tmov.b64 y, {%3, %4};\n\t"
        "setp.ne.b32 p, %6, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %5, p;\n\t}" ::"r"(d),
        "r"(a), "r"(a_hi), "r"(b), "r"(b_hi), "r"(idesc), "n"(ADD)
        : "memory");
}
template <bool ADD>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t b_hi, uint32_t idesc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\tmov.b64 y, {%2, %3};\n\t"
        "setp.ne.b32 p, %5, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(b_hi), "r"(idesc), "n"(ADD)
        : "memory");
}
__device__ __forceinline__ bool elected() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e != 0;
}
__device__ __forceinline__ void commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

#define QMM_R8(r, i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), "=r"(r[i + 4]), "=r"(r[i + 5]), \
                     "=r"(r[i + 6]), "=r"(r[i + 7])
#define QMM_U8(r, i) "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]), \
                     "+r"(r[i + 6]), "+r"(r[i + 7])
#define QMM_I8(r, i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3]), "r"(r[i + 4]), "r"(r[i + 5]), \
                     "r"(r[i + 6]), "r"(r[i + 7])

// 32 columns of this thread's lane; the registers are named again at the
// wait, so that no use of them moves before it.
__device__ __forceinline__ void ld32(uint32_t at, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
        "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : QMM_R8(r, 0), QMM_R8(r, 8), QMM_R8(r, 16), QMM_R8(r, 24)
        : "r"(at));
}
__device__ __forceinline__ void wait_ld(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : QMM_U8(r, 0), QMM_U8(r, 8), QMM_U8(r, 16), QMM_U8(r, 24)
                 :
                 : "memory");
}
__device__ __forceinline__ void st16(uint32_t at, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
            at),
        QMM_I8(r, 0), QMM_I8(r, 8)
        : "memory");
}
__device__ __forceinline__ void ld16(uint32_t at, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : QMM_R8(r, 0), QMM_R8(r, 8)
        : "r"(at));
}
__device__ __forceinline__ void wait_ld(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" : QMM_U8(r, 0), QMM_U8(r, 8) : : "memory");
}

// A bounded wait.  The hardware holds a try back for 1 to 2 us (whatever time it is
// asked for), so counting tries bounds no time: the clock does, by its low 32 bits.
// The loop is short because its copies crowd the instruction cache: with the
// 64-bit clock and an abort flag of the CTA in it, 509 queries over 8190 tokens
// took 172 us instead of 162.  Lanes may disagree where a phase ends at the limit:
// callers vote.
constexpr unsigned MAX_WAIT_NS = 4000000000u;
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, unsigned limit_ns) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .u32 t, t0;\n\tmov.u32 t0, 0;\n"
        "AGAIN:\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "@p bra DONE;\n\t"
        "mov.u32 t, %globaltimer_lo;\n\t"
        "setp.eq.u32 q, t0, 0;\n\t"
        "@q mov.u32 t0, t;\n\t"
        "sub.u32 t, t, t0;\n\t"
        "setp.lt.u32 q, t, %3;\n\t"
        "@q bra AGAIN;\n"
        "DONE:\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(limit_ns)
        : "memory");
    return ok != 0;
}

constexpr float MAX_SCALE = 8188.f;  // 8 MAX_SCALE is the largest fp16
constexpr float WIDE = 16.f;         // what codes are divided by beyond it

// Two codes times a pair of scales: nibbles 0 and 4 of w.  `magic` is the fp16
// pair that the nibbles are OR-ed into, 1024 or (sixteenths) 64, and eight units of
// its last place are u = 8.
__device__ __forceinline__ unsigned magic_codes(bool sixteenths) { return sixteenths ? 0x54005400u : 0x64006400u; }
__device__ __forceinline__ unsigned scaled_codes(unsigned w, __half2 d, unsigned magic, __half2 eight) {
    unsigned bits;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(bits) : "r"(w), "n"(0x000F000Fu), "r"(magic));
    return attn::as_bits(__hmul2(__hsub2(attn::as_half2(bits), eight), d));
}

struct Place {  // where a walk stands
    int entry, head, unit, u;
    unsigned steps, segments, tile1_steps, walked;
};

template <int NB>
__global__ void __launch_bounds__(THREADS, 1) attn_tc_kernel(const __grid_constant__ AttnArgs a) {
    using SM = Smem<NB>;
    constexpr int D = SM::D, REC = SM::REC;
    constexpr int BLOCK_ROWS = ATTN_TC_ROWS;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ attn::Share<THREADS / 32> sh;
    __shared__ uint64_t raw_full[2][8], raw_empty[2][8];  // [K, V][slot]
    __shared__ uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_full[2], o_full, drain;
    // records that are not there; of eight steps: a softmax reads the flags of a step while later ones are copied
    // (a copy is at most four steps ahead of the products of a step, which follow its softmax)
    __shared__ int s_gone[2][8][STEP_RECORDS];
    __shared__ uint64_t q_full;
    __shared__ uint32_t s_tmem;
    // of a segment and the next: a warp may still read one when another sets the other
    __shared__ int s_abort[2];
    __shared__ unsigned s_large[2];  // the segment (walked + 1) that has scales above MAX_SCALE
    __shared__ Place s_place;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        for (int i = 0; i < 8; ++i) {
            mbar_init(&raw_full[0][i], 1);
            mbar_init(&raw_full[1][i], 1);
            mbar_init(&raw_empty[0][i], 1);
            mbar_init(&raw_empty[1][i], V_WARPS / STEP_RECORDS);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&k_full[i], K_WARPS);
            mbar_init(&k_empty[i], 1);
            mbar_init(&v_full[i], V_WARPS);
            mbar_init(&v_empty[i], 1);
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 4);
        }
        mbar_init(&o_full, 1);
        mbar_init(&q_full, SOFTMAX_WARPS);
        mbar_init(&drain, 1);
        s_abort[0] = s_abort[1] = 0;
        s_large[0] = s_large[1] = 0;
        fence_mbar_init();
    }
    if (warp == WARP_MMA) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)),
                     "r"(TMEM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = s_tmem;

    const bool cut = a.mode == ATTN_CUT;
    int entry0 = 0, head0 = 0, unit0 = 0, u0 = 0, u1 = 1;
    attn::Cut shares = {};
    if (cut) {
        attn::find_share<THREADS>(a, BLOCK_ROWS, STEP_RECORDS, sh, u0, u1, shares);
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
        if (u0 < u1) {
            entry0 = sh.entry;
            head0 = (u0 - sh.start) / sh.units;
            unit0 = u0 - sh.start - head0 * sh.units;
        }
    } else {  // later row blocks (more keys) first
        const int e = blockIdx.x / a.kv_heads, b = e / a.blocks;
        head0 = blockIdx.x - e * a.kv_heads;
        entry0 = b * a.blocks + (a.blocks - 1 - (e - b * a.blocks));
    }

    // The walk over the CTA's segments, once for each kind of warp (their register budgets differ), and
    // once more from a segment with large scales on, which is then done in sixteenths: true where the first
    // walk met one, and where it stood is in shared memory.  (One walk that can turn back: 4 x 512 queries
    // 81.2 us instead of 78.8, by registers that were spilled.)
    const auto walk = [&](auto softmax_role, auto turns_back) {
    constexpr bool SOFTMAX = decltype(softmax_role)::value, TURNS_BACK = decltype(turns_back)::value;
    Place at = {entry0, head0, unit0, u0, 0, 0, 0, 0};
    if constexpr (TURNS_BACK) at = s_place;
    int entry = at.entry, head = at.head, unit = at.unit;
    unsigned steps = at.steps, segments = at.segments;  // before this segment: phases of the barriers
    unsigned tile1_steps = at.tile1_steps;              // of them, those of tile 1
    unsigned walked = at.walked;                        // segments, those without keys among them
    bool wide = TURNS_BACK;                             // this segment is done in sixteenths
    for (int u = at.u; u < u1;) {
        const int b = a.blocks == 1 ? entry : entry / a.blocks, block = entry - b * a.blocks;
        const Seq seq = attn::sequence(a, b, !cut && tid == 0);
        const Span sp = attn::span_of(a, seq, block, BLOCK_ROWS, STEP_RECORDS);
        if (sp.units == 0) {
            if (!cut) break;
            ++entry, head = 0, unit = 0;
            continue;
        }
        int counts = 0, unit_end = sp.units;
        if (cut) {  // `unit` is a count: a.start before unit 0
            counts = min(sp.units + a.start - unit, u1 - u);
            unit_end = unit + counts - a.start;
            if (unit_end <= 0) break;  // the share ends before the item's first unit
            unit = max(unit - a.start, 0);
        }
        const int rec0 = sp.lo / GROUP + unit * STEP_RECORDS;
        const int rec_end = min((sp.hi + GROUP - 1) / GROUP, sp.lo / GROUP + unit_end * STEP_RECORDS);
        const int n = rec_end > rec0 ? (rec_end - rec0 + STEP_RECORDS - 1) / STEP_RECORDS : 0;
        const int rows = seq.n * a.group, first_row = block * BLOCK_ROWS;
        const int tiles = rows - first_row > 128 ? 2 : 1;

        // ---- the softmax warps lay down their rows of Q, whole rows a load; the others start at once
        const int tile = warp >> 2;  // of a softmax warp
        const int row = first_row + (tile << 7) + (tid & 127);
        const bool live = SOFTMAX && row < rows;
        const int qi = live ? row / a.group : 0, qh = head * a.group + (live ? row - qi * a.group : 0);
        float f = 1.f;  // from the row's S to its scores
        if (SOFTMAX && tile < tiles && n) {  // without keys the rows' zeros are written in this place at once
            // The warp's rows as they are, in the operand's order of values: a load takes 32 bytes of
            // each of 8 rows, which its store spreads over all banks.
            const int sub = lane >> 2, quarter = lane & 3;
            const int64_t my_row = live ? (int64_t)(seq.q0 + qi) * a.q.ts + (int64_t)qh * a.q.hs : -1;
            uint8_t* q_tile = smem + SM::Q + tile * (128 * D * 2) + (warp & 3) * (4 * D * 16);
            const unsigned short* q = reinterpret_cast<const unsigned short*>(a.q.data) + 4 * quarter;
#pragma unroll 2
            for (int r8 = 0; r8 < 4; ++r8) {
                const int64_t at = __shfl_sync(FULL, my_row, r8 * 8 + sub);
                const unsigned short* p = q + max(at, (int64_t)0);  // without a row, the first one's
                uint2 bits[2 * NB];
                if (a.q.wide) {  // no branch between the loads: each would wait for the one before
#pragma unroll
                    for (int i = 0; i < 2 * NB; ++i) bits[i] = __ldg(reinterpret_cast<const uint2*>(p + 16 * i));
                } else {
#pragma unroll
                    for (int i = 0; i < 2 * NB; ++i)
                        bits[i] = make_uint2(p[16 * i] | (unsigned)p[16 * i + 1] << 16,
                                             p[16 * i + 2] | (unsigned)p[16 * i + 3] << 16);
                }
                uint8_t* to = q_tile + r8 * (D * 16) + quarter * 128 + sub * 16;
#pragma unroll
                for (int i = 0; i < 2 * NB; ++i) {
                    if (at < 0) bits[i] = make_uint2(0, 0);
                    *reinterpret_cast<uint2*>(to + (i >> 1) * 512 + (i & 1) * 8) =
                        make_uint2(__byte_perm(bits[i].x, bits[i].y, 0x5410), __byte_perm(bits[i].x, bits[i].y, 0x7632));
                }
            }
            __syncwarp();
            // this thread's row, times a power of two, as fp16 in its place
            uint8_t* mine = q_tile + (lane >> 3) * (D * 16) + (lane & 7) * 16;
            uint4 raw[NB * 4];
            float top = 0.f;
#pragma unroll
            for (int k = 0; k < NB * 4; ++k) {
                raw[k] = lds128(mine + k * 128);
                const unsigned w[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float x[2];
                    unpack2(w[i], QMM_BF16, x);
                    top = fmaxf(top, fmaxf(fabsf(x[0]), fabsf(x[1])));
                }
            }
            // top * 2^up in [2^13, 2^14); a negative scale goes into q', a scale of 0 makes it 0
            const int up = top > 0.f ? 13 - min(max(ilogbf(top), -100), 100) : 0;
            const float mul = a.scale_log2 == 0.f ? 0.f : copysignf(exp2f((float)up), a.scale_log2);
            f = a.scale_log2 == 0.f ? 1.f : fabsf(a.scale_log2) * exp2f((float)-up);
            if (wide) f *= WIDE;
#pragma unroll
            for (int k = 0; k < NB * 4; ++k) {
                unsigned w[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float x[2];
                    unpack2(w[i], QMM_BF16, x);
                    w[i] = attn::pack_half(x[0] * mul, x[1] * mul);
                }
                *reinterpret_cast<uint4*>(mine + k * 128) = make_uint4(w[0], w[1], w[2], w[3]);
            }
            fence_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(&q_full);
        } else if (SOFTMAX) {
            if (lane == 0) mbar_arrive(&q_full);
        }

        bool ok = true;
        unsigned issued = 0;  // of a loading warp: records whose copies are under way or done
        const auto voted = [&](uint64_t* bar, uint32_t parity) {
            return __all_sync(FULL, wait(bar, parity, a.wait_ns_tc)) != 0;
        };
        if constexpr (!SOFTMAX) {
        if (warp == WARP_LOAD_K || warp == WARP_LOAD_V) {
            // ---------------- records: four a step, two steps in flight; codes and scales of K or of V
            const int kv = warp - WARP_LOAD_K;
            const int* table = a.pages + (int64_t)b * a.pages_stride;
            const unsigned slots = kv ? V_SLOTS : K_SLOTS;
            uint8_t* ring = smem + SM::RAW + kv * (K_SLOTS * SM::PART);
            issued = steps * STEP_RECORDS;  // one after the other over all segments
            for (int t = 0; t < n && ok; ++t) {
                const unsigned it = steps + t;
                const int rec = rec0 + t * STEP_RECORDS + lane;
                int place = -2;  // no record here
                if (lane < STEP_RECORDS && rec < rec_end) {
                    const int pg = rec / a.page_groups, page = table[pg];
                    const bool gone = page < 0 || page >= a.n_pages;
                    if (gone) atomicOr(a.err, ERR_BAD_INDEX);
                    place = gone ? -1 : (page * a.kv_heads + head) * a.page_groups + rec - pg * a.page_groups;
                }
                if (lane < STEP_RECORDS) s_gone[kv][it & 7][lane] = place < 0;
                __syncwarp();
                for (int r = 0; r < STEP_RECORDS; ++r) {
                    const unsigned i = it * STEP_RECORDS + r, slot = i % slots;
                    if (i >= slots) ok = voted(&raw_empty[kv][slot], (i / slots - 1) & 1);
                    if (!ok || (a.withhold && t == n - 1 && r == STEP_RECORDS - 1)) break;
                    if (lane == r) {
                        uint64_t* full = &raw_full[kv][slot];
                        if (place < 0) {
                            mbar_arrive(full);
                        } else {
                            uint8_t* to = ring + slot * SM::PART;
                            const uint8_t* from = a.cache + (int64_t)place * REC;
                            mbar_arrive_expect_tx(full, SM::PART);
                            bulk_g2s(to, from + kv * (NB * 512), NB * 512, full);
                            bulk_g2s(to + NB * 512, from + NB * 1024 + kv * (NB * 64), NB * 64, full);
                        }
                    }
                    __syncwarp();
                    issued = i + 1;
                }
            }
        } else if (warp == WARP_MMA) {
            // ---------------- products
            const int un = __shfl_sync(FULL, n, 0), ut = __shfl_sync(FULL, tiles, 0);  // uniform
            const unsigned us = __shfl_sync(FULL, steps, 0), us1 = __shfl_sync(FULL, tile1_steps, 0);
            const bool one = elected();
            constexpr uint32_t IDESC_S = (1u << 4) | ((STEP >> 3) << 17) | ((128 >> 4) << 24);
            constexpr uint32_t IDESC_O = (1u << 4) | ((uint32_t)(D >> 3) << 17) | ((128 >> 4) << 24);
            constexpr uint32_t QK_HI = desc_hi(D * 16), V_HI = desc_hi(STEP * 16), BUFFER = (STEP * D * 2) >> 4;
            const uint32_t ud = __shfl_sync(FULL, tmem, 0);
            const uint32_t q_lo = desc_lo(smem_u32(smem + SM::Q)), k_lo = desc_lo(smem_u32(smem + SM::K));
            const uint32_t v_lo = desc_lo(smem_u32(smem + SM::V));
            const auto scores = [&](int x, unsigned it) {
                const uint32_t to = ud + S_COL + x * 128, q = q_lo + x * ((128 * D * 2) >> 4);
                const uint32_t k0 = k_lo + (it & 1) * BUFFER;
                if (one) {
                    mma_ss<false>(to, q, QK_HI, k0, QK_HI, IDESC_S);
#pragma unroll
                    for (int k = 1; k < D / 16; ++k) mma_ss<true>(to, q + k * 16, QK_HI, k0 + k * 16, QK_HI, IDESC_S);
                    commit(&s_full[x]);
                    if (x == ut - 1) commit(&k_empty[it & 1]);
                }
                __syncwarp();
            };
            if (un) {
                ok = __all_sync(FULL, wait(&q_full, walked & 1, a.wait_ns_tc) && wait(&k_full[us & 1], (us / 2) & 1, a.wait_ns_tc));
                fence_after();
                for (int x = 0; x < ut && ok; ++x) scores(x, us);
            }
            for (int t = 0; t < un && ok; ++t) {
                const unsigned it = us + t;
                const uint32_t v0 = v_lo + (it & 1) * BUFFER;
                for (int x = 0; x < ut && ok; ++x) {
                    bool there = x != 0 || wait(&v_full[it & 1], (it / 2) & 1, a.wait_ns_tc);
                    there = there && wait(&p_full[x], (x ? us1 + t : it) & 1, a.wait_ns_tc);
                    ok = __all_sync(FULL, there);
                    if (!ok) break;
                    fence_after();
                    const uint32_t to = ud + O_COL + x * 128, w = ud + S_COL + x * 128;
                    if (one) {
                        if (t > 0)
                            mma_ts<true>(to, w, v0, V_HI, IDESC_O);
                        else
                            mma_ts<false>(to, w, v0, V_HI, IDESC_O);
#pragma unroll
                        for (int k = 1; k < STEP / 16; ++k) mma_ts<true>(to, w + k * 8, v0 + k * 16, V_HI, IDESC_O);
                        if (x == ut - 1) commit(&v_empty[it & 1]);
                    }
                    __syncwarp();
                    if (t + 1 < un) {
                        if (x == 0) ok = voted(&k_full[(it + 1) & 1], ((it + 1) / 2) & 1);
                        if (!ok) break;
                        fence_after();
                        scores(x, it + 1);
                    }
                }
            }
            if (un && one) {
                if (ok) {
                    commit(&o_full);
                } else {  // products on their way end before tensor memory is freed
                    commit(&drain);
                    wait(&drain, 0, a.wait_ns_tc);
                }
            }
            __syncwarp();
        } else if (warp < WARP_LOAD_K) {
            // ---------------- K or V of a step as operands, a record a warp
            const int kv = warp < WARP_K, rr = kv ? (warp - WARP_V) & 3 : warp - WARP_K, g = lane >> 2, c = lane & 3;
            const int half = (warp - WARP_V) >> 2;  // of the blocks of V
            const unsigned magic = magic_codes(wide);
            const __half2 eight = attn::as_half2(magic + 0x00080008u);
            __half2 top = __float2half2_rn(0.f);  // of the scales that a row may see
            for (int t = 0; t < n; ++t) {
                const unsigned it = steps + t, st = it & 1;
                const unsigned i = it * STEP_RECORDS + rr, slots = kv ? V_SLOTS : K_SLOTS, slot = i % slots;
                bool there = wait(&raw_full[kv][slot], (i / slots) & 1, a.wait_ns_tc);
                if (it >= 2) there = there && wait(kv ? &v_empty[st] : &k_empty[st], (it / 2 - 1) & 1, a.wait_ns_tc);
                ok = __all_sync(FULL, there);
                if (!ok) break;
                const uint8_t* rec = smem + SM::RAW + (kv * K_SLOTS + slot) * SM::PART;
                // which of the record's keys any row may see
                const int key0 = (rec0 + t * STEP_RECORDS + rr) * GROUP;
                const bool gone = s_gone[kv][it & 7][rr] != 0;
                const bool all = !gone && key0 >= sp.lo && key0 + GROUP <= sp.hi;
                const auto seen = [&](int key) { return !gone && key0 + key >= sp.lo && key0 + key < sp.hi; };
                if (kv == 0) {
                    uint8_t* to = smem + SM::K + st * (STEP * D * 2) + rr * (4 * D * 16) + c * 128 + g * 16;
#pragma unroll 1
                    for (int kb = 0; kb < NB; ++kb) {
                        const uint4 w4 = lds128(rec + kb * 512 + lane * 16);
                        const uint4 d4 = lds128(rec + NB * 512 + kb * 64 + (g >> 1) * 16);
                        const unsigned ws[4] = {w4.x, w4.y, w4.z, w4.w}, ds[4] = {d4.x, d4.y, d4.z, d4.w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            unsigned one = __byte_perm(ds[j], 0, g & 1 ? 0x3232 : 0x1010);
                            if (!all && !seen(8 * j + g)) one = 0;
                            const __half2 d = attn::as_half2(one);
                            top = __hmax2(top, __habs2(d));
                            *reinterpret_cast<uint4*>(to + kb * 512 + j * (D * 16)) =
                                make_uint4(scaled_codes(ws[j], d, magic, eight), scaled_codes(ws[j] >> 8, d, magic, eight),
                                           scaled_codes(ws[j] >> 4, d, magic, eight), scaled_codes(ws[j] >> 12, d, magic, eight));
                        }
                    }
                } else {
                    uint8_t* to = smem + SM::V + st * (STEP * D * 2) + rr * (4 * 128) + g * 16 + c * 4;
#pragma unroll 1
                    for (int kb = half; kb < NB; kb += 2) {
                        const uint4 w4 = lds128(rec + kb * 512 + lane * 16);
                        const uint4 d4 = lds128(rec + NB * 512 + kb * 64 + c * 16);
                        const unsigned ws[4] = {w4.x, w4.y, w4.z, w4.w}, ds[4] = {d4.x, d4.y, d4.z, d4.w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            unsigned two = ds[j];
                            if (!all) {
                                if (!seen(8 * j + 2 * c)) two &= 0xFFFF0000u;
                                if (!seen(8 * j + 2 * c + 1)) two &= 0x0000FFFFu;
                            }
                            const __half2 d = attn::as_half2(two);
                            top = __hmax2(top, __habs2(d));
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                *reinterpret_cast<unsigned*>(to + (kb * 4 + e) * (STEP * 16) + j * 128) =
                                    scaled_codes(ws[j] >> (4 * e), d, magic, eight);
                        }
                    }
                }
                if (__hgt2_mask(top, __float2half2_rn(MAX_SCALE))) s_large[walked & 1] = walked + 1;
                fence_async();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(kv ? &v_full[st] : &k_full[st]);
                    mbar_arrive(&raw_empty[kv][slot]);
                }
            }
        }
        } else if (tile < tiles) {
            // ---------------- softmax: this thread's row
            const uint32_t s_at = tmem + ((uint32_t)((warp & 3) * 32) << 16) + S_COL + tile * 128;
            const uint32_t o_at = tmem + ((uint32_t)((warp & 3) * 32) << 16) + O_COL + tile * 128;
            const int p = seq.L - seq.n + qi;
            const int hi = live && a.causal ? min(seq.L, p + 1) : sp.hi;
            const int lo = live && a.window ? p - a.window + 1 : sp.lo;
            float ref = -INFINITY, l = 0.f;
            uint32_t r[2][32];
            for (int t = 0; t < n; ++t) {
                __syncwarp();
                ok = voted(&s_full[tile], (tile ? tile1_steps + t : steps + t) & 1);
                if (!ok) break;
                fence_after();
                const int key0 = (rec0 + t * STEP_RECORDS) * GROUP;
                bool whole = key0 >= lo && key0 + STEP <= hi;
                const int* gone = s_gone[0][(steps + t) & 7];
#pragma unroll
                for (int q = 0; q < STEP_RECORDS; ++q) whole &= !gone[q];
                const bool masked = __any_sync(FULL, !whole);
                const auto chunk = [&](int q, uint32_t(&s)[32], uint32_t(&next)[32]) {
                    wait_ld(s);
                    if (q < 3) ld32(s_at + 32 * (q + 1), next);
                    if (masked) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            const int key = key0 + 32 * q + e;
                            if (key < lo || key >= hi || gone[q]) s[e] = 0xFF800000u;
                        }
                    }
                    float m4[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        m4[e] = fmaxf(fmaxf(fmaxf(__uint_as_float(s[e]), __uint_as_float(s[e + 4])),
                                            fmaxf(__uint_as_float(s[e + 8]), __uint_as_float(s[e + 12]))),
                                      fmaxf(fmaxf(__uint_as_float(s[e + 16]), __uint_as_float(s[e + 20])),
                                            fmaxf(__uint_as_float(s[e + 24]), __uint_as_float(s[e + 28]))));
                    const float m = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * f;
                    if (__any_sync(FULL, m > ref + SLACK)) {
                        // O holds the steps before (this S was issued after their products); all that
                        // the row has so far, P of this step included, moves to the new reference
                        const float now = fmaxf(ref, m);
                        const float alpha = now == -INFINITY ? 0.f : attn::exp2_fast(ref - now);
                        ref = now;
                        l *= alpha;
                        uint32_t x[16];
                        if (t > 0) {
#pragma unroll
                            for (int i = 0; i < 2 * NB; ++i) {
                                ld16(o_at + 16 * i, x);
                                wait_ld(x);
#pragma unroll
                                for (int e = 0; e < 16; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * alpha);
                                st16(o_at + 16 * i, x);
                            }
                        }
                        wait_st();
                        for (int i = 0; i < q; ++i) {
                            ld16(s_at + 16 * i, x);
                            wait_ld(x);
#pragma unroll
                            for (int e = 0; e < 16; ++e) {  // in fp32: alpha may be far below fp16's least
                                const float2 w = attn::mul2(attn::unpack_half(x[e]), make_float2(alpha, alpha));
                                x[e] = attn::pack_half(w.x, w.y);
                            }
                            st16(s_at + 16 * i, x);
                        }
                    }
                    const float by = ref == -INFINITY ? LIFT : LIFT - ref;
                    uint32_t packed[16];
                    float2 sum = make_float2(0.f, 0.f);
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        float2 x = attn::fma2(make_float2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])),
                                              make_float2(f, f), make_float2(by, by));
                        x = make_float2(attn::exp2_fast(x.x), attn::exp2_fast(x.y));
                        sum = attn::add2(sum, x);
                        packed[e / 2] = attn::pack_half(x.x, x.y);
                    }
                    l += sum.x + sum.y;
                    st16(s_at + 16 * q, packed);  // P over the part of S that has been read
                };
                ld32(s_at, r[0]);
#pragma unroll 1
                for (int q = 0; q < 4; q += 2) {
                    chunk(q, r[0], r[1]);
                    chunk(q + 1, r[1], r[0]);
                }
                wait_st();
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[tile]);
            }
            // ---- the row's output, or its part
            if (ok && n) ok = voted(&o_full, segments & 1);
            fence_after();
            if (wide || *(volatile unsigned*)&s_large[walked & 1] != walked + 1) {
            const bool uncut = unit == 0 && unit_end == sp.units;
            const float inv = l > 0.f ? 1.f / l : 0.f;
            float* part = a.part + (((int64_t)blockIdx.x * 2 + (u != u0)) * BLOCK_ROWS + row - first_row) * attn_part_floats(D);
            const int64_t yat = ((int64_t)(seq.q0 + qi) * ((int64_t)a.kv_heads * a.group) + qh) * NB;
            // rows by way of shared memory (the operands are read), so that a warp stores whole rows
            constexpr int PITCH = D + 4;
            float* buf = reinterpret_cast<float*>(smem) + warp * (32 * PITCH);
            __syncwarp();
#pragma unroll
            for (int kb = 0; kb < NB; ++kb) {
                uint32_t(&v)[32] = r[kb & 1];
                if (ok && n) {
                    ld32(o_at + 32 * kb, v);
                    wait_ld(v);
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] = 0;
                }
                const float by = (uncut ? inv : 1.f) * (wide ? WIDE : 1.f);
#pragma unroll
                for (int e = 0; e < 32; e += 4)
                    *reinterpret_cast<float4*>(buf + lane * PITCH + kb * 32 + e) =
                        make_float4(__uint_as_float(v[e]) * by, __uint_as_float(v[e + 1]) * by,
                                    __uint_as_float(v[e + 2]) * by, __uint_as_float(v[e + 3]) * by);
            }
            __syncwarp();
            const int warp_row = first_row + warp * 32, there = min(32, rows - warp_row);  // rows of this warp
            if (!uncut) {
                float* to = a.part + (((int64_t)blockIdx.x * 2 + (u != u0)) * BLOCK_ROWS + warp * 32) * attn_part_floats(D);
                for (int i = lane; i < there * (D / 4); i += 32) {
                    const int rr = i / (D / 4), e = 4 * (i - rr * (D / 4));
                    *reinterpret_cast<float4*>(to + rr * attn_part_floats(D) + e) =
                        *reinterpret_cast<const float4*>(buf + rr * PITCH + e);
                }
            } else if (a.out.data) {
                for (int i = lane; i < there * (D / 8); i += 32) {
                    const int rr = i / (D / 8), e = 8 * (i - rr * (D / 8));
                    const int gi = (warp_row + rr) / a.group, gh = head * a.group + warp_row + rr - gi * a.group;
                    float o[8];
                    *reinterpret_cast<float4*>(o) = *reinterpret_cast<const float4*>(buf + rr * PITCH + e);
                    *reinterpret_cast<float4*>(o + 4) = *reinterpret_cast<const float4*>(buf + rr * PITCH + e + 4);
                    storen<8>(a.out.data, (int64_t)(seq.q0 + gi) * a.out.ts + (int64_t)gh * a.out.hs + e, QMM_BF16,
                              a.out.wide, o);
                }
            }
            if (uncut && a.yq && live) {
                const float* o = buf + lane * PITCH;
                for (int kb = 0; kb < NB; ++kb) {
                    float top = 0.f;
                    for (int e = 0; e < 32; ++e) top = fmaxf(top, fabsf(o[kb * 32 + e]));
                    const float d = __fdiv_rn(top, 127.0f);
                    for (int e = 0; e < 32; ++e) {
                        const float q =
                            d > 0.f ? fminf(fmaxf(roundf(__fdiv_rn(o[kb * 32 + e], d)), -127.f), 127.f) : 0.f;
                        a.yq[(yat + kb) * 32 + e] = (int8_t)(int)q;
                    }
                    a.yd[yat + kb] = f32_to_f16_bits(d);
                }
            }
            if (!uncut && live) part[D] = ref - LIFT, part[D + 1] = l;
            fence_async();  // the buffers are operands again
            }
        }
        if (!ok) {
            if (lane == 0) {
                atomicOr(a.err, ERR_TIMEOUT);
                s_abort[walked & 1] = 1;
            }
        }
        fence_before();
        __syncthreads();
        fence_after();
        if (s_abort[walked & 1]) {
            if constexpr (!SOFTMAX) {
                if (n && lane == 0 && (warp == WARP_LOAD_K || warp == WARP_LOAD_V)) {
                    // copies on their way land before the CTA ends, or their own limit passes
                    const unsigned slots = warp == WARP_LOAD_V ? V_SLOTS : K_SLOTS;
                    for (unsigned i = issued - min(issued, slots); i < issued; ++i)
                        if (!wait(&raw_full[warp - WARP_LOAD_K][i % slots], (i / slots) & 1, a.wait_ns_tc)) break;
                }
            }
            break;
        }
        const bool again = !wide && *(volatile unsigned*)&s_large[walked & 1] == walked + 1;
        steps += n;
        if (tiles == 2) tile1_steps += n;
        segments += n > 0;
        ++walked;
        if (again) unit = cut ? unit_end - counts + a.start : 0;
        if constexpr (TURNS_BACK) {
            wide = again;
            if (again) continue;
        } else if (again) {
            if (tid == 0) s_place = Place{entry, head, unit, u, steps, segments, tile1_steps, walked};
            __syncthreads();
            return true;
        }
        if (cut && tid == 0 && unit == 0) {
            const bool uncut = unit_end == sp.units;
            const int first = (int)blockIdx.x, last = uncut ? first - 1 : shares.cta_of(u + counts + sp.units - unit_end - 1);
            a.meta[(int64_t)entry * a.kv_heads + head] = AttnMeta{first, last, u != u0, 0};
        }
        u += counts;
        unit = 0;
        if (++head == a.kv_heads) head = 0, ++entry;
        if (!cut) break;
    }
    return false;
    };
    if (warp < SOFTMAX_WARPS) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(SOFTMAX_REGS));
        if (walk(std::true_type{}, std::false_type{})) walk(std::true_type{}, std::true_type{});
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(OTHER_REGS));
        if (walk(std::false_type{}, std::false_type{})) walk(std::false_type{}, std::true_type{});
    }
    __syncthreads();
    if (warp == WARP_MMA)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TMEM_COLS));
}

}  // namespace attn_tc

AttnKernel attn_tc_kernel(int NB) {
    static constexpr AttnKernel kernels[ATTN_TC_MAX_NB] = {
        attn_tc::attn_tc_kernel<1>, attn_tc::attn_tc_kernel<2>, attn_tc::attn_tc_kernel<3>, attn_tc::attn_tc_kernel<4>};
    return kernels[NB - 1];
}

int attn_tc_smem(int NB) {
    static constexpr int bytes[ATTN_TC_MAX_NB] = {attn_tc::Smem<1>::BYTES, attn_tc::Smem<2>::BYTES,
                                                  attn_tc::Smem<3>::BYTES, attn_tc::Smem<4>::BYTES};
    return bytes[NB - 1];
}

int attn_tc_threads() { return attn_tc::THREADS; }

unsigned attn_tc_wait_ns(unsigned long long limit_ns) {
    return (unsigned)std::min<unsigned long long>(limit_ns, attn_tc::MAX_WAIT_NS);
}

}  // namespace qmm
