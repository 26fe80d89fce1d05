// qmm_attn.cu -- qmm_attn_q4_0 on the host: argument checks, the plan of a
// launch, and the kernel that joins items cut over several CTAs.
#include <algorithm>
#include <cmath>
#include <mutex>

#include "qmm.h"
#include "qmm_attn.cuh"
#include "qmm_attn_tc.h"
#include "qmm_internal.h"

namespace qmm {
namespace {

struct Plan {
    bool tc;  // the tensor-memory kernel (qmm_attn_tc.cu)
    int tiles;  // of 8 rows (the other kernel)
    int mode, unit, block_rows, blocks;  // unit: its records
    int ctas, cluster, start;  // CTAs of a cut launch, of a cluster; counts before an item's units
    int64_t items;
    size_t meta_bytes, part_bytes;
    int ring_bytes, part_at, smem;
};

constexpr int DEFAULT_SMS = 152;
constexpr int64_t MAX_CTAS = 1024;  // the join kernel's parts of an item
// The largest cluster (above 8 a kernel has to be opted in).  One token of 32
// heads of 64 over 4096 keys, fp32: 8.9 us on clusters of 8, 7.7 of 16.
constexpr int MAX_CLUSTER = 16;
// Units of a CTA up to which items stay whole or on clusters of c CTAs: cutting
// costs a second launch, and every CTA's share then spans several items where
// there are many.  (64 heads on 8 of 128, us uncut and cut.  32 fp32 tokens over
// 900, c = 1, 8 units: 16.9 and 20.5; ragged up to 1500, 12 units: 18.7 and
// 17.4; 8 over 2000, c = 4, 4 units: 12.3 and 14.5; 4 over 5000, c = 8, 5 units:
// 14.0 and 15.6; 8 ragged up to 3500, c = 4, 7 units: 16.3 and 15.3; 2 over
// 8192, c = 16, 4 units: 15.0 and 13.2.)  Fewer where CTAs would stay idle
// beside the largest clusters (one token over 6000, 3 units: 11.4 and 10.0).
int64_t units_uncut(int64_t c, bool idle) { return idle ? 2 : c <= 2 ? 8 : c <= 8 ? 6 : 3; }

// A call's counts (the units of all items, and ATTN_START an item) in row
// blocks of 16, a CTA of the kernel for them: what there is to do.
//
// With this many, 16 rows of a CTA share what is unpacked; with fewer, blocks
// of 8 make more CTAs and shorter ones.  (fp32, 4 key/value heads of 64, group
// 8.  128 queries over 301 keys, 3 counts: 9.7 us in blocks of 16, 8.7 in
// blocks of 8; 16 over 8000, 4.6: 19.6 and 18.8; 32 sequences of 2 over 4000,
// 2 heads of 256, 7.4: 30.8 and 27.8; 8 of 8 over 4000, 9.8: 20.8 and 22.4; 512
// over 2048, 43: 78 and 93.)
constexpr int64_t WIDE_MIN_COUNTS = 8;
// The tensor-memory kernel takes bf16 calls with this many rows a key/value
// head (its tile has 256; with half as many, 8 x 4 queries over 4096 keys, D =
// 128, it takes 51 us, the other 32), and this many counts, because it takes
// 17 us for the smallest call.  (8 key/value heads, D = 128.  16 queries over
// 8190 keys, 14 counts: 30 us, the other 29; 64 queries of 2 sequences of 512,
// 13 counts: 27 and 22; of 1024, 20 counts: 31 and 37; 509 over 8190, 451
// counts: 161 and 630.)
constexpr int64_t TC_MIN_ROWS = 64;
constexpr int64_t TC_MIN_COUNTS = 15;

Plan plan_of(const qmm_attn_op& op, int sms) {
    Plan p = {};
    const int D = op.cache.head_dim, NB = D / QK, group = op.q.n_heads / op.cache.n_heads;
    const int64_t rows = (int64_t)op.max_q * group;
    const int64_t steps = (op.max_kv + GROUP * ATTN_WARPS - 1) / (GROUP * ATTN_WARPS);
    const int64_t counts = (int64_t)op.n_seqs * op.cache.n_heads * ((rows + 15) / 16) * (steps + ATTN_START);
    const int64_t ctas = (int64_t)sms * attn_ctas(NB, 2);
    p.tiles = rows > 8 && counts >= WIDE_MIN_COUNTS * ctas ? 2 : 1;
    p.tc = op.q.dtype == QMM_BF16 && NB <= ATTN_TC_MAX_NB && rows >= TC_MIN_ROWS && counts >= TC_MIN_COUNTS * ctas;
    p.unit = p.tc ? ATTN_TC_RECORDS : ATTN_WARPS;
    p.block_rows = p.tc ? ATTN_TC_ROWS : p.tiles * 8;
    p.blocks = (int)((rows + p.block_rows - 1) / p.block_rows);
    p.items = (int64_t)op.n_seqs * p.blocks * op.cache.n_heads;
    p.ring_bytes = attn_ring_bytes(D, p.tiles);
    p.part_at = p.smem = p.ring_bytes + attn_q_bytes(D, p.tiles, op.q.dtype);
    const int64_t units = ((op.max_kv + GROUP - 1) / GROUP + p.unit - 1) / p.unit;
    const int64_t slots = p.tc ? sms : (int64_t)sms * attn_ctas(NB, p.tiles);
    if (p.tc) p.smem = std::max(attn_tc_smem(NB), 120 * 1024);  // one CTA an SM: each takes all of tensor memory
    // As many CTAs an item as find room at once, up to one a unit, while none has
    // much to do; beyond that equal shares, whose parts cost a second launch.
    int64_t c = 1;
    while (2 * c <= MAX_CLUSTER && c < units && 2 * c * p.items <= slots) c *= 2;
    const bool idle = c < units && 2 * c * p.items <= slots;
    if (p.tc) {
        // Whole items where they fill the SMs' rounds to three quarters; else
        // equal shares, whose parts cost a second launch.
        const int64_t rounds = (p.items + slots - 1) / slots;
        c = 1;
        p.mode = units <= 2 || 4 * p.items >= 3 * rounds * slots ? ATTN_WHOLE : ATTN_CUT;
        p.cluster = 1;
    } else if ((units + c - 1) / c <= units_uncut(c, idle)) {
        p.mode = c > 1 ? ATTN_CLUSTER : ATTN_WHOLE;
        p.cluster = (int)c;
        if (c > 1) p.smem += p.block_rows * attn_part_floats(D) * 4;
    } else {
        p.mode = ATTN_CUT;
    }
    // shares are counted in 31 bits; that many items fill the device whole, too
    if (p.mode == ATTN_CUT && p.items * (units + 1 + ATTN_START) >= int64_t(1) << 31) {
        p.mode = ATTN_WHOLE;
        p.cluster = 1;
    }
    if (p.mode == ATTN_CUT) {
        p.ctas = (int)std::min<int64_t>({slots, p.items * units, MAX_CTAS});
        p.start = p.items * units <= slots ? 0 : ATTN_START;
        p.meta_bytes = ((size_t)p.items * sizeof(AttnMeta) + 255) / 256 * 256;
        p.part_bytes = (size_t)p.ctas * 2 * p.block_rows * attn_part_floats(D) * 4;
    }
    return p;
}

qmm_status check(const qmm_attn_op& op, bool pointers) {
    if (op.n_seqs < 0 || op.T < 0 || op.max_q < 0 || op.max_kv < 0 || op.window < 0 || !std::isfinite(op.scale))
        return QMM_ERR_ARG;
    if (qmm_status s = check_cache(op.cache, pointers)) return s;
    if (op.q.n_heads <= 0 || (op.q.dtype != QMM_F32 && op.q.dtype != QMM_F16 && op.q.dtype != QMM_BF16))
        return QMM_ERR_ARG;
    if (op.q.n_heads % op.cache.n_heads) return QMM_ERR_SHAPE;
    const int64_t group = op.q.n_heads / op.cache.n_heads;
    if (op.max_kv > 1 << 28 || op.max_q > 1 << 28 || op.max_q * group > 1 << 28 || op.T > 1 << 28 ||
        (int64_t)op.n_seqs * op.max_q * op.q.n_heads > int64_t(1) << 30)
        return QMM_ERR_SHAPE;
    if (!op.q_start && op.T != (int64_t)op.n_seqs * op.max_q) return QMM_ERR_SHAPE;
    if (op.pages_stride < (op.max_kv + op.cache.page_size - 1) / op.cache.page_size) return QMM_ERR_SHAPE;
    if (!pointers) return QMM_OK;
    if (qmm_status s = check_heads(op.q, 0)) return s;
    if (op.out.data) {
        if (qmm_status s = check_output(op.out, op.q.n_heads, op.T, op.cache.head_dim)) return s;
        if (op.out.dtype != op.q.dtype) return QMM_ERR_ARG;
    }
    if ((!op.yq) != (!op.yd) || (!op.out.data && !op.yq)) return QMM_ERR_ARG;
    if (!op.kv_len || (op.max_kv > 0 && !op.pages)) return QMM_ERR_ARG;
    const auto off = [](const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; };
    if (off(op.kv_len, 4) || off(op.q_start, 4) || off(op.pages, 4) || off(op.yd, 2)) return QMM_ERR_ALIGN;
    return QMM_OK;
}

AttnKernel kernel_of(int dtype, int NB, int tiles) {
    if (dtype == QMM_F32) return tiles == 1 ? attn_kernel_f32_1(NB) : attn_kernel_f32_2(NB);
    if (dtype == QMM_F16) return tiles == 1 ? attn_kernel_f16_1(NB) : attn_kernel_f16_2(NB);
    return tiles == 1 ? attn_kernel_bf16_1(NB) : attn_kernel_bf16_2(NB);
}

// Opts a kernel into `most` bytes of dynamic shared memory and clusters of 16,
// once a device.
bool prepared(AttnKernel k, int kind, int NB, int most) {
    static std::mutex mu;
    static bool done[64][7][8];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
    std::lock_guard<std::mutex> lk(mu);
    bool& d = done[dev][kind][NB - 1];
    if (!d)
        d = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, most) == cudaSuccess &&
            cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
            cudaFuncSetAttribute(k, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared) ==
                cudaSuccess;
    if (!d) cudaGetLastError();
    return d;
}

using JoinKernel = void (*)(AttnArgs, int);

template <int TEAM>
JoinKernel join_kernel(int NB) {
    static constexpr JoinKernel kernels[8] = {
        attn::attn_join_kernel<1, TEAM>, attn::attn_join_kernel<2, TEAM>, attn::attn_join_kernel<3, TEAM>,
        attn::attn_join_kernel<4, TEAM>, attn::attn_join_kernel<5, TEAM>, attn::attn_join_kernel<6, TEAM>,
        attn::attn_join_kernel<7, TEAM>, attn::attn_join_kernel<8, TEAM>};
    return kernels[NB - 1];
}

}  // namespace
}  // namespace qmm

using namespace qmm;

extern "C" {

qmm_status qmm_attn_workspace_size(const qmm_attn_op* op, size_t* bytes) {
    if (!op || !bytes) return QMM_ERR_ARG;
    if (qmm_status s = check(*op, false)) return s;
    int sms = DEFAULT_SMS, optin = 0;
    device_facts(&sms, &optin);
    const Plan p = plan_of(*op, sms);
    *bytes = op->n_seqs && op->T && op->max_q ? p.meta_bytes + p.part_bytes : 0;
    return QMM_OK;
}

qmm_status qmm_debug_attn_plan(const qmm_attn_op* op, int* kernel, int* mode) {
    if (!op || !kernel || !mode) return QMM_ERR_ARG;
    if (qmm_status s = check(*op, false)) return s;
    int sms = DEFAULT_SMS, optin = 0;
    device_facts(&sms, &optin);
    const Plan p = plan_of(*op, sms);
    *kernel = p.tc ? QMM_ATTN_KERNEL_TMEM : p.tiles == 2 ? QMM_ATTN_KERNEL_ROWS_16 : QMM_ATTN_KERNEL_ROWS_8;
    *mode = p.mode;
    return QMM_OK;
}

qmm_status qmm_attn_q4_0(const qmm_attn_op* op, void* stream) {
    if (!op) return QMM_ERR_ARG;
    const bool empty = op->n_seqs == 0 || op->T == 0 || op->max_q == 0;
    if (qmm_status s = check(*op, !empty)) return s;
    if (empty) return QMM_OK;
    int sms = 0, optin = 0;
    const bool device = device_facts(&sms, &optin);
    const Plan p = plan_of(*op, device ? sms : DEFAULT_SMS);
    const size_t need = p.meta_bytes + p.part_bytes;
    if (need && (!op->workspace || op->workspace_bytes < need || reinterpret_cast<uintptr_t>(op->workspace) % 16))
        return QMM_ERR_WORKSPACE;
    if (!device) return QMM_ERR_DEVICE;
    AttnArgs a = {};
    a.cache = op->cache.data;
    a.q = kernel_heads(op->q);
    a.out = kernel_heads(op->out);
    a.yq = op->yq;
    a.yd = op->yd;
    a.q_start = op->q_start;
    a.kv_len = op->kv_len;
    a.pages = op->pages;
    a.pages_stride = op->pages_stride;
    a.T = op->T;
    a.n_pages = op->cache.n_pages;
    a.page_groups = op->cache.page_size / GROUP;
    a.kv_heads = op->cache.n_heads;
    a.group = op->q.n_heads / op->cache.n_heads;
    a.n_seqs = op->n_seqs;
    a.max_q = op->max_q;
    a.max_kv = op->max_kv;
    a.causal = op->causal != 0;
    a.window = std::min(op->window, 1 << 29);
    a.scale_log2 = op->scale * 1.4426950408889634f;
    a.ring_bytes = p.ring_bytes;
    a.blocks = p.blocks;
    a.mode = p.mode;
    a.cluster = p.cluster;
    a.start = p.start;
    a.ctas = p.ctas;
    a.part_at = p.part_at;
    a.meta = static_cast<AttnMeta*>(op->workspace);
    a.part = reinterpret_cast<float*>(static_cast<char*>(op->workspace) + p.meta_bytes);
    a.err = device_error_word();
    const WaitSettings wait = wait_settings();
    a.wait_ns = wait.limit_ns;
    a.wait_ns_tc = attn_tc_wait_ns(wait.limit_ns);
    a.withhold = wait.withhold;
    const int NB = op->cache.head_dim / QK;
    const AttnKernel kernel = p.tc ? attn_tc_kernel(NB) : kernel_of(op->q.dtype, NB, p.tiles);
    if (!prepared(kernel, p.tc ? 6 : 2 * op->q.dtype + p.tiles - 1, NB, p.tc ? p.smem : optin - 4096)) return QMM_ERR_CUDA;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.mode == ATTN_CUT ? p.ctas : p.items * p.cluster));
    cfg.blockDim = dim3(p.tc ? attn_tc_threads() : ATTN_THREADS);
    cfg.dynamicSmemBytes = p.smem;
    cfg.stream = st;
    cudaLaunchAttribute attr;
    if (p.mode == ATTN_CLUSTER) {
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = p.cluster;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
    }
    if (cudaLaunchKernelEx(&cfg, kernel, a) != cudaSuccess) {
        cudaGetLastError();
        return QMM_ERR_CUDA;
    }
    if (p.mode == ATTN_CUT) {
        // a block's eight warps share a row of many parts, or take a row each of few
        // (64 bf16 queries over 8190 tokens, two parts a row: 65 us shared, 51 apart)
        const bool shared = p.ctas > 16 * p.items;
        const int64_t at_once = shared ? 1 : attn::JOIN_WARPS;
        const int64_t y = std::min<int64_t>((p.block_rows + at_once - 1) / at_once,
                                            std::max<int64_t>(16, 4096 / p.items));
        cfg.gridDim = dim3((unsigned)p.items, (unsigned)y);
        cfg.blockDim = dim3(attn::JOIN_WARPS * 32);
        cfg.dynamicSmemBytes = 0;
        attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr.val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        const JoinKernel join = shared ? join_kernel<attn::JOIN_WARPS>(NB) : join_kernel<1>(NB);
        if (cudaLaunchKernelEx(&cfg, join, a, p.block_rows) != cudaSuccess) {
            cudaGetLastError();
            return QMM_ERR_CUDA;
        }
    }
    return QMM_OK;
}

}  // extern "C"
