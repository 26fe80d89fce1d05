// qmm_lora.cu -- qmm_lora on the host: argument checks and the launch.
#include <cuda_runtime.h>

#include <algorithm>
#include <mutex>

#include "qmm.h"
#include "qmm_internal.h"
#include "qmm_lora.h"

namespace qmm {
namespace {

bool off(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

size_t size_of(int dtype) { return dtype == QMM_F32 ? 4 : 2; }

bool known(int dtype) { return dtype == QMM_F32 || dtype == QMM_F16 || dtype == QMM_BF16; }

// Rows of a matrix start on `bytes` boundaries.
bool even(const void* p, int64_t stride, size_t size, size_t bytes) {
    return !off(p, bytes) && (stride * size) % bytes == 0;
}

qmm_status check(const qmm_lora_op& op) {
    if (op.T < 0 || op.N <= 0 || op.n_segs < 0 || op.n_adapters <= 0 || op.max_rank <= 0) return QMM_ERR_ARG;
    if (!known(op.x_dtype) || !known(op.w_dtype) || (op.y_dtype != op.x_dtype && op.y_dtype != QMM_F32))
        return QMM_ERR_ARG;
    if (op.ldx < op.K || op.lda < op.K || op.ldb < op.max_rank || op.a_stride < 0 || op.b_stride < 0 ||
        op.ldy < op.N || (op.base && op.ld_base < op.N))
        return QMM_ERR_ARG;
    const int64_t far = int64_t(1) << 40;
    if (op.K <= 0 || op.K % 32 || op.K > 1 << 24 || op.N > 1 << 28 || op.T > 1 << 28 || op.n_segs > 1 << 16 ||
        op.max_rank > QMM_LORA_MAX_RANK || op.ldx > far || op.lda > far || op.ldb > far || op.a_stride > far ||
        op.b_stride > far || op.ldy > far || op.ld_base > far)
        return QMM_ERR_SHAPE;
    if (!op.seg_start && op.n_segs && (op.T % op.n_segs || op.T / op.n_segs > 1 << 28)) return QMM_ERR_SHAPE;
    if (op.T == 0 || op.n_segs == 0) return QMM_OK;
    if (!op.x || !op.a || !op.b || !op.y || !op.seg_adapter) return QMM_ERR_ARG;
    if (op.base == op.y && op.ld_base != op.ldy && op.T > 1) return QMM_ERR_SHAPE;  // in place: one stride
    const size_t xs = size_of(op.x_dtype), ws = size_of(op.w_dtype), ys = size_of(op.y_dtype);
    if (!even(op.x, op.T > 1 ? op.ldx : 0, xs, 16) || !even(op.a, op.lda, ws, 16) || (op.a_stride * ws) % 16 ||
        off(op.b, ws) || off(op.y, ys) || off(op.base, ys) || off(op.ranks, 4) || off(op.scales, 4) ||
        off(op.seg_start, 4) || off(op.seg_adapter, 4))
        return QMM_ERR_ALIGN;
    return QMM_OK;
}

LoraKernel kernel_of(int x, int w, bool f32, bool whole, int tile) {
    static LoraKernel (*const kernels[3][3])(bool, bool, int) = {
        {lora_kernel_f32_f32, lora_kernel_f32_f16, lora_kernel_f32_bf16},
        {lora_kernel_f16_f32, lora_kernel_f16_f16, lora_kernel_f16_bf16},
        {lora_kernel_bf16_f32, lora_kernel_bf16_f16, lora_kernel_bf16_bf16}};
    static_assert(QMM_F32 == 0 && QMM_F16 == 1 && QMM_BF16 == 2, "the order of the types");
    return kernels[x][w](f32, whole, tile);
}

// Opts a kernel into the device's shared memory, once a device.
bool prepared(LoraKernel k, int kind, int optin) {
    static std::mutex mu;
    static bool done[64][108];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
    std::lock_guard<std::mutex> lk(mu);
    bool& d = done[dev][kind];
    if (!d)
        d = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, optin - 1024) == cudaSuccess;
    if (!d) cudaGetLastError();
    return d;
}

}  // namespace
}  // namespace qmm

using namespace qmm;

extern "C" qmm_status qmm_lora(const qmm_lora_op* op, void* stream) {
    if (!op) return QMM_ERR_ARG;
    if (qmm_status s = check(*op)) return s;
    if (op->T == 0 || op->n_segs == 0) return QMM_OK;
    int sms = 0, optin = 0;
    if (!device_facts(&sms, &optin)) return QMM_ERR_DEVICE;
    LoraArgs a = {};
    a.x = op->x;
    a.a = op->a;
    a.b = op->b;
    a.base = op->base;
    a.y = op->y;
    a.ldx = op->ldx;
    a.lda = op->lda;
    a.a_stride = op->a_stride;
    a.ldb = op->ldb;
    a.b_stride = op->b_stride;
    a.ld_base = op->ld_base;
    a.ldy = op->ldy;
    a.ranks = op->ranks;
    a.scales = op->scales;
    a.seg_start = op->seg_start;
    a.seg_adapter = op->seg_adapter;
    a.T = op->T;
    a.N = (int)op->N;
    a.K = (int)op->K;
    a.n_segs = op->n_segs;
    a.seg_rows = (int)(op->T / op->n_segs);
    a.n_adapters = op->n_adapters;
    a.max_rank = op->max_rank;
    a.err = device_error_word();
    const WaitSettings wait = wait_settings();
    a.wait_ns = wait.limit_ns;
    a.withhold = wait.withhold;
    const bool f32 = op->y_dtype == QMM_F32;
    const int tile = op->max_rank <= 16 ? 0 : op->max_rank <= 32 ? 1 : 2, rt = 16 << tile;
    const int room = (op->max_rank + rt - 1) / rt * rt;
    const int xs = size_of(op->x_dtype), ws = size_of(op->w_dtype), ys = size_of(op->y_dtype);
    const auto even_b = [&](int to) { return even(op->b, op->ldb, ws, to) && (op->b_stride * ws) % to == 0; };
    a.vec_b = even_b(16) ? 16 : even_b(4) ? 4 : 0;
    a.vec_out = even(op->y, op->T > 1 ? op->ldy : 0, ys, 16) &&
                (!op->base || even(op->base, op->T > 1 ? op->ld_base : 0, ys, 16));
    // Outputs of 16 bytes, with base through the ring: a kernel of its own.  (One for
    // both had the registers and the code of both: 4093 rows of 8192 -> 28672, bf16,
    // 173 us instead of 164, 2039 rows of 5632 -> 8192, fp32, 54 instead of 48.)
    const bool whole = a.vec_out && a.N % 8 == 0;
    // Tiles: of each segment's rows, the last one short; fewer rows while all find an
    // SM for each of their CTAs (33 rows of 8192 -> 1024, rank 16, 16.7 and 10.0 us; 34 of
    // 5632 -> 1024, rank 128, 34.8 and 21.6).
    const int64_t rows = op->seg_start ? op->T : a.seg_rows;
    const auto tiles_of = [&](int n) {
        return op->seg_start ? std::min(op->T, op->n_segs + op->T / n) : op->n_segs * ((rows + n - 1) / n);
    };
    a.tile_rows = room > 128 ? 32 : 64;
    while (a.tile_rows > 16 && tiles_of(a.tile_rows / 2) * LORA_MAX_CLUSTER <= sms) a.tile_rows /= 2;
    const int64_t tiles = tiles_of(a.tile_rows);
    const int tile_rows = (int)std::min<int64_t>(rows, a.tile_rows), mtiles = (tile_rows + 15) / 16;
    // CTAs of a tile: eight while the tiles find room at once (short segments
    // count half: their CTAs are done early), else four: a CTA's start, its share of h
    // and the barriers take 8 us whatever it has to do.  (us with four and with
    // eight: one row of 2048 -> 2048, rank 16, 6.8 and 6.4; 48 of 8192 -> 8192, rank
    // 16, 17.3 and 13.6; 2039 rows of 5632 -> 8192 66 and 45; 64 segments of one row of
    // 2048 -> 5632, rank 64, 22.5 and 29.0; 4093 rows of 8192 -> 28672 163 and 172; these
    // and the figures of the rules below are of the day each was chosen.)
    const int64_t room_for = (int64_t)sms * (tile == 0 ? 3 : 2);
    const int64_t busy = op->seg_start ? std::min(tiles, op->T / a.tile_rows + op->n_segs / 2) : tiles;
    int64_t c = busy * LORA_MAX_CLUSTER <= room_for ? LORA_MAX_CLUSTER : 4;
    while (c > 1 && c * LORA_CHUNK > op->K) c /= 2;
    while ((1 << a.cluster_shift) < c) ++a.cluster_shift;
    // Clusters of a tile: more while all find room at once and a CTA keeps 256 columns,
    // or 1024 where h is dear and B's copies are not.  (One row of 5632 -> 8192, rank
    // 14, 16.4 and 9.2 us, 206 of 10112 -> 28672, rank 64, 73.5 and 42.8; 645 of 4096
    // -> 8066, rank 128, 77.9 and with 512 columns 105; 9 of 8192 -> 5632, rank 85, rows
    // of B on 4 bytes, 101 and with 352 75.)
    const int64_t blocks = (op->N + 31) / 32, keep = room > 64 && a.vec_b == 16 ? 32 : 8;
    while ((tiles * c << (a.parts_shift + 1)) <= room_for && blocks >> (a.cluster_shift + a.parts_shift + 1) >= keep)
        ++a.parts_shift;
    // Shared memory: the parts of h (of 16-row blocks, one to four of a tile's and
    // four in all at most), its fragments, and the ring.
    const int m2 = mtiles > 2 ? 4 : mtiles;
    const int frag = op->w_dtype == QMM_BF16 ? (f32 ? 6 : 4) : 8;
    a.frag_at = 4 * 16 * (room + 8) * 4;
    a.ring_at = (a.frag_at + mtiles * 16 * room * frag + 127) / 128 * 128;
    const int chunk = LORA_CHUNK * (mtiles * 16 * xs + rt * ws);
    const int block = 32 * (room * ws + (whole && op->base ? tile_rows * ys : 0));
    const int64_t ctas = tiles * c << a.parts_shift;
    // One CTA an SM, two, three: few CTAs have deeper rings.  (us with two or three and
    // with one: 6 rows of one of 2048 -> 2048, rank 128, fp32, 28.1 and 19.8; 18 of 6144
    // -> 2048, rank 64, fp16, 16.4 and 12.3; the rule loses at 645 of 4096 -> 8066, rank
    // 128, 77.9 and 84.8.)  Where two slots at least do not fit beside h a CTA has more
    // than its share: fp32 rows with fp32 adapters of 33 to 64 ranks, 64 rows a tile,
    // need 116,736 bytes and are one CTA an SM.
    const int total = (ctas <= sms ? 220 : tile || ctas <= 2 * sms ? 110 : 72) * 1024;
    const int least = (std::max(chunk, block) + 127) / 128 * 128, most = std::max(4 * chunk, 8 / m2 * block);
    const int share = (total - a.ring_at) / 4 / 128 * 128;
    a.slot_bytes = std::max(least, std::min(most, share));
    a.depth = std::max(2, std::min(4, (total - a.ring_at) / a.slot_bytes));
    const size_t smem = a.ring_at + (size_t)a.depth * a.slot_bytes;
    const LoraKernel kernel = kernel_of(op->x_dtype, op->w_dtype, f32, whole, tile);
    if (!prepared(kernel, (((op->x_dtype * 3 + op->w_dtype) * 2 + f32) * 2 + whole) * 3 + tile, optin)) return QMM_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles * c << a.parts_shift));
    cfg.blockDim = dim3(256 + 32 * (rt == 16 ? LORA_COPIERS<16> : LORA_COPIERS<64>));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)c;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, kernel, a) != cudaSuccess) {
        cudaGetLastError();
        return QMM_ERR_CUDA;
    }
    return QMM_OK;
}
