// qmm_moe_group.cuh -- the tables that group routed slots by expert, and the
// block-wide code that builds them (shared by the expert GEMVs, the sigmoid
// router and qmm_moe_route).
#pragma once

#include "qmm_device.cuh"

namespace qmm {

// Workspace (int32 words): counts[E] | offsets[E+1] | cursor[E] | active[E]
// | n_active[1] | slot_list[T*k].  counts and offsets are per expert id;
// active[i] is the i-th routed expert (ascending id), cursor[i] the start of
// its slots in slot_list (i < n_active; its end is cursor[i + 1], or
// offsets[E] for the last), so a kernel can read its routing in one round
// of independent loads.
struct MoeWs {
    int* counts;
    int* offsets;
    int* cursor;
    int* active;
    int* n_active;
    int* slots;
};

__host__ __device__ inline MoeWs moe_ws(void* base, int E) {
    MoeWs w;
    w.counts = reinterpret_cast<int*>(base);
    w.offsets = w.counts + E;
    w.cursor = w.offsets + E + 1;
    w.active = w.cursor + E;
    w.n_active = w.active + E;
    w.slots = w.n_active + 1;
    return w;
}

__host__ __device__ inline size_t moe_ws_bytes(int E, int64_t nslots) {
    size_t words = (size_t)E * 4 + 2 + (size_t)nslots;
    return (words * 4 + 15) / 16 * 16;
}

// One CTA.  Counting sort of slots by expert id; slots inside one expert's
// list come out in any order (each slot's output is computed on its own,
// so the order does not change any result).
constexpr int GROUP_THREADS = 1024;

// The whole block builds the tables.  ids may have been written earlier in
// the same kernel by this block (plain loads after a block barrier).  The
// counts and cursors live in shared memory while the sort runs (up to
// GROUP_SMEM_E experts; beyond that in the workspace itself), so the only
// global-memory traffic is the final tables, written once.
constexpr int GROUP_SMEM_E = 2048;

// Few slots (one token's top-k, up to 32): each thread derives the tables of
// its experts directly from the slot ids -- counts, offsets and active
// positions by comparing against every slot -- with no scan, no atomics and
// two block barriers.  Slots of one expert keep their slot order.
constexpr int GROUP_FEW = 32;

// The tables of a few slots (nslots <= GROUP_FEW) built from their ids by
// the whole block: warp 0 holds one slot per lane and finds, with warp
// intrinsics, each slot's first occurrence and its place in the slot list;
// then every thread derives the counts, offsets and active position of its
// experts by comparing against the slots (fixed-trip, unrolled).  Every
// word the workspace layout defines is written.  f_id / f_first: GROUP_FEW
// ints of shared memory each.
__device__ __forceinline__ void moe_group_few_tables(const int32_t* ids, int nslots, int E, MoeWs w, int* f_id,
                                                     int* f_first, int* err) {
    if (threadIdx.x < 32) {
        const int s = threadIdx.x;
        int e = s < nslots ? ids[s] : -1;
        if (s < nslots && (e < 0 || e >= E)) {
            atomicOr(err, ERR_BAD_EXPERT);
            e = -1;
        }
        const unsigned same = __match_any_sync(FULL, e);
        const bool first = e >= 0 && (__ffs(same) - 1) == s;
        f_id[s] = e;
        f_first[s] = first ? 1 : 0;
        // place in the slot list: every valid slot of a lower expert, then the
        // earlier slots of the same expert
        int pos = __popc(same & ((1u << s) - 1u));
#pragma unroll
        for (int t = 0; t < GROUP_FEW; ++t) {
            const int v = __shfl_sync(FULL, e, t);
            pos += v >= 0 && v < e;
        }
        if (e >= 0) w.slots[pos] = s;
    }
    __syncthreads();
    for (int e = threadIdx.x; e <= E; e += blockDim.x) {
        int cnt = 0, below = 0, dist_below = 0;
#pragma unroll
        for (int t = 0; t < GROUP_FEW; ++t) {
            const int v = f_id[t];  // -1 past nslots
            cnt += v == e;
            below += v >= 0 && v < e;
            dist_below += f_first[t] && v < e;
        }
        if (e == E) {  // every valid slot, every routed expert
            w.offsets[E] = below;
            *w.n_active = dist_below;
            continue;
        }
        w.offsets[e] = below;
        w.counts[e] = cnt;
        if (cnt > 0) {
            w.active[dist_below] = e;
            w.cursor[dist_below] = below;
        }
    }
}

__device__ __forceinline__ void moe_group_few(const int32_t* ids, int nslots, int E, MoeWs w, int* err) {
    __shared__ int f_id[GROUP_FEW];     // slot id, or -1 (none, or an id outside [0, E))
    __shared__ int f_first[GROUP_FEW];  // 1 if no earlier slot has the same id
    moe_group_few_tables(ids, nslots, E, w, f_id, f_first, err);
}

__device__ __forceinline__ void moe_group_block(const int32_t* ids, int nslots, int E, MoeWs w, int* err) {
    if (nslots <= GROUP_FEW) {
        moe_group_few(ids, nslots, E, w, err);
        return;
    }
    __shared__ int s_cnt[GROUP_SMEM_E];
    __shared__ int s_cur[GROUP_SMEM_E];
    const bool in_smem = E <= GROUP_SMEM_E;
    int* cnt = in_smem ? s_cnt : w.counts;
    int* cur = in_smem ? s_cur : w.cursor;
    for (int e = threadIdx.x; e < E; e += blockDim.x) cnt[e] = 0;
    __syncthreads();
    for (int s = threadIdx.x; s < nslots; s += blockDim.x) {
        const int e = ids[s];
        if (e < 0 || e >= E) {
            atomicOr(err, ERR_BAD_EXPERT);
            continue;
        }
        atomicAdd(&cnt[e], 1);
    }
    __syncthreads();
    // Exclusive scans of counts (-> offsets) and of (counts > 0) (-> active
    // positions), each thread owning a contiguous chunk of experts.
    const int per = (E + blockDim.x - 1) / blockDim.x;
    const int e0 = min(E, (int)threadIdx.x * per), e1 = min(E, e0 + per);
    int csum = 0, asum = 0;
    for (int e = e0; e < e1; ++e) {
        csum += cnt[e];
        asum += cnt[e] > 0;
    }
    // block-wide exclusive scan of (csum, asum) packed into one 64-bit lane value
    long long v = ((long long)csum << 32) | (unsigned)asum;
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    long long incl = v;
    for (int o = 1; o < 32; o <<= 1) {
        long long n = __shfl_up_sync(FULL, incl, o);
        if (lane >= o) incl += n;
    }
    __shared__ long long wsum[32];
    if (lane == 31) wsum[wid] = incl;
    __syncthreads();
    if (wid == 0) {
        long long t = (lane < (int)(blockDim.x >> 5)) ? wsum[lane] : 0;
        for (int o = 1; o < 32; o <<= 1) {
            long long n = __shfl_up_sync(FULL, t, o);
            if (lane >= o) t += n;
        }
        wsum[lane] = t;  // inclusive over warps
    }
    __syncthreads();
    long long excl = incl - v + (wid > 0 ? wsum[wid - 1] : 0);
    int coff = (int)(excl >> 32), aoff = (int)(excl & 0xffffffff);
    for (int e = e0; e < e1; ++e) {
        const int c = cnt[e];
        if (in_smem) w.counts[e] = c;
        w.offsets[e] = coff;
        cur[e] = coff;
        if (c > 0) w.active[aoff++] = e;
        coff += c;
    }
    if (threadIdx.x == blockDim.x - 1) {
        w.offsets[E] = coff;
        *w.n_active = aoff;
    }
    __syncthreads();
    for (int s = threadIdx.x; s < nslots; s += blockDim.x) {
        const int e = ids[s];
        if (e < 0 || e >= E) continue;
        const int pos = atomicAdd(&cur[e], 1);
        w.slots[pos] = s;
    }
    // cursor[i]: the start of the i-th active expert's slots (the sort's own
    // cursors are no longer needed)
    __syncthreads();
    const int na = *w.n_active;
    for (int i = threadIdx.x; i < na; i += blockDim.x) w.cursor[i] = w.offsets[w.active[i]];
}

}  // namespace qmm
