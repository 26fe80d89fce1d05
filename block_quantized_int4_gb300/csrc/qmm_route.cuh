// qmm_route.cuh -- routing to experts in general form: softmax or sigmoid
// scores, a bias that enters the choice alone, groups of experts, top-k,
// renormalised and scaled gates.
//
// The choice is that of the scores in 64 bits: c_e = s_e + b_e, the group
// scores, and equal values to the lower index.  Without a bias c is replaced
// by the logit (both scores are strictly increasing).  A warp takes a token;
// each lane holds PER experts of one group:
//  - a logit's own order is exact; c and the sums of two are computed in fp32,
//    with a bound on their error.  Where two values whose order decides anything
//    are closer than that bound and not of equal operands (about one token in a
//    thousand of sigmoid scores with a bias, 256 experts), these are computed
//    again as sums of two fp32 numbers, and what these do not order either, in 64
//    bits (route_slow).  (All of the close ones in 64 bits, at 16 cycles an
//    instruction, took 10 us more for 32003 tokens of 256 experts in 8 groups, a
//    bound of four times the width 5.)
//  - the k-th largest of the 32 lanes' best bounds the k-th largest from below,
//    so that only experts from there on are candidates: about 1.3 k of them, one
//    a lane, each ranked against all others.  More than 32, as with most experts
//    switched off or in few lanes: k rounds over all.
// What bounds it: the logits pass once (65521 tokens of 512, fp32: 44 us, 3.1
// TB/s), but a token takes some 530 warp instructions, 890 with sigmoid, bias and
// groups (32003 tokens of 256: 36 us; 15 of them reach spilled registers),
// comparisons most of them: their pipe is 53% and 61% busy at 28 warps an SM, which
// registers limit.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <climits>

#include "qmm_device.cuh"
#include "qmm_moe_group.cuh"
#include "qmm_route.h"
#include "qmm_route_pair.cuh"

namespace qmm {
namespace route {

constexpr int MAX_K = 64;
constexpr int WARPS = ROUTE_WARPS;

__device__ __forceinline__ float as_float(float v) { return v; }
__device__ __forceinline__ float as_float(__half v) { return __half2float(v); }
__device__ __forceinline__ float as_float(__nv_bfloat16 v) { return __bfloat162float(v); }

// Ordered keys.
__device__ __forceinline__ uint32_t key32(float v) {
    const int u = __float_as_int(v + 0.f);  // -0 as +0
    return (uint32_t)(u ^ ((u >> 31) | (int)0x80000000));
}
__device__ __forceinline__ unsigned long long key64(double v) {
    const unsigned long long u = __double_as_longlong(v + 0.0);
    return max(u ^ ((u >> 63) ? ~0ull : 1ull << 63), 2ull);
}

// A warp's candidates and choice.
struct __align__(16) Chosen {
    float c[36];       // of candidates, then -inf up to a multiple of four
    int cand[32];
    int id[MAX_K + 1];  // the chosen in order; one more where the border is checked
    union {
        float value[MAX_K + 1];  // and their c
        float2 pair[32];
    };
};

// Where a lane's experts lie: four (two, one) side by side, and again behind
// those of the other lanes of the group, so that loads and stores of a warp are
// contiguous.  (With all of a lane's experts side by side 65521 tokens of 512
// fp32 logits were bound by the shared memory's data path, 82% of its peak: 62 us
// instead of 49.)
template <int PER>
constexpr int BESIDE = PER < 4 ? PER : 4;
struct Place {
    int first, lanes, group;  // lanes: of a group
    int shift, step;
    uint32_t there;  // those that there are

    __device__ __forceinline__ int expert(int i) const { return first + (i >> shift) * step + (i & ((1 << shift) - 1)); }
};

template <int PER>
__device__ __forceinline__ Place place_of(const RouteArgs& a, int lane) {
    constexpr int V = BESIDE<PER>;
    Place p;
    p.lanes = 32 / a.n_groups;
    p.group = lane / p.lanes;
    const int at = (lane - p.group * p.lanes) * V;
    p.first = p.group * a.group_size + at;
    p.shift = V == 4 ? 2 : V - 1;
    p.step = p.lanes * V;
    p.there = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) p.there |= (at + i / V * p.step + i % V < a.group_size ? 1u : 0u) << i;
    return p;
}

template <int BYTES>
struct VecWord;
template <>
struct VecWord<16> {
    using type = uint4;
};
template <>
struct VecWord<8> {
    using type = uint2;
};
template <>
struct VecWord<4> {
    using type = uint32_t;
};
template <>
struct VecWord<2> {
    using type = unsigned short;
};

// A lane's logits as fp32; experts that are not there as -inf.
template <int PER, typename T>
__device__ __forceinline__ void load_logits(const RouteArgs& a, const T* row, const Place& p, float (&l)[PER]) {
    constexpr int V = BESIDE<PER>;
    union alignas(V * sizeof(T)) Vec {
        T e[V];
        typename VecWord<V * (int)sizeof(T)>::type word;
    };
    if (a.vec == 2) {
#pragma unroll
        for (int i = 0; i < PER; i += V) {
            Vec v;
            v.word = *reinterpret_cast<const decltype(v.word)*>(row + p.first + i / V * p.step);
#pragma unroll
            for (int j = 0; j < V; ++j) l[i + j] = as_float(v.e[j]);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < PER; i += V) {
        const T* src = row + p.first + i / V * p.step;
        if (a.vec) {
            Vec v;
            if (p.there >> i & 1) {
                v.word = *reinterpret_cast<const decltype(v.word)*>(src);
#pragma unroll
                for (int j = 0; j < V; ++j) l[i + j] = as_float(v.e[j]);
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j) l[i + j] = -INFINITY;
            }
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) l[i + j] = p.there >> (i + j) & 1 ? as_float(src[j]) : -INFINITY;
        }
    }
}
// Experts that take no part (-inf, NaN) as -inf.
template <int PER>
__device__ __forceinline__ void no_nan(float (&l)[PER]) {
#pragma unroll
    for (int i = 0; i < PER; ++i) l[i] = fmaxf(l[i], -INFINITY);
}

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// NaNs do not count.
__device__ __forceinline__ float warp_max(float v) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float warp_min(float v) {
    float r;
    asm volatile("redux.sync.min.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

// Logits in 64 bits -> score (0 of -inf).
__device__ __forceinline__ double score64(const RouteArgs& a, float l, double top, double sum) {
    const double e = exp(a.softmax ? (double)l - top : -(double)l);
    return a.softmax ? (l > -INFINITY ? e / sum : 0.0) : 1.0 / (1.0 + e);
}

// The 64-bit largest logit and sum of exponentials of a token's softmax.
template <int PER>
__device__ __forceinline__ void softmax64(const float (&l)[PER], double& top, double& sum) {
    top = -INFINITY;
    sum = 0.0;
#pragma unroll
    for (int i = 0; i < PER; ++i) top = fmax(top, (double)l[i]);
    for (int o = 16; o > 0; o >>= 1) top = fmax(top, __shfl_xor_sync(FULL, top, o));
#pragma unroll 1
    for (int i = 0; i < PER; ++i)
        if (l[i] > -INFINITY) sum += exp((double)l[i] - top);
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(FULL, sum, o);
}

// Whether the group of a lane stays, in 64 bits; c: each expert's score and
// bias (its logit where these do not enter the choice).
template <int PER>
__device__ __forceinline__ bool groups64(const RouteArgs& a, const Place& p, const float (&l)[PER], double (&c)[PER]) {
    const bool top2 = a.n_groups > 1 && a.top2;
    if (a.bias || top2) {
        double top = 0.0, sum = 1.0;
        if (a.softmax) softmax64(l, top, sum);
#pragma unroll 1
        for (int i = 0; i < PER; ++i) c[i] = score64(a, l[i], top, sum);
        if (a.bias) {
#pragma unroll
            for (int i = 0; i < PER; ++i) c[i] += p.there >> i & 1 ? (double)a.bias[p.expert(i)] : 0.0;
        }
    } else {
#pragma unroll
        for (int i = 0; i < PER; ++i) c[i] = l[i];
    }
    double first = -INFINITY, second = -INFINITY;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const double v = l[i] > -INFINITY ? c[i] : -INFINITY;
        second = v > first ? first : v > second ? v : second;
        first = v > first ? v : first;
    }
    for (int o = p.lanes >> 1; o > 0; o >>= 1) {
        const double f = __shfl_xor_sync(FULL, first, o), s = __shfl_xor_sync(FULL, second, o);
        second = fmax(fmin(first, f), fmax(second, s));
        first = fmax(first, f);
    }
    const double mine = top2 && second > -INFINITY ? first + second : first;
    const int g = p.group;
    int before = 0;
    for (int h = 0; h < a.n_groups; ++h) {
        const double v = __shfl_sync(FULL, mine, h * p.lanes);
        before += v > mine || (v == mine && h < g);
    }
    return before < a.top_groups;
}

// The whole choice with 64-bit keys, by k rounds over all experts.  Every lane
// of the warp; leaves the chosen experts in out.id.
template <int PER, typename T>
__device__ __noinline__ void route_slow(const RouteArgs& a, const T* row, Chosen& out) {
    const int lane = threadIdx.x & 31;
    const Place p = place_of<PER>(a, lane);
    float l[PER];
    load_logits<PER, T>(a, row, p, l);
    no_nan(l);
    double c[PER];
    const bool stays = groups64(a, p, l, c);
    unsigned long long key[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i)
        key[i] = stays && p.there >> i & 1 ? l[i] > -INFINITY ? key64(a.bias ? c[i] : (double)l[i]) : 1ull : 0ull;
    for (int j = 0; j < a.k; ++j) {
        unsigned long long best = 0;
        int at = 0;
        for (int i = PER - 1; i >= 0; --i)
            if (key[i] >= best) {
                best = key[i];
                at = i;
            }
        unsigned long long most = best;
        for (int o = 16; o > 0; o >>= 1) most = max(most, __shfl_xor_sync(FULL, most, o));
        // (a lane's experts and the places in it rise together)
        const int e = p.expert(at);
        if (__reduce_min_sync(FULL, best == most ? e : INT_MAX) == e && best == most) {
            out.id[j] = e;
            for (int i = 0; i < PER; ++i)
                if (i == at) key[i] = 0;
        }
    }
    __syncwarp();
}

// Experts of this lane in `mask` become candidates, the first of every lane, then
// the second ..; how many there are (more than 32: not all are written).
template <int PER>
__device__ __forceinline__ int collect(uint32_t mask, const Place& p, const float* values, Chosen& out) {
    constexpr int V = BESIDE<PER>;
    const int lane = threadIdx.x & 31;
    int total = 0;
    __syncwarp();
    for (uint32_t some; (some = __ballot_sync(FULL, mask != 0)) != 0; total += __popc(some)) {
        const int at = total + __popc(some & ((1u << lane) - 1u)), i = __ffs(mask) - 1;
        if (mask && at < 32) {
            out.cand[at] = p.expert(i);
            out.c[at] = fmaxf(values[i / V * 32 * V + lane * V + i % V], -INFINITY) + 0.f;  // -0 as +0
        }
        mask &= mask - 1;
    }
    if (total <= 32 && lane < 4) out.c[total + lane] = -INFINITY;
    __syncwarp();
    return total;
}

// The n first of the experts that are `there` by n rounds over all: where more than
// 32 may be among them.
template <int PER>
__device__ __noinline__ void pick(uint32_t there, const Place p, const float* values, int n, Chosen& out) {
    constexpr int V = BESIDE<PER>;
    const int lane = threadIdx.x & 31;
    uint32_t key[PER];
    __syncwarp();
#pragma unroll
    for (int i = 0; i < PER; ++i)
        key[i] = there >> i & 1 ? key32(fmaxf(values[i / V * 32 * V + lane * V + i % V], -INFINITY)) : 0u;
#pragma unroll 1
    for (int r = 0; r < n; ++r) {
        uint32_t best = 0;
        int at = 0;
#pragma unroll
        for (int i = PER - 1; i >= 0; --i)
            if (key[i] >= best) best = key[i], at = i;
        const uint32_t most = __reduce_max_sync(FULL, best);
        // (a lane's experts and the places in it rise together)
        const int e = p.expert(at), first = __reduce_min_sync(FULL, best == most ? e : INT_MAX);
        if (best == most && e == first) {
            out.id[r] = e;
            out.value[r] = __uint_as_float(most ^ ((most >> 31) ? 0x80000000u : 0xFFFFFFFFu));
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (i == at) key[i] = 0;
        }
    }
    __syncwarp();
}

// Scores as pairs: their largest error, 2^-42 of `unit` (1, or a softmax's
// largest score) and 2^-46 of what they are added to, with a margin of 8.
struct Scores {
    float top;
    Pair inverse;  // of the softmax's sum
    float unit;

    template <typename T>
    __device__ __forceinline__ Scores(const RouteArgs& a, const T* row, const Place& p)
        : top(0.f), inverse{1.f, 0.f}, unit(1.f) {
        if (!a.softmax) return;
        top = -INFINITY;
#pragma unroll 1
        for (uint32_t m = p.there; m; m &= m - 1) top = fmaxf(top, as_float(row[p.expert(__ffs(m) - 1)]));
        top = warp_max(top);
        if (!(top > -INFINITY)) return;
        Pair sum = {0.f, 0.f};
#pragma unroll 1
        for (uint32_t m = p.there; m; m &= m - 1) sum = add(sum, power(as_float(row[p.expert(__ffs(m) - 1)])));
        for (int o = 16; o > 0; o >>= 1)
            sum = add(sum, Pair{__shfl_xor_sync(FULL, sum.hi, o), __shfl_xor_sync(FULL, sum.lo, o)});
        inverse = reciprocal(sum);
        unit = inverse.hi;
    }
    __device__ __forceinline__ Pair power(float l) const {
        return l - top > -87.f ? exp_pair(two_sum(l, -top)) : Pair{0.f, 0.f};  // -inf and NaN, too
    }
    // With the bias; -inf of an expert that takes no part.
    __device__ __forceinline__ Pair of(const RouteArgs& a, float l, float bias) const {
        if (!(l > -INFINITY)) return {-INFINITY, 0.f};
        return add(a.softmax ? mul(power(l), inverse) : sigmoid_pair(l), bias);
    }
    __device__ __forceinline__ float tolerance(float size) const { return 0x1p-39f * unit + 0x1p-43f * size; }
};

// Whether the lane's group stays, where fp32 does not tell; `close`: pairs do
// not, either.  mask: experts that may be among their group's best.  (Short loops:
// code that runs for few tokens comes from afar; with eight experts side by side
// 4864 tokens of 256 in 8 groups took 15.3 us, so 11.0, of which these tokens 3.)
template <typename T>
__device__ __noinline__ bool groups_again(const RouteArgs& a, const T* row, const Place p, uint32_t mask, bool& close) {
    const Scores s(a, row, p);
    Pair first = {-INFINITY, 0.f}, second = first;
#pragma unroll 1
    for (; mask; mask &= mask - 1) {
        const int e = p.expert(__ffs(mask) - 1);
        const Pair v = s.of(a, as_float(row[e]), a.bias ? a.bias[e] : 0.f);
        if (before(v, first)) {
            second = first;
            first = v;
        } else if (before(v, second)) {
            second = v;
        }
    }
    for (int o = p.lanes >> 1; o > 0; o >>= 1) {
        const Pair f = {__shfl_xor_sync(FULL, first.hi, o), __shfl_xor_sync(FULL, first.lo, o)};
        const Pair g = {__shfl_xor_sync(FULL, second.hi, o), __shfl_xor_sync(FULL, second.lo, o)};
        const Pair low = before(first, f) ? f : first, rest = before(second, g) ? second : g;
        first = before(f, first) ? f : first;
        second = before(low, rest) ? low : rest;
    }
    const Pair mine = a.top2 && second.hi > -INFINITY ? add(first, second) : first;
    const float size = first.hi > -INFINITY ? fabsf(first.hi) + (second.hi > -INFINITY ? fabsf(second.hi) : 0.f) : 0.f;
    const float tolerance = s.tolerance(warp_max(size));
    const int g = p.group;
    int ahead = 0;
    for (int h = 0; h < a.n_groups; ++h) {
        const Pair v = {__shfl_sync(FULL, mine.hi, h * p.lanes), __shfl_sync(FULL, mine.lo, h * p.lanes)};
        ahead += before(v, mine) || (!before(mine, v) && h < g);
    }
    const bool in = ahead < a.top_groups;
    bool near = false;
    for (int h = 0; h < a.n_groups; ++h) {
        const Pair v = {__shfl_sync(FULL, mine.hi, h * p.lanes), __shfl_sync(FULL, mine.lo, h * p.lanes)};
        const bool other = __shfl_sync(FULL, (int)in, h * p.lanes) != (int)in;
        near |= other && unsure(mine, v, tolerance);
    }
    close = __any_sync(FULL, near);
    return in;
}

// The order of the candidates, each as a pair on a lane of its own, where fp32
// does not tell (all that may be among the k largest and take part are there);
// false: pairs do not, either.
template <typename T>
__device__ __noinline__ bool order_again(const RouteArgs& a, const T* row, const Place p, int total, Chosen& out) {
    const int lane = threadIdx.x & 31;
    const Scores s(a, row, p);
    const int e = lane < total ? out.cand[lane] : 0;
    const float l = fmaxf(as_float(row[e]), -INFINITY), bias = a.bias ? a.bias[e] : 0.f;
    const Pair mine = s.of(a, l, bias);
    out.pair[lane] = make_float2(mine.hi, mine.lo);
    __syncwarp();
    int rank = 0;
    bool near = false;
    for (int d = 0; d < total; ++d) {
        const float2 q = out.pair[d];
        const Pair v = {q.x, q.y};
        rank += before(v, mine) || (!before(mine, v) && out.cand[d] < e);
        const float l_d = __shfl_sync(FULL, l, d), bias_d = __shfl_sync(FULL, bias, d);
        const bool same = l_d == l && bias_d == bias;
        near |= !same && unsure(mine, v, s.tolerance(fabsf(mine.hi)));
    }
    if (lane < total && rank < a.k) out.id[rank] = e;
    __syncwarp();
    return !__any_sync(FULL, near && lane < total && rank < a.k);
}

// One token.  SCORES: the choice takes scores (a bias, or groups by the sum of
// two), not logits alone.  values: 32 * PER words of shared memory.
template <int PER, typename T, bool SCORES>
__device__ __forceinline__ void route_one(const RouteArgs& a, int t, const Place& p, const float (&bias)[PER],
                                          float* values, Chosen& out) {
    const int lane = threadIdx.x & 31;
    const T* row = static_cast<const T*>(a.logits) + (int64_t)t * a.ld;
    const bool grouped = a.n_groups > 1, top2 = grouped && a.top2;
    float l[PER];
    load_logits<PER, T>(a, row, p, l);

    // softmax: the largest logit and the sum of exponentials
    float top = 0.f, sum = 1.f;
    if (a.softmax && (SCORES || !a.renorm)) {
        no_nan(l);
        float m = l[0];
#pragma unroll
        for (int i = 1; i < PER; ++i) m = fmaxf(m, l[i]);
        top = warp_max(m);
        sum = 0.f;
        if (top > -INFINITY) {
#pragma unroll
            for (int i = 0; i < PER; ++i) sum += ex2((l[i] - top) * 1.4426950408889634f);
        }
        sum = warp_sum(sum);
    }

    // what decides, with the error that a score may have.  A sigmoid's exponential
    // is off by 2^-22 and by 1.5 |x| 2^-24 of its exponent, which weighs s (1 - s)
    // (1/4 at most, 0.23 / |x|), 1 + e by 2^-24, its reciprocal by 2^-23: together
    // below 4.4 * 2^-24.  A softmax's sum of up to 1024 and its reciprocal are off by
    // 60 * 2^-24 (the terms by 4 and 2.5 |x|, with |x| 6.9 on average at most, 36
    // additions, 2), the same for all scores, so that the difference of two has that
    // once, and 6 * 2^-24 of the largest score for either.
    const float unit = a.softmax && SCORES ? rcp(sum) : 1.f, slack = unit * (a.softmax ? 0x1p-18f : 0x1p-21f);
    float c[PER];  // NaN here and there where it is the logit
    float first = -INFINITY, second = -INFINITY;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        c[i] = l[i];
        if constexpr (SCORES) {
            const float e = ex2((a.softmax ? l[i] - top : -l[i]) * 1.4426950408889634f);
            float v = (a.softmax ? e * unit : rcp(1.f + e)) + bias[i];
            v = l[i] > -INFINITY ? v : -INFINITY;
            if (a.bias) c[i] = v;
            if (top2) second = fmaxf(second, fminf(first, v));
            first = fmaxf(first, v);
        }
    }
    float best = -INFINITY;
#pragma unroll
    for (int i = 0; i < PER; ++i) best = fmaxf(best, c[i]);
    bool stays = p.there != 0, again = false;
    if (grouped) {
        if constexpr (!SCORES) first = best;
        for (int o = p.lanes >> 1; o > 0; o >>= 1) {
            const float f = __shfl_xor_sync(FULL, first, o);
            if (top2) {
                const float s = __shfl_xor_sync(FULL, second, o);
                second = fmaxf(fminf(first, f), fmaxf(second, s));
            }
            first = fmaxf(first, f);
        }
        const float mine = top2 && second > -INFINITY ? first + second : first;
        const uint32_t key = key32(mine);
        const int g = p.group;
        uint32_t* keys = reinterpret_cast<uint32_t*>(out.c);
        if (lane == g * p.lanes) keys[g] = key;
        if (lane < 2) keys[a.n_groups + lane] = 0;
        __syncwarp();
        int before = 0;
        for (int h = 0; h < a.n_groups; h += 4) {
            const uint4 v = *reinterpret_cast<const uint4*>(keys + h);
            before += (v.x >= key + (h >= g)) + (v.y >= key + (h + 1 >= g)) + (v.z >= key + (h + 2 >= g)) +
                      (v.w >= key + (h + 3 >= g));
        }
        __syncwarp();
        bool in = before < a.top_groups;
        if constexpr (SCORES) {
            // groups on either side of the border that are too close
            const float hi = warp_min(in ? mine : INFINITY), lo = warp_max(in ? -INFINITY : mine);
            const float size = first > -INFINITY ? fabsf(first) + (second > -INFINITY ? fabsf(second) : 0.f) : 0.f;
            const float largest = warp_max(size);
            // (sums of two biases may pass fp32: below all others they are in order with
            // them, but not among themselves or with groups that have no experts left)
            const bool open = lo > -INFINITY ? !(hi - lo > 4.f * slack + 0x1p-21f * largest)
                                             : largest == INFINITY && hi <= -0x1p127f;
            if (open && largest == INFINITY) {
                again = true;
            } else if (open) {
                // of these, all that may be among the best (the two best) of a group
                const float least = (top2 ? second : first) - (2.f * slack + 0x1p-22f * size);
                uint32_t mask = p.there;
                if (a.bias) {
#pragma unroll
                    for (int i = 0; i < PER; ++i) mask &= ~((c[i] < least ? 1u : 0u) << i);
                }
                in = groups_again(a, row, p, mask, again);
            }
        }
        stays = stays && in;
    }

    // candidates: experts from the n-th best of the lanes' best on (n = k, and one
    // more where the border is checked)
    const int n = a.k + (SCORES && a.bias ? 1 : 0);
    const uint32_t there = stays ? p.there : 0u;
#pragma unroll
    for (int i = 0; i < PER; i += BESIDE<PER>) {
        float* to = values + 32 * i + lane * BESIDE<PER>;
        if constexpr (PER >= 4)
            *reinterpret_cast<float4*>(to) = make_float4(c[i], c[i + 1], c[i + 2], c[i + 3]);
        else if constexpr (PER == 2)
            *reinterpret_cast<float2*>(to) = make_float2(c[0], c[1]);
        else
            *to = c[0];
    }
    const auto from = [&](float floor) {
        uint32_t mask = there;
        if (floor > -INFINITY) {
            mask = 0;
#pragma unroll
            for (int i = 0; i < PER; ++i) mask |= (c[i] >= floor ? 1u : 0u) << i;
            mask &= there;
        }
        return collect<PER>(mask, p, values, out);
    };
    float floor = -INFINITY;
    if (n <= 32) {
        // the smallest of those that fewer than n are larger than
        const float mine = stays ? best : -INFINITY;
        out.c[lane] = mine;
        __syncwarp();
        float larger = 0.f;  // (counted by the other pipe than the comparisons')
#pragma unroll
        for (int d = 0; d < 32; d += 4) {
            const float4 v = *reinterpret_cast<const float4*>(out.c + d);
            if (v.x > mine) larger += 1.f;
            if (v.y > mine) larger += 1.f;
            if (v.z > mine) larger += 1.f;
            if (v.w > mine) larger += 1.f;
        }
        floor = warp_min(larger < (float)n ? mine : INFINITY);
    }
    int total = from(floor);
    if (total > 32) {
        __syncwarp();
        pick<PER>(there, p, values, n, out);
    } else {
        const float mine = lane < total ? out.c[lane] : -INFINITY;
        float larger = 0.f;
        for (int d = 0; d < total; d += 4) {
            const float4 v = *reinterpret_cast<const float4*>(out.c + d);
            if (v.x > mine) larger += 1.f;
            if (v.y > mine) larger += 1.f;
            if (v.z > mine) larger += 1.f;
            if (v.w > mine) larger += 1.f;
        }
        int rank = (int)larger;
        // of equal ones the lower expert first
        uint32_t same = __match_any_sync(FULL, __float_as_uint(mine)) & ~(1u << lane);
        if (lane < total)
            for (same &= 0xFFFFFFFFu >> (32 - total); same; same &= same - 1)
                rank += out.cand[__ffs(same) - 1] < out.cand[lane];
        if (lane < total && rank < n) {
            out.id[rank] = out.cand[lane];
            if (SCORES && a.bias) out.value[rank] = mine;
        }
        __syncwarp();
    }
    if (SCORES && a.bias) {
        // neighbours that are too close, but for equal logits with equal biases
        // among the chosen (at the border a third may be close to both)
        bool close = false;
        for (int j = lane; j < min(total, n) - 1; j += 32) {
            const float hi = out.value[j], lo = out.value[j + 1];
            if (lo > -INFINITY && !(hi - lo > 2.f * slack + 0x1p-23f * (fabsf(hi) + fabsf(lo)))) {
                bool differ = true;
                if (j + 1 < a.k) {
                    const int e = out.id[j], f = out.id[j + 1];
                    differ = !(as_float(row[e]) == as_float(row[f]) && a.bias[e] == a.bias[f]);
                }
                close = close || differ;
            }
        }
        if (!again && __any_sync(FULL, close)) {
            // all that may be among the k largest, as pairs; of fewer than k that take part
            // these alone: the others are in order behind them
            const float kth = out.value[a.k - 1];
            total = from(fmaxf(kth - (2.f * slack + 0x1p-21f * fabsf(kth)), -0x1.fffffep127f));
            again = total > 32 || !order_again(a, row, p, total, out);
        }
    }
    if (again) route_slow<PER, T>(a, row, out);

    // gates of the chosen: lane j has the j-th and the (j + 32)-th
    const int halves = a.k > 32 ? 2 : 1;
    float lj[2], s[2];
    int id[2];
    float most = -INFINITY;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        lj[r] = -INFINITY;
        if (r >= halves) break;
        const int j = lane + 32 * r;
        id[r] = j < a.k ? out.id[j] : 0;
        lj[r] = j < a.k ? as_float(row[id[r]]) : -INFINITY;
        lj[r] = lj[r] > -INFINITY ? lj[r] : -INFINITY;
        most = fmaxf(most, lj[r]);
    }
    if (a.renorm) most = warp_max(most);
    // renormalised, softmax needs no sum over all; neither do sigmoids that
    // are e^l to the last bit (below e^-30), whose quotients fp32 would lose
    const bool exps = a.softmax || (a.renorm && most < -30.f);
    const float ref = a.renorm ? most : a.softmax ? top : 0.f;
    float part = 0.f;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        if (r >= halves) break;
        s[r] = lj[r] > -INFINITY ? (exps ? expf(lj[r] - ref) : 1.f / (1.f + expf(-lj[r]))) : 0.f;
        part += s[r];
    }
    float div = a.softmax ? sum : 1.f;
    if (a.renorm) div = warp_sum(part);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int j = lane + 32 * r;
        if (r < halves && j < a.k) {
            a.ids[(int64_t)t * a.k + j] = id[r];
            a.gates[(int64_t)t * a.k + j] = s[r] > 0.f ? s[r] / div * a.scale : 0.f;
        }
    }
    __syncwarp();  // out is written again for the next token
}

template <int PER, typename T, bool SCORES, bool GROUP>
__global__ void __launch_bounds__((GROUP ? route_group_warps(PER) : WARPS) * 32, GROUP ? 1 : PER <= 16 ? 4 : 3)
    route_kernel(const __grid_constant__ RouteArgs a, MoeWs ws, int* err) {
    // launched after the kernel that writes the logits, possibly early
    // (programmatic dependent launch): nothing is read before it completes
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    constexpr int NW = GROUP ? route_group_warps(PER) : WARPS;
    __shared__ Chosen chosen[NW];
    __shared__ __align__(16) float values[NW][32 * PER];
    const int warp = threadIdx.x >> 5;
    const Place p = place_of<PER>(a, threadIdx.x & 31);
    float bias[PER];  // of this lane's experts, whatever the token
#pragma unroll
    for (int i = 0; i < PER; ++i)  // a NaN puts its expert last
        bias[i] = SCORES && a.bias && p.there >> i & 1 ? fmaxf(a.bias[p.expert(i)], -INFINITY) : 0.f;
    for (int64_t t = (int64_t)blockIdx.x * NW + warp; t < a.T; t += (int64_t)gridDim.x * NW)
        route_one<PER, T, SCORES>(a, (int)t, p, bias, values[warp], chosen[warp]);
    if constexpr (GROUP) {
        __syncthreads();
        moe_group_block(a.ids, a.T * a.k, a.n_groups * a.group_size, ws, err);
    }
}

// The kernels of one type, by the experts of a lane (1, 2, 4, .. 32).
template <typename T, bool SCORES, bool GROUP>
RouteKernel kernel_of(int slot) {
    static constexpr RouteKernel kernels[6] = {
        route_kernel<1, T, SCORES, GROUP>, route_kernel<2, T, SCORES, GROUP>,  route_kernel<4, T, SCORES, GROUP>,
        route_kernel<8, T, SCORES, GROUP>, route_kernel<16, T, SCORES, GROUP>, route_kernel<32, T, SCORES, GROUP>};
    return kernels[slot];
}
template <typename T>
RouteKernel kernel_of(int slot, bool scores, bool group) {
    return group ? scores ? kernel_of<T, true, true>(slot) : kernel_of<T, false, true>(slot)
                 : scores ? kernel_of<T, true, false>(slot)
                          : kernel_of<T, false, false>(slot);
}

}  // namespace route
}  // namespace qmm
