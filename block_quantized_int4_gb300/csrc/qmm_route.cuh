// qmm_route.cuh -- routing to experts in general form: softmax or sigmoid
// scores, a bias that enters the choice alone, groups of experts, top-k,
// renormalised and scaled gates.
//
// The choice is that of the scores in 64 bits: c_e = s_e + b_e, the group
// scores, and equal values to the lower index.  Without a bias c is replaced
// by the logit (both scores are strictly increasing).  A warp takes a token;
// each lane holds PER consecutive experts of one group and an ordered 32-bit
// key of each:
//  - a logit's own order is exact in 32 bits; c and the sums of two are
//    computed in fp32, with a bound on their error.  Where two values whose
//    order decides anything are closer than that bound and not of equal
//    operands (about three tokens in a thousand of sigmoid scores with a bias,
//    256 experts), these are computed again as sums of two fp32 numbers, and
//    what these do not order either, in 64 bits (route_slow).  (All of the close
//    ones in 64 bits, at 16 cycles an instruction: 32003 tokens of 256 experts in
//    8 groups 44 us, with these 10 us the last of them.)
//  - the k-th largest of the 32 lanes' best keys bounds the k-th largest key
//    from below, so that only keys from there on are candidates: about 1.3 k
//    of them, one a lane, each ranked against all others.  (More than 32, as
//    with most experts switched off: route_slow, too.)
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

// Ordered keys.  An expert that takes no part has -inf; 0: taken or not there.
constexpr uint32_t KEY_OUT = 0x007FFFFFu;
__device__ __forceinline__ uint32_t key32(float v) {
    const int u = __float_as_int(v + 0.f);  // -0 as +0
    return (uint32_t)(u ^ ((u >> 31) | (int)0x80000000));
}
__device__ __forceinline__ float value32(uint32_t k) {
    return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}
__device__ __forceinline__ unsigned long long key64(double v) {
    const unsigned long long u = __double_as_longlong(v + 0.0);
    return max(u ^ ((u >> 63) ? ~0ull : 1ull << 63), 2ull);
}

// A warp's candidates and choice.
struct __align__(16) Chosen {
    uint32_t key[36];  // of candidates, then zeros up to a multiple of four
    int cand[32];
    int id[MAX_K];     // the chosen in order; one more where the border is checked
    float value[33];   // and their keys
    float2 pair[32];
};

// Where a lane's experts lie: `count` of them from `first` on.
struct Place {
    int first, count, lanes;  // lanes: of a group
};

__device__ __forceinline__ Place place_of(const RouteArgs& a, int lane) {
    Place p;
    p.lanes = 32 / a.n_groups;
    const int g = lane / p.lanes, at = (lane - g * p.lanes) * a.per;
    p.first = g * a.group_size + at;
    p.count = max(0, min(a.per, a.group_size - at));
    return p;
}

// A lane's logits as fp32; experts that take no part (-inf, NaN) as -inf.
template <int PER, typename T>
__device__ __forceinline__ void load_logits(const RouteArgs& a, const T* row, const Place& p, float (&l)[PER]) {
    constexpr int BYTES = PER * (int)sizeof(T), V = BYTES < 16 ? BYTES : 16, N = V / (int)sizeof(T);
    union Vec {
        T e[N];
        uint4 q;
        uint2 d;
        uint32_t w;
        unsigned short h;
    };
    if (a.vec && p.count == PER) {
#pragma unroll
        for (int i = 0; i < PER; i += N) {
            Vec v;
            const T* src = row + p.first + i;
            if constexpr (V == 16) v.q = *reinterpret_cast<const uint4*>(src);
            if constexpr (V == 8) v.d = *reinterpret_cast<const uint2*>(src);
            if constexpr (V == 4) v.w = *reinterpret_cast<const uint32_t*>(src);
            if constexpr (V == 2) v.h = *reinterpret_cast<const unsigned short*>(src);
#pragma unroll
            for (int j = 0; j < N; ++j) l[i + j] = as_float(v.e[j]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < PER; ++i) l[i] = i < p.count ? as_float(row[p.first + i]) : -INFINITY;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) l[i] = fmaxf(l[i], -INFINITY);  // of a NaN: -inf
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

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(FULL, v, o));
    return v;
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
            for (int i = 0; i < PER; ++i) c[i] += i < p.count ? (double)a.bias[p.first + i] : 0.0;
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
    const int g = (threadIdx.x & 31) / p.lanes;
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
    const Place p = place_of(a, lane);
    float l[PER];
    load_logits<PER, T>(a, row, p, l);
    double c[PER];
    const bool stays = groups64(a, p, l, c);
    unsigned long long key[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i)
        key[i] = stays && i < p.count ? l[i] > -INFINITY ? key64(a.bias ? c[i] : (double)l[i]) : 1ull : 0ull;
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
        const int owner = __ffs(__ballot_sync(FULL, best == most)) - 1;
        if (lane == owner) {
            out.id[j] = p.first + at;
            for (int i = 0; i < PER; ++i)
                if (i == at) key[i] = 0;
        }
    }
    __syncwarp();
}

// Experts of this lane in `mask` become candidates, in index order over the
// lanes; how many there are (more than 32: none is written).
__device__ __forceinline__ int collect(uint32_t mask, int first, const uint32_t* key, Chosen& out) {
    const int lane = threadIdx.x & 31, have = __popc(mask);
    int end = have;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(FULL, end, o);
        if (lane >= o) end += v;
    }
    const int total = __shfl_sync(FULL, end, 31);
    if (total > 32) return total;
    __syncwarp();
    for (int at = end - have; mask; ++at, mask &= mask - 1) {
        const int i = __ffs(mask) - 1;
        out.cand[at] = first + i;
        out.key[at] = key[i];
    }
    if (lane < 4) out.key[total + lane] = 0;
    __syncwarp();
    return total;
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
        for (int i = 0; i < p.count; ++i) top = fmaxf(top, as_float(row[p.first + i]));
        top = warp_max(top);
        if (!(top > -INFINITY)) return;
        Pair sum = {0.f, 0.f};
#pragma unroll 1
        for (int i = 0; i < p.count; ++i) sum = add(sum, power(as_float(row[p.first + i])));
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

__device__ __forceinline__ float distance(Pair a, Pair b) {
    return fabsf(__fadd_rn(__fadd_rn(a.hi, -b.hi), __fadd_rn(a.lo, -b.lo)));  // NaN of two -inf
}

// Whether the lane's group stays, where fp32 does not tell; `close`: pairs do
// not, either.  (Short loops: code that runs for few tokens comes from afar, and
// eight experts side by side took 15 us where these take 5.)
template <typename T>
__device__ __noinline__ bool groups_again(const RouteArgs& a, const T* row, bool& close) {
    const Place p = place_of(a, threadIdx.x & 31);
    const Scores s(a, row, p);
    Pair first = {-INFINITY, 0.f}, second = first;
#pragma unroll 1
    for (int i = 0; i < p.count; ++i) {
        const Pair v = s.of(a, as_float(row[p.first + i]), a.bias ? a.bias[p.first + i] : 0.f);
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
    const int g = (threadIdx.x & 31) / p.lanes;
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
        near |= other && distance(v, mine) <= tolerance;
    }
    close = __any_sync(FULL, near);
    return in;
}

// The order of the candidates, each as a pair on a lane of its own, where fp32
// does not tell (all that may be among the k largest are there); false: pairs do
// not, either.
template <typename T>
__device__ __noinline__ bool order_again(const RouteArgs& a, const T* row, int total, Chosen& out) {
    const int lane = threadIdx.x & 31;
    const Scores s(a, row, place_of(a, lane));
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
        rank += before(v, mine) || (!before(mine, v) && d < lane);
        const float l_d = __shfl_sync(FULL, l, d), bias_d = __shfl_sync(FULL, bias, d);
        const bool same = l_d == l && bias_d == bias;
        near |= !same && distance(v, mine) <= s.tolerance(fabsf(mine.hi));
    }
    if (lane < total && rank < a.k) out.id[rank] = e;
    __syncwarp();
    return !__any_sync(FULL, near && lane < total && rank < a.k);
}

// One token.  SCORES: the choice takes scores (a bias, or groups by the sum of
// two), not logits alone.  keys: 32 * PER words of shared memory.
template <int PER, typename T, bool SCORES>
__device__ __forceinline__ void route_one(const RouteArgs& a, int t, const Place& p, const float (&bias)[PER],
                                          uint32_t* keys, Chosen& out) {
    const int lane = threadIdx.x & 31;
    const T* row = static_cast<const T*>(a.logits) + (int64_t)t * a.ld;
    const bool grouped = a.n_groups > 1, top2 = grouped && a.top2;
    float l[PER];
    load_logits<PER, T>(a, row, p, l);

    // softmax: the largest logit and the sum of exponentials
    float top = 0.f, sum = 1.f;
    if (a.softmax && (SCORES || !a.renorm)) {
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

    // keys; and the error that c and group scores may have.  Exponentials and
    // reciprocals are off by 2^-21 of the largest score at most (an exponent's
    // rounding, |x| 2^-24, weighs s or s (1 - s), below 0.4 / |x|), softmax by
    // the sum's own error besides; c by its own rounding.
    const float unit = a.softmax && SCORES ? rcp(sum) : 1.f, slack = unit * (a.softmax ? 0x1p-18f : 0x1p-19f);
    uint32_t key[PER];
    float first = -INFINITY, second = -INFINITY;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        float c = l[i];
        if constexpr (SCORES) {
            const float e = ex2((a.softmax ? l[i] - top : -l[i]) * 1.4426950408889634f);
            float v = a.softmax ? e * unit : rcp(1.f + e);
            v += bias[i];
            v = l[i] > -INFINITY ? fmaxf(v, -INFINITY) : -INFINITY;
            if (a.bias) c = v;
            if (top2) second = fmaxf(second, fminf(first, v));
            first = fmaxf(first, v);
        }
        key[i] = key32(c);
    }
    uint32_t best = key[0];
#pragma unroll
    for (int i = 1; i < PER; ++i) best = max(best, key[i]);
    bool stays = p.count > 0, again = false;
    if (grouped) {
        if constexpr (!SCORES) first = p.count > 0 ? value32(best) : -INFINITY;
        for (int o = p.lanes >> 1; o > 0; o >>= 1) {
            const float f = __shfl_xor_sync(FULL, first, o);
            if (top2) {
                const float s = __shfl_xor_sync(FULL, second, o);
                second = fmaxf(fminf(first, f), fmaxf(second, s));
            }
            first = fmaxf(first, f);
        }
        const float mine = top2 && second > -INFINITY ? first + second : first;
        const int g = lane / p.lanes;
        int before = 0;
#pragma unroll 1
        for (int h = 0; h < a.n_groups; ++h) {
            const float v = __shfl_sync(FULL, mine, h * p.lanes);
            before += v > mine || (v == mine && h < g);
        }
        bool in = before < a.top_groups;
        if constexpr (SCORES) {
            // groups on either side of the border that are too close
            const float hi = value32(__reduce_min_sync(FULL, in ? key32(mine) : 0xFFFFFFFFu));
            const uint32_t no = __reduce_max_sync(FULL, in ? 0u : key32(mine));
            const float lo = no ? value32(no) : -INFINITY;
            const float size = first > -INFINITY ? fabsf(first) + (second > -INFINITY ? fabsf(second) : 0.f) : 0.f;
            if (lo > -INFINITY && !(hi - lo > 4.f * slack + 0x1p-21f * warp_max(size)))
                in = groups_again(a, row, again);
        }
        stays = stays && in;
    }

    // candidates: keys from the n-th best of the lanes' best on (n = k, and one
    // more where the border is checked)
    const int n = a.k + (SCORES && a.bias ? 1 : 0);
    const uint32_t there = !stays ? 0u : PER == 32 && p.count == 32 ? 0xFFFFFFFFu : (1u << p.count) - 1u;
#pragma unroll
    for (int i = 0; i < PER; i += PER < 4 ? PER : 4) {
        if constexpr (PER >= 4)
            *reinterpret_cast<uint4*>(keys + lane * PER + i) = make_uint4(key[i], key[i + 1], key[i + 2], key[i + 3]);
        else if constexpr (PER == 2)
            *reinterpret_cast<uint2*>(keys + lane * PER) = make_uint2(key[0], key[1]);
        else
            keys[lane] = key[0];
    }
    const auto from = [&](uint32_t floor_key) {
        uint32_t mask = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) mask |= (key[i] >= floor_key ? 1u : 0u) << i;
        return collect(mask & there, p.first, keys + lane * PER, out);
    };
    uint32_t floor_key = KEY_OUT;
    if (n <= 32) {
        // the smallest of those that fewer than n are larger than
        const uint32_t mine = stays ? best : 0u;
        out.key[lane] = mine;
        __syncwarp();
        int larger = 0;
#pragma unroll
        for (int d = 0; d < 32; d += 4) {
            const uint4 v = *reinterpret_cast<const uint4*>(out.key + d);
            larger += (v.x > mine) + (v.y > mine) + (v.z > mine) + (v.w > mine);
        }
        floor_key = max(__reduce_min_sync(FULL, larger < n ? mine : 0xFFFFFFFFu), KEY_OUT);
    }
    int total = from(floor_key);
    again = again || total > 32;
    if (!again) {
        // candidates lie in index order: of equal keys the earlier ranks first
        const uint32_t mine = lane < total ? out.key[lane] : 0u;
        int rank = 0;
        for (int d = 0; d < total; d += 4) {
            const uint4 v = *reinterpret_cast<const uint4*>(out.key + d);
            rank += (v.x >= mine + (d >= lane)) + (v.y >= mine + (d + 1 >= lane)) + (v.z >= mine + (d + 2 >= lane)) +
                    (v.w >= mine + (d + 3 >= lane));
        }
        if (lane < total && rank < n) {
            out.id[rank] = out.cand[lane];
            if (SCORES && a.bias) out.value[rank] = value32(mine);
        }
        __syncwarp();
        if (SCORES && a.bias) {
            // neighbours that are too close, but for equal logits with equal biases
            // among the chosen (at the border a third may be close to both)
            bool close = false;
            if (lane < min(total, n) - 1) {
                const float hi = out.value[lane], lo = out.value[lane + 1];
                if (lo > -INFINITY && !(hi - lo > 2.f * slack + 0x1p-22f * (fabsf(hi) + fabsf(lo)))) {
                    close = true;
                    if (lane + 1 < a.k) {
                        const int e = out.id[lane], f = out.id[lane + 1];
                        close = !(as_float(row[e]) == as_float(row[f]) && a.bias[e] == a.bias[f]);
                    }
                }
            }
            if (__any_sync(FULL, close)) {
                // all that may be among the k largest, as pairs
                const float kth = out.value[a.k - 1];
                total = from(max(KEY_OUT, key32(kth - (2.f * slack + 0x1p-21f * fabsf(kth)))));
                again = total > 32 || !order_again(a, row, total, out);
            }
        }
    }
    if (again) route_slow<PER, T>(a, row, out);

    // gates of the chosen: lane j has the j-th and the (j + 32)-th
    float lj[2], s[2];
    int id[2];
    float most = -INFINITY;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
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
        s[r] = lj[r] > -INFINITY ? (exps ? expf(lj[r] - ref) : 1.f / (1.f + expf(-lj[r]))) : 0.f;
        part += s[r];
    }
    float div = a.softmax ? sum : 1.f;
    if (a.renorm) div = warp_sum(part);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int j = lane + 32 * r;
        if (j < a.k) {
            a.ids[(int64_t)t * a.k + j] = id[r];
            a.gates[(int64_t)t * a.k + j] = s[r] > 0.f ? s[r] / div * a.scale : 0.f;
        }
    }
    __syncwarp();  // out is written again for the next token
}

template <int PER, typename T, bool SCORES, bool GROUP>
__global__ void __launch_bounds__((GROUP ? route_group_warps(PER) : WARPS) * 32, GROUP ? 1 : PER <= 16 ? 4 : 3) route_kernel(const __grid_constant__ RouteArgs a, MoeWs ws,
                                                                                           int* err) {
    // launched after the kernel that writes the logits, possibly early
    // (programmatic dependent launch): nothing is read before it completes
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    constexpr int NW = GROUP ? route_group_warps(PER) : WARPS;
    __shared__ Chosen chosen[NW];
    __shared__ __align__(16) uint32_t keys[NW][32 * PER];
    const int warp = threadIdx.x >> 5;
    const Place p = place_of(a, threadIdx.x & 31);
    float bias[PER];  // of this lane's experts, whatever the token
#pragma unroll
    for (int i = 0; i < PER; ++i) bias[i] = SCORES && a.bias && i < p.count ? a.bias[p.first + i] : 0.f;
    for (int64_t t = (int64_t)blockIdx.x * NW + warp; t < a.T; t += (int64_t)gridDim.x * NW)
        route_one<PER, T, SCORES>(a, (int)t, p, bias, keys[warp], chosen[warp]);
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
