// route.cu -- routing of tokens to experts: the choice of k experts for each token, their weights, and the
// order of the chosen rows by expert; and the gradient of the logits.
//
// With l the logits of a token, s = softmax(l) or 1 / (1 + e^-l), b the bias:
//   c = s + b, or l where there is no bias (s rises with l)
//   group score = c_1 [+ c_2], the largest of the group; the top_groups best groups stay
//   the k largest c of what stays, the lowest index first among equals
//   w = scale * s, renormalised: scale * s / (sum of s over the chosen)
// Renormalised weights come from the chosen logits alone and cannot underflow together: for softmax
// e^(l - max) / sum, for the sigmoid e^(min(l, 0) - max) / (1 + e^-|l|) / sum, the maxima over the chosen.
//
// A warp takes a token.  Its lanes hold the experts in ascending order, a group on a power of two of lanes
// (32 / groups), so that what is reduced within a group stays within neighbouring lanes and a lower lane holds lower
// indices.  The k-th largest of the lanes' largest values bounds the k-th largest of all from below: what is not under it (a dozen
// of 256 for k = 8) is gathered, one candidate a lane, and each candidate's place is the number of those before it.  That is a
// third of the instructions of k rounds of "largest of all, then remove it", which bounded the kernel.
//
// The choice is that of the definition in fp64.  Where c is the logit itself its order is exact.  Otherwise c
// is evaluated in fp32 (the error bound stands at kTauSigmoid), and where two neighbours in the order lie closer than the bound
// the candidates near it are compared in fp64 (about 1 token in 1000 of 256 experts with sigmoid scores), as are groups whose
// scores are too close (groups_slow).  More than 32 candidates are looked through one by one, in fp64 (choose_slow): many equal
// values, or more wanted than the lanes that stay give to the bound (one value each, with groups two).  Random logits, 16384
// tokens: 256 experts 21 us with k = 8, 112 with 20 (17 % of the tokens), 203 with 24 (91 %), 269 with 32 (all); 512 experts
// with k = 8 55 us in the 4 best of 8 groups, 221 in the best one (4 lanes: all).
//
// Rows: a warp takes neighbouring tokens and counts each expert's choices as it goes, so that a choice's rank
// among the warp's is there at once; the ranks are joined over the block's warps, and over the blocks by a
// second kernel, which reads every block's counts.  No atomics on memory: the order is that of the tokens.
// One block does it all for few tokens.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cfloat>
#include <cstdint>

#include "nvfp4_device.cuh"
#include "nvfp4_internal.h"
#include "sm100_ptx.cuh"

namespace nvfp4 {

constexpr uint32_t kAll = 0xFFFFFFFFu;
constexpr float kNone = -INFINITY;   // an expert that may not be chosen

// Two values of c that differ by no more than tau + |c| * kTauC may be out of order in fp32.
// Sigmoid: __expf errs by 2 + 1.173 |l| ulp, which enters s with a factor s (1 - s) (0.8 ulp of 1 at most, as
// |l| s (1 - s) < 0.23), the sum and the quotient by 3 ulp of s: 3.8 * 2^-23 for one value, less than 2^-20 for
// two.  Softmax: a term errs by s (4 + 1.173 |l - max|) ulp; the error of the sum is common to all, at most
// 50 ulp of it (37 adds of a lane and the lanes, and the terms' errors), and enters the difference of two c with a factor |s - s'|: together
// less than 2^-16 of the largest s.  Adding the bias errs by half an ulp of c each.
constexpr float kTauSigmoid = 1.9073486e-6f;   // 2^-19
constexpr float kTauSoftmax = 1.5258789e-5f;   // 2^-16, times the largest s
constexpr float kTauC = 4.7683716e-7f;         // 2^-21

struct RouteKernelParams {
    RouteProblem r;
    int32_t size;        // experts per group
    int32_t lanes_log2;  // lanes of a group, a power of two
    int32_t per_lane;    // experts of a lane
    int32_t vec;         // a lane's logits can be read 16 bytes at a time
    int32_t block_tokens, warp_tokens;
    int32_t stride;      // of the warps' counts: odd
    int32_t held;        // choices that shared memory keeps, 0: they are read back from rows and chosen
};

__device__ __forceinline__ uint32_t order_key(float c) {   // ascends with c; 0 for none
    const uint32_t b = __float_as_uint(c);
    return c > kNone ? b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u) : 0u;   // NaN too is none
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return k ? __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k) : kNone;
}
// a logit as it counts: NaN is none, what is above the largest number is that number, -0 is 0
__device__ __forceinline__ float logit_of(float v) { return v == v ? fminf(v, FLT_MAX) + 0.0f : kNone; }

template <typename T>
__device__ __forceinline__ float raw_logit(const T* row, int e) {
    if constexpr (sizeof(T) == 2) return __uint_as_float((uint32_t)__ldg(row + e) << 16);
    else return __ldg(row + e);
}

// The two largest of a and of b, merged
template <typename F>
__device__ __forceinline__ void merge_top2(F& a1, F& a2, F b1, F b2) {
    const F lo = a1 < b1 ? a1 : b1, hi = a1 < b1 ? b1 : a1, second = a2 < b2 ? b2 : a2;
    a1 = hi;
    a2 = lo < second ? second : lo;
}
// Whether the group of this lane is among the top_groups best, the lowest index first among equals
template <typename F>
__device__ __forceinline__ bool group_stays(F score, const RouteKernelParams& p, int lane) {
    const int g = lane >> p.lanes_log2;
    int before = 0;
#pragma unroll 4
    for (int i = 0; i < p.r.groups; ++i) {
        const F other = __shfl_sync(kAll, score, i << p.lanes_log2);
        before += i < g ? other >= score : other > score;
    }
    return before < p.r.top_groups && score > (F)kNone && g < p.r.groups;
}

// c in fp64; the softmax's largest logit and sum
__device__ __forceinline__ double value64(const RouteKernelParams& p, float l, int e, float top, double sum) {
    if (!(l > kNone)) return (double)kNone;
    const double s = p.r.sigmoid ? 1.0 / (1.0 + exp(-(double)l)) : exp((double)l - (double)top) / sum;
    const double c = p.r.bias ? s + (double)__ldg(p.r.bias + e) : s;
    return c == c ? c : (double)kNone;
}
template <typename T>
__device__ __noinline__ double sum64(const RouteKernelParams& p, const T* row, float top) {
    double part = 0.0;
    for (int e = threadIdx.x & 31; e < p.r.experts; e += 32) {
        const float l = logit_of(raw_logit(row, e));
        if (l > kNone) part += exp((double)l - (double)top);
    }
    for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(kAll, part, o);
    return part;
}

// The groups' choice in fp64
template <typename T>
__device__ __noinline__ bool groups_slow(const RouteKernelParams& p, const T* row, float top) {
    const int lane = threadIdx.x & 31, g = lane >> p.lanes_log2, first = (lane & ((1 << p.lanes_log2) - 1)) * p.per_lane;
    const int count = g < p.r.groups ? max(0, min(p.per_lane, p.size - first)) : 0, e0 = g * p.size + first;
    const double sum = p.r.sigmoid ? 1.0 : sum64(p, row, top);
    double a1 = kNone, a2 = kNone;
    for (int i = 0; i < count; ++i) merge_top2(a1, a2, value64(p, logit_of(raw_logit(row, e0 + i)), e0 + i, top, sum), (double)kNone);
    for (int o = 1; o < 1 << p.lanes_log2; o <<= 1) merge_top2(a1, a2, __shfl_xor_sync(kAll, a1, o), __shfl_xor_sync(kAll, a2, o));
    return group_stays(p.r.group_top == 2 ? a1 + a2 : a1, p, lane);
}

// The experts' choice in fp64 within the groups that stay: lane j returns the j-th expert, or -1
template <int VMAX, typename T>
__device__ __noinline__ int choose_slow(const RouteKernelParams& p, const T* row, float top, bool stays) {
    const int lane = threadIdx.x & 31, g = lane >> p.lanes_log2, first = (lane & ((1 << p.lanes_log2) - 1)) * p.per_lane;
    const int count = stays ? max(0, min(p.per_lane, p.size - first)) : 0, e0 = g * p.size + first;
    const double sum = p.r.sigmoid || !p.r.bias ? 1.0 : sum64(p, row, top);
    double c[VMAX];
    for (int i = 0; i < count; ++i) {
        const float l = logit_of(raw_logit(row, e0 + i));
        c[i] = p.r.bias ? value64(p, l, e0 + i, top, sum) : (double)l;
    }
    int mine = -1, last_e = -1;
    double last = INFINITY;
    for (int j = 0; j < p.r.k; ++j) {   // what comes next in order behind the one before
        double best = kNone;
        int at = -1;
        for (int i = 0; i < count; ++i) {
            const int e = e0 + i;
            if ((c[i] < last || (c[i] == last && e > last_e)) && c[i] > best) {
                best = c[i];
                at = e;
            }
        }
        for (int o = 16; o > 0; o >>= 1) {
            const double b = __shfl_xor_sync(kAll, best, o);
            const int e = __shfl_xor_sync(kAll, at, o);
            if (e >= 0 && (at < 0 || b > best || (b == best && e < at))) {
                best = b;
                at = e;
            }
        }
        if (at < 0) break;
        if (lane == j) mine = at;
        last = best;
        last_e = at;
    }
    return mine;
}

// One candidate a lane, the first `count` lanes, in ascending order of their indices: the place of each in descending
// order of c, the lowest index first among equals
template <typename F>
__device__ __forceinline__ int place_of(F c, int count, int lane) {
    int before = 0;
#pragma unroll 4
    for (int i = 0; i < count; ++i) before += __shfl_sync(kAll, c, i) > c;
    // equals have come to one place
    return before + __popc(__match_any_sync(kAll, lane < count ? before : 64) & ((1u << lane) - 1u));
}
template <typename T>
__device__ __noinline__ int places_slow(const RouteKernelParams& p, const T* row, int e, float top, int count) {
    const double sum = p.r.sigmoid ? 1.0 : sum64(p, row, top);
    const int lane = threadIdx.x & 31;
    return place_of(lane < count ? value64(p, logit_of(raw_logit(row, e)), e, top, sum) : (double)kNone, count, lane);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}
__device__ __forceinline__ float warp_max(float v) {
    return key_value(__reduce_max_sync(kAll, order_key(v)));
}

// The weights of the chosen: lane j's expert has logit l (none: kNone).  `top` and `sum` are the softmax's.
__device__ __forceinline__ float chosen_weight(const RouteProblem& r, float l, float top, float sum) {
    const bool held = l > kNone;
    if (!r.renormalize) {
        if (!held) return 0.0f;
        return r.scale * (r.sigmoid ? 1.0f / (1.0f + expf(-l)) : expf(l - top) / sum);
    }
    const float z = r.sigmoid ? fminf(l, 0.0f) : l;
    const float most = warp_max(held ? z : kNone);
    float v = held ? expf(z - most) : 0.0f;
    if (r.sigmoid && held) v /= 1.0f + expf(-fabsf(l));
    const float all = warp_sum(v);
    return held ? r.scale * __fdividef(v, all) : 0.0f;   // all: 0.5 to 32 (a sigmoid's largest term is 1 / (1 + e^-|l|))
}

struct RouteWarp {       // a warp's candidates, then the same in order: c, the expert
    float2 found[32], sorted[32];
};

// VMAX: experts of a lane at most; T: the logits' type.  WARPS: at most
template <int VMAX, int WARPS, typename T>
__global__ void __launch_bounds__(32 * WARPS) route_choose_kernel(const __grid_constant__ RouteKernelParams p) {
    extern __shared__ int32_t smem[];
    __shared__ RouteWarp scratch[WARPS];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int k = p.r.k, E = p.r.experts;
    int32_t* counts = smem;                               // [warps][stride]
    int32_t* base = smem + warps * p.stride;              // [experts + 1]: one block's offsets
    uint32_t* held = reinterpret_cast<uint32_t*>(base + E + 1);   // rank << 11 | expert + 1 of the block's choices
    RouteWarp& own = scratch[warp];
    for (int i = threadIdx.x; i < warps * p.stride; i += blockDim.x) counts[i] = 0;
    ptx::griddep_launch();
    const int t0 = blockIdx.x * p.block_tokens, t1 = min(p.r.tokens, t0 + p.block_tokens);
    const int g = lane >> p.lanes_log2, first = (lane & ((1 << p.lanes_log2) - 1)) * p.per_lane, e0 = g * p.size + first;
    const int count = g < p.r.groups ? max(0, min(p.per_lane, p.size - first)) : 0;
    const bool by_logit = !p.r.bias;
    const bool scores = !by_logit || (p.r.groups > 1 && p.r.group_top == 2);
    const bool soft = !p.r.sigmoid && (scores || !p.r.renormalize);
    bool odd = false;
    int32_t* mine_counts = counts + warp * p.stride;
    // the bias, -inf for what is none whatever its logit
    const auto bias_of = [&](int i) {
        float b = i < count ? 0.0f : kNone;
        if (p.r.bias && i < count) b = __ldg(p.r.bias + e0 + i);
        return b == b ? b : kNone;
    };
    float bias[VMAX <= 8 ? VMAX : 1];
    if constexpr (VMAX <= 8) {
#pragma unroll
        for (int i = 0; i < VMAX; ++i) bias[i] = bias_of(i);
    }
    const auto load = [&](int t, float (&l)[VMAX]) {   // places without an expert: -inf
        const T* row = reinterpret_cast<const T*>(p.r.logits) + (int64_t)t * p.r.ld;
        if (p.vec) {
            constexpr int per = 16 / (int)sizeof(T);
            constexpr uint32_t none = sizeof(T) == 4 ? 0xFF800000u : 0xFF80FF80u;
#pragma unroll
            for (int i = 0; i < VMAX; i += per) {
                uint4 v = make_uint4(none, none, none, none);
                if (i < count) v = __ldg(reinterpret_cast<const uint4*>(row + e0 + i));
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int j = 0; j < per && i + j < VMAX; ++j)
                    l[i + j] = sizeof(T) == 4 ? __uint_as_float(w[j & 3]) : (j & 1 ? bf16_hi(w[(j >> 1) & 3]) : bf16_lo(w[(j >> 1) & 3]));
            }
        } else {
#pragma unroll
            for (int i = 0; i < VMAX; ++i) l[i] = i < count ? raw_logit(row, e0 + i) : kNone;
        }
    };
    const int w1 = min(t1, t0 + (warp + 1) * p.warp_tokens);
    int t = t0 + warp * p.warp_tokens;
    float next[VMAX <= 8 ? VMAX : 1];   // the next token's logits, on their way
    if constexpr (VMAX <= 8) {
        if (t < w1) load(t, next);
    }
    __syncthreads();
    for (; t < w1; ++t) {
        float l[VMAX];
        if constexpr (VMAX <= 8) {
#pragma unroll
            for (int i = 0; i < VMAX; ++i) l[i] = next[i];
            if (t + 1 < w1) load(t + 1, next);
        } else {
            load(t, l);
        }
        int mine = -1;
        float weight = 0.0f;
        if (!p.r.valid || __ldg(p.r.valid + t)) {
            const T* row = reinterpret_cast<const T*>(p.r.logits) + (int64_t)t * p.r.ld;
            bool strange = false;   // NaN or an infinity, here where there is no expert too
#pragma unroll
            for (int i = 0; i < VMAX; ++i) strange |= !(fabsf(l[i]) <= FLT_MAX);
            if (strange) {
#pragma unroll
                for (int i = 0; i < VMAX; ++i) {
                    odd |= !(l[i] <= FLT_MAX);
                    l[i] = logit_of(l[i]);
                }
            }
            float top = 0.0f, sum = 1.0f;
            if (soft) {
                top = kNone;
#pragma unroll
                for (int i = 0; i < VMAX; ++i) top = fmaxf(top, l[i]);
                top = warp_max(top);
                if (!(top > kNone)) top = 0.0f;   // no expert at all
                sum = 0.0f;
#pragma unroll
                for (int i = 0; i < VMAX; ++i) sum += __expf(l[i] - top);
                sum = warp_sum(sum);
            }
            // c, and the lane's largest two
            float c[VMAX];
            const float tau = p.r.sigmoid ? kTauSigmoid : kTauSoftmax / sum;
            if (scores) {
                const float per_sum = 1.0f / sum;
                const auto bias_at = [&](int i) { return VMAX <= 8 ? bias[VMAX <= 8 ? i : 0] : bias_of(i); };
                if (p.r.sigmoid) {
#pragma unroll
                    for (int i = 0; i < VMAX; ++i) c[i] = __fdividef(1.0f, 1.0f + __expf(-l[i])) + bias_at(i);
                } else {
#pragma unroll
                    for (int i = 0; i < VMAX; ++i) c[i] = fmaf(__expf(l[i] - top), per_sum, bias_at(i));
                }
                if (strange) {
#pragma unroll
                    for (int i = 0; i < VMAX; ++i) c[i] = l[i] > kNone && c[i] == c[i] ? c[i] : kNone;
                }
            } else {
#pragma unroll
                for (int i = 0; i < VMAX; ++i) c[i] = l[i];
            }
            bool stays = g < p.r.groups;
            float a1 = kNone, a2 = kNone;
            if (p.r.groups > 1) {
#pragma unroll
                for (int i = 0; i < VMAX; ++i) {
                    a2 = fmaxf(a2, fminf(a1, c[i]));
                    a1 = fmaxf(a1, c[i]);
                }
                float b1 = a1, b2 = a2;
                for (int o = 1; o < 1 << p.lanes_log2; o <<= 1) {
                    const float d1 = __shfl_xor_sync(kAll, b1, o), d2 = __shfl_xor_sync(kAll, b2, o);
                    b2 = fmaxf(fminf(b1, d1), fmaxf(b2, d2));
                    b1 = fmaxf(b1, d1);
                }
                // a sum of two that are no less than the lowest number is above -inf: it is held there, where groups are as close as can be
                const float score = p.r.group_top == 1 ? b1 : b2 > kNone ? fmaxf(b1 + b2, -FLT_MAX) : kNone;
                stays = group_stays(score, p, lane);
                if (scores) {
                    // what a score may err by: a sum of two by both and by its rounding, relative to the larger of them, since they may cancel
                    const float err = p.r.group_top == 1 ? 0.5f * tau + kTauC * fabsf(b1) : tau + kTauC * fmaxf(fabsf(b1), fabsf(b2));
                    const uint32_t least = __reduce_min_sync(kAll, stays ? order_key(score - err) : kAll);
                    const uint32_t most = __reduce_max_sync(kAll, stays || g >= p.r.groups ? 0u : order_key(score + err));
                    if (most && least != kAll && !(key_value(least) > key_value(most))) stays = groups_slow(p, row, top);
                }
                if (by_logit && scores) {   // the groups went by scores, the experts go by logits
                    a1 = a2 = kNone;
#pragma unroll
                    for (int i = 0; i < VMAX; ++i) {
                        c[i] = l[i];
                        a2 = fmaxf(a2, fminf(a1, c[i]));
                        a1 = fmaxf(a1, c[i]);
                    }
                }
                if (!stays) a1 = a2 = kNone;
            } else {
#pragma unroll
                for (int i = 0; i < VMAX; ++i) a1 = fmaxf(a1, c[i]);
            }
            // a bound that as many values reach as are wanted: k, and where c has errors one more, to see its distance
            const int wanted = by_logit ? k : k + 1;
            uint32_t x = order_key(a1), y = p.r.groups > 1 ? order_key(a2) : 0u, bound = 0;
#pragma unroll 4
            for (int j = 0; j < wanted; ++j) {   // 0: fewer than that, so all that there are
                bound = __reduce_max_sync(kAll, x);
                if (x == bound) {
                    x = y;
                    y = 0;
                }
            }
            float at_least = bound ? key_value(bound) : -FLT_MAX;
            int all = 0;
            const auto gather = [&]() {   // what reaches at_least, one a lane, in ascending order of the experts
                int n = 0;
                const float least = stays ? at_least : __int_as_float(0x7FC00000);   // NaN: nothing reaches it
#pragma unroll
                for (int i = 0; i < VMAX; ++i) n += c[i] >= least;
                int before = n;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int u = __shfl_up_sync(kAll, before, o);
                    if (lane >= o) before += u;
                }
                all = __shfl_sync(kAll, before, 31);
                if (all > 32) return make_float2(kNone, 0.0f);
                float2* to = own.found + (before - n);
#pragma unroll
                for (int i = 0; i < VMAX; ++i)
                    if (c[i] >= least) *to++ = make_float2(c[i], __int_as_float(e0 + i));
                __syncwarp();
                return lane < all ? own.found[lane] : make_float2(kNone, 0.0f);
            };
            float2 found = gather();
            float logit = kNone;
            if (all <= 32) {
                int place = place_of(found.x, all, lane);
                if (lane < all) own.sorted[place] = found;
                __syncwarp();
                float2 at = own.sorted[lane];
                if (!by_logit) {
                    const float2 behind = own.sorted[min(lane + 1, 31)];
                    const int e1 = __float_as_int(at.y), e2 = __float_as_int(behind.y);
                    bool close = lane < k && lane + 1 < all && !(at.x - behind.x > tau + kTauC * fabsf(at.x));
                    // the same logit and bias give the same c, and the lower index came first
                    if (close && lane + 1 < k) close = raw_logit(row, e1) != raw_logit(row, e2) || __ldg(p.r.bias + e1) != __ldg(p.r.bias + e2);
                    if (__any_sync(kAll, close)) {
                        // all that may be among the first k, compared in fp64
                        const float last = own.sorted[min(k, all) - 1].x;
                        // (next to the lowest number the difference is -inf, which places without an expert and experts that may
                        // not be chosen would reach too)
                        at_least = fmaxf(fminf(at_least, last - 2.0f * (tau + kTauC * fabsf(last))), -FLT_MAX);
                        __syncwarp();
                        found = gather();
                        if (all <= 32) {
                            place = places_slow(p, row, __float_as_int(found.y), top, all);
                            if (lane < all) own.sorted[place] = found;
                            __syncwarp();
                            at = own.sorted[lane];
                        }
                    }
                }
                if (all <= 32 && lane < k && lane < all) {
                    mine = __float_as_int(at.y);
                    logit = by_logit ? at.x : logit_of(raw_logit(row, mine));
                }
                __syncwarp();
            }
            if (all > 32) {
                mine = choose_slow<VMAX>(p, row, top, stays);
                logit = mine >= 0 ? logit_of(raw_logit(row, mine)) : kNone;
            }
            weight = chosen_weight(p.r, logit, top, sum);
        }
        int rank = 0;
        if (mine >= 0) rank = mine_counts[mine]++;   // a token's experts differ
        __syncwarp();
        if (lane < k) {
            const int64_t at = (int64_t)t * k + lane;
            p.r.chosen[at] = mine;
            p.r.weights[at] = weight;
            if (p.held) held[(t - t0) * k + lane] = (uint32_t)rank << 11 | (uint32_t)(mine + 1);
            else p.r.rows[at] = rank;
        }
    }
    if (__any_sync(kAll, odd) && lane == 0) atomicOr(p.r.flags, kFlagNonFinite);
    __syncthreads();
    // ranks within the block: the warps before
    const bool alone = gridDim.x == 1;
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
        int before = 0;
#pragma unroll 8
        for (int w = 0; w < warps; ++w) {
            const int c = counts[w * p.stride + e];
            counts[w * p.stride + e] = before;
            before += c;
        }
        if (alone) base[e] = before;
        else p.r.scratch[blockIdx.x * route_count_stride(E) + e] = before;
    }
    __syncthreads();
    if (alone) {
        if (warp == 0) {   // the offsets: lane by lane a run of experts
            const int per = (E + 31) / 32, lo = min(E, lane * per), hi = min(E, lo + per);
            int sum = 0;
            for (int e = lo; e < hi; ++e) sum += base[e];
            int before = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(kAll, before, o);
                if (lane >= o) before += u;
            }
            before -= sum;
            for (int e = lo; e < hi; ++e) {
                const int c = base[e];
                base[e] = before;
                p.r.offsets[e] = before;
                before += c;
            }
            if (lane == 31) {
                base[E] = before;
                p.r.offsets[E] = before;
            }
        }
        __syncthreads();
    }
    const int64_t c0 = (int64_t)t0 * k;
    const int choices = max(0, t1 - t0) * k, per_warp = k * p.warp_tokens;   // of a block: less than 2^30
    for (int i = threadIdx.x; i < choices; i += blockDim.x) {
        const uint32_t h = p.held ? held[i] : 0u;
        const int e = p.held ? (int)(h & 2047u) - 1 : p.r.chosen[c0 + i];
        int row = -1;
        if (e >= 0) {
            row = (p.held ? (int)(h >> 11) : p.r.rows[c0 + i]) + counts[(int)((uint32_t)i / (uint32_t)per_warp) * p.stride + e];
            if (alone) {
                row += base[e];
                p.r.sources[row] = (int32_t)(c0 + i);
            }
        }
        p.r.rows[c0 + i] = row;
    }
    if (alone)
        for (int i = base[E] + threadIdx.x; i < choices; i += blockDim.x) p.r.sources[i] = -1;
}

constexpr int kPlaceThreads = 1024;

// The blocks' counts joined: each block's first row of every expert, and with it the rows of its choices
__global__ void __launch_bounds__(kPlaceThreads) route_place_kernel(const RouteKernelParams p, int blocks) {
    __shared__ int32_t total[kMaxExperts + 1], before[kMaxExperts];
    const int E = p.r.experts, k = p.r.k, lane = threadIdx.x & 31;
    for (int e = threadIdx.x; e < E; e += kPlaceThreads) total[e] = before[e] = 0;
    __syncthreads();
    ptx::griddep_wait();
    const int t0 = blockIdx.x * p.block_tokens, t1 = min(p.r.tokens, t0 + p.block_tokens);
    const int64_t c0 = (int64_t)t0 * k + threadIdx.x, c1 = (int64_t)t1 * k;
    // the block's first choices are on their way during the sums
    const int chosen0 = c0 < c1 ? __ldcg(p.r.chosen + c0) : -1, rank0 = c0 < c1 ? __ldcg(p.r.rows + c0) : 0;
    // four experts of every parts-th block a thread
    int wide = 8, shift = 3;
    while (4 * wide < E) {
        wide <<= 1;
        ++shift;
    }
    const int e = 4 * (threadIdx.x & (wide - 1)), parts = kPlaceThreads >> shift;
    if (e < E) {
        int4 all = make_int4(0, 0, 0, 0), prior = all;
#pragma unroll 10
        for (int b = threadIdx.x >> shift; b < blocks; b += parts) {
            const int4 c = __ldcg(reinterpret_cast<const int4*>(p.r.scratch + b * route_count_stride(E) + e));
            const int m = b < (int)blockIdx.x ? -1 : 0;
            all.x += c.x; all.y += c.y; all.z += c.z; all.w += c.w;
            prior.x += c.x & m; prior.y += c.y & m; prior.z += c.z & m; prior.w += c.w & m;
        }
        const int a4[4] = {all.x, all.y, all.z, all.w}, p4[4] = {prior.x, prior.y, prior.z, prior.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (e + i >= E) break;            // what a row of counts has behind the last expert is nobody's
            atomicAdd(&total[e + i], a4[i]);  // whole numbers: no order to depend on
            atomicAdd(&before[e + i], p4[i]);
        }
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        const int per = (E + 31) / 32, lo = min(E, lane * per), hi = min(E, lo + per);
        int sum = 0;
        for (int i = lo; i < hi; ++i) sum += total[i];
        int at = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(kAll, at, o);
            if (lane >= o) at += u;
        }
        at -= sum;
        for (int i = lo; i < hi; ++i) {
            const int c = total[i];
            total[i] = at;
            before[i] += at;
            at += c;
        }
        if (lane == 31) total[E] = at;
    }
    __syncthreads();
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i <= E; i += kPlaceThreads) p.r.offsets[i] = total[i];
    for (int64_t i = c0; i < c1; i += kPlaceThreads) {
        const int c = i == c0 ? chosen0 : __ldcg(p.r.chosen + i);
        if (c < 0) continue;
        const int row = (i == c0 ? rank0 : __ldcg(p.r.rows + i)) + before[c];
        p.r.rows[i] = row;
        p.r.sources[row] = (int32_t)i;
    }
    const int64_t end = (int64_t)p.r.tokens * k;
    for (int64_t i = total[E] + (int64_t)blockIdx.x * kPlaceThreads + threadIdx.x; i < end; i += (int64_t)blocks * kPlaceThreads)
        p.r.sources[i] = -1;
}

// ---------------------------------------------------------------------------------------
// the gradient of the logits
//   softmax      dl_i = s_i (g_i - sum_j g_j s_j), g_j = scale * dw_j for the chosen, 0 for the others
//   sigmoid      dl_j = g_j s_j (1 - s_j)
//   renormalised, n_j the weights without the scale: softmax dl_j = n_j (g_j - sum g n), sigmoid that times
//                (1 - s_j); nothing for those that are not chosen
// A warp takes a token: it writes the row for those that are not chosen, then the chosen ones' places.
// ---------------------------------------------------------------------------------------
template <typename T>
__device__ __forceinline__ void put_logit(T* row, int e, float v) {
    if constexpr (sizeof(T) == 2) row[e] = (uint16_t)f32x2_to_bf16x2(v, 0.0f);
    else row[e] = v;
}

template <typename T>
__global__ void __launch_bounds__(256) route_bwd_kernel(const RouteBwd p) {
    const int lane = threadIdx.x & 31, k = p.r.k, E = p.r.experts;
    const int t = blockIdx.x * 8 + (threadIdx.x >> 5);
    if (t >= p.r.tokens) return;
    const T* row = reinterpret_cast<const T*>(p.r.logits) + (int64_t)t * p.r.ld;
    T* out = reinterpret_cast<T*>(p.dlogits) + (int64_t)t * p.ldd;
    const bool whole = !p.r.renormalize && !p.r.sigmoid;
    constexpr int per = 16 / (int)sizeof(T);
    if (!whole) {   // the zeros are under way during the rest
        if (p.vec) {
            for (int i = lane * per; i < E; i += 32 * per) *reinterpret_cast<uint4*>(out + i) = make_uint4(0, 0, 0, 0);
        } else {
            for (int i = lane; i < E; i += 32) put_logit(out, i, 0.0f);
        }
    }
    int mine = -1;
    float g = 0.0f;
    if (lane < k) {
        mine = __ldg(p.r.chosen + (int64_t)t * k + lane);
        if (mine < 0 || mine >= E) mine = -1;
        if (mine >= 0) g = p.r.scale * __ldg(p.dweights + (int64_t)t * k + lane);
    }
    const float l = mine >= 0 ? logit_of(raw_logit(row, mine)) : kNone;
    const bool held = l > kNone;
    float d = 0.0f;
    if (p.r.renormalize) {
        const float z = p.r.sigmoid ? fminf(l, 0.0f) : l, most = warp_max(held ? z : kNone);
        float n = held ? expf(z - most) : 0.0f;
        const float small = expf(-fabsf(l));   // 1 - s = small / (1 + small) for l >= 0, 1 / (1 + small) below
        if (p.r.sigmoid && held) n /= 1.0f + small;
        const float all = warp_sum(n);
        n = held ? n / all : 0.0f;
        const float mean = warp_sum(held ? g * n : 0.0f);
        d = held ? n * (g - mean) : 0.0f;
        if (p.r.sigmoid && held) d *= (l >= 0.0f ? small : 1.0f) / (1.0f + small);
    } else if (p.r.sigmoid) {
        const float small = expf(-fabsf(l)), one = 1.0f + small;
        d = held ? g * (small / one) / one : 0.0f;
    }
    if (whole && !__any_sync(kAll, held)) {
        for (int i = lane; i < E; i += 32) put_logit(out, i, 0.0f);
    } else if (whole) {
        float top = kNone;
        for (int i = lane; i < E; i += 32) top = fmaxf(top, logit_of(raw_logit(row, i)));
        top = warp_max(top);
        float sum = 0.0f;
        for (int i = lane; i < E; i += 32) sum += expf(logit_of(raw_logit(row, i)) - top);
        sum = warp_sum(sum);
        const float s = held ? expf(l - top) / sum : 0.0f;
        const float mean = warp_sum(held ? g * s : 0.0f);
        d = s * (g - mean);
        for (int i = lane; i < E; i += 32) put_logit(out, i, -mean * (expf(logit_of(raw_logit(row, i)) - top) / sum));
    }
    __syncwarp();   // the row before the chosen places of it
    if (mine >= 0) put_logit(out, mine, d);
}

// ---------------------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------------------
constexpr int kRouteHeld = 8192;   // choices of a block that shared memory keeps

template <int VMAX, int WARPS, typename T>
static cudaError_t launch_choose(const RouteKernelParams& p, int blocks, int warps, cudaStream_t s) {
    static std::atomic<uint64_t> attr{0};
    auto kern = route_choose_kernel<VMAX, WARPS, T>;
    if (cudaError_t e = host::ensure_smem(reinterpret_cast<const void*>(kern), (WARPS * (kMaxExperts + 1) + kMaxExperts + 1 + kRouteHeld) * 4, attr)) return e;
    kern<<<blocks, 32 * warps, (warps * p.stride + p.r.experts + 1 + p.held) * 4, s>>>(p);
    return cudaGetLastError();
}
// 28 of 8 experts a lane: 72 registers, where 32 leave 64 and spill (16384 tokens of 256 experts, softmax: 20.5 us, with 32 21.6, with
// 24 21.7).  32 save a round from 4145 to 4736 tokens, among others, which is worth what the spills cost: 4144 tokens 12.4 to 12.6 us, 12.8
// to 13.3 with 32; 4700 13.6 to 14.7, 13.3 to 13.7; 9000 16.5 to 17.7, 16.8 to 16.9.
static int most_warps(int per_lane) { return per_lane <= 4 ? 32 : per_lane <= 8 ? 28 : per_lane <= 16 ? 16 : 8; }
template <typename T>
static cudaError_t launch_choose(const RouteKernelParams& p, int blocks, int warps, cudaStream_t s) {
    const int v = p.per_lane;
    if (v <= 1) return launch_choose<1, 32, T>(p, blocks, warps, s);
    if (v <= 2) return launch_choose<2, 32, T>(p, blocks, warps, s);
    if (v <= 4) return launch_choose<4, 32, T>(p, blocks, warps, s);
    if (v <= 8) return launch_choose<8, 28, T>(p, blocks, warps, s);
    if (v <= 16) return launch_choose<16, 16, T>(p, blocks, warps, s);
    return launch_choose<64, 8, T>(p, blocks, warps, s);
}

cudaError_t launch_route(const RouteProblem& r, cudaStream_t s) {
    RouteKernelParams p{};
    p.r = r;
    p.size = r.experts / r.groups;
    p.lanes_log2 = 5;
    while ((32 >> p.lanes_log2) < r.groups) --p.lanes_log2;
    const int lanes = 1 << p.lanes_log2;
    p.per_lane = (p.size + lanes - 1) / lanes;
    const int esz = r.bf16 ? 2 : 4;
    p.vec = p.per_lane * esz % 16 == 0 && p.size % p.per_lane == 0 && r.ld * esz % 16 == 0;
    int warps = most_warps(p.per_lane), blocks = 1;
    // One block by itself as long as a warp takes one token: 28 tokens of 256 experts 7.3 us, 40 by two kernels 7.2; 8 tokens 5.3 and
    // 8.0.  More tokens go over as many blocks as leave each 8 (of 512 experts and more: a token for each of its warps), since joining the
    // warps' counts is what a block of few tokens spends its time on: 300 tokens of 256 experts by blocks of 28 9.9 us, of 8 7.8.
    const int least = p.per_lane <= 8 ? 8 : warps;
    if (r.tokens > warps) blocks = std::min(kRouteBlocks, (r.tokens + least - 1) / least);
    p.block_tokens = std::max(1, (r.tokens + blocks - 1) / blocks);
    warps = std::min(warps, p.block_tokens);
    blocks = std::max(1, (r.tokens + p.block_tokens - 1) / p.block_tokens);
    p.warp_tokens = (p.block_tokens + warps - 1) / warps;
    p.stride = r.experts | 1;
    p.held = (int64_t)p.block_tokens * r.k <= kRouteHeld ? p.block_tokens * r.k : 0;
    if (cudaError_t e = r.bf16 ? launch_choose<uint16_t>(p, blocks, warps, s) : launch_choose<float>(p, blocks, warps, s)) return e;
    if (blocks == 1) return cudaSuccess;
    cudaLaunchAttribute pdl{};
    pdl.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(kPlaceThreads);
    cfg.stream = s;
    cfg.attrs = &pdl;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, route_place_kernel, p, blocks);
}

cudaError_t launch_route_bwd(const RouteBwd& b, cudaStream_t s) {
    RouteBwd p = b;
    const int esz = p.r.bf16 ? 2 : 4;
    p.vec = p.r.experts * esz % 16 == 0 && p.ldd * esz % 16 == 0;
    const unsigned blocks = (unsigned)((p.r.tokens + 7) / 8);
    if (p.r.bf16) route_bwd_kernel<uint16_t><<<blocks, 256, 0, s>>>(p);
    else route_bwd_kernel<float><<<blocks, 256, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace nvfp4
