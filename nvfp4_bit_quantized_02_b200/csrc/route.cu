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
// (32 / groups), so that what is reduced within a group stays within neighbouring lanes and the lowest lane
// with a value holds the lowest index.  Values are compared as unsigned words that order as they do.
//
// The choice is that of the definition in fp64.  Where c is the logit itself its order is exact.  Otherwise c
// is evaluated in fp32 (the error bound stands at kTau), and a token whose order is not certain, because
// two neighbours in it lie closer than the bound, is decided again in fp64 (choose_slow): about 1 token in 300
// of 256 experts with sigmoid scores.
//
// Rows: a warp takes neighbouring tokens and counts each expert's choices as it goes, so that a choice's rank
// among the warp's is there at once; the ranks are joined over the block's warps, and over the blocks by a
// second kernel, which reads every block's counts.  No atomics: the order is that of the tokens.
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
    int32_t lanes;       // of a group, a power of two
    int32_t per_lane;    // experts of a lane
    int32_t vec;         // a lane's logits can be read 16 bytes at a time
    int32_t block_tokens, warp_tokens;
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
    const int g = lane / p.lanes;
    int before = 0;
    for (int i = 0; i < p.r.groups; ++i) {
        const F other = __shfl_sync(kAll, score, i * p.lanes);
        before += other > score || (other == score && i < g);
    }
    return before < p.r.top_groups && score > (F)kNone && g < p.r.groups;
}

// The choice in fp64: lane j returns the j-th expert, or -1.  Nothing is kept: each pick looks through the
// row for what comes next in order behind the one before.
template <typename T>
__device__ __noinline__ int choose_slow(const RouteKernelParams& p, const T* row, float top) {
    const int lane = threadIdx.x & 31, g = lane / p.lanes, first = (lane % p.lanes) * p.per_lane;
    const int count = g < p.r.groups ? max(0, min(p.per_lane, p.size - first)) : 0, e0 = g * p.size + first;
    double sum = 1.0;
    const auto value = [&](int e) {
        const float l = logit_of(raw_logit(row, e));
        if (!(l > kNone)) return (double)kNone;
        const double s = p.r.sigmoid ? 1.0 / (1.0 + exp(-(double)l)) : exp((double)l - (double)top) / sum;
        const double c = p.r.bias ? s + (double)__ldg(p.r.bias + e) : s;
        return c == c ? c : (double)kNone;
    };
    if (!p.r.sigmoid) {
        double part = 0.0;
        for (int i = 0; i < count; ++i) {
            const float l = logit_of(raw_logit(row, e0 + i));
            if (l > kNone) part += exp((double)l - (double)top);
        }
        for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(kAll, part, o);
        sum = part;
    }
    bool open = true;
    if (p.r.groups > 1) {
        double a1 = kNone, a2 = kNone;
        for (int i = 0; i < count; ++i) merge_top2(a1, a2, value(e0 + i), (double)kNone);
        for (int o = 1; o < p.lanes; o <<= 1) merge_top2(a1, a2, __shfl_xor_sync(kAll, a1, o), __shfl_xor_sync(kAll, a2, o));
        open = group_stays(p.r.group_top == 2 ? a1 + a2 : a1, p, lane);
    }
    // without a bias the groups alone go by scores, the experts by their logits
    const auto order = [&](int e) { return p.r.bias ? value(e) : (double)logit_of(raw_logit(row, e)); };
    int mine = -1, last_e = -1;
    double last = INFINITY;
    for (int j = 0; j < p.r.k; ++j) {
        double best = kNone;
        int at = -1;
        if (open)
            for (int i = 0; i < count; ++i) {
                const int e = e0 + i;
                const double c = order(e);
                if ((c < last || (c == last && e > last_e)) && c > best) {
                    best = c;
                    at = e;
                }
            }
        for (int o = 16; o > 0; o >>= 1) {
            const double c = __shfl_xor_sync(kAll, best, o);
            const int e = __shfl_xor_sync(kAll, at, o);
            if (e >= 0 && (at < 0 || c > best || (c == best && e < at))) {
                best = c;
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
    return held ? r.scale * (v / all) : 0.0f;
}

// VMAX: experts of a lane at most; T: the logits' type
template <int VMAX, int WARPS, typename T>
__global__ void __launch_bounds__(32 * WARPS) route_choose_kernel(const RouteKernelParams p) {
    extern __shared__ int32_t smem[];
    int32_t* counts = smem;                               // [WARPS][experts]
    int32_t* base = smem + WARPS * p.r.experts;           // [experts + 1]: one block's offsets
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int k = p.r.k, E = p.r.experts;
    for (int i = threadIdx.x; i < WARPS * E; i += 32 * WARPS) counts[i] = 0;
    __syncthreads();
    ptx::griddep_launch();
    const int t0 = blockIdx.x * p.block_tokens, t1 = min(p.r.tokens, t0 + p.block_tokens);
    const int g = lane / p.lanes, first = (lane % p.lanes) * p.per_lane, e0 = g * p.size + first;
    const int count = g < p.r.groups ? max(0, min(p.per_lane, p.size - first)) : 0;
    const bool by_logit = !p.r.bias;
    const bool scores = !by_logit || (p.r.groups > 1 && p.r.group_top == 2);
    bool odd = false;
    int32_t* mine_counts = counts + warp * E;
    const int w1 = min(t1, t0 + (warp + 1) * p.warp_tokens);
    for (int t = t0 + warp * p.warp_tokens; t < w1; ++t) {
        int mine = -1;
        float weight = 0.0f;
        if (!p.r.valid || __ldg(p.r.valid + t)) {
            const T* row = reinterpret_cast<const T*>(p.r.logits) + (int64_t)t * p.r.ld;
            float l[VMAX];
            if (p.vec) {
                constexpr int per = 16 / (int)sizeof(T);
#pragma unroll
                for (int i = 0; i < VMAX; i += per) {
                    uint4 v = make_uint4(0, 0, 0, 0);
                    if (i < count) v = __ldg(reinterpret_cast<const uint4*>(row + e0 + i));
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int j = 0; j < per && i + j < VMAX; ++j)
                        l[i + j] = sizeof(T) == 4 ? __uint_as_float(w[j & 3]) : (j & 1 ? bf16_hi(w[(j >> 1) & 3]) : bf16_lo(w[(j >> 1) & 3]));
                }
            } else {
#pragma unroll
                for (int i = 0; i < VMAX; ++i) l[i] = i < count ? raw_logit(row, e0 + i) : 0.0f;
            }
            float top = kNone;
#pragma unroll
            for (int i = 0; i < VMAX; ++i) {
                const bool in = i < count;
                odd |= in && !(l[i] <= FLT_MAX);
                l[i] = in ? logit_of(l[i]) : kNone;
                top = fmaxf(top, l[i]);
            }
            float sum = 1.0f;
            const bool soft = !p.r.sigmoid && (scores || !p.r.renormalize);
            if (soft) {
                top = warp_max(top);
                sum = 0.0f;
#pragma unroll
                for (int i = 0; i < VMAX; ++i) sum += l[i] > kNone ? __expf(l[i] - top) : 0.0f;
                sum = warp_sum(sum);
            }
            // c, and what of it the groups go by
            uint32_t key[VMAX];
            bool certain = true;
            const float tau = p.r.sigmoid ? kTauSigmoid : kTauSoftmax / sum;
            if (scores) {
                const float per_sum = 1.0f / sum;
#pragma unroll
                for (int i = 0; i < VMAX; ++i) {
                    float c = p.r.sigmoid ? __fdividef(1.0f, 1.0f + __expf(-l[i])) : __expf(l[i] - top) * per_sum;
                    if (p.r.bias && i < count) c += __ldg(p.r.bias + e0 + i);
                    key[i] = l[i] > kNone ? order_key(c) : 0u;
                }
            } else {
#pragma unroll
                for (int i = 0; i < VMAX; ++i) key[i] = order_key(l[i]);
            }
            if (p.r.groups > 1) {
                float a1 = kNone, a2 = kNone;
#pragma unroll
                for (int i = 0; i < VMAX; ++i) merge_top2(a1, a2, key_value(key[i]), kNone);
                for (int o = 1; o < p.lanes; o <<= 1) merge_top2(a1, a2, __shfl_xor_sync(kAll, a1, o), __shfl_xor_sync(kAll, a2, o));
                const float score = p.r.group_top == 2 ? a1 + a2 : a1;
                const bool stays = group_stays(score, p, lane);
                if (scores) {
                    const uint32_t least = __reduce_min_sync(kAll, stays ? order_key(score) : kAll);
                    const uint32_t most = __reduce_max_sync(kAll, stays || g >= p.r.groups ? 0u : order_key(score));
                    const float lo = key_value(least);
                    // a sum of two errs by both, and by its rounding
                    if (most && least != kAll) certain = lo - key_value(most) > 2.0f * (tau + kTauC * fabsf(lo));
                }
#pragma unroll
                for (int i = 0; i < VMAX; ++i) key[i] = !stays ? 0u : by_logit ? order_key(l[i]) : key[i];
            }
            uint32_t best = 0;
#pragma unroll
            for (int i = 0; i < VMAX; ++i) best = max(best, key[i]);
            // k picks, and where the order is that of c in fp32 one more, to see its distance
            float last = INFINITY;
            int last_e = -1;
            const int picks = by_logit ? k : k + 1;
            for (int j = 0; j < picks && certain; ++j) {
                const uint32_t most = __reduce_max_sync(kAll, best);
                if (!most) break;
                const int winner = __ffs(__ballot_sync(kAll, best == most)) - 1;
                int at = 0;
                if (lane == winner) {
                    bool found = false;
                    best = 0;
#pragma unroll
                    for (int i = 0; i < VMAX; ++i) {
                        const bool here = !found && key[i] == most;
                        found |= here;
                        if (here) {
                            at = i;
                            key[i] = 0;
                        }
                        best = max(best, key[i]);
                    }
                    at += e0;
                }
                at = __shfl_sync(kAll, at, winner);
                if (!by_logit) {
                    const float c = key_value(most);
                    if (j > 0 && !(last - c > tau + kTauC * fabsf(last))) {
                        // the same logit and bias give the same c: the lower index came first
                        certain = j < k && raw_logit(row, at) == raw_logit(row, last_e) && __ldg(p.r.bias + at) == __ldg(p.r.bias + last_e);
                    }
                    last = c;
                    last_e = at;
                }
                if (lane == j && j < k) mine = at;
            }
            if (!certain) {
                if (p.r.sigmoid) top = 0.0f;
                mine = choose_slow(p, row, top);
            }
            weight = chosen_weight(p.r, mine >= 0 ? logit_of(raw_logit(row, mine)) : kNone, top, sum);
        }
        int rank = 0;
        if (mine >= 0) rank = mine_counts[mine]++;   // a token's experts differ
        __syncwarp();
        if (lane < k) {
            const int64_t at = (int64_t)t * k + lane;
            p.r.chosen[at] = mine;
            p.r.weights[at] = weight;
            p.r.rows[at] = rank;
        }
    }
    if (__any_sync(kAll, odd) && lane == 0) atomicOr(p.r.flags, kFlagNonFinite);
    __syncthreads();
    // ranks within the block: the warps before
    for (int e = threadIdx.x; e < E; e += 32 * WARPS) {
        int before = 0;
#pragma unroll 8
        for (int w = 0; w < WARPS; ++w) {
            const int c = counts[w * E + e];
            counts[w * E + e] = before;
            before += c;
        }
        if (gridDim.x == 1) base[e] = before;
        else p.r.scratch[(int64_t)blockIdx.x * E + e] = before;
    }
    __syncthreads();
    const bool alone = gridDim.x == 1;
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
    const int64_t c0 = (int64_t)t0 * k, c1 = (int64_t)t1 * k;
    for (int64_t i = c0 + threadIdx.x; i < c1; i += 32 * WARPS) {
        const int e = p.r.chosen[i];
        const int w = (int)((uint32_t)(i - c0) / (uint32_t)(k * p.warp_tokens));   // a block's choices: less than 2^30
        int row = -1;
        if (e >= 0) {
            row = p.r.rows[i] + counts[w * E + e];
            if (alone) {
                row += base[e];
                p.r.sources[row] = (int32_t)i;
            }
        }
        p.r.rows[i] = row;
    }
    if (alone)
        for (int64_t i = base[E] + threadIdx.x; i < c1; i += 32 * WARPS) p.r.sources[i] = -1;
}

constexpr int kPlaceThreads = 1024;

// The blocks' counts joined: each block's first row of every expert, and with it the rows of its choices
__global__ void __launch_bounds__(kPlaceThreads) route_place_kernel(const RouteKernelParams p, int blocks) {
    __shared__ int32_t total[kMaxExperts + 1], before[kMaxExperts];
    const int E = p.r.experts, k = p.r.k, lane = threadIdx.x & 31;
    for (int e = threadIdx.x; e < E; e += kPlaceThreads) total[e] = before[e] = 0;
    __syncthreads();
    ptx::griddep_wait();
    int wide = 32;
    while (wide < E) wide <<= 1;
    const int e = threadIdx.x & (wide - 1), parts = kPlaceThreads / wide;
    if (e < E) {
        int all = 0, prior = 0;
#pragma unroll 8
        for (int b = threadIdx.x / wide; b < blocks; b += parts) {
            const int c = __ldcg(p.r.scratch + (int64_t)b * E + e);
            all += c;
            prior += b < (int)blockIdx.x ? c : 0;
        }
        atomicAdd(&total[e], all);     // whole numbers: no order to depend on
        atomicAdd(&before[e], prior);
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
    const int t0 = blockIdx.x * p.block_tokens, t1 = min(p.r.tokens, t0 + p.block_tokens);
    for (int64_t i = (int64_t)t0 * k + threadIdx.x; i < (int64_t)t1 * k; i += kPlaceThreads) {
        const int c = __ldcg(p.r.chosen + i);
        if (c < 0) continue;
        const int row = __ldcg(p.r.rows + i) + before[c];
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
    const bool whole = !p.r.renormalize && !p.r.sigmoid;
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
    const int per = 16 / (int)sizeof(T);
    if (!whole || !__any_sync(kAll, held)) {
        if (p.vec) {
            for (int i = lane * per; i < E; i += 32 * per) *reinterpret_cast<uint4*>(out + i) = make_uint4(0, 0, 0, 0);
        } else {
            for (int i = lane; i < E; i += 32) put_logit(out, i, 0.0f);
        }
    } else {
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
template <int VMAX, int WARPS, typename T>
static cudaError_t launch_choose(const RouteKernelParams& p, int blocks, cudaStream_t s) {
    static std::atomic<uint64_t> attr{0};
    auto kern = route_choose_kernel<VMAX, WARPS, T>;
    const int bytes = (WARPS * p.r.experts + p.r.experts + 1) * 4;
    if (cudaError_t e = host::ensure_smem(reinterpret_cast<const void*>(kern), (WARPS * kMaxExperts + kMaxExperts + 1) * 4, attr)) return e;
    kern<<<blocks, 32 * WARPS, bytes, s>>>(p);
    return cudaGetLastError();
}
template <typename T>
static cudaError_t launch_choose(const RouteKernelParams& p, int blocks, cudaStream_t s) {
    const int v = p.per_lane;
    if (v <= 1) return launch_choose<1, 32, T>(p, blocks, s);
    if (v <= 2) return launch_choose<2, 32, T>(p, blocks, s);
    if (v <= 4) return launch_choose<4, 32, T>(p, blocks, s);
    if (v <= 8) return launch_choose<8, 32, T>(p, blocks, s);
    if (v <= 16) return launch_choose<16, 16, T>(p, blocks, s);
    return launch_choose<64, 8, T>(p, blocks, s);
}

constexpr int kAloneTokens = 256;   // tokens that one block takes by itself

cudaError_t launch_route(const RouteProblem& r, cudaStream_t s) {
    RouteKernelParams p{};
    p.r = r;
    p.size = r.experts / r.groups;
    int wide = 1;
    while (wide < r.groups) wide <<= 1;
    p.lanes = 32 / wide;
    p.per_lane = (p.size + p.lanes - 1) / p.lanes;
    const int esz = r.bf16 ? 2 : 4;
    p.vec = p.per_lane * esz % 16 == 0 && p.size % p.per_lane == 0 && r.ld * esz % 16 == 0;
    const int warps = p.per_lane <= 8 ? 32 : p.per_lane <= 16 ? 16 : 8;
    int blocks = 1;
    if (r.tokens > kAloneTokens) blocks = std::min(kRouteBlocks, (r.tokens + warps - 1) / warps);
    p.block_tokens = std::max(1, (r.tokens + blocks - 1) / blocks);
    blocks = std::max(1, (r.tokens + p.block_tokens - 1) / p.block_tokens);
    p.warp_tokens = (p.block_tokens + warps - 1) / warps;
    if (cudaError_t e = r.bf16 ? launch_choose<uint16_t>(p, blocks, s) : launch_choose<float>(p, blocks, s)) return e;
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
