// grouped_few.cu -- fprop of the products grouped by expert for few token rows (a served batch):
// D[t] = A[t] . W_e^T, W_e [N][K].
//
// The rows cost nothing against the weights, each of which is read once: the work is bound by
// memory, and at the smallest sizes by latency.  A CTA takes 16 features of one expert; its warps
// cut K into chunks of 64 and join their sums through shared memory, so that even two experts of a
// few hundred features are spread over most SMs, with no tensor maps, TMEM or clusters to set up.
// The products run on mma.sync m16n8k16 (features x token groups of 8): at these sizes the tensor
// pipe is idle either way, and the fragments come straight from global memory in 16-byte loads.  For
// that the K positions within a chunk are permuted, the same way for both operands: lane (g, t) of a
// warp holds 8 consecutive products of weight row g (and g + 8) and of token g, which serve as its
// fragment slots of two MMAs.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "nvfp4_device.cuh"
#include "nvfp4_internal.h"
#include "sm100_ptx.cuh"

namespace nvfp4 {

constexpr int kFewChunks = kFewMaxExperts / 32;
// Warps that cut K, and so CTAs per SM.  16 serve a K of kFewLongK or more in launches that a single wave
// of CTAs holds, where a CTA's chain of loads is what counts: one expert of 1280 x 5120, 8 rows 6.8 us with
// 16 and 10.0 with 8, 64 rows 21.2 and 31.9.  With more CTAs or a shorter K 8 are better: 48 rows x 14 busy
// experts of 5120 x 1280 (184 MB) 31.4 us, with 16 34.8.  Those take 36.2 with 5 CTAs per SM, and 35.2 with
// the K loop unrolled by 2 (more loads in flight per warp; 42.2 with the registers that it asks for).
constexpr int few_resident(int warps) { return 32 / warps; }

// Products a warp accumulates on the tensor core, which truncates, before it joins them in fp32: 65536
// positive products summed without joining came out 3.5e-5 low, so 8.9e-7.
constexpr int kFewRun = 512;

struct FewParams {
    const uint16_t* a;
    const uint16_t* b;
    void* d;
    const int32_t* offsets;
    int64_t lda, ldb, stride_b, ldd;
    int32_t rows, N, K, experts;
    int32_t out_fp32;
    uint32_t* flags;
};

__device__ __forceinline__ uint4 ld_stream(const uint16_t* p) {   // weights: read once
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
__device__ __forceinline__ void mma_16n8k16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The rows of the j-th expert that owns any: each warp reads all offsets, lane by lane, as their
// running maximum clamped to [0, rows].  Returns the expert, or -1 if fewer own rows.
__device__ __forceinline__ int busy_expert(const FewParams& p, int j, bool report, int& lo_out, int& hi_out) {
    const int lane = threadIdx.x & 31;
    int raw[kFewChunks], next[kFewChunks];
#pragma unroll
    for (int c = 0; c < kFewChunks; ++c) {   // all loads in flight together
        const int e = 32 * c + lane;
        raw[c] = e < p.experts ? __ldg(p.offsets + e) : 0;
        next[c] = e < p.experts ? __ldg(p.offsets + e + 1) : 0;
    }
    int carry = 0, found = -1, before = 0;
    bool bad = false;
#pragma unroll
    for (int c = 0; c < kFewChunks; ++c) {
        if (32 * c >= p.experts) break;
        const bool in = 32 * c + lane < p.experts;
        int v = in ? min(max(raw[c], 0), p.rows) : 0;
#pragma unroll
        for (int s = 1; s < 32; s <<= 1) {
            const int u = __shfl_up_sync(0xFFFFFFFFu, v, s);
            if (lane >= s) v = max(v, u);
        }
        const int lo = max(v, carry), hi = in ? max(lo, min(max(next[c], 0), p.rows)) : lo;
        carry = __shfl_sync(0xFFFFFFFFu, lo, 31);
        bad |= in && (raw[c] != lo || next[c] != hi);
        const uint32_t busy = __ballot_sync(0xFFFFFFFFu, hi > lo);
        const int n = __popc(busy);
        if (found < 0 && j < before + n) {
            const uint32_t it = __ballot_sync(0xFFFFFFFFu, hi > lo && before + __popc(busy & ((1u << lane) - 1u)) == j);
            const int src = __ffs(it) - 1;
            found = 32 * c + src;
            lo_out = __shfl_sync(0xFFFFFFFFu, lo, src);
            hi_out = __shfl_sync(0xFFFFFFFFu, hi, src);
        }
        before += n;
    }
    if (report && bad) atomicOr(p.flags, kFlagOffsets);
    return found;
}

// NG: groups of 8 tokens taken in one pass over the weights; an expert with more rows takes more
// passes (its weights then come from L2)
template <int NG, int WARPS>
__global__ void __launch_bounds__(32 * WARPS, few_resident(WARPS)) grouped_few_kernel(const FewParams p) {
    __shared__ float part[WARPS][NG * 8][17];   // [warp][token][feature], padded
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    int lo = 0, hi = 0;
    const int e = busy_expert(p, blockIdx.y, blockIdx.x == 0 && blockIdx.y == 0 && warp == 0, lo, hi);
    if (e < 0) return;
    const int f0 = blockIdx.x * 16;
    // rows g and g + 8 of the CTA's features (N % 8 == 0: the second eight may be past the end)
    const bool upper = f0 + 8 < p.N;
    const uint16_t* w0 = p.b + e * p.stride_b + (int64_t)(f0 + g) * p.ldb + 8 * t;
    const uint16_t* w1 = w0 + (upper ? 8 * p.ldb : 0);
    const uint4 zero = make_uint4(0, 0, 0, 0);
    for (; lo < hi; lo += 8 * NG) {
        const int tokens = min(8 * NG, hi - lo), groups = (tokens + 7) >> 3;
        const uint16_t* x = p.a + (int64_t)(lo + g) * p.lda + 8 * t;   // token g of each group
        // runs of kFewRun products, joined in the warp's own part of shared memory (registers are full)
#pragma unroll 1
        for (int k = 64 * warp, run = 0; run == 0 || k < p.K; ++run) {
            const int end = min(p.K, k + kFewRun * WARPS);
            float acc[NG][4] = {};
#pragma unroll 1
            for (; k < end; k += 64 * WARPS) {
                const bool in0 = k + 8 * t < p.K, in1 = k + 32 + 8 * t < p.K;
                const uint4 a00 = in0 ? ld_stream(w0 + k) : zero, a01 = in1 ? ld_stream(w0 + k + 32) : zero;
                const uint4 a10 = in0 && upper ? ld_stream(w1 + k) : zero, a11 = in1 && upper ? ld_stream(w1 + k + 32) : zero;
#pragma unroll
                for (int i = 0; i < NG; ++i) {
                    if (i >= groups) break;
                    const bool tok = 8 * i + g < tokens;
                    const uint16_t* xi = x + (int64_t)(8 * i) * p.lda + k;
                    const uint4 b0 = tok && in0 ? __ldg(reinterpret_cast<const uint4*>(xi)) : zero;
                    const uint4 b1 = tok && in1 ? __ldg(reinterpret_cast<const uint4*>(xi + 32)) : zero;
                    mma_16n8k16(acc[i], a00.x, a10.x, a00.y, a10.y, b0.x, b0.y);
                    mma_16n8k16(acc[i], a00.z, a10.z, a00.w, a10.w, b0.z, b0.w);
                    mma_16n8k16(acc[i], a01.x, a11.x, a01.y, a11.y, b1.x, b1.y);
                    mma_16n8k16(acc[i], a01.z, a11.z, a01.w, a11.w, b1.z, b1.w);
                }
            }
#pragma unroll
            for (int i = 0; i < NG; ++i) {
                if (i >= groups) break;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float& s = part[warp][8 * i + 2 * t + (j & 1)][g + 4 * (j & 2)];
                    s = run == 0 ? acc[i][j] : s + acc[i][j];
                }
            }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < 256; i += 32 * WARPS) {   // 16 tokens at most
            const int f = i & 15, tok = i >> 4;
            if (tok >= tokens || f0 + f >= p.N) continue;
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) s += part[w][tok][f];
            const int64_t at = (int64_t)(lo + tok) * p.ldd + f0 + f;
            if (p.out_fp32)
                reinterpret_cast<float*>(p.d)[at] = s;
            else
                reinterpret_cast<uint16_t*>(p.d)[at] = (uint16_t)f32x2_to_bf16x2(s, 0.0f);
        }
        __syncthreads();   // the next pass writes `part` again
    }
}

template <int NG, int WARPS>
static void launch_few(const FewParams& p, dim3 grid, cudaStream_t s) {
    grouped_few_kernel<NG, WARPS><<<grid, 32 * WARPS, 0, s>>>(p);
}

cudaError_t launch_gemm_grouped_few(const GroupedGemm& g, cudaStream_t s) {
    if (g.b_kn || g.rows < 1 || g.rows > kFewMaxRows || g.experts > kFewMaxExperts) return cudaErrorInvalidValue;
    FewParams p{};
    p.a = g.a;
    p.b = g.b;
    p.d = g.d;
    p.offsets = g.offsets;
    p.lda = g.lda;
    p.ldb = g.ldb;
    p.stride_b = g.stride_b;
    p.ldd = g.ldd;
    p.rows = (int32_t)g.rows;
    p.N = (int32_t)g.N;
    p.K = (int32_t)g.K;
    p.experts = g.experts;
    p.out_fp32 = g.out_fp32;
    p.flags = g.flags;
    const dim3 grid((unsigned)((g.N + 15) / 16), (unsigned)std::min<int64_t>(g.rows, g.experts));
    const bool long_k = p.K >= kFewLongK && (int64_t)grid.x * grid.y <= host::sm_count() * few_resident(16);
    if (g.rows <= 8)
        long_k ? launch_few<1, 16>(p, grid, s) : launch_few<1, 8>(p, grid, s);
    else
        long_k ? launch_few<2, 16>(p, grid, s) : launch_few<2, 8>(p, grid, s);
    return cudaGetLastError();
}

}  // namespace nvfp4
