// grouped.cu -- bf16 products grouped by expert: D[t] = A[t] . W_e^T and the weight gradients
// dW_e (+)= sum_t A[t]^T B[t] over each expert's rows.
//
// First form: one kernel for all three products, 64 x 64 output tiles by 256 threads (4 x 4 fp32
// sums each), the operands read through their strides into shared memory 16 products deep.
#include <cuda_runtime.h>

#include <cstdint>

#include "nvfp4_device.cuh"
#include "nvfp4_internal.h"

namespace nvfp4 {

struct SimpleParams {
    const uint16_t *a, *b;
    void* d;
    const int32_t* offsets;
    int64_t a_m, a_k, b_n, b_k;   // element strides of A by output row / product, of B by output column / product
    int64_t stride_b, ldd, stride_d;
    int64_t rows, M, N, K;        // M, K: of the dimension that is not the token rows
    int experts, wgrad, accumulate, out_fp32;
    uint32_t* flags;
};

// The rows of expert e as the running maximum of the clamped offsets
__device__ void expert_rows(const SimpleParams& p, int e, int64_t& lo, int64_t& hi) {
    int64_t run = 0;
    bool bad = false;
    for (int i = 0; i <= e + 1; ++i) {
        const int64_t o = p.offsets[i];
        bad |= o < run || o > p.rows || o < 0;
        lo = run;
        run = max(run, min(max(o, (int64_t)0), p.rows));
        if (i == 0) lo = run;
    }
    hi = run;
    if (bad) atomicOr(p.flags, kFlagOffsets);
}

__global__ void __launch_bounds__(256) grouped_simple_kernel(const SimpleParams p) {
    __shared__ float as[16][65], bs[16][65];
    __shared__ int64_t s_lo, s_hi;
    __shared__ int s_e;
    const int64_t n0 = (int64_t)blockIdx.x * 64;
    if (threadIdx.x == 0) {
        int64_t lo = 0, hi = 0;
        if (p.wgrad) {
            s_e = blockIdx.z;
            expert_rows(p, blockIdx.z, lo, hi);
        } else {   // row tile blockIdx.y of the experts' tiles in order
            int64_t left = blockIdx.y;
            s_e = -1;
            for (int e = 0; e < p.experts; ++e) {
                expert_rows(p, e, lo, hi);
                const int64_t tiles = (hi - lo + 63) / 64;
                if (left < tiles) {
                    s_e = e;
                    lo += left * 64;
                    break;
                }
                left -= tiles;
            }
        }
        s_lo = lo;
        s_hi = hi;
    }
    __syncthreads();
    const int e = s_e;
    if (e < 0) return;
    const int64_t lo = s_lo, hi = s_hi;
    const int64_t m0 = p.wgrad ? (int64_t)blockIdx.y * 64 : lo;
    const int64_t m_end = p.wgrad ? p.M : hi, k0 = p.wgrad ? lo : 0, k_end = p.wgrad ? hi : p.K;
    if (p.wgrad && p.accumulate && lo == hi) return;
    const uint16_t* b = p.b + (p.wgrad ? 0 : e * p.stride_b);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float acc[4][4] = {}, sum[4][4] = {};
    for (int64_t k = k0; k < k_end; k += 16) {
        for (int i = threadIdx.x; i < 1024; i += 256) {
            const int kk = p.wgrad ? i >> 6 : i & 15, r = p.wgrad ? i & 63 : i >> 4;
            const bool kin = k + kk < k_end;
            as[kk][r] = kin && m0 + r < m_end ? __uint_as_float((uint32_t)p.a[(m0 + r) * p.a_m + (k + kk) * p.a_k] << 16) : 0.0f;
            bs[kk][r] = kin && n0 + r < p.N ? __uint_as_float((uint32_t)b[(n0 + r) * p.b_n + (k + kk) * p.b_k] << 16) : 0.0f;
        }
        __syncthreads();
#pragma unroll
        for (int kk = 0; kk < 16; ++kk)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(as[kk][ty + 16 * i], bs[kk][tx + 16 * j], acc[i][j]);
        __syncthreads();
        if (((k - k0) & 511) == 496 || k + 16 >= k_end) {   // runs of 512 products are joined
            for (int i = 0; i < 4; ++i)
                for (int j = 0; j < 4; ++j) {
                    sum[i][j] += acc[i][j];
                    acc[i][j] = 0.0f;
                }
        }
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
            if (m >= m_end || n >= p.N) continue;
            const int64_t at = (p.wgrad ? e * p.stride_d : 0) + m * p.ldd + n;
            if (!p.out_fp32) {
                reinterpret_cast<uint16_t*>(p.d)[at] = (uint16_t)f32x2_to_bf16x2(sum[i][j], 0.0f);
            } else {
                float* d = reinterpret_cast<float*>(p.d) + at;
                *d = p.accumulate ? *d + sum[i][j] : sum[i][j];
            }
        }
}

cudaError_t launch_gemm_grouped(const GroupedGemm& g, cudaStream_t s) {
    SimpleParams p{};
    p.a = g.a;
    p.b = g.b;
    p.d = g.d;
    p.offsets = g.offsets;
    p.a_m = g.lda;
    p.a_k = 1;
    p.b_n = g.b_kn ? 1 : g.ldb;
    p.b_k = g.b_kn ? g.ldb : 1;
    p.stride_b = g.stride_b;
    p.ldd = g.ldd;
    p.rows = g.rows;
    p.N = g.N;
    p.K = g.K;
    p.experts = g.experts;
    p.out_fp32 = g.out_fp32;
    p.flags = g.flags;
    const int64_t tiles = g.rows / 64 + (g.rows < g.experts ? g.rows : g.experts);
    grouped_simple_kernel<<<dim3((unsigned)((g.N + 63) / 64), (unsigned)tiles), 256, 0, s>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_wgrad_grouped(const GroupedWgrad& g, cudaStream_t s) {
    SimpleParams p{};
    p.a = g.a;
    p.b = g.b;
    p.d = g.d;
    p.offsets = g.offsets;
    p.a_m = 1;
    p.a_k = g.lda;
    p.b_n = 1;
    p.b_k = g.ldb;
    p.ldd = g.ldd;
    p.stride_d = g.stride_d;
    p.rows = g.rows;
    p.M = g.M;
    p.N = g.N;
    p.experts = g.experts;
    p.wgrad = 1;
    p.accumulate = g.accumulate;
    p.out_fp32 = 1;
    p.flags = g.flags;
    grouped_simple_kernel<<<dim3((unsigned)((g.N + 63) / 64), (unsigned)((g.M + 63) / 64), g.experts), 256, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace nvfp4
