// tokens.cu -- token rows into the experts' order (dispatch) and back (combine), and combine's gradient.
//
//   dispatch      xs[r(t, j)] = x[t]
//   combine       y[t] = residual[t] + sum_j w(t, j) ys[r(t, j)]          (w = 1 without weights)
//   its gradient  dys[r(t, j)] = w(t, j) dy[t],  dw(t, j) = dy[t] . ys[r(t, j)]
//
// All of them go by token: a token's row is read once for its k rows, and the sums of combine are a thread's
// own, in fp32, in the order of the choices, with no atomics and one rounding.  They are bound by memory.
// A choice without a row (-1) is skipped; rows that no choice names are left as they are.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "nvfp4_device.cuh"
#include "nvfp4_internal.h"
#include "sm100_ptx.cuh"

namespace nvfp4 {

constexpr int kMoveThreads = 128;

// How the 16-byte pieces (8 elements) of the token rows are dealt out: a block takes `pieces` pieces of one
// token (grid.y cuts its row), or whole rows of `tokens` tokens.
struct MoveGrid {
    int32_t vecs;      // pieces of a row
    int32_t pieces;    // of a block, per token
    int32_t tokens;    // of a block
};

__device__ __forceinline__ int64_t row_of(const TokenRows& m, int64_t choice) {
    const int64_t r = __ldg(m.rows + choice);
    return r >= 0 && r < m.rows_total ? r : -1;
}

__device__ __forceinline__ void widen(const uint4& v, float (&f)[8]) {
    f[0] = bf16_lo(v.x); f[1] = bf16_hi(v.x); f[2] = bf16_lo(v.y); f[3] = bf16_hi(v.y);
    f[4] = bf16_lo(v.z); f[5] = bf16_hi(v.z); f[6] = bf16_lo(v.w); f[7] = bf16_hi(v.w);
}
__device__ __forceinline__ uint4 narrow(const float (&f)[8]) {
    return make_uint4(f32x2_to_bf16x2(f[0], f[1]), f32x2_to_bf16x2(f[2], f[3]), f32x2_to_bf16x2(f[4], f[5]), f32x2_to_bf16x2(f[6], f[7]));
}
// SHARED: the memory may be the output's (a residual that the sum replaces)
template <bool FP32, bool SHARED = false>
__device__ __forceinline__ void load8(const void* base, int64_t at, float (&f)[8]) {
    if constexpr (FP32) {
        const float4* q = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(base) + at);
        const float4 a = SHARED ? q[0] : __ldg(q), b = SHARED ? q[1] : __ldg(q + 1);
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    } else {
        const uint4* q = reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(base) + at);
        widen(SHARED ? *q : __ldg(q), f);
    }
}
template <bool FP32>
__device__ __forceinline__ void store8(void* base, int64_t at, const float (&f)[8]) {
    if constexpr (FP32) {
        float4* q = reinterpret_cast<float4*>(reinterpret_cast<float*>(base) + at);
        q[0] = make_float4(f[0], f[1], f[2], f[3]);
        q[1] = make_float4(f[4], f[5], f[6], f[7]);
    } else {
        *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(base) + at) = narrow(f);
    }
}

__global__ void __launch_bounds__(kMoveThreads) dispatch_kernel(const TokenRows m, const uint16_t* x, int64_t ldx, uint16_t* xs, int64_t ldxs, const MoveGrid g) {
    const int64_t t0 = (int64_t)blockIdx.x * g.tokens;
    const int v0 = blockIdx.y * g.pieces, width = min(g.pieces, g.vecs - v0);
    const int tokens = (int)min((int64_t)g.tokens, m.tokens - t0);
    for (int i = threadIdx.x; i < tokens * width; i += kMoveThreads) {
        const int a = i / width, v = v0 + i - a * width;
        const int64_t t = t0 + a;
        const uint4 w = __ldg(reinterpret_cast<const uint4*>(x + t * ldx) + v);
        for (int j = 0; j < m.k; ++j) {
            const int64_t r = row_of(m, t * m.k + j);
            if (r >= 0) reinterpret_cast<uint4*>(xs + r * ldxs)[v] = w;
        }
    }
}

template <bool YS32, bool Y32>
__global__ void __launch_bounds__(kMoveThreads) combine_kernel(const Combine c, const MoveGrid g) {
    const TokenRows& m = c.m;
    const int64_t t0 = (int64_t)blockIdx.x * g.tokens;
    const int v0 = blockIdx.y * g.pieces, width = min(g.pieces, g.vecs - v0);
    const int tokens = (int)min((int64_t)g.tokens, m.tokens - t0);
    for (int i = threadIdx.x; i < tokens * width; i += kMoveThreads) {
        const int a = i / width, col = 8 * (v0 + i - a * width);
        const int64_t t = t0 + a;
        float y[8] = {};
        if (c.residual) load8<Y32, true>(c.residual, t * c.ldr + col, y);
        for (int j = 0; j < m.k; ++j) {
            const int64_t r = row_of(m, t * m.k + j);
            if (r < 0) continue;
            const float w = m.weights ? __ldg(m.weights + t * m.k + j) : 1.0f;
            float f[8];
            load8<YS32>(c.ys, r * c.ldys + col, f);
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = fmaf(w, f[e], y[e]);
        }
        store8<Y32>(c.y, t * c.ldy + col, y);
    }
}

// One block per token
constexpr int kGradThreads = 128;
template <int KMAX, bool YS32>
__global__ void __launch_bounds__(kGradThreads) combine_bwd_kernel(const CombineBwd c) {
    __shared__ float part[kGradThreads / 32][KMAX];
    const TokenRows& m = c.m;
    const int64_t t = blockIdx.x;
    const int vecs = (int)(m.d >> 3), lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float dot[KMAX];
#pragma unroll
    for (int j = 0; j < KMAX; ++j) dot[j] = 0.0f;
    for (int v = threadIdx.x; v < vecs; v += kGradThreads) {
        float g[8];
        load8<false>(c.dy, t * c.lddy + 8 * v, g);
#pragma unroll
        for (int j = 0; j < KMAX; ++j) {
            const int64_t r = j < m.k ? row_of(m, t * m.k + j) : -1;
            if (r < 0) continue;
            const float w = __ldg(m.weights + t * m.k + j);
            float f[8], o[8];
            load8<YS32>(c.ys, r * c.ldys + 8 * v, f);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                dot[j] = fmaf(g[e], f[e], dot[j]);
                o[e] = w * g[e];
            }
            store8<false>(c.dys, r * c.lddys + 8 * v, o);
        }
    }
#pragma unroll
    for (int j = 0; j < KMAX; ++j) {
        if (j >= m.k) break;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) dot[j] += __shfl_xor_sync(0xFFFFFFFFu, dot[j], o);
        if (lane == 0) part[warp][j] = dot[j];
    }
    __syncthreads();
    if (threadIdx.x < m.k) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kGradThreads / 32; ++w) s += part[w][threadIdx.x];
        c.dweights[t * m.k + threadIdx.x] = s;
    }
}

// ---------------------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------------------
static dim3 move_grid(const TokenRows& m, MoveGrid& g) {
    g.vecs = (int32_t)(m.d / 8);
    // 4 pieces for each thread, 1 where there are few
    const int64_t all = m.tokens * g.vecs;
    const int per_block = all >= (int64_t)4 * kMoveThreads * host::sm_count() * 8 ? 4 * kMoveThreads : kMoveThreads;
    if (g.vecs >= per_block) {
        const int cuts = (g.vecs + per_block - 1) / per_block;
        g.pieces = (g.vecs + cuts - 1) / cuts;
        g.tokens = 1;
        return dim3((unsigned)m.tokens, (unsigned)((g.vecs + g.pieces - 1) / g.pieces));
    }
    g.pieces = g.vecs;
    g.tokens = per_block / g.vecs;
    return dim3((unsigned)((m.tokens + g.tokens - 1) / g.tokens));
}

cudaError_t launch_dispatch(const TokenRows& m, const uint16_t* x, int64_t ldx, uint16_t* xs, int64_t ldxs, cudaStream_t s) {
    MoveGrid g;
    const dim3 grid = move_grid(m, g);
    dispatch_kernel<<<grid, kMoveThreads, 0, s>>>(m, x, ldx, xs, ldxs, g);
    return cudaGetLastError();
}

cudaError_t launch_combine(const Combine& c, cudaStream_t s) {
    MoveGrid g;
    const dim3 grid = move_grid(c.m, g);
    if (c.ys_fp32) {
        if (c.y_fp32) combine_kernel<true, true><<<grid, kMoveThreads, 0, s>>>(c, g);
        else combine_kernel<true, false><<<grid, kMoveThreads, 0, s>>>(c, g);
    } else {
        if (c.y_fp32) combine_kernel<false, true><<<grid, kMoveThreads, 0, s>>>(c, g);
        else combine_kernel<false, false><<<grid, kMoveThreads, 0, s>>>(c, g);
    }
    return cudaGetLastError();
}

template <int KMAX>
static void launch_combine_bwd(const CombineBwd& c, cudaStream_t s) {
    if (c.ys_fp32) combine_bwd_kernel<KMAX, true><<<(unsigned)c.m.tokens, kGradThreads, 0, s>>>(c);
    else combine_bwd_kernel<KMAX, false><<<(unsigned)c.m.tokens, kGradThreads, 0, s>>>(c);
}
cudaError_t launch_combine_bwd(const CombineBwd& c, cudaStream_t s) {
    const int k = c.m.k;
    if (k <= 2) launch_combine_bwd<2>(c, s);
    else if (k <= 4) launch_combine_bwd<4>(c, s);
    else if (k <= 8) launch_combine_bwd<8>(c, s);
    else launch_combine_bwd<kRouteMaxK>(c, s);
    return cudaGetLastError();
}

}  // namespace nvfp4
