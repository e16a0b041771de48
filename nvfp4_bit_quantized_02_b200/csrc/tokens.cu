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

constexpr int kMoveThreads = 128, kCombineThreads = 256;

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
__device__ __forceinline__ void widen(const uint4 (&v)[1], float (&f)[8]) { widen(v[0], f); }   // 8 elements as loaded: bf16
__device__ __forceinline__ void widen(const uint4 (&v)[2], float (&f)[8]) {                      // or fp32
    f[0] = __uint_as_float(v[0].x); f[1] = __uint_as_float(v[0].y); f[2] = __uint_as_float(v[0].z); f[3] = __uint_as_float(v[0].w);
    f[4] = __uint_as_float(v[1].x); f[5] = __uint_as_float(v[1].y); f[6] = __uint_as_float(v[1].z); f[7] = __uint_as_float(v[1].w);
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

// A block takes a piece of one token's row (narrow rows: a row of threads for each of several tokens), so that the rows and
// weights of its choices are looked up once; the loads of J choices and U pieces are issued
// before the first is used.  8192 tokens x 2 x 5120, bf16 rows with a residual: 69 us (4.8 TB/s).
template <int J, int U, bool YS32, bool Y32>
__global__ void __launch_bounds__(kCombineThreads) combine_kernel(const Combine c, int pieces) {
    constexpr int Q = YS32 ? 2 : 1;
    const TokenRows& m = c.m;
    const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    if (t >= m.tokens) return;
    const int end = min((int)(blockIdx.y + 1) * pieces, (int)(m.d >> 3));
    int64_t r[J];
    float w[J];
    const auto look_up = [&](int j0) {
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const bool in = j0 + j < m.k;
            r[j] = in ? row_of(m, t * m.k + j0 + j) : -1;
            w[j] = in && m.weights ? __ldg(m.weights + t * m.k + j0 + j) : 1.0f;
        }
    };
    look_up(0);
    for (int v0 = blockIdx.y * pieces + threadIdx.x; v0 < end; v0 += U * blockDim.x) {
        float y[U][8];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int v = v0 + u * blockDim.x;
#pragma unroll
            for (int e = 0; e < 8; ++e) y[u][e] = 0.0f;
            if (c.residual && v < end) load8<Y32, true>(c.residual, t * c.ldr + 8 * v, y[u]);
        }
        for (int j0 = 0; j0 < m.k; j0 += J) {
            if (m.k > J) look_up(j0);
            uint4 f[U][J][Q];
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int v = v0 + u * blockDim.x;
                    if (r[j] >= 0 && v < end) {
                        const uint4* q = reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(c.ys) + (r[j] * c.ldys + 8 * v) * (YS32 ? 4 : 2));
#pragma unroll
                        for (int h = 0; h < Q; ++h) f[u][j][h] = __ldg(q + h);
                    }
                }
#pragma unroll
            for (int j = 0; j < J; ++j)
                if (r[j] >= 0) {
#pragma unroll
                    for (int u = 0; u < U; ++u) {   // past the end: what is in the registers, and is not stored
                        float x[8];
                        widen(f[u][j], x);
#pragma unroll
                        for (int e = 0; e < 8; ++e) y[u][e] = fmaf(w[j], x[e], y[u][e]);
                    }
                }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int v = v0 + u * blockDim.x;
            if (v < end) store8<Y32>(c.y, t * c.ldy + 8 * v, y[u]);
        }
    }
}

// One block per token, as many threads as its row has pieces, up to 256 (narrow rows: up to 32 threads a token, several tokens a
// block).  The loads of up to 8 choices' rows are issued before the first is used.
constexpr int kGradThreads = 256;
template <int KMAX, bool YS32>
__global__ void __launch_bounds__(kGradThreads) combine_bwd_kernel(const CombineBwd c) {
    constexpr int J = KMAX < 8 ? KMAX : 8, Q = YS32 ? 2 : 1;
    __shared__ float part[kGradThreads / 32][KMAX];
    const TokenRows& m = c.m;
    const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const bool in = t < m.tokens;
    const int vecs = (int)(m.d >> 3), lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    for (int j0 = 0; j0 < m.k; j0 += J) {
        int64_t r[J];
        float w[J], dot[J];
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const bool choice = in && j0 + j < m.k;
            r[j] = choice ? row_of(m, t * m.k + j0 + j) : -1;
            w[j] = choice ? __ldg(m.weights + t * m.k + j0 + j) : 0.0f;
            dot[j] = 0.0f;
        }
        for (int v = threadIdx.x; v < vecs && in; v += blockDim.x) {
            const uint4 g4 = __ldg(reinterpret_cast<const uint4*>(c.dy + t * c.lddy) + v);
            uint4 f[J][Q];
#pragma unroll
            for (int j = 0; j < J; ++j)
                if (r[j] >= 0) {
                    const uint4* q = reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(c.ys) + (r[j] * c.ldys + 8 * v) * (YS32 ? 4 : 2));
#pragma unroll
                    for (int h = 0; h < Q; ++h) f[j][h] = __ldg(q + h);
                }
            float g[8];
            widen(g4, g);
#pragma unroll
            for (int j = 0; j < J; ++j)
                if (r[j] >= 0) {
                    float x[8], o[8];
                    widen(f[j], x);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        dot[j] = fmaf(g[e], x[e], dot[j]);
                        o[e] = w[j] * g[e];
                    }
                    store8<false>(c.dys, r[j] * c.lddys + 8 * v, o);
                }
        }
        __syncwarp();
        const int span = min((int)blockDim.x, 32);   // lanes of a token in a warp, a power of two
#pragma unroll
        for (int j = 0; j < J; ++j) {
            if (j0 + j >= m.k) break;
            for (int o = span >> 1; o > 0; o >>= 1) dot[j] += __shfl_xor_sync(0xFFFFFFFFu, dot[j], o);
            if (blockDim.x <= 32) {
                if (threadIdx.x == 0 && in) c.dweights[t * m.k + j0 + j] = dot[j];
            } else if (lane == 0) {
                part[warp][j0 + j] = dot[j];
            }
        }
    }
    if (blockDim.x <= 32) return;
    __syncthreads();
    if (threadIdx.x < m.k) {
        float s = 0.0f;
        for (int i = 0; i < warps; ++i) s += part[i][threadIdx.x];
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

// Threads for `vecs` pieces: as even a cut into rounds of at most `most` threads as warps allow; up to 32 pieces a power of two
// of threads, and as many tokens as make 128
static dim3 even_threads(int vecs, int most) {
    if (vecs <= 32) {
        unsigned x = 1;
        while ((int)x < vecs) x <<= 1;
        return dim3(x, 128 / x);
    }
    const int rounds = (vecs + most - 1) / most, each = (vecs + rounds - 1) / rounds;
    return dim3((unsigned)((each + 31) / 32 * 32));
}
template <int J>
static void launch_combine(const Combine& c, cudaStream_t s) {
    const int vecs = (int)(c.m.d / 8);
    // few tokens: their rows cut over blocks, a piece a thread
    const int64_t want = (8 * host::sm_count() + c.m.tokens - 1) / c.m.tokens;
    const int cuts = (int)std::max<int64_t>(1, std::min<int64_t>((vecs + 127) / 128, want));
    const int pieces = (vecs + cuts - 1) / cuts;
    const bool two = !c.ys_fp32 && pieces > 128;   // pieces a thread at a time
    const dim3 threads = even_threads(two ? (pieces + 1) / 2 : pieces, kCombineThreads);
    const dim3 grid((unsigned)((c.m.tokens + threads.y - 1) / threads.y), (unsigned)((vecs + pieces - 1) / pieces));
    if (c.ys_fp32) {
        if (c.y_fp32) combine_kernel<J, 1, true, true><<<grid, threads, 0, s>>>(c, pieces);
        else combine_kernel<J, 1, true, false><<<grid, threads, 0, s>>>(c, pieces);
    } else if (two) {
        if (c.y_fp32) combine_kernel<J, 2, false, true><<<grid, threads, 0, s>>>(c, pieces);
        else combine_kernel<J, 2, false, false><<<grid, threads, 0, s>>>(c, pieces);
    } else {
        if (c.y_fp32) combine_kernel<J, 1, false, true><<<grid, threads, 0, s>>>(c, pieces);
        else combine_kernel<J, 1, false, false><<<grid, threads, 0, s>>>(c, pieces);
    }
}
cudaError_t launch_combine(const Combine& c, cudaStream_t s) {
    if (c.m.k <= 2) launch_combine<2>(c, s);
    else launch_combine<4>(c, s);
    return cudaGetLastError();
}

template <int KMAX>
static void launch_combine_bwd(const CombineBwd& c, cudaStream_t s) {
    const dim3 threads = even_threads((int)(c.m.d / 8), kGradThreads);   // more than 32, the bound of k, or several tokens
    const unsigned blocks = (unsigned)((c.m.tokens + threads.y - 1) / threads.y);
    if (c.ys_fp32) combine_bwd_kernel<KMAX, true><<<blocks, threads, 0, s>>>(c);
    else combine_bwd_kernel<KMAX, false><<<blocks, threads, 0, s>>>(c);
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
