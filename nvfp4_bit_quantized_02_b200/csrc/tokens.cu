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
#include <atomic>
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
// before the first is used.  8192 tokens x 2 x 5120 in fp32, with a residual: 99 us (6.8 TB/s).
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
// Many tokens: warps that stay, each thread with a ring of its own in shared memory that cp.async fills kRing - 1 steps ahead.
// What a thread copies it reads itself, so that nothing waits for another thread, and the rows and weights of a token are on
// their way during the one before.  A block for each token has to look its rows up, then load, then store, with as many bytes in
// flight as registers hold.  8192 tokens x 2 x 5120 with a residual: 53 us (6.3 TB/s; 69 by blocks), the gradient of 3001 x 3 x 1032
// 12.1 us (14.2).  Rows of fp32 are left to the blocks: pieces of 32 bytes copied 16 at a time fill half of each request
// (8192 x 2 x 5120 in fp32: 99 us by blocks, 181 by rings).
// ---------------------------------------------------------------------------------------
constexpr int kRing = 4, kRingWarps = 4;

struct RingGrid {
    int32_t rounds;        // of 32 pieces, of a unit
    int32_t cuts;          // units of a token
    int32_t warps;         // all of the launch
    int32_t step_tokens, step_cuts;   // warps = step_tokens * cuts + step_cuts
};

// A unit: `rounds` rounds of 32 pieces of a token, taken by one warp
template <int J, bool Y32>
__global__ void __launch_bounds__(32 * kRingWarps) combine_ring_kernel(const Combine c, const RingGrid g) {
    extern __shared__ __align__(16) uint8_t ring[];
    constexpr int R = Y32 ? 2 : 1, kSlot = 16 * 32 * kRingWarps;
    const TokenRows& m = c.m;
    const uint16_t* ys = reinterpret_cast<const uint16_t*>(c.ys);
    const int lane = threadIdx.x & 31, k = m.k, vecs = (int)(m.d >> 3);
    const int warp = blockIdx.x * kRingWarps + (threadIdx.x >> 5);
    const int slots = k + (c.residual ? R : 0);
    const uint32_t own = ptx::smem_u32(ring) + 16 * threadIdx.x, stage = slots * kSlot;
    const int64_t t0 = warp / g.cuts;
    const int cut0 = warp - (int)t0 * g.cuts;

    // one walk over the warp's units for what is asked for, one for what is used
    struct Walk {
        int64_t t;
        int cut, round;
    };
    const auto advance = [&](int64_t& t, int& cut) {
        t += g.step_tokens;
        cut += g.step_cuts;
        if (cut >= g.cuts) {
            cut -= g.cuts;
            ++t;
        }
    };
    const auto rows = [&](int64_t t, int32_t (&r)[J]) {
#pragma unroll
        for (int j = 0; j < J; ++j) r[j] = t < m.tokens && j < k ? (int32_t)row_of(m, t * k + j) : -1;
    };
    const auto weights = [&](int64_t t, float (&w)[J]) {
#pragma unroll
        for (int j = 0; j < J; ++j) w[j] = t < m.tokens && j < k && m.weights ? __ldg(m.weights + t * k + j) : 1.0f;
    };
    Walk in{t0, cut0, 0}, out{t0, cut0, 0};
    int32_t r[J], r_next[J], used[J], used_next[J];
    float w[J], w_next[J];
    const auto follow = [&](const Walk& a, int32_t (&rn)[J]) {   // the next unit's rows
        int64_t t = a.t;
        int cut = a.cut;
        advance(t, cut);
        rows(t, rn);
        return t;
    };
    rows(t0, r);
    follow(in, r_next);
    const auto ask = [&](int s) {
        const int v = (in.cut * g.rounds + in.round) * 32 + lane;
        if (in.t < m.tokens && v < vecs) {
            uint32_t to = own + s * stage;
#pragma unroll
            for (int j = 0; j < J; ++j) {
                if (j < k) {
                    if (r[j] >= 0) ptx::copy16(to, ys + (int64_t)r[j] * c.ldys + 8 * v);
                    to += kSlot;
                }
            }
            if (c.residual) {
                const uint8_t* from = reinterpret_cast<const uint8_t*>(c.residual) + (in.t * c.ldr + 8 * v) * (Y32 ? 4 : 2);
#pragma unroll
                for (int q = 0; q < R; ++q) ptx::copy16(to + q * kSlot, from + 16 * q);
            }
        }
        ptx::copies_end();
        if (++in.round == g.rounds) {
            in.round = 0;
            advance(in.t, in.cut);
#pragma unroll
            for (int j = 0; j < J; ++j) r[j] = r_next[j];
            follow(in, r_next);
        }
    };
#pragma unroll
    for (int s = 0; s < kRing - 1; ++s) ask(s);
    rows(t0, used);
    weights(t0, w);
    weights(follow(out, used_next), w_next);
    for (int s = 0; out.t < m.tokens; s = s + 1 == kRing ? 0 : s + 1) {
        ask(s == 0 ? kRing - 1 : s - 1);
        ptx::copies_wait<kRing - 1>();
        const int v = (out.cut * g.rounds + out.round) * 32 + lane;
        if (v < vecs) {
            uint32_t at = own + s * stage;
            float y[8] = {}, x[8];
            if (c.residual) {
                uint4 f[R];
#pragma unroll
                for (int q = 0; q < R; ++q) f[q] = ptx::take16(at + (k + q) * kSlot);
                widen(f, y);
            }
#pragma unroll
            for (int j = 0; j < J; ++j) {
                if (used[j] >= 0) {
                    widen(ptx::take16(at + j * kSlot), x);
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[e] = fmaf(w[j], x[e], y[e]);
                }
            }
            store8<Y32>(c.y, out.t * c.ldy + 8 * v, y);
        }
        if (++out.round == g.rounds) {
            out.round = 0;
            advance(out.t, out.cut);
#pragma unroll
            for (int j = 0; j < J; ++j) {
                used[j] = used_next[j];
                w[j] = w_next[j];
            }
            weights(follow(out, used_next), w_next);
        }
    }
}

// A token by a block's warps
template <int J>
__global__ void __launch_bounds__(256) combine_bwd_ring_kernel(const CombineBwd c, int rounds) {
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ float part[2][8][J];
    const TokenRows& m = c.m;
    const uint16_t* ys = reinterpret_cast<const uint16_t*>(c.ys);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5, k = m.k, vecs = (int)(m.d >> 3);
    const uint32_t slot = 16 * blockDim.x, stage = (1 + k) * slot, own = ptx::smem_u32(ring) + 16 * threadIdx.x;
    const auto rows = [&](int64_t t, int32_t (&r)[J]) {
#pragma unroll
        for (int j = 0; j < J; ++j) r[j] = t < m.tokens && j < k ? (int32_t)row_of(m, t * k + j) : -1;
    };
    const auto weights = [&](int64_t t, float (&w)[J]) {
#pragma unroll
        for (int j = 0; j < J; ++j) w[j] = t < m.tokens && j < k ? __ldg(m.weights + t * k + j) : 0.0f;
    };
    int64_t in = blockIdx.x, out = blockIdx.x;
    int in_round = 0, round = 0, buffer = 0;
    int32_t r[J], r_next[J], used[J], used_next[J];
    float w[J], w_next[J], dot[J] = {};
    rows(in, r);
    rows(in + gridDim.x, r_next);
    const auto ask = [&](int s) {
        const int v = in_round * (int)blockDim.x + (int)threadIdx.x;
        if (in < m.tokens && v < vecs) {
            uint32_t to = own + s * stage;
            ptx::copy16(to, c.dy + in * c.lddy + 8 * v);
#pragma unroll
            for (int j = 0; j < J; ++j) {
                if (r[j] >= 0) ptx::copy16(to + (1 + j) * slot, ys + (int64_t)r[j] * c.ldys + 8 * v);
            }
        }
        ptx::copies_end();
        if (++in_round == rounds) {
            in_round = 0;
            in += gridDim.x;
#pragma unroll
            for (int j = 0; j < J; ++j) r[j] = r_next[j];
            rows(in + gridDim.x, r_next);
        }
    };
#pragma unroll
    for (int s = 0; s < kRing - 1; ++s) ask(s);
    rows(out, used);
    weights(out, w);
    rows(out + gridDim.x, used_next);
    weights(out + gridDim.x, w_next);
    for (int s = 0; out < m.tokens; s = s + 1 == kRing ? 0 : s + 1) {
        ask(s == 0 ? kRing - 1 : s - 1);
        ptx::copies_wait<kRing - 1>();
        const int v = round * (int)blockDim.x + (int)threadIdx.x;
        if (v < vecs) {
            const uint32_t at = own + s * stage;
            float g[8];
            widen(ptx::take16(at), g);
#pragma unroll
            for (int j = 0; j < J; ++j) {
                if (used[j] >= 0) {
                    float x[8], o[8];
                    widen(ptx::take16(at + (1 + j) * slot), x);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        dot[j] = fmaf(g[e], x[e], dot[j]);
                        o[e] = w[j] * g[e];
                    }
                    store8<false>(c.dys, (int64_t)used[j] * c.lddys + 8 * v, o);
                }
            }
        }
        if (++round < rounds) continue;
        round = 0;
        __syncwarp();
#pragma unroll
        for (int j = 0; j < J; ++j) {
            if (j >= k) break;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) dot[j] += __shfl_xor_sync(0xFFFFFFFFu, dot[j], o);
            if (lane == 0) {
                if (warps == 1) c.dweights[out * k + j] = dot[j];
                else part[buffer][warp][j] = dot[j];
            }
            dot[j] = 0.0f;
        }
        if (warps > 1) {   // two buffers: the sums are read before the next token's barrier, this buffer is written behind it
            __syncthreads();
            if ((int)threadIdx.x < k) {
                float sum = 0.0f;
                for (int i = 0; i < warps; ++i) sum += part[buffer][i][threadIdx.x];
                c.dweights[out * k + threadIdx.x] = sum;
            }
            buffer ^= 1;
        }
        out += gridDim.x;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            used[j] = used_next[j];
            w[j] = w_next[j];
        }
        rows(out + gridDim.x, used_next);
        weights(out + gridDim.x, w_next);
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
constexpr int kRingSmem = 200 * 1024;   // of an SM's, for the rings of its blocks

template <int J, bool Y32>
static cudaError_t launch_combine_ring(const Combine& c, const RingGrid& g, int blocks, int smem, cudaStream_t s) {
    static std::atomic<uint64_t> attr{0};
    auto kern = combine_ring_kernel<J, Y32>;
    if (cudaError_t e = host::ensure_smem(reinterpret_cast<const void*>(kern), kRingSmem, attr)) return e;
    kern<<<blocks, 32 * kRingWarps, smem, s>>>(c, g);
    return cudaGetLastError();
}
cudaError_t launch_combine(const Combine& c, cudaStream_t s) {
    // Rings from 24 MB on, for up to 4 choices and rows of 512 elements.  us by blocks and by rings, bf16 with a residual: 1024 x 2 x
    // 2048 (17 MB) 5.9, 6.2; 2048 x 2 x 2048 (34 MB) 9.8, 9.0; 16384 x 2 x 2048 54, 43; 16384 x 2 x 256 10.0, 10.7; 4096 x 4 x 5120 46, 42;
    // 2048 x 8 x 5120 41, 49 (what is held of a token leaves an SM few warps).
    const int64_t bytes = c.m.tokens * c.m.d * (2 * c.m.k + (c.y_fp32 ? 4 : 2) * (c.residual ? 2 : 1));
    if (!c.ys_fp32 && c.m.k <= 4 && c.m.d >= 512 && bytes >= 24 << 20) {
        const int slots = c.m.k + (c.residual ? c.y_fp32 ? 2 : 1 : 0);
        const int smem = kRing * slots * 16 * 32 * kRingWarps;   // 48 KB at most
        const int blocks = host::sm_count() * std::min(8, kRingSmem / (smem + 1024));
        RingGrid g{};
        g.warps = blocks * kRingWarps;
        const int all = (int)((c.m.d / 8 + 31) / 32);   // rounds of a token
        g.cuts = (all + 4) / 5;
        g.rounds = (all + g.cuts - 1) / g.cuts;
        g.step_tokens = g.warps / g.cuts;
        g.step_cuts = g.warps % g.cuts;
        if (c.m.k <= 2) return c.y_fp32 ? launch_combine_ring<2, true>(c, g, blocks, smem, s) : launch_combine_ring<2, false>(c, g, blocks, smem, s);
        return c.y_fp32 ? launch_combine_ring<4, true>(c, g, blocks, smem, s) : launch_combine_ring<4, false>(c, g, blocks, smem, s);
    }
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
template <int J>
static cudaError_t launch_combine_bwd_ring(const CombineBwd& c, int blocks, int warps, int rounds, int smem, cudaStream_t s) {
    static std::atomic<uint64_t> attr{0};
    auto kern = combine_bwd_ring_kernel<J>;
    if (cudaError_t e = host::ensure_smem(reinterpret_cast<const void*>(kern), kRingSmem, attr)) return e;
    kern<<<blocks, 32 * warps, smem, s>>>(c, rounds);
    return cudaGetLastError();
}
cudaError_t launch_combine_bwd(const CombineBwd& c, cudaStream_t s) {
    const int k = c.m.k;
    // Rings from 16 MB and 512 tokens on, for up to 8 choices and rows of 512 elements.  us by blocks and by rings: 1024 x 2 x 1032
    // (11 MB) 4.4, 4.8; 2048 x 2 x 1032 (21 MB) 7.8, 7.1; 16384 x 8 x 1024 137, 104; 16384 x 8 x 256 38, 49; 256 x 8 x 2048 7.8, 9.8;
    // 2048 x 8 x 2048 40, 29; 8192 x 2 x 5120 73, 72.
    if (!c.ys_fp32 && k <= 8 && c.m.tokens >= 512 && c.m.d >= 512 && c.m.tokens * c.m.d * (4 * k + 2) >= 16 << 20) {
        const int all = (int)((c.m.d / 8 + 31) / 32);   // rounds of one warp
        const int warps = std::min(8, (all + 4) / 5), rounds = (all + warps - 1) / warps;
        const int smem = kRing * (1 + k) * 16 * 32 * warps;   // 144 KB at most
        const int blocks = (int)std::min<int64_t>(c.m.tokens, host::sm_count() * std::min(32 / warps, kRingSmem / (smem + 1024)));
        if (k <= 2) return launch_combine_bwd_ring<2>(c, blocks, warps, rounds, smem, s);
        if (k <= 4) return launch_combine_bwd_ring<4>(c, blocks, warps, rounds, smem, s);
        return launch_combine_bwd_ring<8>(c, blocks, warps, rounds, smem, s);
    }
    if (k <= 2) launch_combine_bwd<2>(c, s);
    else if (k <= 4) launch_combine_bwd<4>(c, s);
    else if (k <= 8) launch_combine_bwd<8>(c, s);
    else launch_combine_bwd<kRouteMaxK>(c, s);
    return cudaGetLastError();
}

}  // namespace nvfp4
