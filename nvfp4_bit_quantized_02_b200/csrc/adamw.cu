// adamw.cu -- one AdamW step over many tensors: fp32 master weights, fp32 or bf16 gradients,
// moments in fp32 or as E4M3 codes with a scale per 256 elements, bf16 weights out.
//
// The step reads each tensor once and writes it once; with ~30 fp32 operations per 30 bytes it is
// bound by memory.  The work is cut into chunks of 2048 elements (one CTA's 8 warps x 256
// elements), numbered through all tensors of the launch; a CTA takes a consecutive run of chunks,
// so it looks its first tensor up once and then walks.  The tensor table travels in the kernel's
// parameters (constant bank): no device copy that a captured graph or a second call could share.
//
// A warp owns a block of 256 consecutive elements, lane l the elements 4 l + 128 j + (0..3),
// j = 0, 1: every fp32 access is one 16-byte piece per lane and 512 consecutive bytes per warp, the
// codes' are 4 bytes and 128, and a block of an 8-bit moment is one warp's registers, so its amax is
// a warp reduction.
// Compiled without contraction: the update's fp32 operations are single IEEE operations in the
// order the header states, so the codes can be reproduced bit for bit.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "nvfp4_device.cuh"
#include "nvfp4_internal.h"

namespace nvfp4 {

constexpr int kAdamThreads = 256;
constexpr int kAdamBlock = 256;                                // elements per warp and per scale
constexpr int kAdamChunk = kAdamThreads / 32 * kAdamBlock;     // elements per CTA and step

template <int CAP>
struct AdamwTable {
    AdamwEntry t[CAP];
    int32_t count;
    uint32_t chunks;
};

// Two E4M3 codes (low byte first) to fp32, exact
__device__ __forceinline__ void e4m3x2_decode(uint32_t pair, float& lo, float& hi) {
    uint32_t h;
    asm("{\n\t.reg .b16 c;\n\tcvt.u16.u32 c, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, c;\n\t}" : "=r"(h) : "r"(pair & 0xFFFFu));
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(lo), "=f"(hi)
        : "r"(h));
}

// E4M3 code of x * per (per = 448 * (1 / amax) of the block), sign kept.  For u = |x| * per >= 2^-6 the
// code is the top bits of u's fp32 pattern; below, u + 2^-6 lies in a binade whose 3-bit step is
// the subnormal step 2^-9, so the same bits give the subnormal code plus 8.  Adding `round` to the
// 20 bits that are cut off carries into the code where it rounds up: 2^20 - 1 - 16 r16 does so iff
// r16 < f * 2^16 (f = the cut-off bits / 2^20), half a step less the parity bit gives nearest even.
__device__ __forceinline__ uint32_t e4m3_encode(float x, float per, bool sr, uint32_t r16) {
    const float u = __fmul_rn(fabsf(x), per);
    const bool low = u < 0.015625f;
    const uint32_t bits = __float_as_uint(low ? __fadd_rn(u, 0.015625f) : u);
    const uint32_t round = sr ? 0xFFFFFu - (r16 << 4) : 0x7FFFFu + ((bits >> 20) & 1u);
    const uint32_t code = min(((bits + round) >> 20) - (low ? 968u : 960u), 0x7Eu);
    return code | ((__float_as_uint(x) >> 24) & 0x80u);
}

// The four 16-bit fields of each of a lane's two element quads.  A Philox block serves eight
// consecutive elements, i.e. the quads of two neighbouring lanes: the even lane computes the block
// of the pair's j = 0 quads, the odd lane that of the j = 1 quads, and each hands the other half over.
__device__ __forceinline__ void quad_words(uint32_t (&w)[2][2], uint64_t block_base, uint32_t stream, uint32_t tensor,
                                           uint32_t k0, uint32_t k1) {
    const uint32_t lane = threadIdx.x & 31;
    const uint64_t g = (block_base + 4u * (lane & ~1u) + 128u * (lane & 1u)) >> 3;
    const U4 r = philox4x32_10((uint32_t)g, (uint32_t)(g >> 32), stream, tensor, k0, k1);
    const bool odd = lane & 1u;
    const uint32_t g0 = __shfl_xor_sync(0xFFFFFFFFu, odd ? r.x : r.z, 1);
    const uint32_t g1 = __shfl_xor_sync(0xFFFFFFFFu, odd ? r.y : r.w, 1);
    w[0][0] = odd ? g0 : r.x;
    w[0][1] = odd ? g1 : r.y;
    w[1][0] = odd ? r.z : g0;
    w[1][1] = odd ? r.w : g1;
}

// Encodes one moment's block: the scale, then the lane's two words of four codes
__device__ __forceinline__ void encode_block(const float (&x)[8], uint32_t (&codes)[2], float& scale, bool sr,
                                             uint64_t block_base, uint32_t stream, uint32_t tensor, uint32_t k0,
                                             uint32_t k1) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(x[i]) & 0x7FFFFFFFu);
    top = __reduce_max_sync(0xFFFFFFFFu, top);   // magnitudes order as integers, NaN above Inf above the rest
    const bool finite = top < 0x7F800000u, held = finite && top >= 0x0D800000u;   // 2^-100
    const float amax = __uint_as_float(top);
    scale = held ? __fmul_rn(amax, 1.0f / 448.0f) : finite ? 0.0f : __uint_as_float(0x7FC00000u);
    const float per = held ? __fmul_rn(448.0f, __frcp_rn(amax)) : 0.0f;
    uint32_t r[2][2] = {};
    if (sr) quad_words(r, block_base, stream, tensor, k0, k1);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        uint32_t c = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t r16 = (i & 1) ? r[j][i >> 1] >> 16 : r[j][i >> 1] & 0xFFFFu;
            const float v = finite ? x[4 * j + i] : 0.0f;
            c |= e4m3_encode(v, per, sr, r16) << (8 * i);
        }
        codes[j] = c;
    }
}

template <bool FP8, int CAP>
__global__ void __launch_bounds__(kAdamThreads)
    adamw_kernel(const __grid_constant__ AdamwTable<CAP> tab, const AdamwScalars sc, uint32_t* flags) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t c0 = (uint32_t)((uint64_t)tab.chunks * blockIdx.x / gridDim.x);
    const uint32_t c1 = (uint32_t)((uint64_t)tab.chunks * (blockIdx.x + 1) / gridDim.x);
    if (c0 >= c1) return;
    float keep = sc.keep, size = sc.step_size, fix = sc.v_fix, gs = sc.grad_scale;
    uint32_t k0 = (uint32_t)sc.sr_seed, k1 = (uint32_t)(sc.sr_seed >> 32);
    if (sc.dynamic) {
        const float4 d = __ldg(reinterpret_cast<const float4*>(sc.dynamic));
        const uint2 k = __ldg(reinterpret_cast<const uint2*>(sc.dynamic) + 2);
        keep = d.x;
        size = d.y;
        fix = d.z;
        gs = d.w;
        k0 = k.x;
        k1 = k.y;
    }
    // the tensor of chunk c0: the last entry whose first chunk is <= c0 (every entry has chunks)
    int ti = 0;
    for (int lo = 0, hi = tab.count; hi - lo > 1;) {
        const int mid = (lo + hi) >> 1;
        if (tab.t[mid].first_chunk <= c0) lo = mid; else hi = mid;
        ti = lo;
    }
    uint32_t am = 0;   // |w| bits of this thread's elements of the current tensor
    for (uint32_t c = c0; c < c1; ++c) {
        while (ti + 1 < tab.count && tab.t[ti + 1].first_chunk <= c) ++ti;
        const AdamwEntry& e = tab.t[ti];
        const int64_t base = (int64_t)(c - e.first_chunk) * kAdamChunk + warp * kAdamBlock;
        const int64_t n = e.n;
        if (base < n) {
            const bool full = base + kAdamBlock <= n;
            const int64_t at = base + 4 * lane;
            float p[8], g[8], m[8], v[8];
            if (full) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float4 x = *reinterpret_cast<const float4*>(e.p + at + 128 * j);
                    p[4 * j] = x.x; p[4 * j + 1] = x.y; p[4 * j + 2] = x.z; p[4 * j + 3] = x.w;
                    if ((e.index_g & 1)) {
                        const uint2 y = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint16_t*>(e.g) + at + 128 * j);
                        g[4 * j] = bf16_lo(y.x); g[4 * j + 1] = bf16_hi(y.x); g[4 * j + 2] = bf16_lo(y.y); g[4 * j + 3] = bf16_hi(y.y);
                    } else {
                        const float4 y = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(e.g) + at + 128 * j);
                        g[4 * j] = y.x; g[4 * j + 1] = y.y; g[4 * j + 2] = y.z; g[4 * j + 3] = y.w;
                    }
                    if (!FP8) {
                        const float4 a = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(e.m) + at + 128 * j);
                        const float4 b = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(e.v) + at + 128 * j);
                        m[4 * j] = a.x; m[4 * j + 1] = a.y; m[4 * j + 2] = a.z; m[4 * j + 3] = a.w;
                        v[4 * j] = b.x; v[4 * j + 1] = b.y; v[4 * j + 2] = b.z; v[4 * j + 3] = b.w;
                    } else {
                        const uint32_t a = *reinterpret_cast<const uint32_t*>(reinterpret_cast<const uint8_t*>(e.m) + at + 128 * j);
                        const uint32_t b = *reinterpret_cast<const uint32_t*>(reinterpret_cast<const uint8_t*>(e.v) + at + 128 * j);
                        e4m3x2_decode(a, m[4 * j], m[4 * j + 1]);
                        e4m3x2_decode(a >> 16, m[4 * j + 2], m[4 * j + 3]);
                        e4m3x2_decode(b, v[4 * j], v[4 * j + 1]);
                        e4m3x2_decode(b >> 16, v[4 * j + 2], v[4 * j + 3]);
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int64_t k = at + 128 * (i >> 2) + (i & 3);
                    const bool in = k < n;
                    p[i] = in ? e.p[k] : 0.0f;
                    g[i] = !in ? 0.0f : (e.index_g & 1) ? __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(e.g)[k] << 16)
                                                 : reinterpret_cast<const float*>(e.g)[k];
                    if (!FP8) {
                        m[i] = in ? reinterpret_cast<const float*>(e.m)[k] : 0.0f;
                        v[i] = in ? reinterpret_cast<const float*>(e.v)[k] : 0.0f;
                    } else {
                        float unused;
                        e4m3x2_decode(in ? reinterpret_cast<const uint8_t*>(e.m)[k] : 0u, m[i], unused);
                        e4m3x2_decode(in ? reinterpret_cast<const uint8_t*>(e.v)[k] : 0u, v[i], unused);
                    }
                }
            }
            if (FP8) {
                const float ms = e.m_scale[base / kAdamBlock], vs = e.v_scale[base / kAdamBlock];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const bool in = full || at + 128 * (i >> 2) + (i & 3) < n;   // a NaN scale stays out of the padding
                    m[i] = in ? __fmul_rn(m[i], ms) : 0.0f;
                    const float r = in ? __fmul_rn(v[i], vs) : 0.0f;
                    v[i] = __fmul_rn(r, r);
                }
            }
            float root[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float gi = __fmul_rn(g[i], gs);
                m[i] = __fadd_rn(__fmul_rn(m[i], sc.beta1), __fmul_rn(gi, sc.one_beta1));
                v[i] = __fadd_rn(__fmul_rn(v[i], sc.beta2), __fmul_rn(__fmul_rn(gi, sc.one_beta2), gi));
                root[i] = __fsqrt_rn(v[i]);
                const float q = __fdiv_rn(m[i], __fadd_rn(__fmul_rn(root[i], fix), sc.eps));
                p[i] = __fsub_rn(__fmul_rn(p[i], keep), __fmul_rn(q, size));
            }
            uint32_t wb[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) wb[i] = f32x2_to_bf16x2(p[2 * i], p[2 * i + 1]);
            uint32_t mc[2], vc[2];
            if (FP8) {
                float ms, vs;
                const uint32_t tensor = (uint32_t)e.index_g >> 1;
                encode_block(m, mc, ms, sc.sr, (uint64_t)base, kStreamMoment1, tensor, k0, k1);
                encode_block(root, vc, vs, sc.sr, (uint64_t)base, kStreamMoment2, tensor, k0, k1);
                if (lane == 0) {
                    e.m_scale[base / kAdamBlock] = ms;
                    e.v_scale[base / kAdamBlock] = vs;
                }
            }
            if (full) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    *reinterpret_cast<float4*>(e.p + at + 128 * j) = make_float4(p[4 * j], p[4 * j + 1], p[4 * j + 2], p[4 * j + 3]);
                    if (e.w) *reinterpret_cast<uint2*>(e.w + at + 128 * j) = make_uint2(wb[2 * j], wb[2 * j + 1]);
                    if (!FP8) {
                        *reinterpret_cast<float4*>(reinterpret_cast<float*>(e.m) + at + 128 * j) =
                            make_float4(m[4 * j], m[4 * j + 1], m[4 * j + 2], m[4 * j + 3]);
                        *reinterpret_cast<float4*>(reinterpret_cast<float*>(e.v) + at + 128 * j) =
                            make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
                    } else {
                        *reinterpret_cast<uint32_t*>(reinterpret_cast<uint8_t*>(e.m) + at + 128 * j) = mc[j];
                        *reinterpret_cast<uint32_t*>(reinterpret_cast<uint8_t*>(e.v) + at + 128 * j) = vc[j];
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int64_t k = at + 128 * (i >> 2) + (i & 3);
                    if (k >= n) continue;
                    e.p[k] = p[i];
                    if (e.w) e.w[k] = (uint16_t)(wb[i >> 1] >> (16 * (i & 1)));
                    if (!FP8) {
                        reinterpret_cast<float*>(e.m)[k] = m[i];
                        reinterpret_cast<float*>(e.v)[k] = v[i];
                    } else {
                        reinterpret_cast<uint8_t*>(e.m)[k] = (uint8_t)(mc[i >> 2] >> (8 * (i & 3)));
                        reinterpret_cast<uint8_t*>(e.v)[k] = (uint8_t)(vc[i >> 2] >> (8 * (i & 3)));
                    }
                }
            }
            if (e.amax) {
                // elements past n hold p = 0 - 0 * size: no effect on the maximum (or NaN, from
                // eps = 0, so they are masked)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const bool in = full || at + 128 * (i >> 2) + (i & 3) < n;
                    const uint32_t b = (wb[i >> 1] >> (16 * (i & 1))) & 0x7FFFu;
                    am = max(am, in ? b : 0u);
                }
            }
        }
        // the run of this tensor ends here: its maximum so far
        if (e.amax && (c + 1 == c1 || (ti + 1 < tab.count && tab.t[ti + 1].first_chunk == c + 1))) {
            const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, am);
            am = 0;
            if (lane == 0 && top) {
                atomicMax(e.amax, top << 16);
                if (top >= 0x7F80u) atomicOr(flags, kFlagNonFinite);
            }
        }
    }
}

template <int CAP>
__global__ void adamw_reset_amax_kernel(const __grid_constant__ AdamwTable<CAP> tab) {
    const int i = threadIdx.x + blockIdx.x * blockDim.x;
    if (i < tab.count && tab.t[i].amax) *tab.t[i].amax = 0u;
}

static int sm_count_adamw() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
        return 148;
    return n;
}

template <bool FP8, int CAP>
static cudaError_t launch_table(const AdamwEntry* entries, int count, const AdamwScalars& sc,
                                uint32_t* flags, cudaStream_t s) {
    AdamwTable<CAP> tab;
    uint64_t chunks = 0;
    bool any_amax = false;
    for (int i = 0; i < count; ++i) {
        tab.t[i] = entries[i];
        tab.t[i].first_chunk = (uint32_t)chunks;
        chunks += (uint64_t)((entries[i].n + kAdamChunk - 1) / kAdamChunk);
        any_amax |= entries[i].amax != nullptr;
    }
    if (chunks > 0xFFFFFFFFull) return cudaErrorInvalidValue;
    tab.count = count;
    tab.chunks = (uint32_t)chunks;
    if (any_amax) adamw_reset_amax_kernel<CAP><<<(CAP + 127) / 128, 128, 0, s>>>(tab);
    const uint64_t most = (uint64_t)sm_count_adamw() * 4;
    adamw_kernel<FP8, CAP><<<(unsigned)std::min<uint64_t>(chunks, most), kAdamThreads, 0, s>>>(tab, sc, flags);
    return cudaGetLastError();
}

cudaError_t launch_adamw(const AdamwEntry* entries, int count, bool fp8, const AdamwScalars& sc, uint32_t* flags, cudaStream_t s) {
    if (count < 1 || count > kAdamMaxTensors) return cudaErrorInvalidValue;
    // two table sizes: a launch copies its whole parameter block (80 bytes per tensor)
    if (count <= 16)
        return fp8 ? launch_table<true, 16>(entries, count, sc, flags, s)
                   : launch_table<false, 16>(entries, count, sc, flags, s);
    return fp8 ? launch_table<true, kAdamMaxTensors>(entries, count, sc, flags, s)
               : launch_table<false, kAdamMaxTensors>(entries, count, sc, flags, s);
}

}  // namespace nvfp4
