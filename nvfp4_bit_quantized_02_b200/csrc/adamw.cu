// adamw.cu -- one AdamW step over many tensors: fp32 master weights, fp32 or bf16 gradients,
// moments in fp32 or as E4M3 codes with a scale per 256 elements, bf16 weights out.
//
// The step reads each tensor once and writes it once: 30 bytes an element with fp32 moments and
// gradients, 16 to 18 with 8-bit moments.  The work is cut into chunks of 1024 elements (one CTA's 4
// warps x 256 elements), numbered through all tensors of the launch; a CTA takes a consecutive run of
// chunks, so it looks its first tensor up once and then walks with running addresses (looking every
// chunk's addresses up again cost 15 of 115 instructions an element).  One wave of CTAs, 8 of 128
// threads per SM.  The tensor table travels in the kernel's parameters (constant bank): no device
// copy that a captured graph or a second call could share.
//
// Measured: 2 x 104857600 elements, fp32 moments, 1040 us, 6.05 TB/s, 92 % of the copy bandwidth: bound by
// memory.  200 tensors of 1000 to 4.8 M elements (107 M in all), E4M3 moments, bf16 gradients, 385 us,
// 4.8 TB/s (rounded to nearest 371): bound by instruction issue and load latency together, ~83 instructions
// an element (Philox and the rounding's random bits 19, square root and quotient 23), two thirds of the
// issue slots taken.  These are replays after a pause; a call among others takes 1056 to 1064 and 411 to 418.
// Without effect there: the next block's loads ahead in registers (530 us when the rest took 443), by an
// L2 prefetch (481) or by asynchronous copies into shared memory (425 when the rest took 384), streaming
// loads and stores (387), the approximate quotient (2 %); 7 or 9 CTAs per SM 394, 4 of 256 threads 4 % more.
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
#include "sm100_ptx.cuh"

namespace nvfp4 {

constexpr int kAdamThreads = 128;
constexpr int kAdamBlock = 256;                                // elements per warp and per scale
constexpr int kAdamChunk = kAdamThreads / 32 * kAdamBlock;     // elements per CTA and step

template <int CAP>
struct AdamwTable {
    AdamwEntry t[CAP];
    int32_t count;
    uint32_t chunks;
    uint32_t key0[10], key1[10];   // Philox round keys of the arguments' seed (constant-bank operands)
};

// Decodes the four codes of a word times `scale`, one rounding each (a code is exact in fp16).
__device__ __forceinline__ void decode4(uint32_t w, float scale, float* x) {
    uint32_t h[2];
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\tcvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
        : "=r"(h[0]), "=r"(h[1])
        : "r"(w));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float lo, hi;
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}" : "=f"(lo), "=f"(hi) : "r"(h[i]));
        f2_split(f2_mul(f2(lo, hi), f2c(scale)), x[2 * i], x[2 * i + 1]);
    }
}

// E4M3 code of u = |x| * per (per = 448 * (1 / amax) of the block) in the top byte, from the fp32
// pattern of x * per * 2^-120, whose bits 20-26 are the code's fields (below 2^-6 the number is an fp32
// subnormal, rounded to the step that u + 2^-6 would have).  Four places to the left, where the sign
// falls out, 24 bits are cut off.  Adding `cut` to them carries into the code where it rounds up:
// 2^24 - 1 - 256 r16 does so iff r16 < f * 2^16 (f = the cut-off bits / 2^24), half a step less the
// parity bit gives nearest even.
template <bool SR>
__device__ __forceinline__ uint32_t e4m3_code(float scaled, uint32_t cut) {
    const uint32_t bits = __float_as_uint(scaled);
    if (!SR) cut = 0x7FFFFFu + ((bits >> 20) & 1u);
    return 16u * bits + cut;
}
// The top bytes of four codes, at most 0x7E (u may exceed 448 by its rounding)
__device__ __forceinline__ uint32_t pack_codes(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3) {
    const uint32_t lo = __vminu2(__byte_perm(c0, c1, 0x7632), 0x7EFF7EFFu), hi = __vminu2(__byte_perm(c2, c3, 0x7632), 0x7EFF7EFFu);
    return __byte_perm(lo, hi, 0x7531);
}

// The Philox words of a lane's two element quads.  A block of four words serves eight consecutive
// elements, i.e. the quads of two neighbouring lanes: the even lane computes the block of the pair's
// j = 0 quads, the odd lane that of the j = 1 quads, and each hands the other half over.
__device__ __forceinline__ void quad_words(uint32_t (&w)[2][2], uint64_t block_base, uint32_t stream, uint32_t tensor,
                                           const uint32_t* key0, const uint32_t* key1) {
    const uint32_t lane = threadIdx.x & 31;
    const uint64_t g = (block_base + 4u * (lane & ~1u) + 128u * (lane & 1u)) >> 3;
    uint32_t c0 = (uint32_t)g, c1 = (uint32_t)(g >> 32), c2 = stream, c3 = tensor;
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t p0 = (uint64_t)0xD2511F53u * c0, p1 = (uint64_t)0xCD9E8D57u * c2;
        const uint32_t n0 = (uint32_t)(p1 >> 32) ^ c1 ^ key0[r], n2 = (uint32_t)(p0 >> 32) ^ c3 ^ key1[r];
        c1 = (uint32_t)p1;
        c3 = (uint32_t)p0;
        c0 = n0;
        c2 = n2;
    }
    const bool odd = lane & 1u;
    const uint32_t h0 = __shfl_xor_sync(0xFFFFFFFFu, odd ? c0 : c2, 1);
    const uint32_t h1 = __shfl_xor_sync(0xFFFFFFFFu, odd ? c1 : c3, 1);
    w[0][0] = odd ? h0 : c0;
    w[0][1] = odd ? h1 : c1;
    w[1][0] = odd ? c2 : h0;
    w[1][1] = odd ? c3 : h1;
}

// max(a, |b|, |c|), a >= 0, NaN where there is one
__device__ __forceinline__ float max3_abs_nan(float a, float b, float c) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(fabsf(b)), "f"(fabsf(c)));
    return r;
}

// Encodes one moment's block: the scale, then the lane's two words of four codes
template <bool SR, bool SIGNED>
__device__ __forceinline__ void encode_block(const float (&x)[8], uint32_t (&codes)[2], float& scale, uint64_t block_base,
                                             uint32_t stream, uint32_t tensor, const uint32_t* key0,
                                             const uint32_t* key1) {
    float t0 = max3_abs_nan(fabsf(x[0]), x[1], x[2]), t1 = max3_abs_nan(fabsf(x[3]), x[4], x[5]);
    t0 = max3_abs_nan(t0, x[6], x[7]);
    uint32_t top = __float_as_uint(max3_abs_nan(t0, t1, t1)) & 0x7FFFFFFFu;
    top = __reduce_max_sync(0xFFFFFFFFu, top);   // magnitudes order as integers, NaN above Inf above the rest
    if (top >= 0x7F800000u) {
        scale = __uint_as_float(0x7FC00000u);
        codes[0] = codes[1] = 0u;
        return;
    }
    const bool held = top >= 0x0D800000u;   // 2^-100
    const float amax = __uint_as_float(top);
    scale = held ? __fmul_rn(amax, 1.0f / 448.0f) : 0.0f;
    const float per = held ? __fmul_rn(448.0f, __frcp_rn(amax)) : 0.0f;
    uint32_t r[2][2] = {};
    if (SR) quad_words(r, block_base, stream, tensor, key0, key1);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        uint32_t c[4];
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
            float lo, hi;
            f2_split(f2_mul(f2_mul(f2(x[4 * j + i], x[4 * j + i + 1]), f2c(per)), f2c(0x1p-120f)), lo, hi);
            // 2^24 - 1 - 256 r16: r16's complement and a byte of ones
            const uint32_t n = ~r[j][i >> 1];
            c[i] = e4m3_code<SR>(lo, __byte_perm(n, 0xFFu, 0x5104));
            c[i + 1] = e4m3_code<SR>(hi, __byte_perm(n, 0xFFu, 0x5324));
        }
        codes[j] = pack_codes(c[0], c[1], c[2], c[3]);
        if (SIGNED) {
            const uint32_t s01 = __byte_perm(__float_as_uint(x[4 * j]), __float_as_uint(x[4 * j + 1]), 0x0073);
            const uint32_t s23 = __byte_perm(__float_as_uint(x[4 * j + 2]), __float_as_uint(x[4 * j + 3]), 0x0073);
            codes[j] |= __byte_perm(s01, s23, 0x5410) & 0x80808080u;
        }
    }
}

// The step's scalars and the tensor's constants as one chunk uses them
struct StepValues {
    float keep, size, fix, gs;
};

// This thread's places in the current chunk of a tensor: lane l of a warp owns elements 4 l + 128 j +
// (0..3), j = 0, 1, of the warp's block.  They advance by whole chunks.
template <bool FP8>
struct Places {
    float* p;
    const uint8_t* g;
    uint16_t* w;
    uint8_t *m, *v;            // fp32, or codes
    float *m_scale, *v_scale;  // of the warp's block
    bool g_bf16;
    __device__ __forceinline__ Places(const AdamwEntry& e, int64_t chunk) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        const int64_t at = chunk * kAdamChunk + warp * kAdamBlock + 4 * lane;
        g_bf16 = e.index_g & 1;
        p = e.p + at;
        g = reinterpret_cast<const uint8_t*>(e.g) + at * (g_bf16 ? 2 : 4);
        w = e.w ? e.w + at : nullptr;
        m = reinterpret_cast<uint8_t*>(e.m) + at * (FP8 ? 1 : 4);
        v = reinterpret_cast<uint8_t*>(e.v) + at * (FP8 ? 1 : 4);
        m_scale = e.m_scale + chunk * (kAdamChunk / kAdamBlock) + warp;
        v_scale = e.v_scale + chunk * (kAdamChunk / kAdamBlock) + warp;
    }
    __device__ __forceinline__ void next() {
        p += kAdamChunk;
        g += kAdamChunk * (g_bf16 ? 2 : 4);
        if (w) w += kAdamChunk;
        m += kAdamChunk * (FP8 ? 1 : 4);
        v += kAdamChunk * (FP8 ? 1 : 4);
        if (FP8) {
            m_scale += kAdamChunk / kAdamBlock;
            v_scale += kAdamChunk / kAdamBlock;
        }
    }
};

// One warp's block.  FULL: all its 256 elements are there; otherwise `left` (> 0) of them, counted
// from the block's first.  `first` is the block's first element's index, for the random fields.
template <bool FP8, bool SR, bool FULL>
__device__ __forceinline__ void block_step(const Places<FP8>& at, int64_t first, int left, uint32_t tensor, const AdamwScalars& sc,
                                           const StepValues& sv, const uint32_t* key0, const uint32_t* key1, bool amax,
                                           uint32_t& am) {
    const int lane = threadIdx.x & 31;
    const auto in = [&](int i) { return FULL || 4 * lane + 128 * (i >> 2) + (i & 3) < left; };
    const auto off = [](int i) { return 128 * (i >> 2) + (i & 3); };
    float p[8], g[8], m[8], v[8];
    uint32_t mc[2] = {0u, 0u}, vc[2] = {0u, 0u};   // codes of the 8-bit moments
    if (FULL) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float4 x = *reinterpret_cast<const float4*>(at.p + 128 * j);
            p[4 * j] = x.x; p[4 * j + 1] = x.y; p[4 * j + 2] = x.z; p[4 * j + 3] = x.w;
            if (at.g_bf16) {
                const uint2 y = *reinterpret_cast<const uint2*>(at.g + 256 * j);
                g[4 * j] = bf16_lo(y.x); g[4 * j + 1] = bf16_hi(y.x); g[4 * j + 2] = bf16_lo(y.y); g[4 * j + 3] = bf16_hi(y.y);
            } else {
                const float4 y = *reinterpret_cast<const float4*>(at.g + 512 * j);
                g[4 * j] = y.x; g[4 * j + 1] = y.y; g[4 * j + 2] = y.z; g[4 * j + 3] = y.w;
            }
            if (FP8) {
                mc[j] = *reinterpret_cast<const uint32_t*>(at.m + 128 * j);
                vc[j] = *reinterpret_cast<const uint32_t*>(at.v + 128 * j);
            } else {
                const float4 a = *reinterpret_cast<const float4*>(at.m + 512 * j);
                const float4 b = *reinterpret_cast<const float4*>(at.v + 512 * j);
                m[4 * j] = a.x; m[4 * j + 1] = a.y; m[4 * j + 2] = a.z; m[4 * j + 3] = a.w;
                v[4 * j] = b.x; v[4 * j + 1] = b.y; v[4 * j + 2] = b.z; v[4 * j + 3] = b.w;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const bool ok = in(i);
            p[i] = ok ? at.p[off(i)] : 0.0f;
            g[i] = !ok ? 0.0f : at.g_bf16 ? __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(at.g)[off(i)] << 16)
                                          : reinterpret_cast<const float*>(at.g)[off(i)];
            if (FP8) {
                mc[i >> 2] |= (ok ? at.m[off(i)] : 0u) << (8 * (i & 3));
                vc[i >> 2] |= (ok ? at.v[off(i)] : 0u) << (8 * (i & 3));
            } else {
                m[i] = ok ? reinterpret_cast<const float*>(at.m)[off(i)] : 0.0f;
                v[i] = ok ? reinterpret_cast<const float*>(at.v)[off(i)] : 0.0f;
            }
        }
    }
    if (FP8) {
        const float ms = *at.m_scale, vs = *at.v_scale;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            decode4(mc[j], ms, m + 4 * j);
            decode4(vc[j], vs, v + 4 * j);   // the root
        }
        if (!FULL) {   // a NaN scale stays out of the padding
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (!in(i)) m[i] = v[i] = 0.0f;
        }
    }
    // Products on pairs (an f32x2 product is two single IEEE products), sums one by one: a pair's
    // product that feeds a pair's sum would be fused with it, whatever the flags.
    float root[8];
    const uint64_t gs2 = f2c(sv.gs), b1 = f2c(sc.beta1), nb1 = f2c(sc.one_beta1), b2 = f2c(sc.beta2), nb2 = f2c(sc.one_beta2);
    const uint64_t fix2 = f2c(sv.fix), keep2 = f2c(sv.keep), size2 = f2c(sv.size);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        float x0, x1, y0, y1;
        const uint64_t gi = f2_mul(f2(g[i], g[i + 1]), gs2);
        f2_split(f2_mul(f2(m[i], m[i + 1]), b1), x0, x1);
        f2_split(f2_mul(gi, nb1), y0, y1);
        m[i] = __fadd_rn(x0, y0);
        m[i + 1] = __fadd_rn(x1, y1);
        uint64_t vi = f2(v[i], v[i + 1]);
        if (FP8) vi = f2_mul(vi, vi);
        f2_split(f2_mul(vi, b2), x0, x1);
        f2_split(f2_mul(f2_mul(gi, nb2), gi), y0, y1);
        v[i] = __fadd_rn(x0, y0);
        v[i + 1] = __fadd_rn(x1, y1);
        root[i] = __fsqrt_rn(v[i]);
        root[i + 1] = __fsqrt_rn(v[i + 1]);
    }
    // The divisor's roots.  A root below one code may have been held as zero while its m was not, and with
    // a zero gradient the quotient would be m / eps: such a root divides as the smallest code it can have
    // been held as.  (The search for one costs 2 us of the 385 above, a select per element 9.)
    float r[8], low = 1.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        r[i] = root[i];
        low = fminf(low, root[i]);
    }
    if (FP8 && low == 0.0f) {
        const float code = *at.v_scale * 0x1p-9f;   // the old scale: the new one is written below
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (root[i] == 0.0f) r[i] = code;
    }
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        float x0, x1, y0, y1;
        f2_split(f2_mul(f2(r[i], r[i + 1]), fix2), x0, x1);
        const uint64_t q = f2(__fdiv_rn(m[i], __fadd_rn(x0, sc.eps)), __fdiv_rn(m[i + 1], __fadd_rn(x1, sc.eps)));
        f2_split(f2_mul(f2(p[i], p[i + 1]), keep2), x0, x1);
        f2_split(f2_mul(q, size2), y0, y1);
        p[i] = __fsub_rn(x0, y0);
        p[i + 1] = __fsub_rn(x1, y1);
    }
    // p and w leave at once: the encode below needs their registers
    uint32_t wb[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) wb[i] = f32x2_to_bf16x2(p[2 * i], p[2 * i + 1]);
    if (FULL) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            *reinterpret_cast<float4*>(at.p + 128 * j) = make_float4(p[4 * j], p[4 * j + 1], p[4 * j + 2], p[4 * j + 3]);
            if (at.w) *reinterpret_cast<uint2*>(at.w + 128 * j) = make_uint2(wb[2 * j], wb[2 * j + 1]);
            if (!FP8) {
                *reinterpret_cast<float4*>(at.m + 512 * j) = make_float4(m[4 * j], m[4 * j + 1], m[4 * j + 2], m[4 * j + 3]);
                *reinterpret_cast<float4*>(at.v + 512 * j) = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (!in(i)) continue;
            at.p[off(i)] = p[i];
            if (at.w) at.w[off(i)] = (uint16_t)(wb[i >> 1] >> (16 * (i & 1)));
            if (!FP8) {
                reinterpret_cast<float*>(at.m)[off(i)] = m[i];
                reinterpret_cast<float*>(at.v)[off(i)] = v[i];
            }
        }
    }
    if (amax) {
        // elements past the end are masked: their p is 0 - 0 * size, or NaN where eps = 0
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t b = (wb[i >> 1] >> (16 * (i & 1))) & 0x7FFFu;
            am = max(am, in(i) ? b : 0u);
        }
    }
    if (FP8) {
        float ms, vs;
        encode_block<SR, true>(m, mc, ms, (uint64_t)first, kStreamMoment1, tensor, key0, key1);
        encode_block<SR, false>(root, vc, vs, (uint64_t)first, kStreamMoment2, tensor, key0, key1);
        if (lane == 0) {
            *at.m_scale = ms;
            *at.v_scale = vs;
        }
        if (FULL) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                *reinterpret_cast<uint32_t*>(at.m + 128 * j) = mc[j];
                *reinterpret_cast<uint32_t*>(at.v + 128 * j) = vc[j];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (!in(i)) continue;
                at.m[off(i)] = (uint8_t)(mc[i >> 2] >> (8 * (i & 3)));
                at.v[off(i)] = (uint8_t)(vc[i >> 2] >> (8 * (i & 3)));
            }
        }
    }
}

constexpr int kAdamResident = 8;   // CTAs per SM

// DYN: the step's values and the seed are read from device memory
template <bool FP8, bool SR, bool DYN, int CAP>
__global__ void __launch_bounds__(kAdamThreads, kAdamResident)
    adamw_kernel(const __grid_constant__ AdamwTable<CAP> tab, const AdamwScalars sc, uint32_t* flags) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t c0 = (uint32_t)((uint64_t)tab.chunks * blockIdx.x / gridDim.x);
    const uint32_t c1 = (uint32_t)((uint64_t)tab.chunks * (blockIdx.x + 1) / gridDim.x);
    if (c0 >= c1) return;
    StepValues sv{sc.keep, sc.step_size, sc.v_fix, sc.grad_scale};
    PhiloxKeys dyn_keys;
    if (DYN) {
        const float4 d = __ldg(reinterpret_cast<const float4*>(sc.dynamic));
        const uint2 k = __ldg(reinterpret_cast<const uint2*>(sc.dynamic) + 2);
        sv = StepValues{d.x, d.y, d.z, d.w};
        dyn_keys = philox_keys((uint64_t)k.y << 32 | k.x);
    }
    const uint32_t *key0 = DYN ? dyn_keys.k0 : tab.key0, *key1 = DYN ? dyn_keys.k1 : tab.key1;
    // the tensor of chunk c0: the last entry whose first chunk is <= c0 (every entry has chunks)
    int ti = 0;
    for (int lo = 0, hi = tab.count; hi - lo > 1;) {
        const int mid = (lo + hi) >> 1;
        if (tab.t[mid].first_chunk <= c0) lo = mid; else hi = mid;
        ti = lo;
    }
    for (uint32_t c = c0; c < c1; ++ti) {   // this CTA's run, tensor by tensor
        const AdamwEntry& e = tab.t[ti];
        const uint32_t end = min(c1, ti + 1 < tab.count ? tab.t[ti + 1].first_chunk : tab.chunks);
        const uint32_t tensor = (uint32_t)e.index_g >> 1;
        const bool amax = e.amax != nullptr;
        const int64_t n = e.n;
        Places<FP8> at(e, c - e.first_chunk);
        int64_t first = (int64_t)(c - e.first_chunk) * kAdamChunk + warp * kAdamBlock;
        uint32_t am = 0;   // |w| bits of this thread's elements
#pragma unroll 1
        for (; c < end; ++c, first += kAdamChunk, at.next()) {
            if (first + kAdamBlock <= n)
                block_step<FP8, SR, true>(at, first, kAdamBlock, tensor, sc, sv, key0, key1, amax, am);
            else if (first < n)
                block_step<FP8, SR, false>(at, first, (int)(n - first), tensor, sc, sv, key0, key1, amax, am);
        }
        if (amax) {
            const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, am);
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

template <bool FP8, bool SR, bool DYN, int CAP>
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
    for (int r = 0; r < 10; ++r) {   // Weyl sequences of the seed's two words
        tab.key0[r] = (uint32_t)sc.sr_seed + 0x9E3779B9u * r;
        tab.key1[r] = (uint32_t)(sc.sr_seed >> 32) + 0xBB67AE85u * r;
    }
    if (any_amax) adamw_reset_amax_kernel<CAP><<<(CAP + 127) / 128, 128, 0, s>>>(tab);
    const uint64_t most = (uint64_t)host::sm_count() * kAdamResident;   // one wave: a CTA takes its whole run
    adamw_kernel<FP8, SR, DYN, CAP><<<(unsigned)std::min<uint64_t>(chunks, most), kAdamThreads, 0, s>>>(tab, sc, flags);
    return cudaGetLastError();
}

template <bool FP8, bool SR, int CAP>
static cudaError_t launch_values(const AdamwEntry* entries, int count, const AdamwScalars& sc, uint32_t* flags, cudaStream_t s) {
    return sc.dynamic ? launch_table<FP8, SR, true, CAP>(entries, count, sc, flags, s)
                      : launch_table<FP8, SR, false, CAP>(entries, count, sc, flags, s);
}

template <int CAP>
static cudaError_t launch_state(const AdamwEntry* entries, int count, bool fp8, const AdamwScalars& sc, uint32_t* flags,
                                cudaStream_t s) {
    if (!fp8) return launch_values<false, false, CAP>(entries, count, sc, flags, s);
    return sc.sr ? launch_values<true, true, CAP>(entries, count, sc, flags, s)
                 : launch_values<true, false, CAP>(entries, count, sc, flags, s);
}

cudaError_t launch_adamw(const AdamwEntry* entries, int count, bool fp8, const AdamwScalars& sc, uint32_t* flags,
                         cudaStream_t s) {
    if (count < 1 || count > kAdamMaxTensors) return cudaErrorInvalidValue;
    // Table sizes: a launch copies its whole parameter block, 80 bytes per tensor (24 tensors in the table
    // of 384 took the host 18 us a call, in one of 64 10.5 us; 9 tensors in that of 16 6.2 us).
    if (count <= 16) return launch_state<16>(entries, count, fp8, sc, flags, s);
    if (count <= 32) return launch_state<32>(entries, count, fp8, sc, flags, s);
    if (count <= 96) return launch_state<96>(entries, count, fp8, sc, flags, s);
    return launch_state<kAdamMaxTensors>(entries, count, fp8, sc, flags, s);
}

}  // namespace nvfp4
