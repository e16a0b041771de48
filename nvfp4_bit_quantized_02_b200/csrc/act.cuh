// act.cuh -- the activations of the products' epilogues and their slopes, in fp32.
//
//   relu  max(h, 0)      relu2  max(h, 0)^2      gelu  h Phi(h)      silu  h / (1 + e^-h)
//
// By the approximate reciprocal and 2^x, Phi from the Chebyshev fit of erfc published by Press, Teukolsky, Vetterling
// and Flannery (Numerical Recipes, 2nd ed., section 6.2), relative error below 1.2e-7.  The exponential's argument, rounded to
// fp32, makes it 1e-6 for |h| < 3 and 1e-5 at 12, of a term that has become small there: gelu and silu err by less than 2^-20 |h|, for
// fp32 outputs too (expf, normcdff and IEEE quotients took a tile of 16 rows 1.2 to 4 us longer, the quotient of a zero most of
// all).  Below -30 all of gelu and its slope are zero in fp32 (Phi(-30) = 5e-198).
#pragma once

#include <cstdint>

#include "nvfp4_device.cuh"

namespace nvfp4 {

enum : int { kActNone = 0, kActRelu = 1, kActRelu2 = 2, kActGelu = 3, kActSilu = 4 };

namespace act {

__device__ __forceinline__ float rcp(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float exp2a(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
constexpr float kLog2e = 1.4426950408889634f;

// min(|h|, 30), NaN kept
__device__ __forceinline__ float capped(float h) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(h)), "f"(30.0f));
    return r;
}
// erfc(a / sqrt 2) of a pair, a = capped(h): t e^(-a^2 / 2 + c(t)), t = 1 / (1 + a / sqrt 8); the fit's coefficients
// times log2 e, for 2^x
__device__ __forceinline__ uint64_t erfc_of(float al, float ah) {
    const uint64_t a = f2(al, ah);
    float dl, dh;
    f2_split(f2_fma(a, f2c(0.35355339059327376f), f2c(1.0f)), dl, dh);
    const uint64_t t = f2(rcp(dl), rcp(dh));
    uint64_t p = f2c((float)(0.17087277 * 1.4426950408889634));
    p = f2_fma(t, p, f2c((float)(-0.82215223 * 1.4426950408889634)));
    p = f2_fma(t, p, f2c((float)(1.48851587 * 1.4426950408889634)));
    p = f2_fma(t, p, f2c((float)(-1.13520398 * 1.4426950408889634)));
    p = f2_fma(t, p, f2c((float)(0.27886807 * 1.4426950408889634)));
    p = f2_fma(t, p, f2c((float)(-0.18628806 * 1.4426950408889634)));
    p = f2_fma(t, p, f2c((float)(0.09678418 * 1.4426950408889634)));
    p = f2_fma(t, p, f2c((float)(0.37409196 * 1.4426950408889634)));
    p = f2_fma(t, p, f2c((float)(1.00002368 * 1.4426950408889634)));
    p = f2_fma(t, p, f2c((float)(-1.26551223 * 1.4426950408889634)));
    float xl, xh;
    f2_split(f2_fma(f2_mul(a, f2c(-0.5f * kLog2e)), a, p), xl, xh);
    return f2_mul(t, f2(exp2a(xl), exp2a(xh)));
}

// a pair of activations, in place
template <int ACT>
__device__ __forceinline__ void pair(float& x, float& y) {
    if (ACT == kActRelu || ACT == kActRelu2) {
        x = x < 0.0f ? 0.0f : x;
        y = y < 0.0f ? 0.0f : y;
        if (ACT == kActRelu2) {
            x *= x;
            y *= y;
        }
    } else if (ACT == kActGelu) {   // max(h, 0) - |h| erfc(|h| / sqrt 2) / 2
        const float al = capped(x), ah = capped(y);
        f2_split(f2_fma(f2_mul(f2(al, ah), f2c(-0.5f)), erfc_of(al, ah), f2(fmaxf(x, 0.0f), fmaxf(y, 0.0f))), x, y);
    } else if (ACT == kActSilu) {
        x = x * rcp(1.0f + exp2a(x * -kLog2e));
        y = y * rcp(1.0f + exp2a(y * -kLog2e));
    }
}
__device__ __forceinline__ float one(int act, float h) {
    float z = 0.0f;
    switch (act) {
        case kActRelu: pair<kActRelu>(h, z); break;
        case kActRelu2: pair<kActRelu2>(h, z); break;
        case kActGelu: pair<kActGelu>(h, z); break;
        case kActSilu: pair<kActSilu>(h, z); break;
    }
    return h;
}

// a pair of slopes
template <int ACT>
__device__ __forceinline__ void slope_pair(float& x, float& y) {
    if (ACT == kActNone) {
        x = y = 1.0f;
    } else if (ACT == kActRelu) {
        x = x > 0.0f ? 1.0f : (x <= 0.0f ? 0.0f : x);
        y = y > 0.0f ? 1.0f : (y <= 0.0f ? 0.0f : y);
    } else if (ACT == kActRelu2) {
        x = x < 0.0f ? 0.0f : 2.0f * x;
        y = y < 0.0f ? 0.0f : 2.0f * y;
    } else if (ACT == kActGelu) {   // Phi(h) + h phi(h)
        const float al = capped(x), ah = capped(y);
        const uint64_t e = erfc_of(al, ah), a = f2(al, ah);
        const uint64_t cdf = f2_fma(f2(x >= 0.0f ? -0.5f : 0.5f, y >= 0.0f ? -0.5f : 0.5f), e,
                                    f2(x >= 0.0f ? 1.0f : 0.0f, y >= 0.0f ? 1.0f : 0.0f));
        float ml, mh;
        f2_split(f2_mul(f2_mul(a, f2c(-0.5f * kLog2e)), a), ml, mh);
        const uint64_t hc = f2_mul(f2(x < 0.0f ? -al : al, y < 0.0f ? -ah : ah), f2c(0.39894228040143268f));
        f2_split(f2_fma(hc, f2(exp2a(ml), exp2a(mh)), cdf), x, y);
    } else {                        // s (1 + h (1 - s)), s = 1 / (1 + e^-h); h (1 - s) = h e^-|h| / (1 + e^-|h|) where it is small
        const float el = exp2a(fabsf(x) * -kLog2e), eh = exp2a(fabsf(y) * -kLog2e);
        const float rl = rcp(1.0f + el), rh = rcp(1.0f + eh);
        const float cl = x > 100.0f ? 100.0f : (x < -100.0f ? -100.0f : x), ch = y > 100.0f ? 100.0f : (y < -100.0f ? -100.0f : y);
        const float sl = (x >= 0.0f ? 1.0f : el) * rl, sh = (y >= 0.0f ? 1.0f : eh) * rh;
        const float ol = (x >= 0.0f ? el : 1.0f) * rl, oh = (y >= 0.0f ? eh : 1.0f) * rh;
        x = sl * fmaf(cl, ol, 1.0f);
        y = sh * fmaf(ch, oh, 1.0f);
    }
}

}  // namespace act
}  // namespace nvfp4
