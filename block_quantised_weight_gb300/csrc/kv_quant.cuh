// Scales and codes of the 8-bit cache: what the appends share (the definitions
// are qgkv_append's; each step is one correctly rounded fp32 operation).
#pragma once
#include "kv_common.cuh"

namespace qg {

// Code of y = x / scale.
template <bool INT8>
__device__ __forceinline__ uint32_t code_of(float y) {
    if (INT8) {
        if (!(y == y)) return 0u;
        return static_cast<uint32_t>(__float2int_rn(fminf(fmaxf(y, -127.f), 127.f))) & 0xFFu;
    }
    unsigned short r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(y));
    return r & 0xFFu;
}

// Four codes of int8 by division: out of line, the way there is rare.
static __device__ __noinline__ uint32_t codes_by_division(float x0, float x1, float x2, float x3, float scale) {
    const float x[4] = {x0, x1, x2, x3};
    uint32_t r = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bool finite = fabsf(x[i]) <= 3.4028235e38f;
        r |= code_of<true>(scale == 0.f ? (finite ? 0.f : x[i]) : __fdiv_rn(x[i], scale)) << (8 * i);
    }
    return r;
}

// Codes of four values.  inv: 1 / scale rounded (for e4m3 a power of two,
// exact), 0 for a zero block.
template <bool INT8>
__device__ __forceinline__ uint32_t codes_of(float x0, float x1, float x2, float x3, float scale, float inv) {
    if (!INT8) {
        if (scale == 0.f) inv = 1.f;  // zeros stay zeros, infinities and NaN keep their codes
        unsigned short lo, hi;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(x1 * inv), "f"(x0 * inv));
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(x3 * inv), "f"(x2 * inv));
        return lo | static_cast<uint32_t>(hi) << 16;
    }
    const float x[4] = {x0, x1, x2, x3};
    uint32_t z[4];
    bool sure = true;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float y = x[i] * inv;
        const float big = y + 12582912.f;  // 1.5 * 2^23: the sum's low bits are y rounded to an integer
        z[i] = __float_as_uint(big);
        // further than 2^-15 from a tie; false for NaN and infinities
        sure &= fabsf(fabsf(y - (big - 12582912.f)) - 0.5f) > 0x1p-15f;
    }
    if (!sure) return codes_by_division(x0, x1, x2, x3, scale);
    return prmt(prmt(z[0], z[1], 0x0040u), prmt(z[2], z[3], 0x0040u), 0x5410u);
}

template <bool INT8>
__device__ __forceinline__ float scale_for(float amax) {
    if (INT8) return __fdiv_rn(amax, 127.f);
    if (!(amax > 0.f)) return 0.f;
    // smallest e >= -126 with amax <= 1.75 * 2^(8 + e)
    const uint32_t u = __float_as_uint(amax);
    int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    e = max(e, -126);
    return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// Four codes of a word, rescaled by f = old scale / new scale.
template <bool INT8>
__device__ __forceinline__ uint32_t rescaled(uint32_t x, float f) {
    uint32_t r = 0;
    if (INT8) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            r |= code_of<true>(__fmul_rn(static_cast<float>(static_cast<signed char>(x >> (8 * j))), f)) << (8 * j);
    } else {
        const f2 lo = h2_to_f2(e4m3x2_f16x2(x & 0xFFFFu)), hi = h2_to_f2(e4m3x2_f16x2(x >> 16));
        r = code_of<false>(__fmul_rn(lo.x, f)) | code_of<false>(__fmul_rn(lo.y, f)) << 8 |
            code_of<false>(__fmul_rn(hi.x, f)) << 16 | code_of<false>(__fmul_rn(hi.y, f)) << 24;
    }
    return r;
}

}  // namespace qg
