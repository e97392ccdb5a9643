// e4m3.hpp -- codes in 8-bit floating point (e4m3, largest value 448) of blocks
// of values that share a scale, each the code nearest to the exact quotient.
#pragma once

#include "device.hpp"

namespace archead {

constexpr float kE4m3Max = 448.f;

__device__ __forceinline__ float block_scale(float amax)
{
    return amax > 0.f ? fmaxf(amax * (1.f / kE4m3Max), 1.17549435e-38f) : 0.f;
}

// x / s with the last bit set where the quotient is not exact, so that the
// rounding to e4m3 that follows never sees a tie that is not one: the
// division's remainder x - q s is exact in one fma and says on which side of
// q the quotient lies.
__device__ __forceinline__ float sticky_quotient(float x, float s)
{
    float q, rem;
    if (s < 7.9e-31f) { // 2^-100: the remainder could fall below fp32's range
        const double d = (double)x / (double)s;
        q = (float)d;
        rem = (float)(d - (double)q);
    } else {
        q = x / s;
        rem = __builtin_fmaf(-q, s, x);
    }
    uint32_t b = __float_as_uint(q);
    if (rem != 0.f && (b & 1u) == 0u && fabsf(q) < 3.0e38f) {
        const bool outward = (rem > 0.f) == (q > 0.f);
        b = outward ? b + 1 : b - 1;
    }
    return q == 0.f ? q : __uint_as_float(b);
}

// eight codes in order
__device__ __forceinline__ u32x2 codes8_exact(const float v[8], float s)
{
    float q[8];
    uint32_t nan = 0;
    for (int i = 0; i < 8; ++i) {
        const float t = s > 0.f ? sticky_quotient(v[i], s) : 0.f;
        const bool is_nan = v[i] != v[i] || t != t;
        nan |= (uint32_t)is_nan << i;
        q[i] = is_nan ? 0.f : fminf(fmaxf(t, -kE4m3Max), kE4m3Max);
    }
    u32x2 o;
    for (int h = 0; h < 2; ++h) {
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * h], q[4 * h + 1], 0, false);
        o[h] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q[4 * h + 2], q[4 * h + 3], w, true);
        for (int i = 0; i < 4; ++i)
            if (nan >> (4 * h + i) & 1)
                o[h] |= 0x7Fu << (8 * i);
    }
    return o;
}

// The same at a fifth of the work: the quotient by the scale's reciprocal is within
// 2^-22 of the exact one, so where it converts alike 2^-21 below and above itself,
// that is the code.  The others (one vector of fp32 values in some 2^14; more of bf16
// ones, whose quotients are true ties at times), NaN (its code is 0x7f without a sign)
// and the ends of the scales' range go the exact way.
__device__ __forceinline__ u32x2 codes8(const float v[8], float s)
{
    const float r = __builtin_amdgcn_rcpf(s);
    u32x2 o;
    bool sure = s > 7.9e-31f && s < 1.2e30f;
    for (int h = 0; h < 2; ++h) {
        float lo[4], hi[4];
        for (int i = 0; i < 4; ++i) {
            const float t = v[4 * h + i] * r;
            lo[i] = t * (1.f - 4.76837158e-7f);
            hi[i] = t * (1.f + 4.76837158e-7f);
        }
        int a = __builtin_amdgcn_cvt_pk_fp8_f32(lo[0], lo[1], 0, false);
        a = __builtin_amdgcn_cvt_pk_fp8_f32(lo[2], lo[3], a, true);
        int b = __builtin_amdgcn_cvt_pk_fp8_f32(hi[0], hi[1], 0, false);
        b = __builtin_amdgcn_cvt_pk_fp8_f32(hi[2], hi[3], b, true);
        o[h] = (uint32_t)a;
        sure = sure && a == b && (((uint32_t)a & 0x7F7F7F7Fu) + 0x01010101u & 0x80808080u) == 0;
    }
    return sure ? o : codes8_exact(v, s);
}

} // namespace archead
