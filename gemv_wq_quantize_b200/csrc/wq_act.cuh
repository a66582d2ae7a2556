// wq_act.cuh -- device helpers of the operators around the matmuls (RMS norm, key / value
// cache): conversions of the 16-bit types, and 8-bit codes of binary32 values.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include "wq_device.cuh"

namespace wq {

__device__ __forceinline__ float act_f(__half v) { return __half2float(v); }
__device__ __forceinline__ float act_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T act_t(float v);
template <>
__device__ __forceinline__ __half act_t<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 act_t<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// Two 16-bit values in a word as binary32, and back (round to nearest even).
template <typename T>
__device__ __forceinline__ float2 act_f2(uint32_t w)
{
    T e[2];
    memcpy(e, &w, 4);
    return make_float2(act_f(e[0]), act_f(e[1]));
}
template <typename T>
__device__ __forceinline__ uint32_t act_t2(float a, float b);
// (one packed conversion: two single ones would go through the slow conversion pipe)
template <>
__device__ __forceinline__ uint32_t act_t2<__half>(float a, float b)
{
    const __half2 v = __floats2half2_rn(a, b);
    uint32_t w;
    memcpy(&w, &v, 4);
    return w;
}
template <>
__device__ __forceinline__ uint32_t act_t2<__nv_bfloat16>(float a, float b)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    uint32_t w;
    memcpy(&w, &v, 4);
    return w;
}

// The scale of a largest magnitude m is m * kInvQmax, one binary32 product: no division on the
// way from a reduction to the codes, at most 1.5 binary32 steps from m / qmax (the code of m
// itself is still qmax: codes are clipped).
template <bool F8>
constexpr float kInvQmax = F8 ? 1.f / 448.f : 1.f / 127.f;

// 8-bit codes of v / s (the IEEE quotient, then nearest, ties to even) without a division per
// value: with r = 1 / s correctly rounded, v r (1 - 2^-21) and v r (1 + 2^-21) enclose v / s (r,
// its factor and the products are off by 2^-24 each), and rounding to codes is monotone, so where
// both give the same code it is the quotient's.  Only four values of which one lies that near to a
// border between codes are divided.
struct CodeScale {
    float s, lo, hi;
    bool divide;  // a scale whose reciprocal is not a normal number
};
__device__ __forceinline__ CodeScale code_scale(float s)
{
    const float r = s != 0.f ? __frcp_rn(s) : 0.f;
    return {s, __fmul_rn(r, 1.f - 0x1p-21f), __fmul_rn(r, 1.f + 0x1p-21f), s != 0.f && !(s >= 0x1p-126f && s <= 0x1p126f)};
}

// Four e4m3 codes: nearest, ties to even, values beyond 448 saturate, a zero result is +0 (the
// convention of act_quant_fp8).
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d)
{
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}
__device__ __forceinline__ uint32_t e4m3_plus_zero(uint32_t w)
{
    const uint32_t nonzero = (w & 0x7f7f7f7fu) + 0x7f7f7f7fu;  // bit 7 of a byte: its magnitude is not 0
    return w & (nonzero | 0x7f7f7f7fu);
}

// Four INT8 codes of v * r for |v * r| < 128: 1.5 * 2^23 + v r leaves the nearest integer in the
// low byte of the sum's pattern.
__device__ __forceinline__ uint32_t i8x4(const float (&v)[4], float r)
{
    uint32_t b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = __float_as_uint(__fmaf_rn(v[i], r, 12582912.f));
    return prmt(prmt(b[0], b[1], 0x0040), prmt(b[2], b[3], 0x0040), 0x5410);
}

// Codes of four values with |v| <= qmax * s up to rounding (0 where s is 0).
template <bool F8>
__device__ __forceinline__ uint32_t codes4(const float (&v)[4], const CodeScale &c)
{
    uint32_t lo, hi;
    if constexpr (F8) {
        lo = e4m3x4(v[0] * c.lo, v[1] * c.lo, v[2] * c.lo, v[3] * c.lo);
        hi = e4m3x4(v[0] * c.hi, v[1] * c.hi, v[2] * c.hi, v[3] * c.hi);
    } else {
        lo = i8x4(v, c.lo);
        hi = i8x4(v, c.hi);
    }
    if (lo != hi || c.divide) {
        float q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) q[i] = fminf(fmaxf(__fdiv_rn(v[i], c.s), F8 ? -448.f : -127.f), F8 ? 448.f : 127.f);
        lo = F8 ? e4m3x4(q[0], q[1], q[2], q[3]) : i8x4(q, 1.f);
    }
    return F8 ? e4m3_plus_zero(lo) : lo;
}

// The value of code i (byte i of w).
template <bool F8>
__device__ __forceinline__ float code_value(uint32_t w, int i)
{
    if constexpr (F8) {
        const uint32_t h = i < 2 ? e4m3x2_to_f16x2<0>(w) : e4m3x2_to_f16x2<1>(w);
        __half2 p;
        memcpy(&p, &h, 4);
        return __half2float((i & 1) ? __high2half(p) : __low2half(p));
    } else {
        return float(int8_t(w >> (8 * i)));
    }
}

// binary16 pair of two 8-bit codes: bytes HALF * 2 and HALF * 2 + 1 of w.  INT8 comes with its
// sign bits flipped (c + 128 in 0..255): 0x6400 | byte is 1024 + byte, less 1152.
template <bool F8, int HALF>
__device__ __forceinline__ uint32_t widen(uint32_t w)
{
    if constexpr (F8) return e4m3x2_to_f16x2<HALF>(w);
    else return h2_add(prmt(w, 0x64646464u, HALF ? 0x4342 : 0x4140), 0xE480E480u);
}

__device__ __forceinline__ float exp2_approx(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ uint32_t warp_umax(uint32_t v) { return __reduce_max_sync(0xffffffffu, v); }

}  // namespace wq
