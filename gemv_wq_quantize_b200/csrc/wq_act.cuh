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
__device__ __forceinline__ uint32_t act_t2(float a, float b)
{
    const T e[2] = {act_t<T>(a), act_t<T>(b)};
    uint32_t w;
    memcpy(&w, e, 4);
    return w;
}

// The scale of a largest magnitude m is m * kInvQmax, one binary32 product: no division on the
// way from a reduction to the codes, at most 1.5 binary32 steps from m / qmax (the code of m
// itself is still qmax: codes are clipped).
template <bool F8>
constexpr float kInvQmax = F8 ? 1.f / 448.f : 1.f / 127.f;

// INT8 code of a finite v for the scale s > 0: clip(rint(v / s), -127, 127) with the IEEE
// quotient.  quant_i8 forms it from the reciprocal r of s (with a division next to ties
// only); a scale at or below 2^-128 has no finite reciprocal and divides.
__device__ __forceinline__ int code_i8(float v, float s, float r)
{
    if (isinf(r)) return int(fminf(fmaxf(rintf(__fdiv_rn(v, s)), -127.f), 127.f));
    return quant_i8(v, s, r);
}

// Four e4m3 codes of a, b, c, d (already divided by their scale): nearest, ties to even,
// values beyond 448 saturate, a zero result is +0 (the convention of act_quant_fp8).
__device__ __forceinline__ uint32_t codes_e4m3(float a, float b, float c, float d)
{
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    const uint32_t w = lo | (hi << 16);
    const uint32_t nonzero = (w & 0x7f7f7f7fu) + 0x7f7f7f7fu;  // bit 7 of a byte: its magnitude is not 0
    return w & (nonzero | 0x7f7f7f7fu);
}

// Four codes of finite values for one scale s >= 0 with reciprocal r (INT8; unused for
// e4m3, whose quotients are IEEE divisions): 0 where s is 0.
template <bool F8>
__device__ __forceinline__ uint32_t codes4(const float (&v)[4], float s, float r)
{
    if (s == 0.f) return 0u;
    if constexpr (F8) {
        return codes_e4m3(__fdiv_rn(v[0], s), __fdiv_rn(v[1], s), __fdiv_rn(v[2], s), __fdiv_rn(v[3], s));
    } else {
        uint32_t w = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) w |= (uint32_t(code_i8(v[i], s, r)) & 0xffu) << (8 * i);
        return w;
    }
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
