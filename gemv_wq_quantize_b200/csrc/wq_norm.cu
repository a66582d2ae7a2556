// wq_norm.cu -- RMS norm with the residual's addition and a per-token 8-bit output
// (rmsnorm_quant_int8, rmsnorm_quant_fp8) for sm_100a.
//
// Mathematics, for one token x of K elements (T: binary16 or bfloat16):
//   h = T(x + residual)                                  rounded once; the new residual stream
//   y = (h * rstd) * gamma,  rstd = binary32(1 / sqrt(mean(h^2) + eps))
//   a_scale = max|y| * binary32(1 / 127 or 1 / 448),  code = the 8-bit code of y / a_scale
// The squares and their sum are binary64: a sum of K <= 2^31 squares of 8- or 11-bit
// mantissas then has an error far below one binary32 step, so rstd (and with it every code)
// does not depend on how the row is split over threads, and the codes are bit-exact with any
// other implementation of the same reading.  All products of y are single binary32 roundings.
//
// One block per token; the row is read once and stays in registers through both reductions
// (sum of squares, then max|y|).  Bound by memory where there are many rows, else by the launch and
// the chain of one read, two reductions and one write.
// Measured (device time, calls back to back in a graph), with a residual: 8192 rows of 4096, bfloat16 to
// INT8: 45.3 us, 5.2 TB/s (binary32 squares: 0.5 less, so binary64 is not what bounds it), to e4m3 46.8; 128
// rows of 3200: 3.2 us; one row of 4096: 2.2 us.
#include <cuda_runtime.h>
#include <stdint.h>

#include <cmath>

#include "wq_act.cuh"
#include "wq_host.h"

namespace wq {
namespace {

constexpr int kNormThreads = 512;  // rows of up to 4 vectors of 8 elements a thread (16384) are held whole

struct NormArgs {
    const void *X, *residual, *gamma;
    void *h;
    uint8_t *Aq;
    float *a_scale;
    int64_t K8;  // vectors of 8 elements in a row
    float eps;
};

template <typename T>
__device__ __forceinline__ uint4 add8(const uint4 &a, const uint4 &b)
{
    const uint32_t *x = &a.x, *y = &b.x;
    uint4 o;
    uint32_t *w = &o.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 p = act_f2<T>(x[i]), q = act_f2<T>(y[i]);
        w[i] = act_t2<T>(__fadd_rn(p.x, q.x), __fadd_rn(p.y, q.y));
    }
    return o;
}

template <typename T>
__device__ __forceinline__ double squares8(const uint4 &a, double sum)
{
    const uint32_t *x = &a.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 p = act_f2<T>(x[i]);
        sum = fma(double(p.x), double(p.x), sum);
        sum = fma(double(p.y), double(p.y), sum);
    }
    return sum;
}

template <typename T>
__device__ __forceinline__ void scaled8(const uint4 &h, const uint4 &g, float rstd, float (&y)[8])
{
    const uint32_t *x = &h.x, *w = &g.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 p = act_f2<T>(x[i]), q = act_f2<T>(w[i]);
        y[2 * i] = __fmul_rn(__fmul_rn(p.x, rstd), q.x);
        y[2 * i + 1] = __fmul_rn(__fmul_rn(p.y, rstd), q.y);
    }
}

// max over |y| as ordered bit patterns: infinities and NaN compare above every finite value.
__device__ __forceinline__ uint32_t absmax8(const float (&y)[8], uint32_t m)
{
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(y[i]) & 0x7fffffffu);
    return m;
}

template <bool F8>
__device__ __forceinline__ uint2 codes8(const float (&y)[8], const CodeScale &c)
{
    const float lo[4] = {y[0], y[1], y[2], y[3]}, hi[4] = {y[4], y[5], y[6], y[7]};
    return make_uint2(codes4<F8>(lo, c), codes4<F8>(hi, c));
}

// V: vectors a thread holds (0: the row is too long to hold; h is read back for the two
// later passes).
template <typename T, bool F8, bool RES, int V>
__global__ void __launch_bounds__(kNormThreads) rmsnorm_quant_kernel(const __grid_constant__ NormArgs a)
{
    const int64_t row = blockIdx.x;
    const int tid = threadIdx.x, nt = blockDim.x;
    const uint4 *x = static_cast<const uint4 *>(a.X) + row * a.K8;
    const uint4 *res = RES ? static_cast<const uint4 *>(a.residual) + row * a.K8 : nullptr;
    uint4 *h = RES ? static_cast<uint4 *>(a.h) + row * a.K8 : nullptr;
    const uint4 *gamma = static_cast<const uint4 *>(a.gamma);
    uint2 *q = reinterpret_cast<uint2 *>(a.Aq) + row * a.K8;
    __shared__ double red_sum[32];
    __shared__ uint32_t red_max[32];
    __shared__ float s_rstd;
    grid_dep_launch();
    grid_dep_wait();  // X and residual may be written, and the outputs read, by the kernel before

    constexpr int VH = V ? V : 1;
    uint4 hv[VH], gv[VH];
    double sum = 0;
    if constexpr (V > 0) {
        uint4 rv[VH];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int64_t j = tid + int64_t(i) * nt;
            hv[i] = j < a.K8 ? x[j] : make_uint4(0, 0, 0, 0);
            if constexpr (RES) rv[i] = j < a.K8 ? res[j] : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int64_t j = tid + int64_t(i) * nt;
            gv[i] = j < a.K8 ? gamma[j] : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int64_t j = tid + int64_t(i) * nt;
            if constexpr (RES) {
                hv[i] = add8<T>(hv[i], rv[i]);
                if (j < a.K8) h[j] = hv[i];
            }
            sum = squares8<T>(hv[i], sum);
        }
    } else {
        for (int64_t j = tid; j < a.K8; j += nt) {
            uint4 v = x[j];
            if constexpr (RES) {
                v = add8<T>(v, res[j]);
                h[j] = v;
            }
            sum = squares8<T>(v, sum);
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if ((tid & 31) == 0) red_sum[tid >> 5] = sum;
    __syncthreads();
    if (tid < 32) {
        double t = tid < (nt >> 5) ? red_sum[tid] : 0.0;
#pragma unroll
        for (int o = 16; o; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
        if (tid == 0) s_rstd = float(1.0 / sqrt(t / double(a.K8 * 8) + double(a.eps)));
    }
    __syncthreads();
    const float rstd = s_rstd;

    uint32_t amax = 0;
    const uint4 *back = RES ? h : x;  // each thread reads back only what it wrote itself
    if constexpr (V > 0) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float y[8];
            scaled8<T>(hv[i], gv[i], rstd, y);
            amax = absmax8(y, amax);
        }
    } else {
        for (int64_t j = tid; j < a.K8; j += nt) {
            float y[8];
            scaled8<T>(back[j], gamma[j], rstd, y);
            amax = absmax8(y, amax);
        }
    }
    amax = warp_umax(amax);
    if ((tid & 31) == 0) red_max[tid >> 5] = amax;
    __syncthreads();
    amax = warp_umax((tid & 31) < (nt >> 5) ? red_max[tid & 31] : 0u);
    // a row that holds an infinity or NaN: scale NaN (its products are NaN), codes 0
    const bool finite = amax < 0x7f800000u;
    const float sc = finite ? __fmul_rn(__uint_as_float(amax), kInvQmax<F8>) : __uint_as_float(0x7fc00000u);
    const CodeScale cs = code_scale(finite ? sc : 0.f);
    if (tid == 0) a.a_scale[row] = sc;
    if constexpr (V > 0) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int64_t j = tid + int64_t(i) * nt;
            float y[8];
            scaled8<T>(hv[i], gv[i], rstd, y);
            if (j < a.K8) q[j] = finite ? codes8<F8>(y, cs) : make_uint2(0, 0);
        }
    } else {
        for (int64_t j = tid; j < a.K8; j += nt) {
            float y[8];
            scaled8<T>(back[j], gamma[j], rstd, y);
            q[j] = finite ? codes8<F8>(y, cs) : make_uint2(0, 0);
        }
    }
}

template <typename T, bool F8, bool RES>
const void *norm_kernel(int v)
{
    switch (v) {
    case 1: return reinterpret_cast<const void *>(rmsnorm_quant_kernel<T, F8, RES, 1>);
    case 2: return reinterpret_cast<const void *>(rmsnorm_quant_kernel<T, F8, RES, 2>);
    case 4: return reinterpret_cast<const void *>(rmsnorm_quant_kernel<T, F8, RES, 4>);
    }
    return reinterpret_cast<const void *>(rmsnorm_quant_kernel<T, F8, RES, 0>);
}

wq_status rmsnorm_quant(bool f8, const void *X, const void *residual, const void *gamma, wq_dtype dt, float eps,
                        int64_t M, int64_t K, void *h, uint8_t *Aq, float *a_scale, cudaStream_t stream)
{
    if (M <= 0 || K <= 0) return fail(WQ_ERR_INVALID_ARG, "M and K must be positive");
    if (M > 0x7fffffff || K > 0x7fffffff) return fail(WQ_ERR_INVALID_ARG, "sizes exceed int32");
    if (!X || !gamma || !Aq || !a_scale) return fail(WQ_ERR_INVALID_ARG, "X, gamma, Aq and a_scale must be non-null");
    if (dt != WQ_F16 && dt != WQ_BF16) return fail(WQ_ERR_INVALID_ARG, "dt must be WQ_F16 or WQ_BF16");
    if ((residual != nullptr) != (h != nullptr))
        return fail(WQ_ERR_INVALID_ARG, "residual and h are given together or not at all");
    if (!(eps > 0.f) || !std::isfinite(eps)) return fail(WQ_ERR_INVALID_ARG, "eps must be positive and finite");
    if (K % 8) return fail(WQ_ERR_INVALID_ARG, "K %% 8 != 0");
    if (!aligned16(X) || !aligned16(gamma) || !aligned16(Aq) || (residual && (!aligned16(residual) || !aligned16(h))))
        return fail(WQ_ERR_ALIGNMENT, "X, residual, gamma, h and Aq must be 16-byte aligned");
    if (reinterpret_cast<uintptr_t>(a_scale) & 3) return fail(WQ_ERR_ALIGNMENT, "a_scale must be 4-byte aligned");

    NormArgs a{X, residual, gamma, h, Aq, a_scale, K / 8, eps};
    // Few tokens: a vector a thread, for latency.  Many: four vectors a thread, so that more rows are
    // in flight on an SM and a reduction joins fewer warps (8192 tokens of 4096: 55.8 -> 46.6 us;
    // 128 tokens of 3200 would go from 3.2 to 3.6).
    const int most = M > 2 * int64_t(device_info().sm_count) ? 128 : kNormThreads;
    int v = 0, threads = kNormThreads;
    for (int t : {1, 2, 4})
        if (!v && a.K8 <= int64_t(t) * (t < 4 ? most : kNormThreads)) {
            v = t;
            threads = int(((a.K8 + t - 1) / t + 31) / 32 * 32);
        }
    const bool bf = dt == WQ_BF16, res = residual != nullptr;
    const void *fn = bf ? (f8 ? (res ? norm_kernel<__nv_bfloat16, true, true>(v) : norm_kernel<__nv_bfloat16, true, false>(v))
                              : (res ? norm_kernel<__nv_bfloat16, false, true>(v) : norm_kernel<__nv_bfloat16, false, false>(v)))
                        : (f8 ? (res ? norm_kernel<__half, true, true>(v) : norm_kernel<__half, true, false>(v))
                              : (res ? norm_kernel<__half, false, true>(v) : norm_kernel<__half, false, false>(v)));
    PreparedLaunch L;
    L.set(fn, dim3(unsigned(M)), dim3(unsigned(threads)), 0, a);
    return launch_prepared(L, stream, "rmsnorm_quant_kernel");
}

}  // namespace
}  // namespace wq

extern "C" wq_status rmsnorm_quant_int8(const void *X, const void *residual, const void *gamma, wq_dtype dt, float eps,
                                        int64_t M, int64_t K, void *h, int8_t *Aq, float *a_scale, cudaStream_t stream)
{
    return wq::rmsnorm_quant(false, X, residual, gamma, dt, eps, M, K, h, reinterpret_cast<uint8_t *>(Aq), a_scale,
                             stream);
}

extern "C" wq_status rmsnorm_quant_fp8(const void *X, const void *residual, const void *gamma, wq_dtype dt, float eps,
                                       int64_t M, int64_t K, void *h, uint8_t *Aq, float *a_scale, cudaStream_t stream)
{
    return wq::rmsnorm_quant(true, X, residual, gamma, dt, eps, M, K, h, Aq, a_scale, stream);
}
