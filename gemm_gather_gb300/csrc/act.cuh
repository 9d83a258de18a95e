// 16-bit elements, and activations with their slopes, in float32: the epilogues of the linear
// layer and the kernels that apply an activation by itself.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "../../include/gemm_gather.h"
#include "f32x2.cuh"

namespace gg {

__device__ __forceinline__ float load16(const void *p, int64_t at, int bf16)
{
    const uint16_t u = reinterpret_cast<const uint16_t *>(p)[at];
    return bf16 ? __uint_as_float((uint32_t)u << 16) : __half2float(__ushort_as_half(u));
}

__device__ __forceinline__ void store16(void *p, int64_t at, float v, int bf16)
{
    reinterpret_cast<uint16_t *>(p)[at] =
        bf16 ? __bfloat16_as_ushort(__float2bfloat16_rn(v)) : __half_as_ushort(__float2half_rn(v));
}

// Activations in float32, on pairs (two neighbouring tokens of a feature) where
// the arithmetic comes in pairs.  relu keeps NaN (its slope there is 0).  gelu_tanh's 0.5 (1 + tanh u) is
// the logistic function of 2u, which keeps its relative precision for u << 0.
// gelu's normal distribution function has Abramowitz and Stegun's form (7.1.26),
//     Phi(-x) = P(t) exp(-x^2 / 2),  t = 1 / (1 + 0.35 x),  x >= 0,
// P of degree 7 without a constant, fitted here for the least relative error (a linear
// program over 3000 points of [0, 13.5]): 1.5e-7 (1 + x^2 / 4), and 5e-7 at x < 1, 1.7e-6
// at 6 as evaluated.  So Y = max(z, 0) - |z| Phi(-|z|) is as near in the left tail, where
// it is tiny, as the power of two itself.  (7.1.26's own coefficients are within 7.5e-8 of
// Phi, which at z = -4 is a float16's half ulp of Y and at -7 more than a bfloat16's ulp.)
// The exponential is also the density that the derivative needs.  (With erff and a float
// division, the epilogue of a 256 x 256 tile took longer than its MMAs at K = 3584.)
__device__ __forceinline__ float ex2_approx(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float rcp_approx(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 1 / (1 + exp(-x))
__device__ __forceinline__ float2 logistic(F2 x)
{
    const float2 e = halves_of(mul2(x, pair_of(-1.44269504f)));
    const float2 d = halves_of(add2(pair_of(ex2_approx(e.x), ex2_approx(e.y)), pair_of(1.0f)));
    return make_float2(rcp_approx(d.x), rcp_approx(d.y));
}

// 2 sqrt(2/pi) (z + 0.044715 z^3)
__device__ __forceinline__ F2 gelu_2u(F2 z, F2 zz)
{
    return mul2(z, fma2(zz, pair_of(0.071354816f), pair_of(1.59576912f)));
}

// Phi(-|z|), and exp(-z^2 / 2) in *e.
__device__ __forceinline__ F2 normal_tail(float2 z, F2 zz, float2 *e)
{
    const float2 y = halves_of(mul2(zz, pair_of(-0.72134752f)));
    *e = make_float2(ex2_approx(y.x), ex2_approx(y.y));
    const float2 d = halves_of(fma2(pair_of(fabsf(z.x), fabsf(z.y)), pair_of(0.35f), pair_of(1.0f)));
    const F2 t = pair_of(rcp_approx(d.x), rcp_approx(d.y));
    F2 q = fma2(t, pair_of(0.0462695388f), pair_of(-0.190911355f));
    q = fma2(t, q, pair_of(0.221250296f));
    q = fma2(t, q, pair_of(0.00082826442f));
    q = fma2(t, q, pair_of(0.146570468f));
    q = fma2(t, q, pair_of(0.136159971f));
    q = fma2(t, q, pair_of(0.139832881f));
    return mul2(mul2(t, q), pair_of(e->x, e->y));
}

template <int ACT>
__device__ __forceinline__ float2 act_value(float2 v)
{
    const F2 z = pair_of(v.x, v.y);
    if constexpr (ACT == GG_ACT_RELU)
        return make_float2(!(v.x <= 0.0f) ? v.x : 0.0f, !(v.y <= 0.0f) ? v.y : 0.0f);
    if constexpr (ACT == GG_ACT_GELU) {
        // max(z, 0) - |z| Phi(-|z|), |z| held below 64, where the product is long 0; NaN is in
        // the tail
        float2 e;
        const F2 tail = normal_tail(v, mul2(z, z), &e);
        const F2 size = pair_of(-fminf(fabsf(v.x), 64.0f), -fminf(fabsf(v.y), 64.0f));
        return halves_of(fma2(size, tail, pair_of(fmaxf(v.x, 0.0f), fmaxf(v.y, 0.0f))));
    }
    if constexpr (ACT == GG_ACT_GELU_TANH || ACT == GG_ACT_SILU) {
        const float2 s = logistic(ACT == GG_ACT_SILU ? z : gelu_2u(z, mul2(z, z)));
        return halves_of(mul2(z, pair_of(s.x, s.y)));
    }
    return v;
}

// x between -128 and 128, where every smooth slope is 0 or 1; NaN stays NaN.
__device__ __forceinline__ float held128(float x)
{
    float y;
    asm("min.NaN.f32 %0, %1, 0f43000000;\n\tmax.NaN.f32 %0, %0, 0fC3000000;" : "=f"(y) : "f"(x));
    return y;
}

// The derivative at z.  A stored Z may be infinite where the sum was not (16 bits), and the
// square of a large one is: the smooth slopes see z held between -128 and 128, so that
// infinity times 0 meets none of them.
template <int ACT>
__device__ __forceinline__ float2 act_slope(float2 v)
{
    if constexpr (ACT != GG_ACT_RELU && ACT != GG_ACT_NONE)
        v = make_float2(held128(v.x), held128(v.y));
    const F2 z = pair_of(v.x, v.y);
    if constexpr (ACT == GG_ACT_RELU)
        return make_float2(v.x > 0.0f ? 1.0f : 0.0f, v.y > 0.0f ? 1.0f : 0.0f);
    if constexpr (ACT == GG_ACT_GELU) {  // Phi + z density
        float2 e;
        const float2 tail = halves_of(normal_tail(v, mul2(z, z), &e));
        const float2 c = make_float2(v.x < 0.0f ? tail.x : 1.0f - tail.x, v.y < 0.0f ? tail.y : 1.0f - tail.y);
        return halves_of(fma2(mul2(z, pair_of(0.39894228f)), pair_of(e.x, e.y), pair_of(c.x, c.y)));
    }
    if constexpr (ACT == GG_ACT_GELU_TANH) {  // d(z s)/dz = s + z s (1 - s) 2u'
        const F2 zz = mul2(z, z);
        const float2 h = logistic(gelu_2u(z, zz));
        const F2 s = pair_of(h.x, h.y), rest = pair_of(1.0f - h.x, 1.0f - h.y);
        const F2 du = fma2(zz, pair_of(0.21406445f), pair_of(1.59576912f));
        return halves_of(fma2(mul2(mul2(z, s), rest), du, s));
    }
    if constexpr (ACT == GG_ACT_SILU) {  // s + z s (1 - s)
        const float2 h = logistic(z);
        const F2 s = pair_of(h.x, h.y), rest = pair_of(1.0f - h.x, 1.0f - h.y);
        return halves_of(fma2(mul2(z, s), rest, s));
    }
    return make_float2(1.0f, 1.0f);
}

// v = act(v) and v *= act'(x), over an even number of values.
template <int ACT, int C>
__device__ __forceinline__ void apply_act(float (&v)[C])
{
#pragma unroll
    for (int u = 0; u < C; u += 2) {
        const float2 y = act_value<ACT>(make_float2(v[u], v[u + 1]));
        v[u] = y.x, v[u + 1] = y.y;
    }
}
template <int ACT, int C>
__device__ __forceinline__ void apply_slope(float (&v)[C], const float (&x)[C])
{
#pragma unroll
    for (int u = 0; u < C; u += 2) {
        const float2 y = act_slope<ACT>(make_float2(x[u], x[u + 1]));
        v[u] *= y.x, v[u + 1] *= y.y;
    }
}

// f(ACT) with the activation as a compile-time constant.
template <typename F>
__device__ __forceinline__ void with_act(int act, F f)
{
    switch (act) {
    case GG_ACT_RELU: f(std::integral_constant<int, GG_ACT_RELU>()); break;
    case GG_ACT_GELU: f(std::integral_constant<int, GG_ACT_GELU>()); break;
    case GG_ACT_GELU_TANH: f(std::integral_constant<int, GG_ACT_GELU_TANH>()); break;
    case GG_ACT_SILU: f(std::integral_constant<int, GG_ACT_SILU>()); break;
    default: f(std::integral_constant<int, GG_ACT_NONE>()); break;
    }
}

}  // namespace gg
