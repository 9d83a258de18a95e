// Activations in 8 bits: e4m3 codes of a row-major matrix, and one float32 power of two for
// every kPackBlock elements of a row (the last block of a row may be shorter).  A value is its
// code times its block's scale.  The scale is the power of two that brings the block's largest
// finite magnitude into (224, 448], 2^-118 at least, so scaling is exact, no code overflows and
// a code's rounding (to nearest, ties to even) is the only one: half a step of four significant
// bits, 2^-4 of the value, or 2^-10 scale below 2^-6 scale.  What is not finite is stored as NaN
// and does not enter the scale.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <cstdint>

#include "../../include/gemm_gather.h"

namespace gg {

constexpr int kPackBlock = GG_PACK_BLOCK;

// Pairs of 16-bit elements (the lower half first).
template <bool BF16>
__device__ __forceinline__ float2 pair16(uint32_t w)
{
    if constexpr (BF16)
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    else
        return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}

template <bool BF16>
__device__ __forceinline__ uint32_t pair16_of(float lo, float hi)
{
    if constexpr (BF16) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&v);
    } else {
        const __half2 v = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
}

__device__ __forceinline__ bool is_finite(float x) { return fabsf(x) <= 3.402823466e38f; }

// The larger magnitude; what is not finite counts as 0.
__device__ __forceinline__ float pack_top(float top, float x) { return is_finite(x) ? fmaxf(top, fabsf(x)) : top; }

// A block's scale 2^e from its largest magnitude (e: 2^e * 224 < top <= 2^e * 448).
__device__ __forceinline__ int pack_exponent(float top)
{
    const int e = ((__float_as_int(top) + 0x1FFFFF) >> 23) - 127 - 8;
    return e < -118 ? -118 : e;
}

__device__ __forceinline__ float power_of_two(int e) { return __int_as_float((e + 127) << 23); }

// Codes of four values, already divided by their scale (|x| <= 448 or not finite).
__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d)
{
    // an infinity would be held at 448
    a = is_finite(a) ? a : __int_as_float(0x7fffffff);
    b = is_finite(b) ? b : __int_as_float(0x7fffffff);
    c = is_finite(c) ? c : __int_as_float(0x7fffffff);
    d = is_finite(d) ? d : __int_as_float(0x7fffffff);
    return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3) |
           (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3) << 16;
}

// The e4m3 values of four codes.
__device__ __forceinline__ void unpack4(uint32_t codes, float (&x)[4])
{
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(codes >> (16 * h)), __NV_E4M3);
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&r));
        x[2 * h] = f.x;
        x[2 * h + 1] = f.y;
    }
}

// A value from its code and scale: rounded up on the way into 8 bits it may lie just beyond the
// 16-bit type's range, and is its largest number then.
template <bool BF16>
__device__ __forceinline__ float held16(float x)
{
    constexpr float kTop = BF16 ? 3.3895313892515355e38f : 65504.0f;
    return x > kTop ? kTop : (x < -kTop ? -kTop : x);
}

// Eight neighbouring elements of a row, of which `left` exist; the others are zero and not read.
__device__ __forceinline__ uint4 load8(const uint16_t *p, int64_t left)
{
    if (left >= 8)
        return *reinterpret_cast<const uint4 *>(p);
    uint32_t w[4] = {};
#pragma unroll
    for (int u = 0; u < 7; ++u)
        if (u < left)
            w[u >> 1] |= (uint32_t)p[u] << (16 * (u & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void store8(uint16_t *p, int64_t left, const uint4 &v)
{
    if (left >= 8) {
        *reinterpret_cast<uint4 *>(p) = v;
        return;
    }
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int u = 0; u < 7; ++u)
        if (u < left)
            p[u] = (uint16_t)(w[u >> 1] >> (16 * (u & 1)));
}

__device__ __forceinline__ uint2 load_codes8(const uint8_t *p, int64_t left)
{
    if (left >= 8)
        return *reinterpret_cast<const uint2 *>(p);
    uint32_t w[2] = {};
#pragma unroll
    for (int u = 0; u < 7; ++u)
        if (u < left)
            w[u >> 2] |= (uint32_t)p[u] << (8 * (u & 3));
    return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ void store_codes8(uint8_t *p, int64_t left, const uint2 &v)
{
    if (left >= 8) {
        *reinterpret_cast<uint2 *>(p) = v;
        return;
    }
    const uint32_t w[2] = {v.x, v.y};
#pragma unroll
    for (int u = 0; u < 7; ++u)
        if (u < left)
            p[u] = (uint8_t)(w[u >> 2] >> (8 * (u & 3)));
}

// Eight values of a 16-lane group's 128: the group's scale exponent and this lane's codes.  The
// whole warp calls it.
__device__ __forceinline__ uint2 pack_group(const float (&x)[8], int *exponent)
{
    float top = 0.0f;
#pragma unroll
    for (int u = 0; u < 8; ++u)
        top = pack_top(top, x[u]);
#pragma unroll
    for (int d = 8; d > 0; d >>= 1)
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    const int e = pack_exponent(top);
    const float inv = power_of_two(-e);
    *exponent = e;
    return make_uint2(pack4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv),
                      pack4(x[4] * inv, x[5] * inv, x[6] * inv, x[7] * inv));
}

// The same for any alignment: a warp and its block, four elements a lane, 32 apart.
__device__ __forceinline__ uint32_t pack_warp(const float (&x)[4], int *exponent)
{
    float top = 0.0f;
#pragma unroll
    for (int u = 0; u < 4; ++u)
        top = pack_top(top, x[u]);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    const int e = pack_exponent(top);
    const float inv = power_of_two(-e);
    *exponent = e;
    return pack4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv);
}

}  // namespace gg
