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
#include "f32x2.cuh"

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

// Codes of two pairs of values, already divided by their scale (|x| <= 448, or NaN).
__device__ __forceinline__ uint32_t pack4(float2 a, float2 b)
{
    uint32_t codes;
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
        "mov.b32 %0, {lo, hi};\n\t}"
        : "=r"(codes)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return codes;
}

// NaN for what is not finite (an infinity would be held at 448).
__device__ __forceinline__ float nan_unless_finite(float x) { return is_finite(x) ? x : __int_as_float(0x7fffffff); }

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
// 16-bit type's range, and is its largest number then.  Only blocks of the largest scale have such.
template <bool BF16>
__device__ __forceinline__ float held16(float x)
{
    constexpr float kTop = BF16 ? 3.3895313892515355e38f : 65504.0f;
    return x > kTop ? kTop : (x < -kTop ? -kTop : x);
}

// The values of eight codes under one scale.
template <bool BF16>
__device__ __forceinline__ void values8(const uint2 &codes, float scale, float (&v)[8])
{
    float x[4], y[4];
    unpack4(codes.x, x);
    unpack4(codes.y, y);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        v[u] = x[u] * scale;
        v[4 + u] = y[u] * scale;
    }
    constexpr float kBig = BF16 ? 1.329227995784916e36f : 256.0f;  // 2^120, 2^8
    if (scale >= kBig) {
#pragma unroll
        for (int u = 0; u < 8; ++u)
            v[u] = held16<BF16>(v[u]);
    }
}

// An exponential between 0 and 1 in 16 bits: five of exponent and eleven of mantissa, to nearest (half a step is
// 2^-12 of it, an eighth of bfloat16's and half of float16's); below 2^-31 it is 0.
__device__ __forceinline__ uint32_t kept_code(float e)
{
    const uint32_t code = (__float_as_uint(e) + 0x800u) >> 12;
    return min(max(code, 96u << 11) - (96u << 11), 0xffffu);
}

__device__ __forceinline__ float kept_value(uint32_t code)
{
    return code == 0 ? 0.0f : __uint_as_float((code + (96u << 11)) << 12);
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

// 16-bit patterns without their signs, two in a word: their order is that of the magnitudes, and from
// kInf16 on they are not finite.
template <bool BF16>
constexpr uint32_t kInf16 = BF16 ? 0x7f80u : 0x7c00u;

// The larger of each half (unsigned).
__device__ __forceinline__ uint32_t max_halves(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// 8 VECS 16-bit values of 128 that a group of 16 / VECS neighbouring lanes holds: the block's scale
// exponent and this lane's codes.  The whole warp calls it.
template <bool BF16, int VECS>
__device__ __forceinline__ void pack_block(const uint4 (&q)[VECS], int *exponent, uint2 (&codes)[VECS])
{
    uint32_t top = 0;
#pragma unroll
    for (int v = 0; v < VECS; ++v) {
        top = max_halves(top, max_halves(q[v].x & 0x7fff7fffu, q[v].y & 0x7fff7fffu));
        top = max_halves(top, max_halves(q[v].z & 0x7fff7fffu, q[v].w & 0x7fff7fffu));
    }
#pragma unroll
    for (int d = 8 / VECS; d > 0; d >>= 1)
        top = max_halves(top, __shfl_xor_sync(0xffffffffu, top, d));
    top = max(top & 0xffffu, top >> 16);
    const float largest = BF16 ? __uint_as_float(top << 16) : __half2float(__ushort_as_half((unsigned short)top));
    int e = pack_exponent(largest);
    const bool odd = __any_sync(0xffffffffu, top >= kInf16<BF16>);
    if (odd) {  // rare: what is not finite stays out of the scale
        float finite = 0.0f;
#pragma unroll
        for (int v = 0; v < VECS; ++v) {
            const uint32_t w[4] = {q[v].x, q[v].y, q[v].z, q[v].w};
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const float2 x = pair16<BF16>(w[u]);
                finite = pack_top(pack_top(finite, x.x), x.y);
            }
        }
#pragma unroll
        for (int d = 8 / VECS; d > 0; d >>= 1)
            finite = fmaxf(finite, __shfl_xor_sync(0xffffffffu, finite, d));
        e = pack_exponent(finite);
    }
    *exponent = e;
    const F2 inv = pair_of(power_of_two(-e));
#pragma unroll
    for (int v = 0; v < VECS; ++v) {
        const uint32_t w[4] = {q[v].x, q[v].y, q[v].z, q[v].w};
        float2 x[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            x[u] = pair16<BF16>(w[u]);
            if (odd)
                x[u] = make_float2(nan_unless_finite(x[u].x), nan_unless_finite(x[u].y));
            x[u] = halves_of(mul2(pair_of(x[u].x, x[u].y), inv));
        }
        codes[v] = make_uint2(pack4(x[0], x[1]), pack4(x[2], x[3]));
    }
}

template <bool BF16>
__device__ __forceinline__ uint2 pack_group(const uint4 &q, int *exponent)
{
    const uint4 one[1] = {q};
    uint2 codes[1];
    pack_block<BF16>(one, exponent, codes);
    return codes[0];
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
    return pack4(make_float2(nan_unless_finite(x[0] * inv), nan_unless_finite(x[1] * inv)),
                 make_float2(nan_unless_finite(x[2] * inv), nan_unless_finite(x[3] * inv)));
}

}  // namespace gg
