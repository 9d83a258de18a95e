// AdamW over many tensors at once, for sm_103a.
//
// Elementwise: m = b1 m + (1-b1) g, v = b2 v + (1-b2) g^2, p = p (1 - lr wd) -
// lr' m / (sqrt(v) k + eps).  Bound: HBM; every array is read once and written
// once.  Measured: 117M float32 parameters with bfloat16 gradients and copies, float32
// states 495 us, 6.6 TB/s; 8-bit states 277 us, 6.8 TB/s (a copy's rate is 6.8); 200
// small tensors 3.1 us.  The tensors' descriptors are the kernel's parameter (up to 256 in a
// launch: no table in device memory, no copy before the launch), and a CTA
// finds its tensor by bisection of the running count of chunks.
//
// A warp works on blocks of 256 elements, each lane on two quads (elements
// 4 lane and 128 + 4 lane on): 16-byte accesses of float arrays, 8-byte ones
// of 16-bit arrays, 4-byte ones of codes, each a whole contiguous piece of the
// warp's block, all loads ahead of the arithmetic.
//
// States in 8 bits.  m and sqrt(v) are e4m3 codes under one power-of-two scale
// per block, the block's largest magnitude found by a warp reduction, so a
// scale costs no mantissa bit and scaling is exact.  sqrt(v), because e4m3
// spans 2^17 and v's range is twice that of g.  Rounding to nearest would
// freeze v: at b2 = 0.999 a step changes sqrt(v) by less than half an e4m3
// step (3%) unless g^2 > 60 v, and v would stay up to 60 times too small.
// So codes are rounded stochastically, and the state follows on average.  The
// random bits are a hash of (seed, step, tensor, element), 16 for m and 16 for
// sqrt(v): a published 32-bit integer mixer (xor-shift-multiply, multipliers
// 0x7feb352d and 0x846ca68b, by C. Wellons), no state to keep.  m, v and
// sqrt(v) are rounded as written in the formulas above, operation by
// operation to nearest, so that codes and scales have one value, whatever
// a compiler contracts; the parameter's update is within float32's rounding.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <mutex>

#include "f32x2.cuh"
#include "gg_internal.h"
#include "gg_ops.h"
#include "ptx.cuh"

namespace gg {
namespace {

constexpr int kSMs = 152;
constexpr int kMaxDevices = 64;
constexpr int kBlock = GG_ADAMW_BLOCK;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kStep = kWarps * kBlock;  // elements of one pass of a CTA

struct Tensor {
    void *param;
    const void *grad;
    void *m, *v;
    float *m_scale, *v_scale;
    void *copy;
    int64_t n;
    uint32_t key;     // hash of (seed, step, position)
    uint16_t copy_bf16, vec;
};

struct Group {
    AdamwStep h;
    int count;
    int chunk;                          // elements of a CTA's share, a multiple of kStep
    uint32_t first[GG_ADAMW_GROUP + 1];  // running count of chunks
    Tensor t[GG_ADAMW_GROUP];
};
static_assert(sizeof(Group) <= 32764, "kernel parameters");

__host__ __device__ __forceinline__ uint32_t mix32(uint32_t x)
{
    x ^= x >> 16;
    x *= 0x7feb352du;
    x ^= x >> 15;
    x *= 0x846ca68bu;
    return x ^ (x >> 16);
}

template <typename T>
__device__ __forceinline__ float to_f32(T x);
template <>
__device__ __forceinline__ float to_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ float to_f32<__half>(__half x) { return __half2float(x); }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

template <typename T>
struct alignas(4 * sizeof(T)) Quad {
    T e[4];
};

// Four consecutive elements; `left` of them exist.
template <typename T>
__device__ __forceinline__ void load4(const void *p, int64_t at, int left, bool vec, float (&x)[4])
{
    const T *q = reinterpret_cast<const T *>(p) + at;
    if (vec && left >= 4) {
        const Quad<T> v = *reinterpret_cast<const Quad<T> *>(q);
#pragma unroll
        for (int u = 0; u < 4; ++u)
            x[u] = to_f32<T>(v.e[u]);
    } else {
#pragma unroll
        for (int u = 0; u < 4; ++u)
            x[u] = u < left ? to_f32<T>(q[u]) : 0.0f;
    }
}

template <typename T>
__device__ __forceinline__ void store4(void *p, int64_t at, int left, bool vec, const float (&x)[4])
{
    T *q = reinterpret_cast<T *>(p) + at;
    if (vec && left >= 4) {
        Quad<T> v;
#pragma unroll
        for (int u = 0; u < 4; ++u)
            v.e[u] = from_f32<T>(x[u]);
        *reinterpret_cast<Quad<T> *>(q) = v;
    } else {
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (u < left)
                q[u] = from_f32<T>(x[u]);
    }
}

// Codes: the e4m3 values of four bytes.
__device__ __forceinline__ void load_codes(const void *p, int64_t at, int left, bool vec, float (&x)[4])
{
    const uint8_t *q = reinterpret_cast<const uint8_t *>(p) + at;
    uint32_t bytes = 0;
    if (vec && left >= 4) {
        bytes = *reinterpret_cast<const uint32_t *>(q);
    } else {
#pragma unroll
        for (int u = 0; u < 4; ++u)
            bytes |= u < left ? (uint32_t)q[u] << (8 * u) : 0u;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(bytes >> (16 * h)), __NV_E4M3);
        const float2 f = __half22float2(__half2(r));
        x[2 * h] = f.x;
        x[2 * h + 1] = f.y;
    }
}

__device__ __forceinline__ void store_codes(void *p, int64_t at, int left, bool vec, const float *x)
{
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[0], x[1]), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[2], x[3]), __NV_SATFINITE, __NV_E4M3);
    const uint32_t bytes = lo | hi << 16;
    uint8_t *q = reinterpret_cast<uint8_t *>(p) + at;
    if (vec && left >= 4) {
        *reinterpret_cast<uint32_t *>(q) = bytes;
    } else {
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (u < left)
                q[u] = (uint8_t)(bytes >> (8 * u));
    }
}

__device__ __forceinline__ bool finite(float x) { return fabsf(x) < INFINITY; }

// The largest magnitude of the warp's block, as bits: not below 0x7f800000
// where a value is not finite.
__device__ __forceinline__ uint32_t block_top(const float (&x)[8])
{
    uint32_t top = 0;
#pragma unroll
    for (int u = 0; u < 8; ++u)
        top = max(top, __float_as_uint(x[u]) & 0x7fffffffu);
    return __reduce_max_sync(~0u, top);
}

// The same over the finite values.
__device__ __forceinline__ uint32_t finite_top(const float (&x)[8])
{
    uint32_t top = 0;
#pragma unroll
    for (int u = 0; u < 8; ++u)
        top = finite(x[u]) ? max(top, __float_as_uint(x[u]) & 0x7fffffffu) : top;
    return __reduce_max_sync(~0u, top);
}

// Exponent k of the scale 2^k with top / 2^k in (224, 448]: 448 = 1.75 * 2^8, so
// adding 0x1fffff to the bits carries into the exponent beyond 1.75.
__device__ __forceinline__ int scale_exp(uint32_t top)
{
    const int k = (int)((top + 0x1fffffu) >> 23) - 127 - 8;
    return k < -118 ? -118 : k;
}

// One of the two e4m3 neighbours of a finite x (|x| <= 448), away from zero with
// the probability of the remainder: 16 random bits are added below the code's
// mantissa and the rest is cut off.  Below 2^-6, where the code's step stays
// 2^-9, the same on |x| + 2^-6.
__device__ __forceinline__ float round_e4m3(float x, uint32_t r16_shifted)
{
    const bool low = fabsf(x) < 0.015625f;
    const float off = __uint_as_float((__float_as_uint(x) & 0x80000000u) | 0x3c800000u);
    const float y = low ? x + off : x;
    const float z = __uint_as_float((__float_as_uint(y) + r16_shifted) & 0xfff00000u);
    return low ? z - off : z;
}

__device__ __forceinline__ float sqrt_approx(float x)
{
    float y;
    asm("sqrt.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// a + b of two products, each rounded, where the sum becomes a code: add2 of mul2's comes
// out as one fused operation, for all its .rn; a scalar sum does not.  sqrt(v) likewise:
// correctly rounded where it becomes a code.  (Fused, and with the approximate root, some
// codes in a million were their other neighbour.  117M parameters take 281.5 us instead of
// 280.7, and 16-bit ones 259 instead of 236.)
template <int BITS>
__device__ __forceinline__ F2 sum_of(F2 a, F2 b)
{
    if (BITS != 8)
        return add2(a, b);
    const float2 x = halves_of(a), y = halves_of(b);
    return pair_of(__fadd_rn(x.x, y.x), __fadd_rn(x.y, y.y));
}

template <int BITS>
__device__ __forceinline__ float root(float v)
{
    return BITS == 8 ? __fsqrt_rn(v) : sqrt_approx(v);
}

__device__ __forceinline__ float rcp_approx(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A step's constants, in pairs.
struct Constants {
    F2 gscale, beta1, omb1, beta2, omb2, ic2, eps, decay, minus_step;
    __device__ __forceinline__ explicit Constants(const AdamwStep &h)
        : gscale(pair_of(h.grad_scale ? *h.grad_scale : 1.0f)), beta1(pair_of(h.beta1)),
          omb1(pair_of(h.one_minus_beta1)), beta2(pair_of(h.beta2)), omb2(pair_of(h.one_minus_beta2)),
          ic2(pair_of(h.inv_sqrt_c2)), eps(pair_of(h.eps)), decay(pair_of(h.decay)),
          minus_step(pair_of(-h.step_size))
    {
    }
};

// One block of a tensor, whole or not, at any alignment.
template <typename P, typename G, int BITS>
__device__ __forceinline__ void any_block(const Tensor &t, const Constants &c, int64_t base, int lane)
{
    const bool vec = t.vec != 0;
    const int64_t block = base / kBlock;
    float p[8], gr[8], m[8], v[8], u[8];
    const float ms = BITS == 8 ? t.m_scale[block] : 0.0f, vs = BITS == 8 ? t.v_scale[block] : 0.0f;
    int left[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int64_t at = base + q * 128 + lane * 4;
        left[q] = t.n - at >= 4 ? 4 : (t.n > at ? (int)(t.n - at) : 0);
        float(&p4)[4] = *reinterpret_cast<float(*)[4]>(p + 4 * q);
        float(&g4)[4] = *reinterpret_cast<float(*)[4]>(gr + 4 * q);
        float(&m4)[4] = *reinterpret_cast<float(*)[4]>(m + 4 * q);
        float(&v4)[4] = *reinterpret_cast<float(*)[4]>(v + 4 * q);
        load4<P>(t.param, at, left[q], vec, p4);
        load4<G>(t.grad, at, left[q], vec, g4);
        if constexpr (BITS == 8) {
            load_codes(t.m, at, left[q], vec, m4);
            load_codes(t.v, at, left[q], vec, v4);
        } else {
            load4<float>(t.m, at, left[q], vec, m4);
            load4<float>(t.v, at, left[q], vec, v4);
        }
    }
    // 8-bit states: m and v are rounded operation by operation, as their definition has
    // them; 32-bit ones and the update need not be
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        const F2 x = mul2(pair_of(gr[e], gr[e + 1]), c.gscale);
        F2 m2 = pair_of(m[e], m[e + 1]), v2 = pair_of(v[e], v[e + 1]);
        if constexpr (BITS == 8) {
            m2 = mul2(m2, pair_of(ms));
            v2 = mul2(v2, pair_of(vs));
            v2 = mul2(v2, v2);
        }
        m2 = sum_of<BITS>(mul2(m2, c.beta1), mul2(x, c.omb1));
        v2 = sum_of<BITS>(mul2(v2, c.beta2), mul2(mul2(x, x), c.omb2));
        const float2 vh = halves_of(v2), mh = halves_of(m2);
        const float2 uh = make_float2(root<BITS>(vh.x), root<BITS>(vh.y));
        const float2 dh = halves_of(fma2(pair_of(uh.x, uh.y), c.ic2, c.eps));
        const F2 q2 = mul2(m2, pair_of(rcp_approx(dh.x), rcp_approx(dh.y)));
        const float2 ph = halves_of(fma2(q2, c.minus_step, mul2(pair_of(p[e], p[e + 1]), c.decay)));
        m[e] = mh.x, m[e + 1] = mh.y;
        v[e] = vh.x, v[e + 1] = vh.y;
        u[e] = uh.x, u[e + 1] = uh.y;
        p[e] = ph.x, p[e + 1] = ph.y;
    }
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int64_t at = base + q * 128 + lane * 4;
        const float(&p4)[4] = *reinterpret_cast<float(*)[4]>(p + 4 * q);
        store4<P>(t.param, at, left[q], vec, p4);
        if (t.copy) {
            if (t.copy_bf16)
                store4<__nv_bfloat16>(t.copy, at, left[q], vec, p4);
            else
                store4<__half>(t.copy, at, left[q], vec, p4);
        }
        if constexpr (BITS == 32) {
            store4<float>(t.m, at, left[q], vec, *reinterpret_cast<float(*)[4]>(m + 4 * q));
            store4<float>(t.v, at, left[q], vec, *reinterpret_cast<float(*)[4]>(v + 4 * q));
        }
    }
    if constexpr (BITS == 8) {
        // elements past the end hold m = v = 0.  The scale of sqrt(v) comes from
        // the largest v: the square root rounds monotonically.
        uint32_t mt = block_top(m), vt = block_top(v);
        const bool odd = mt >= 0x7f800000u || vt >= 0x7f800000u;  // the whole warp's
        if (odd) {
            mt = finite_top(m);
            vt = finite_top(v);
        }
        const int mk = scale_exp(mt);
        const int vk = scale_exp(__float_as_uint(__fsqrt_rn(__uint_as_float(vt))));
        const float ims = __uint_as_float((uint32_t)(127 - mk) << 23);
        const float ivs = __uint_as_float((uint32_t)(127 - vk) << 23);
        if (lane == 0) {
            t.m_scale[block] = __uint_as_float((uint32_t)(127 + mk) << 23);
            t.v_scale[block] = __uint_as_float((uint32_t)(127 + vk) << 23);
        }
        const uint32_t key = mix32((uint32_t)(base >> 32) ^ t.key);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int64_t at = base + q * 128 + lane * 4;
            const uint32_t first = (uint32_t)at ^ key;  // at is a multiple of 4
            float cm[4], cv[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t r = mix32(first ^ (uint32_t)e);
                const float y = m[4 * q + e] * ims, z = u[4 * q + e] * ivs;
                cm[e] = round_e4m3(y, (r & 0xffffu) << 4);
                cv[e] = round_e4m3(z, r >> 16 << 4);
                if (odd) {
                    cm[e] = finite(m[4 * q + e]) ? cm[e] : NAN;
                    cv[e] = finite(v[4 * q + e]) ? cv[e] : NAN;
                }
            }
            store_codes(t.m, at, left[q], vec, cm);
            store_codes(t.v, at, left[q], vec, cv);
        }
    }
}

// Eight consecutive elements of a lane.
template <typename T>
struct Eight;
template <>
struct Eight<float> {
    float4 a, b;
    __device__ __forceinline__ F2 get(int e) const
    {
        const float4 &h = e & 4 ? b : a;
        return e & 2 ? pair_of(h.z, h.w) : pair_of(h.x, h.y);
    }
    __device__ __forceinline__ void set(int e, float2 y)
    {
        float4 &h = e & 4 ? b : a;
        if (e & 2)
            h.z = y.x, h.w = y.y;
        else
            h.x = y.x, h.y = y.y;
    }
    __device__ __forceinline__ void store(void *p, int64_t at) const
    {
        float *q = reinterpret_cast<float *>(p) + at;
        asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(q), "f"(a.x),
                     "f"(a.y), "f"(a.z), "f"(a.w), "f"(b.x), "f"(b.y), "f"(b.z), "f"(b.w)
                     : "memory");
    }
};
template <>
struct Eight<__nv_bfloat16> {
    uint4 w;
    __device__ __forceinline__ F2 get(int e) const
    {
        const uint32_t h = (&w.x)[e >> 1];
        return pair_of(__uint_as_float(h << 16), __uint_as_float(h & 0xffff0000u));
    }
    __device__ __forceinline__ void set(int e, float2 y)
    {
        const __nv_bfloat162 h = __float22bfloat162_rn(y);
        (&w.x)[e >> 1] = *reinterpret_cast<const uint32_t *>(&h);
    }
    __device__ __forceinline__ void store(void *p, int64_t at) const
    {
        *reinterpret_cast<uint4 *>(reinterpret_cast<__nv_bfloat16 *>(p) + at) = w;
    }
};
template <>
struct Eight<__half> {
    uint4 w;
    __device__ __forceinline__ F2 get(int e) const
    {
        const float2 f = __half22float2(reinterpret_cast<const __half2 *>(&w)[e >> 1]);
        return pair_of(f.x, f.y);
    }
    __device__ __forceinline__ void set(int e, float2 y)
    {
        const __half2 h = __float22half2_rn(y);
        (&w.x)[e >> 1] = *reinterpret_cast<const uint32_t *>(&h);
    }
    __device__ __forceinline__ void store(void *p, int64_t at) const
    {
        *reinterpret_cast<uint4 *>(reinterpret_cast<__half *>(p) + at) = w;
    }
};

// A warp's ring of whole blocks with 8-bit states on their way from memory: one
// stage holds param, grad and the codes of m and v, copied in 16- and 8-byte pieces.
// Bytes in flight are what this kernel lives on: with 46 KB of loads in flight
// on an SM it ran at 4.9 TB/s, the latency of a load under its stores 2.5 us.
template <typename P, typename G>
struct Ring {
    static constexpr int kP = kBlock * (int)sizeof(P), kG = kBlock * (int)sizeof(G);
    static constexpr int kStage = kP + kG + 2 * kBlock;
    static constexpr int kDepth = 65536 / (kWarps * kStage);  // 64 KB a CTA, three CTAs an SM
    static constexpr int kWarpBytes = kDepth * kStage;
    static constexpr int kBytes = kWarps * kWarpBytes;

    // Pieces of an array of 32-byte lanes, so that the lanes' 16-byte reads of
    // either half fall on different banks.
    static __device__ __forceinline__ int place(int piece, int bytes)
    {
        return bytes == 1024 ? (piece ^ (piece >> 3 & 1)) * 16 : piece * 16;
    }
    static __device__ __forceinline__ void piece(uint32_t dst, const void *src)
    {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    }
    // The codes come 8 bytes at a time: with 16, tensors in a flat buffer that begin at
    // a multiple of 8 elements went without the ring (16 of 1600001: 106 us, now 67; it costs aligned ones 0.3 %).
    static __device__ __forceinline__ void half_piece(uint32_t dst, const void *src)
    {
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
    }
    // Start the copies of the block at element `base`.
    static __device__ __forceinline__ void start(uint32_t stage, const Tensor &t, int64_t base, int lane)
    {
        const uint8_t *p = reinterpret_cast<const uint8_t *>(t.param) + base * (int64_t)sizeof(P);
        const uint8_t *g = reinterpret_cast<const uint8_t *>(t.grad) + base * (int64_t)sizeof(G);
        const int64_t c = base + lane * 8;
#pragma unroll
        for (int k = 0; k < kP / 512; ++k)
            piece(stage + place(k * 32 + lane, kP), p + (k * 32 + lane) * 16);
#pragma unroll
        for (int k = 0; k < kG / 512; ++k)
            piece(stage + kP + place(k * 32 + lane, kG), g + (k * 32 + lane) * 16);
        half_piece(stage + kP + kG + lane * 8, reinterpret_cast<const uint8_t *>(t.m) + c);
        half_piece(stage + kP + kG + kBlock + lane * 8, reinterpret_cast<const uint8_t *>(t.v) + c);
    }
    static __device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
    // Wait for all but the newest kDepth - 1 groups of this thread's copies.
    static __device__ __forceinline__ void wait()
    {
        asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory");
        __syncwarp();
    }
    template <typename T>
    static __device__ __forceinline__ void read(const uint8_t *at, int lane, Eight<T> &x)
    {
        if constexpr (sizeof(T) == 4) {
            x.a = *reinterpret_cast<const float4 *>(at + place(2 * lane, 1024));
            x.b = *reinterpret_cast<const float4 *>(at + place(2 * lane + 1, 1024));
        } else {
            x.w = *reinterpret_cast<const uint4 *>(at + lane * 16);
        }
    }
};

// A lane's share of a whole block with 8-bit states.
template <typename P, typename G>
struct Lane8 {
    Eight<P> p;
    Eight<G> g;
    uint2 m, v;
    float ms, vs;
    __device__ __forceinline__ void read(const uint8_t *stage, int lane)
    {
        using R = Ring<P, G>;
        R::read(stage, lane, p);
        R::read(stage + R::kP, lane, g);
        m = *reinterpret_cast<const uint2 *>(stage + R::kP + R::kG + lane * 8);
        v = *reinterpret_cast<const uint2 *>(stage + R::kP + R::kG + kBlock + lane * 8);
    }
};

__device__ __forceinline__ F2 codes_at(const uint2 &w, int e)
{
    const uint32_t h = (e & 4 ? w.y : w.x) >> (e & 2 ? 16 : 0);
    const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)h, __NV_E4M3);
    const float2 f = __half22float2(__half2(r));
    return pair_of(f.x, f.y);
}

__device__ __forceinline__ uint32_t codes_of(float a, float b, float c, float d)
{
    return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3) |
           (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3) << 16;
}

// The scale's exponent for sqrt(v) from the largest v's bits: what scale_exp
// gives for its correctly rounded square root.  In a period of 4 of v,
// sqrt(v) passes 1.75 2^j where v passes 3.0625 4^j, which in the 24 bits of
// (exponent parity, mantissa) is 0xc40000; a float above that has a square root
// that rounds above 1.75 2^j.
__device__ __forceinline__ int sqrt_scale_exp(uint32_t vt)
{
    if (vt < 0x00800000u)  // zero or subnormal: the warp takes the long way together
        return scale_exp(__float_as_uint(__fsqrt_rn(__uint_as_float(vt))));
    return (int)((vt + 0x800000u + 0x3bffffu) >> 24) - 72;
}

// One whole block with 8-bit states, already loaded.  Nothing is stored, and
// the answer is false, where a new state is not finite.
template <typename P, typename G>
__device__ __forceinline__ bool whole_block8(const Tensor &t, const Constants &c, Lane8<P, G> &x,
                                             int64_t base, int lane, uint32_t &key, uint32_t &hi32,
                                             float &new_ms, float &new_vs)
{
    const int64_t at = base + lane * 8;
    float m[8], u[8];
    uint32_t mt = 0, vt = 0;
    Eight<P> p;
    uint4 copy;
    const bool copy_bf16 = t.copy_bf16 != 0;
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        const F2 g2 = mul2(x.g.get(e), c.gscale);
        F2 m2 = mul2(codes_at(x.m, e), pair_of(x.ms));
        F2 v2 = mul2(codes_at(x.v, e), pair_of(x.vs));
        v2 = mul2(v2, v2);
        m2 = sum_of<8>(mul2(m2, c.beta1), mul2(g2, c.omb1));
        v2 = sum_of<8>(mul2(v2, c.beta2), mul2(mul2(g2, g2), c.omb2));
        const float2 vh = halves_of(v2), mh = halves_of(m2);
        const float2 uh = make_float2(root<8>(vh.x), root<8>(vh.y));
        const float2 dh = halves_of(fma2(pair_of(uh.x, uh.y), c.ic2, c.eps));
        const F2 q2 = mul2(m2, pair_of(rcp_approx(dh.x), rcp_approx(dh.y)));
        const float2 ph = halves_of(fma2(q2, c.minus_step, mul2(x.p.get(e), c.decay)));
        p.set(e, ph);
        if (copy_bf16) {
            const __nv_bfloat162 h = __float22bfloat162_rn(ph);
            (&copy.x)[e >> 1] = *reinterpret_cast<const uint32_t *>(&h);
        } else {
            const __half2 h = __float22half2_rn(ph);
            (&copy.x)[e >> 1] = *reinterpret_cast<const uint32_t *>(&h);
        }
        m[e] = mh.x, m[e + 1] = mh.y;
        u[e] = uh.x, u[e + 1] = uh.y;
        mt = max(mt, max(__float_as_uint(mh.x) & 0x7fffffffu, __float_as_uint(mh.y) & 0x7fffffffu));
        vt = max(vt, max(__float_as_uint(vh.x), __float_as_uint(vh.y)));
    }
    mt = __reduce_max_sync(~0u, mt);
    vt = __reduce_max_sync(~0u, vt);
    if (mt >= 0x7f800000u || vt >= 0x7f800000u)  // the whole warp's answer
        return false;
    p.store(t.param, at);
    if (t.copy)
        *reinterpret_cast<uint4 *>(reinterpret_cast<uint16_t *>(t.copy) + at) = copy;
    const int mk = scale_exp(mt), vk = sqrt_scale_exp(vt);
    const float ims = __uint_as_float((uint32_t)(127 - mk) << 23);
    const float ivs = __uint_as_float((uint32_t)(127 - vk) << 23);
    new_ms = __uint_as_float((uint32_t)(127 + mk) << 23);
    new_vs = __uint_as_float((uint32_t)(127 + vk) << 23);
    if ((uint32_t)(base >> 32) != hi32) {
        hi32 = (uint32_t)(base >> 32);
        key = mix32(hi32 ^ t.key);
    }
    const uint32_t first = (uint32_t)at ^ key;  // at is a multiple of 8
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uint32_t r = mix32(first ^ (uint32_t)e);
        m[e] = round_e4m3(m[e] * ims, (r & 0xffffu) << 4);
        u[e] = round_e4m3(u[e] * ivs, r >> 16 << 4);
    }
    *reinterpret_cast<uint2 *>(reinterpret_cast<uint8_t *>(t.m) + at) =
        make_uint2(codes_of(m[0], m[1], m[2], m[3]), codes_of(m[4], m[5], m[6], m[7]));
    *reinterpret_cast<uint2 *>(reinterpret_cast<uint8_t *>(t.v) + at) =
        make_uint2(codes_of(u[0], u[1], u[2], u[3]), codes_of(u[4], u[5], u[6], u[7]));
    return true;
}

template <typename P, typename G, int BITS>
__global__ void __launch_bounds__(kThreads, BITS == 8 ? 3 : 4) adamw_kernel(const __grid_constant__ Group g)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int lo = 0, hi = g.count - 1;  // the tensor of this CTA's chunk
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (g.first[mid] <= blockIdx.x)
            lo = mid;
        else
            hi = mid - 1;
    }
    const Tensor &t = g.t[lo];
    const int64_t begin = (int64_t)(blockIdx.x - g.first[lo]) * g.chunk;
    const int64_t end = gg_min64(begin + g.chunk, t.n);
    const Constants c(g.h);

    if constexpr (BITS == 32) {
#pragma unroll 1
        for (int64_t base = begin + warp * kBlock; base < end; base += kStep)
            any_block<P, G, 32>(t, c, base, lane);
    } else {
        // whole, aligned blocks come through the warp's ring; a chunk has at most 32
        // blocks a warp, and lane k keeps the scales of the k-th
        using R = Ring<P, G>;
        extern __shared__ __align__(16) uint8_t smem[];
        uint8_t *ring = smem + warp * R::kWarpBytes;
        const uint32_t ring_at = ptx::smem_addr(ring);
        const int64_t whole = t.vec == 2 ? gg_min64(end, t.n / kBlock * kBlock) : begin;
        const int64_t first = begin + warp * kBlock;
        const int count = first < whole ? (int)((whole - first + kStep - 1) / kStep) : 0;
        const int64_t my_block = first / kBlock + (int64_t)lane * kWarps;
#pragma unroll 1
        for (int k = 0; k < R::kDepth - 1; ++k) {
            if (k < count)
                R::start(ring_at + k * R::kStage, t, first + (int64_t)k * kStep, lane);
            R::commit();
        }
        float ms = 0.0f, vs = 0.0f;
        if (lane < count) {
            ms = t.m_scale[my_block];
            vs = t.v_scale[my_block];
        }
        uint32_t hi32 = (uint32_t)(first >> 32), key = mix32(hi32 ^ t.key);
        uint32_t kept = 0;  // blocks whose scales lane k stores
        int stage = 0;
#pragma unroll 1
        for (int k = 0; k < count; ++k) {
            const int ahead = k + R::kDepth - 1;
            if (ahead < count) {
                const int s = stage == 0 ? R::kDepth - 1 : stage - 1;
                R::start(ring_at + s * R::kStage, t, first + (int64_t)ahead * kStep, lane);
            }
            R::commit();
            R::wait();
            Lane8<P, G> x;
            x.read(ring + stage * R::kStage, lane);
            x.ms = __shfl_sync(~0u, ms, k);
            x.vs = __shfl_sync(~0u, vs, k);
            __syncwarp();  // read by every lane: the next round may fill the stage
            const int64_t base = first + (int64_t)k * kStep;
            float new_ms, new_vs;
            if (whole_block8(t, c, x, base, lane, key, hi32, new_ms, new_vs)) {
                ms = lane == k ? new_ms : ms;
                vs = lane == k ? new_vs : vs;
                kept |= 1u << k;
            } else {
                any_block<P, G, 8>(t, c, base, lane);
            }
            stage = stage + 1 == R::kDepth ? 0 : stage + 1;
        }
        if (kept >> lane & 1u) {
            t.m_scale[my_block] = ms;
            t.v_scale[my_block] = vs;
        }
#pragma unroll 1
        for (int64_t base = first + (int64_t)count * kStep; base < end; base += kStep)
            any_block<P, G, 8>(t, c, base, lane);
    }
}

template <typename P, typename G>
cudaError_t launch_group(const Group &g, int bits, cudaStream_t s)
{
    const unsigned grid = g.first[g.count];
    if (bits == 8) {
        constexpr int kBytes = Ring<P, G>::kBytes;
        static std::once_flag once[kMaxDevices];
        static cudaError_t result[kMaxDevices];
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices)
            dev = 0;
        std::call_once(once[dev], [&] {
            result[dev] = cudaFuncSetAttribute(adamw_kernel<P, G, 8>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
        });
        if (result[dev] != cudaSuccess)
            return result[dev];
        adamw_kernel<P, G, 8><<<grid, kThreads, kBytes, s>>>(g);
    } else {
        adamw_kernel<P, G, 32><<<grid, kThreads, 0, s>>>(g);
    }
    return cudaGetLastError();
}

template <typename P>
cudaError_t launch_param(const Group &g, int grad, int bits, cudaStream_t s)
{
    if (grad == GG_F32)
        return launch_group<P, float>(g, bits, s);
    if (grad == GG_F16)
        return launch_group<P, __half>(g, bits, s);
    return launch_group<P, __nv_bfloat16>(g, bits, s);
}

cudaError_t launch_one(const Group &g, int param, int grad, int bits, cudaStream_t s)
{
    if (g.count == 0)
        return cudaSuccess;
    if (param == GG_F32)
        return launch_param<float>(g, grad, bits, s);
    if (param == GG_F16)
        return launch_param<__half>(g, grad, bits, s);
    return launch_param<__nv_bfloat16>(g, grad, bits, s);
}

// 2: every array holds whole blocks in aligned vectors (32 bytes of float, 16 of
// 16-bit types, 8 of codes); 1: 4 elements in one access; 0: one by one.
int vector_width(const gg_adamw_tensor &x)
{
    const uint64_t param = reinterpret_cast<uint64_t>(x.param), grad = reinterpret_cast<uint64_t>(x.grad);
    const uint64_t state = reinterpret_cast<uint64_t>(x.m) | reinterpret_cast<uint64_t>(x.v);
    const uint64_t copy = reinterpret_cast<uint64_t>(x.copy);
    for (int width = 2; width >= 1; --width) {
        const uint64_t f = 16 * width, h = 8 * width, s = x.state_bits == 8 ? (width == 2 ? 8 : 4) : f;
        if (param % (x.param_dtype == GG_F32 ? f : h) == 0 && grad % (x.grad_dtype == GG_F32 ? f : h) == 0 &&
            state % s == 0 && copy % h == 0)
            return width;
    }
    return 0;
}

}  // namespace

cudaError_t launch_adamw(const gg_adamw_tensor *tensors, int count, const AdamwStep &h, cudaStream_t s)
{
    // Chunks: 8 passes of a CTA once there are enough of them to fill the GPU, so that
    // the search for the tensor is spread over more elements, one pass for small
    // work (longer chunks measured slower: 545 us at 31 passes, 495 at 8, for 117M
    // elements with 32-bit states).
    int64_t total = 0;
    uint32_t kinds = 0;  // combinations of types that occur
    for (int i = 0; i < count; ++i) {
        total += tensors[i].n;
        if (tensors[i].n > 0)
            kinds |= 1u << (tensors[i].param_dtype * 6 + tensors[i].grad_dtype * 2 +
                            (tensors[i].state_bits == 8));
    }
    const int64_t chunk = total >= (int64_t)kSMs * 8 * 8 * kStep ? 8 * kStep : kStep;
    static thread_local Group g;
    g.h = h;
    g.chunk = (int)chunk;
    // one kernel per combination of types, each over its tensors in list order
    for (int kind = 0; kind < 18; ++kind) {
        if (!(kinds >> kind & 1u))
            continue;
        const int param = kind / 6, grad = kind / 2 % 3, bits = kind % 2 ? 8 : 32;
        g.count = 0;
        g.first[0] = 0;
        for (int i = 0; i < count; ++i) {
            const gg_adamw_tensor &x = tensors[i];
            if (x.n == 0 || x.param_dtype != param || x.grad_dtype != grad || x.state_bits != bits)
                continue;
            const int64_t chunks = (x.n + chunk - 1) / chunk;
            if (g.count == GG_ADAMW_GROUP || g.first[g.count] + chunks > 0x7fffffffll) {
                const cudaError_t e = launch_one(g, param, grad, bits, s);
                if (e != cudaSuccess)
                    return e;
                g.count = 0;
            }
            Tensor &t = g.t[g.count];
            t.param = x.param;
            t.grad = x.grad;
            t.m = x.m;
            t.v = x.v;
            t.m_scale = x.m_scale;
            t.v_scale = x.v_scale;
            t.copy = x.copy;
            t.n = x.n;
            t.key = bits == 8 ? mix32(mix32(mix32(mix32((uint32_t)i) ^ h.step) ^ (uint32_t)h.seed) ^
                                      (uint32_t)(h.seed >> 32))
                              : 0;
            t.copy_bf16 = x.copy_dtype == GG_BF16;
            t.vec = (uint16_t)vector_width(x);
            g.first[g.count + 1] = g.first[g.count] + (uint32_t)chunks;
            ++g.count;
        }
        const cudaError_t e = launch_one(g, param, grad, bits, s);
        if (e != cudaSuccess)
            return e;
    }
    return cudaSuccess;
}

}  // namespace gg
