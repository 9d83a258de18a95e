// Root-mean-square norm with the residual's addition and an output in 8 bits, its gradients, and
// the 8-bit form of activations (pack8.cuh) by itself, for sm_103a.
//
//     h = x + residual,  rstd = 1 / sqrt(mean h^2 + eps),  y = h rstd w
//     dh = rstd (g - u mean(g u)) + dh_in,   g = dy w,  u = h rstd;   dw = sum over rows of dy u
//
// All of it is bound by HBM: each matrix is read or written once.  h is rounded to 16 bits before
// the norm is taken, so that the backward pass, which reads the rounded h, differentiates exactly
// what the forward pass computed; y is rounded once, and the codes are those of the rounded y,
// which is what the next layer multiplies by.
//
// Row kernels.  A row belongs to R warps (1 to 32) of a block, VPT vectors of eight elements a
// thread, so that it stays in registers between its sum and its use; blocks of at least eight
// warps take 8 / R rows side by side and walk the rows with the grid's stride.  Rows that are not
// 16-byte aligned, or longer than 32 warps hold, go through kernels that read a row twice.
//
// dw: a thread keeps the sums of its own columns over all its rows in registers; a block adds its
// rows' sums in shared memory and stores them as one row of the workspace, and a second kernel
// adds the blocks' rows.  Fixed orders throughout: the same bits on every run.
#include <cuda_runtime.h>

#include "act.cuh"
#include "gg_internal.h"
#include "gg_ops.h"
#include "pack8.cuh"
#include "ptx.cuh"

namespace gg {
namespace {

constexpr int kSMs = 152;
constexpr int kMaxWarps = 32;
constexpr int kVec = 8;

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

// How a block's warps share rows.
struct RowShape {
    int R;     // warps of a row
    int rows;  // rows of a block
};

// The sum over a row's R warps of each warp's v; every thread of the block calls it.  Two
// buffers in turn, so that one barrier a call is enough.
__device__ __forceinline__ float row_sum(float v, const RowShape &s, float (&buf)[2][kMaxWarps], int turn)
{
    v = warp_sum(v);
    if (s.R == 1)
        return v;
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0)
        buf[turn][warp] = v;
    __syncthreads();
    const int first = warp / s.R * s.R;
    float t = 0.0f;
    for (int k = 0; k < s.R; ++k)
        t += buf[turn][first + k];
    return t;
}

// Eight neighbouring weights.
template <bool BF16>
__device__ __forceinline__ void load_weights(const void *w, int f32, int vec, int64_t n, int64_t left, float (&v)[8])
{
    if (f32) {
        const float *p = reinterpret_cast<const float *>(w) + n;
        if (left >= 8 && vec) {
            const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
            v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
            v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
            return;
        }
#pragma unroll
        for (int u = 0; u < 8; ++u)
            v[u] = u < left ? p[u] : 0.0f;
        return;
    }
    const uint16_t *p = reinterpret_cast<const uint16_t *>(w) + n;
    if (left >= 8 && vec) {
        const uint4 q = *reinterpret_cast<const uint4 *>(p);
        const uint32_t h[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const float2 f = pair16<BF16>(h[u]);
            v[2 * u] = f.x, v[2 * u + 1] = f.y;
        }
        return;
    }
#pragma unroll
    for (int u = 0; u < 8; ++u)
        v[u] = u < left ? load16(p, u, BF16) : 0.0f;
}

template <bool BF16>
__device__ __forceinline__ void floats8(const uint4 &q, float (&v)[8])
{
    const uint32_t h[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const float2 f = pair16<BF16>(h[u]);
        v[2 * u] = f.x, v[2 * u + 1] = f.y;
    }
}

template <bool BF16>
__device__ __forceinline__ uint4 halves8(const float (&v)[8])
{
    return make_uint4(pair16_of<BF16>(v[0], v[1]), pair16_of<BF16>(v[2], v[3]), pair16_of<BF16>(v[4], v[5]),
                      pair16_of<BF16>(v[6], v[7]));
}

// ---- forward ------------------------------------------------------------------------------
template <bool BF16, int VPT>
__global__ void __launch_bounds__(1024) norm_kernel(const __grid_constant__ NormArgs a, const RowShape s)
{
    __shared__ float sums[2][kMaxWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int sub = warp % s.R;
    const int64_t step = (int64_t)gridDim.x * s.rows;
    const uint16_t *x = reinterpret_cast<const uint16_t *>(a.x), *r = reinterpret_cast<const uint16_t *>(a.residual);
    int turn = 0;
    for (int64_t row0 = (int64_t)blockIdx.x * s.rows; row0 < a.M; row0 += step, turn ^= 1) {
        const int64_t row = row0 + warp / s.R;
        const bool live = row < a.M;
        uint4 h[VPT];
        float sq = 0.0f;
        if (live) {
            uint4 q[VPT];
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int64_t n = (int64_t)((k * s.R + sub) * 32 + lane) * kVec;
                h[k] = load8(x + row * a.ldx + n, a.N - n);
                if (r)
                    q[k] = load8(r + row * a.ldr + n, a.N - n);
            }
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                float v[8];
                floats8<BF16>(h[k], v);
                if (r) {
                    float t[8];
                    floats8<BF16>(q[k], t);
#pragma unroll
                    for (int u = 0; u < 8; ++u)
                        v[u] += t[u];
                    h[k] = halves8<BF16>(v);
                    floats8<BF16>(h[k], v);
                }
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    sq = fmaf(v[u], v[u], sq);
            }
            if (a.h) {
#pragma unroll
                for (int k = 0; k < VPT; ++k) {
                    const int64_t n = (int64_t)((k * s.R + sub) * 32 + lane) * kVec;
                    store8(reinterpret_cast<uint16_t *>(a.h) + row * a.ldh + n, a.N - n, h[k]);
                }
            }
        }
        const float total = row_sum(sq, s, sums, turn);
        if (!live)
            continue;
        const float rstd = 1.0f / sqrtf(total / (float)a.N + a.eps);
        if (a.rstd && sub == 0 && lane == 0)
            a.rstd[row] = rstd;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int64_t n = (int64_t)((k * s.R + sub) * 32 + lane) * kVec, left = a.N - n;
            float v[8], w[8];
            floats8<BF16>(h[k], v);
            load_weights<BF16>(a.weight, a.weight_f32, a.weight_vec, n, left, w);
#pragma unroll
            for (int u = 0; u < 8; ++u)
                v[u] = v[u] * rstd * w[u];
            const uint4 y = halves8<BF16>(v);
            if (a.y)
                store8(reinterpret_cast<uint16_t *>(a.y) + row * a.ldy + n, left, y);
            if (a.codes) {
                floats8<BF16>(y, v);
                int e;
                const uint2 c = pack_group(v, &e);
                if (left > 0) {
                    store_codes8(a.codes + row * a.ldc + n, left, c);
                    if ((lane & 15) == 0)
                        a.scales[row * a.lds + n / kPackBlock] = power_of_two(e);
                }
            }
        }
    }
}

// Any alignment and length: a block a row, a warp a block of 128 elements, the row read twice
// (h again where it was stored: x or the residual may be what it was stored over).
template <bool BF16>
__global__ void __launch_bounds__(512) norm_any_kernel(const __grid_constant__ NormArgs a)
{
    __shared__ float sums[2][kMaxWarps];
    const RowShape s{(int)blockDim.x / 32, 1};
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int turn = 0;
    for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x, turn ^= 1) {
        const auto sum_at = [&](int64_t n) {
            float v = load16(a.x, row * a.ldx + n, BF16);
            if (a.residual) {
                v += load16(a.residual, row * a.ldr + n, BF16);
                const uint32_t p = pair16_of<BF16>(v, 0.0f);
                v = pair16<BF16>(p).x;
            }
            return v;
        };
        float sq = 0.0f;
        for (int64_t b = (int64_t)warp * kPackBlock; b < a.N; b += (int64_t)s.R * kPackBlock)
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int64_t n = b + u * 32 + lane;
                if (n < a.N) {
                    const float v = sum_at(n);
                    if (a.h)
                        store16(a.h, row * a.ldh + n, v, BF16);
                    sq = fmaf(v, v, sq);
                }
            }
        const float rstd = 1.0f / sqrtf(row_sum(sq, s, sums, turn) / (float)a.N + a.eps);
        if (a.rstd && threadIdx.x == 0)
            a.rstd[row] = rstd;
        for (int64_t b = (int64_t)warp * kPackBlock; b < a.N; b += (int64_t)s.R * kPackBlock) {
            float y[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int64_t n = b + u * 32 + lane;
                y[u] = 0.0f;
                if (n < a.N) {
                    const float v = a.h ? load16(a.h, row * a.ldh + n, BF16) : sum_at(n);
                    const float w = a.weight_f32 ? reinterpret_cast<const float *>(a.weight)[n] : load16(a.weight, n, BF16);
                    y[u] = pair16<BF16>(pair16_of<BF16>(v * rstd * w, 0.0f)).x;
                    if (a.y)
                        store16(a.y, row * a.ldy + n, y[u], BF16);
                }
            }
            if (a.codes) {
                int e;
                const uint32_t c = pack_warp(y, &e);
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int64_t n = b + u * 32 + lane;
                    if (n < a.N)
                        a.codes[row * a.ldc + n] = (uint8_t)(c >> (8 * u));
                }
                if (lane == 0)
                    a.scales[row * a.lds + b / kPackBlock] = power_of_two(e);
            }
        }
    }
}

// ---- backward -----------------------------------------------------------------------------
template <bool BF16, int VPT>
__global__ void __launch_bounds__(VPT > 2 ? 512 : 1024) norm_backward_kernel(const __grid_constant__ NormBackwardArgs a,
                                                                             const RowShape s)
{
    __shared__ float sums[2][kMaxWarps];
    extern __shared__ float columns[];  // where a block has several rows: their sums
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int sub = warp % s.R;
    const int64_t step = (int64_t)gridDim.x * s.rows;
    const uint16_t *dy = reinterpret_cast<const uint16_t *>(a.dy), *h = reinterpret_cast<const uint16_t *>(a.h),
                   *in = reinterpret_cast<const uint16_t *>(a.dh_in);
    float dw[VPT][8];
#pragma unroll
    for (int k = 0; k < VPT; ++k)
#pragma unroll
        for (int u = 0; u < 8; ++u)
            dw[k][u] = 0.0f;
    int turn = 0;
    for (int64_t row0 = (int64_t)blockIdx.x * s.rows; row0 < a.M; row0 += step, turn ^= 1) {
        const int64_t row = row0 + warp / s.R;
        const bool live = row < a.M;
        uint4 qy[VPT], qh[VPT], qi[VPT];
        float dot = 0.0f, rstd = 0.0f;
        if (live) {
            rstd = a.rstd[row];
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int64_t n = (int64_t)((k * s.R + sub) * 32 + lane) * kVec;
                qy[k] = load8(dy + row * a.lddy + n, a.N - n);
                qh[k] = load8(h + row * a.ldh + n, a.N - n);
                if (in)
                    qi[k] = load8(in + row * a.lddhin + n, a.N - n);
            }
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int64_t n = (int64_t)((k * s.R + sub) * 32 + lane) * kVec;
                float y[8], u8[8], w[8];
                floats8<BF16>(qy[k], y);
                floats8<BF16>(qh[k], u8);
                load_weights<BF16>(a.weight, a.weight_f32, a.weight_vec, n, a.N - n, w);
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const float t = u8[u] * rstd;
                    dot = fmaf(y[u] * w[u], t, dot);
                    dw[k][u] = fmaf(y[u], t, dw[k][u]);
                }
            }
        }
        const float c = row_sum(dot, s, sums, turn) / (float)a.N;
        if (!live || !a.dh)
            continue;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int64_t n = (int64_t)((k * s.R + sub) * 32 + lane) * kVec, left = a.N - n;
            float y[8], v[8], w[8];
            floats8<BF16>(qy[k], y);
            floats8<BF16>(qh[k], v);
            load_weights<BF16>(a.weight, a.weight_f32, a.weight_vec, n, left, w);
#pragma unroll
            for (int u = 0; u < 8; ++u)
                v[u] = rstd * (y[u] * w[u] - v[u] * rstd * c);
            if (in) {
                float t[8];
                floats8<BF16>(qi[k], t);
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    v[u] += t[u];
            }
            store8(reinterpret_cast<uint16_t *>(a.dh) + row * a.lddh + n, left, halves8<BF16>(v));
        }
    }
    if (!a.partial)
        return;
    float *out = a.partial + (int64_t)blockIdx.x * a.N;
    for (int g = 0; g < s.rows; ++g) {  // row group by row group, in order
        if (warp / s.R == g) {
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int64_t n = (int64_t)((k * s.R + sub) * 32 + lane) * kVec;
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    if (n + u < a.N) {
                        const float t = g > 0 ? columns[n + u] + dw[k][u] : dw[k][u];
                        if (g + 1 == s.rows)
                            out[n + u] = t;
                        else
                            columns[n + u] = t;
                    }
            }
        }
        if (g + 1 < s.rows)
            __syncthreads();
    }
}

// Any alignment and length, rows: as norm_any_kernel.
template <bool BF16>
__global__ void __launch_bounds__(512) norm_backward_any_kernel(const __grid_constant__ NormBackwardArgs a)
{
    __shared__ float sums[2][kMaxWarps];
    const RowShape s{(int)blockDim.x / 32, 1};
    int turn = 0;
    const auto weight = [&](int64_t n) {
        return a.weight_f32 ? reinterpret_cast<const float *>(a.weight)[n] : load16(a.weight, n, BF16);
    };
    for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x, turn ^= 1) {
        const float rstd = a.rstd[row];
        float dot = 0.0f;
        for (int64_t n = threadIdx.x; n < a.N; n += blockDim.x)
            dot = fmaf(load16(a.dy, row * a.lddy + n, BF16) * weight(n), load16(a.h, row * a.ldh + n, BF16) * rstd, dot);
        const float c = row_sum(dot, s, sums, turn) / (float)a.N;
        for (int64_t n = threadIdx.x; n < a.N; n += blockDim.x) {
            float v = rstd * (load16(a.dy, row * a.lddy + n, BF16) * weight(n) -
                              load16(a.h, row * a.ldh + n, BF16) * rstd * c);
            if (a.dh_in)
                v += load16(a.dh_in, row * a.lddhin + n, BF16);
            store16(a.dh, row * a.lddh + n, v, BF16);
        }
    }
}

// The same, columns: block (x, y) sums share y of the rows for 256 columns.
template <bool BF16>
__global__ void __launch_bounds__(256) norm_columns_kernel(const __grid_constant__ NormBackwardArgs a)
{
    const int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (n >= a.N)
        return;
    const int64_t from = a.M * blockIdx.y / gridDim.y, to = a.M * (blockIdx.y + 1) / gridDim.y;
    float t = 0.0f;
    for (int64_t row = from; row < to; ++row)
        t = fmaf(load16(a.dy, row * a.lddy + n, BF16), load16(a.h, row * a.ldh + n, BF16) * a.rstd[row], t);
    a.partial[blockIdx.y * a.N + n] = t;
}

// dw from the blocks' rows: 32 columns a block, eight shares of the rows, added in order.
__global__ void __launch_bounds__(256) norm_join_kernel(const float *partial, int parts, int64_t N, void *out, int out_f32,
                                                        int is_bf16, int accumulate)
{
    __shared__ float share[8][32];
    const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
    const int64_t n = (int64_t)blockIdx.x * 32 + lane;
    float t = 0.0f;
    if (n < N) {
        const int from = parts * g / 8, to = parts * (g + 1) / 8;
#pragma unroll 8
        for (int p = from; p < to; ++p)
            t += partial[p * N + n];
    }
    share[g][lane] = t;
    __syncthreads();
    if (g > 0 || n >= N)
        return;
    t = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k)
        t += share[k][lane];
    if (out_f32) {
        float *o = reinterpret_cast<float *>(out) + n;
        *o = accumulate ? *o + t : t;
    } else {
        store16(out, n, accumulate ? load16(out, n, is_bf16) + t : t, is_bf16);
    }
}

// ---- 8-bit activations by themselves --------------------------------------------------------
// 16 lanes a block of 128 elements.
template <bool BF16>
__global__ void __launch_bounds__(256) pack_kernel(const __grid_constant__ PackArgs a)
{
    const int64_t units = (a.N + kPackBlock - 1) / kPackBlock;  // blocks of a row
    const int64_t total = a.M * units;
    const int64_t step = (int64_t)gridDim.x * 16;
    const int lane = threadIdx.x & 15;
    // a warp's two halves end together
    for (int64_t t0 = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 5) * 2; t0 < total; t0 += step) {
        const int64_t t = t0 + ((threadIdx.x >> 4) & 1);
        const int64_t row = t / units, b = t - row * units, n = b * kPackBlock + lane * kVec;
        const int64_t left = t < total ? a.N - n : 0;
        float v[8];
        floats8<BF16>(load8(reinterpret_cast<const uint16_t *>(a.x) + row * a.ldx + n, left), v);
        int e;
        const uint2 c = pack_group(v, &e);
        if (left > 0) {
            store_codes8(a.codes + row * a.ldc + n, left, c);
            if (lane == 0)
                a.scales[row * a.lds + b] = power_of_two(e);
        }
    }
}

template <bool BF16>
__global__ void __launch_bounds__(256) pack_any_kernel(const __grid_constant__ PackArgs a)
{
    const int64_t units = (a.N + kPackBlock - 1) / kPackBlock;
    const int64_t total = a.M * units;
    const int lane = threadIdx.x & 31;
    for (int64_t t = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); t < total; t += (int64_t)gridDim.x * 8) {
        const int64_t row = t / units, b = t - row * units, n0 = b * kPackBlock + lane;
        float v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
            v[u] = n0 + u * 32 < a.N ? load16(a.x, row * a.ldx + n0 + u * 32, BF16) : 0.0f;
        int e;
        const uint32_t c = pack_warp(v, &e);
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (n0 + u * 32 < a.N)
                a.codes[row * a.ldc + n0 + u * 32] = (uint8_t)(c >> (8 * u));
        if (lane == 0)
            a.scales[row * a.lds + b] = power_of_two(e);
    }
}

// V elements per thread and step, as act_backward.
template <bool BF16, int V>
__global__ void __launch_bounds__(256) unpack_kernel(const __grid_constant__ UnpackArgs a)
{
    const int64_t units = (a.N + V - 1) / V;
    const int64_t total = a.M * units;
    const int64_t step = (int64_t)gridDim.x * blockDim.x;
    for (int64_t t = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; t < total; t += step) {
        const int64_t row = t / units, n = (t - row * units) * V;
        const int64_t left = V == 8 ? a.N - n : 1;
        const float scale = a.scales[row * a.lds + n / kPackBlock];
        float v[8] = {};
        {
            const uint8_t *p = a.codes + row * a.ldc + n;
            const uint2 c = V == 8 ? load_codes8(p, left) : make_uint2(*p, 0u);
            float x[4];
            unpack4(c.x, x);
#pragma unroll
            for (int u = 0; u < 4; ++u)
                v[u] = held16<BF16>(x[u] * scale);
            unpack4(c.y, x);
#pragma unroll
            for (int u = 0; u < 4; ++u)
                v[4 + u] = held16<BF16>(x[u] * scale);
        }
        if (a.act != GG_ACT_NONE)
            with_act(a.act, [&](auto k) { apply_act<decltype(k)::value>(v); });
        uint16_t *out = reinterpret_cast<uint16_t *>(a.out) + row * a.ldo + n;
        if (V == 8)
            store8(out, left, halves8<BF16>(v));
        else
            store16(out, 0, v[0], BF16);
    }
}

// ---- host ----------------------------------------------------------------------------------
bool on16(const void *p, int64_t ld) { return ((reinterpret_cast<uint64_t>(p) | (uint64_t)(ld * 2)) & 15) == 0; }
bool on8(const void *p, int64_t ld) { return ((reinterpret_cast<uint64_t>(p) | (uint64_t)ld) & 7) == 0; }

// Warps and vectors a thread for rows of N elements.  Few rows: as many warps as there are, since
// then a row's own latency is the time; many: up to 4 vectors a thread, so that a block has several
// rows' loads in flight.
bool row_shape(int64_t M, int64_t N, int most_vpt_at_1024, RowShape *s, int *vpt)
{
    const int64_t warps = (N + 32 * kVec - 1) / (32 * kVec);  // at one vector a thread
    if (warps > 32 * most_vpt_at_1024)
        return false;
    int v = M <= kSMs ? 1 : 4;
    while (v > 1 && warps < v)
        v /= 2;
    while ((warps + v - 1) / v > (v > most_vpt_at_1024 ? 16 : 32))
        v *= 2;
    int R = 1;
    while (R * v < warps)
        R *= 2;
    *vpt = v;
    s->R = R;
    s->rows = R >= 8 ? 1 : 8 / R;
    return true;
}

int row_blocks(int64_t M, const RowShape &s, int per_sm)
{
    return (int)gg_min64((M + s.rows - 1) / s.rows, (int64_t)kSMs * per_sm);
}

template <bool BF16>
cudaError_t norm_of(const NormArgs &a, cudaStream_t s)
{
    RowShape r;
    int vpt;
    const bool wide = on16(a.x, a.ldx) && (!a.residual || on16(a.residual, a.ldr)) && (!a.h || on16(a.h, a.ldh)) &&
                      (!a.y || on16(a.y, a.ldy)) && (!a.codes || on8(a.codes, a.ldc));
    if (!wide || !row_shape(a.M, a.N, 4, &r, &vpt)) {
        norm_any_kernel<BF16><<<(int)gg_min64(a.M, kSMs * 4), 512, 0, s>>>(a);
        return cudaGetLastError();
    }
    const int threads = 32 * r.R * r.rows;
    const int grid = row_blocks(a.M, r, 2048 / threads);
    if (vpt == 1)
        norm_kernel<BF16, 1><<<grid, threads, 0, s>>>(a, r);
    else if (vpt == 2)
        norm_kernel<BF16, 2><<<grid, threads, 0, s>>>(a, r);
    else
        norm_kernel<BF16, 4><<<grid, threads, 0, s>>>(a, r);
    return cudaGetLastError();
}

template <bool BF16>
cudaError_t norm_backward_of(const NormBackwardArgs &a, cudaStream_t s)
{
    RowShape r;
    int vpt, parts = 0;
    const bool wide = on16(a.dy, a.lddy) && on16(a.h, a.ldh) && (!a.dh_in || on16(a.dh_in, a.lddhin)) &&
                      (!a.dh || on16(a.dh, a.lddh));
    if (a.M == 0) {
        // no rows: the sums are zero
    } else if (wide && row_shape(a.M, a.N, 2, &r, &vpt)) {
        const int threads = 32 * r.R * r.rows;
        const int grid = row_blocks(a.M, r, norm_backward_parts(a.M) / kSMs > 0 ? norm_backward_parts(a.M) / kSMs : 1);
        const int smem = r.rows > 1 ? (int)a.N * 4 : 0;
        parts = grid;
        if (vpt == 1)
            norm_backward_kernel<BF16, 1><<<grid, threads, smem, s>>>(a, r);
        else if (vpt == 2)
            norm_backward_kernel<BF16, 2><<<grid, threads, smem, s>>>(a, r);
        else
            norm_backward_kernel<BF16, 4><<<grid, threads, smem, s>>>(a, r);
    } else {
        if (a.partial) {  // first: dh may lie over what it reads
            parts = norm_backward_parts(a.M);
            norm_columns_kernel<BF16><<<dim3((unsigned)((a.N + 255) / 256), (unsigned)parts), 256, 0, s>>>(a);
        }
        if (a.dh)
            norm_backward_any_kernel<BF16><<<(int)gg_min64(a.M, kSMs * 4), 512, 0, s>>>(a);
    }
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess && a.dweight) {
        norm_join_kernel<<<(int)((a.N + 31) / 32), 256, 0, s>>>(a.partial, parts, a.N, a.dweight, a.grad_f32, BF16,
                                                                 a.accumulate);
        e = cudaGetLastError();
    }
    return e;
}

template <bool BF16>
cudaError_t unpack_of(const UnpackArgs &a, cudaStream_t s)
{
    const bool wide = on16(a.out, a.ldo) && on8(a.codes, a.ldc);
    const int64_t total = a.M * (wide ? (a.N + 7) / 8 : a.N);
    const int grid = (int)gg_min64((total + 255) / 256, kSMs * 8);
    if (wide)
        unpack_kernel<BF16, 8><<<grid, 256, 0, s>>>(a);
    else
        unpack_kernel<BF16, 1><<<grid, 256, 0, s>>>(a);
    return cudaGetLastError();
}

template <bool BF16>
cudaError_t pack_of(const PackArgs &a, cudaStream_t s)
{
    const int64_t blocks = a.M * ((a.N + kPackBlock - 1) / kPackBlock);
    if (on16(a.x, a.ldx) && on8(a.codes, a.ldc))
        pack_kernel<BF16><<<(int)gg_min64((blocks + 15) / 16, kSMs * 8), 256, 0, s>>>(a);
    else
        pack_any_kernel<BF16><<<(int)gg_min64((blocks + 7) / 8, kSMs * 8), 256, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

// Blocks' rows of dw's sums: two blocks an SM.
int norm_backward_parts(int64_t M) { return (int)gg_min64(M, 2 * kSMs); }

cudaError_t launch_norm(const NormArgs &a, cudaStream_t s) { return a.is_bf16 ? norm_of<true>(a, s) : norm_of<false>(a, s); }

cudaError_t launch_norm_backward(const NormBackwardArgs &a, cudaStream_t s)
{
    return a.is_bf16 ? norm_backward_of<true>(a, s) : norm_backward_of<false>(a, s);
}

cudaError_t launch_pack(const PackArgs &a, cudaStream_t s) { return a.is_bf16 ? pack_of<true>(a, s) : pack_of<false>(a, s); }

cudaError_t launch_unpack(const UnpackArgs &a, cudaStream_t s)
{
    return a.is_bf16 ? unpack_of<true>(a, s) : unpack_of<false>(a, s);
}

}  // namespace gg
