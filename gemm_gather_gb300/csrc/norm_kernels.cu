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
// warps take 8 / R rows side by side.  Forward, a block ends with its row group; backward, where dw's
// sums stay in registers, blocks walk the rows with the grid's stride.  Rows that are not
// 16-byte aligned, or longer than 32 warps hold, go through kernels that read a row twice.
//
// dw: a thread keeps the sums of its own columns over all its rows in registers; a block adds its
// rows' sums in shared memory and stores them as one row of the workspace, and a second kernel
// adds the blocks' rows.  Fixed orders throughout: the same bits on every run.
#include <cuda_runtime.h>

#include <mutex>

#include "act.cuh"
#include "gg_internal.h"
#include "gg_ops.h"
#include "launch.cuh"
#include "pack8.cuh"
#include "tc.cuh"

namespace gg {
namespace {

using tc::launch_dependents;
using tc::wait_dependencies;

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

// A sum with what its roundings left: squares of a row, whose sum decides its rstd's last bit, and with it that of
// thousands of elements of y and of their codes.  The sums that are small beside the row's are plain (a warp's where
// it is one of eight or more, else an eighth of it): their roundings hardly show.  rstd is then what an exact sum gives for
// 90 to 94 % of bfloat16 rows (plain sums: 81 to 86 %, 66 % of rows of 32 warps) and 83 to 91 % of float16's (65 to 85 %),
// whose squares' last bits are not evenly spread, so that a thread's own sum loses some; 16384 x 8192 takes 181.8 us for 180.3.
struct Exact {
    float sum, rest;
};

__device__ __forceinline__ Exact plus(Exact a, Exact b)
{
    const float s = a.sum + b.sum, other = s - a.sum;
    const float lost = (a.sum - (s - other)) + (b.sum - other);  // exactly, in either order
    return Exact{s, a.rest + b.rest + lost};
}

__device__ __forceinline__ Exact plus_lane(Exact t, int d)
{
    return plus(t, Exact{__shfl_xor_sync(0xffffffffu, t.sum, d), __shfl_xor_sync(0xffffffffu, t.rest, d)});
}

// The sum over a row's R warps of each thread's v, as row_sum's.  Where it overflows it is infinite, or NaN as one of
// its terms.
__device__ __forceinline__ float row_sum_exact(float v, const RowShape &s, float2 (&buf)[kMaxWarps])
{
#pragma unroll
    for (int d = 16; d > 2; d >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, d);
    Exact t{v, 0.0f};
    if (s.R < 8) {
        t = plus_lane(plus_lane(t, 2), 1);
    } else {
        t.sum += __shfl_xor_sync(0xffffffffu, t.sum, 2);
        t.sum += __shfl_xor_sync(0xffffffffu, t.sum, 1);
    }
    if (s.R > 1) {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        if (lane == 0)
            buf[warp] = make_float2(t.sum, t.rest);
        __syncthreads();
        // the row's warps, side by side in every group of lanes that holds them
        const int at = lane & ((2 << (31 - __clz(s.R - 1))) - 1);
        const float2 own = at < s.R ? buf[warp / s.R * s.R + at] : make_float2(0.0f, 0.0f);
        t = Exact{own.x, own.y};
#pragma unroll
        for (int d = 1; d < 32; d *= 2)
            if (d < s.R)
                t = plus_lane(t, d);
    }
    return t.sum <= 3.402823466e38f ? t.sum + t.rest : t.sum;  // (what infinities leave is NaN)
}

// Eight neighbouring 16-bit elements, or weights, as pairs of floats.
struct Eight {
    F2 v[4];
};

template <bool BF16>
__device__ __forceinline__ Eight eight_of(const uint4 &q)
{
    const uint32_t h[4] = {q.x, q.y, q.z, q.w};
    Eight r;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const float2 f = pair16<BF16>(h[u]);
        r.v[u] = pair_of(f.x, f.y);
    }
    return r;
}

template <bool BF16>
__device__ __forceinline__ uint4 halves8(const Eight &e)
{
    uint32_t w[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const float2 f = halves_of(e.v[u]);
        w[u] = pair16_of<BF16>(f.x, f.y);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// a + b, rounded once to the type.
template <bool BF16>
__device__ __forceinline__ uint32_t add16(uint32_t a, uint32_t b)
{
    if constexpr (BF16) {
        const __nv_bfloat162 v = __hadd2(*reinterpret_cast<const __nv_bfloat162 *>(&a), *reinterpret_cast<const __nv_bfloat162 *>(&b));
        return *reinterpret_cast<const uint32_t *>(&v);
    } else {
        const __half2 v = __hadd2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
        return *reinterpret_cast<const uint32_t *>(&v);
    }
}

template <bool BF16>
__device__ __forceinline__ Eight load_weights(const void *w, int f32, int vec, int n, int left)
{
    Eight r;
    if (f32) {
        const float *p = reinterpret_cast<const float *>(w) + n;
        if (left >= 8 && vec) {
            const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
            r.v[0] = pair_of(a.x, a.y), r.v[1] = pair_of(a.z, a.w);
            r.v[2] = pair_of(b.x, b.y), r.v[3] = pair_of(b.z, b.w);
            return r;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
            r.v[u] = pair_of(2 * u < left ? p[2 * u] : 0.0f, 2 * u + 1 < left ? p[2 * u + 1] : 0.0f);
        return r;
    }
    const uint16_t *p = reinterpret_cast<const uint16_t *>(w) + n;
    if (left >= 8 && vec)
        return eight_of<BF16>(*reinterpret_cast<const uint4 *>(p));
#pragma unroll
    for (int u = 0; u < 4; ++u)
        r.v[u] = pair_of(2 * u < left ? load16(p, 2 * u, BF16) : 0.0f, 2 * u + 1 < left ? load16(p, 2 * u + 1, BF16) : 0.0f);
    return r;
}

// ---- rows in flight ---------------------------------------------------------------------
// Backward, where a block walks several rows, its threads copy the next rows' vectors into slots of their own in
// shared memory (D rows deep, one commit group a row) while they work on the present one; nobody else
// reads a thread's slots, so there is nothing to wait for but its own copies.  D = 1: no
// copies ahead, vectors come straight into registers.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, int bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A thread's slots: vector k of input i of the row in slot d.
template <int VPT, int INPUTS>
struct Slots {
    uint4 *mine;
    __device__ __forceinline__ explicit Slots(uint8_t *smem) : mine(reinterpret_cast<uint4 *>(smem) + threadIdx.x) {}
    __device__ __forceinline__ uint4 *at(int d, int i, int k) const
    {
        return mine + ((d * INPUTS + i) * VPT + k) * (int)blockDim.x;
    }
    __device__ __forceinline__ void clear(int depth) const
    {
        for (int v = 0; v < depth * INPUTS * VPT; ++v)
            mine[v * (int)blockDim.x] = make_uint4(0u, 0u, 0u, 0u);
    }
    // Vector k of a row, `left` elements to the row's end.  WHOLE: rows of whole vectors; one past the end is
    // not copied (its slot holds zeros).  Else a vector's missing elements come as zeros.
    template <bool WHOLE>
    __device__ __forceinline__ void copy(int d, int i, int k, const uint16_t *row, int n, int left) const
    {
        if (WHOLE) {
            if (left > 0)
                copy16(ptx::smem_addr(at(d, i, k)), row + n, 16);
        } else {
            const int bytes = left >= 8 ? 16 : (left > 0 ? left * 2 : 0);
            copy16(ptx::smem_addr(at(d, i, k)), left > 0 ? row + n : row, bytes);
        }
    }
};

template <bool WHOLE>
__device__ __forceinline__ uint4 load_vector(const uint16_t *p, int left)
{
    if (!WHOLE)
        return load8(p, left);
    return left > 0 ? *reinterpret_cast<const uint4 *>(p) : make_uint4(0u, 0u, 0u, 0u);
}

template <bool WHOLE>
__device__ __forceinline__ void store_vector(uint16_t *p, int left, const uint4 &v)
{
    if (!WHOLE)
        store8(p, left, v);
    else if (left > 0)
        *reinterpret_cast<uint4 *>(p) = v;
}

// ---- forward ------------------------------------------------------------------------------
// A block a row group: with a new block's loads starting wherever one has ended, reads and writes mix
// evenly, which HBM rewards: 16384 x 8192 (residual, codes) takes 182 us, at 98 % of the copy rate; blocks that walk
// rows with the next one's loads in flight 215, and 203 without.
template <bool BF16, int VPT, bool RES, bool WHOLE>
__global__ void __launch_bounds__(1024) norm_kernel(const __grid_constant__ NormArgs a, const RowShape s)
{
    __shared__ float2 sums[kMaxWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int sub = warp % s.R, N = (int)a.N;
    const int64_t row = (int64_t)blockIdx.x * s.rows + warp / s.R;
    const bool live = row < a.M;
    const auto column = [&](int k) { return ((k * s.R + sub) * 32 + lane) * kVec; };
    uint4 h[VPT];
    F2 sq = pair_of(0.0f);
    Eight w;
    wait_dependencies();
    if (live) {
        const uint16_t *x = reinterpret_cast<const uint16_t *>(a.x) + row * a.ldx;
        const uint16_t *r = RES ? reinterpret_cast<const uint16_t *>(a.residual) + row * a.ldr : nullptr;
        uint4 q[VPT];
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int n = column(k);
            h[k] = load_vector<WHOLE>(x + n, N - n);
            if (RES)
                q[k] = load_vector<WHOLE>(r + n, N - n);
        }
        if (VPT == 1)  // few rows: the weights' latency beside the row's
            w = load_weights<BF16>(a.weight, a.weight_f32, a.weight_vec, column(0), N - column(0));
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            if (RES)
                h[k] = make_uint4(add16<BF16>(h[k].x, q[k].x), add16<BF16>(h[k].y, q[k].y),
                                  add16<BF16>(h[k].z, q[k].z), add16<BF16>(h[k].w, q[k].w));
            const Eight v = eight_of<BF16>(h[k]);
#pragma unroll
            for (int u = 0; u < 4; ++u)
                sq = fma2(v.v[u], v.v[u], sq);
        }
        if (a.h) {
            uint16_t *out = reinterpret_cast<uint16_t *>(a.h) + row * a.ldh;
#pragma unroll
            for (int k = 0; k < VPT; ++k)
                store_vector<WHOLE>(out + column(k), N - column(k), h[k]);
        }
    }
    const float2 both = halves_of(sq);
    const float total = row_sum_exact(both.x + both.y, s, sums);
    launch_dependents();  // (earlier, the next launch's blocks take places from this one's)
    if (!live)
        return;
    const float rstd = 1.0f / sqrtf(total / (float)N + a.eps);
    if (a.rstd && sub == 0 && lane == 0)
        a.rstd[row] = rstd;
    uint16_t *out = reinterpret_cast<uint16_t *>(a.y) + row * a.ldy;
    uint8_t *codes = a.codes + row * a.ldc;
    float *scales = a.scales + row * a.lds;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const int n = column(k), left = N - n;
        Eight v = eight_of<BF16>(h[k]);
        if (VPT > 1)
            w = load_weights<BF16>(a.weight, a.weight_f32, a.weight_vec, n, left);
#pragma unroll
        for (int u = 0; u < 4; ++u)
            v.v[u] = mul2(mul2(v.v[u], pair_of(rstd)), w.v[u]);
        const uint4 y = halves8<BF16>(v);
        if (a.y)
            store_vector<WHOLE>(out + n, left, y);
        if (a.codes) {
            int e;
            const uint2 c = pack_group<BF16>(y, &e);
            if (left > 0) {
                if (WHOLE)
                    *reinterpret_cast<uint2 *>(codes + n) = c;
                else
                    store_codes8(codes + n, left, c);
                if ((lane & 15) == 0)
                    scales[n / kPackBlock] = power_of_two(e);
            }
        }
    }
}

// Any alignment and length: a block a row, a warp a block of 128 elements, the row read twice
// (h again where it was stored: x or the residual may be what it was stored over).
template <bool BF16>
__global__ void __launch_bounds__(512) norm_any_kernel(const __grid_constant__ NormArgs a)
{
    __shared__ float2 sums[2][kMaxWarps];  // in turn, so that one barrier a row is enough
    const RowShape s{(int)blockDim.x / 32, 1};
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int turn = 0;
    wait_dependencies();
    launch_dependents();
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
        const float rstd = 1.0f / sqrtf(row_sum_exact(sq, s, sums[turn]) / (float)a.N + a.eps);
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
template <bool BF16, int VPT, int D, bool IN, bool WHOLE>
__global__ void __launch_bounds__(D > 1 ? 256 : (VPT > 2 ? 512 : 1024), D > 1 ? 2 : 1)
    norm_backward_kernel(const __grid_constant__ NormBackwardArgs a, const RowShape s)
{
    __shared__ float sums[2][kMaxWarps];
    // the rows in flight; at the end, where a block has several rows at a time, their sums
    extern __shared__ __align__(16) uint8_t ring[];
    constexpr int kInputs = IN ? 3 : 2;
    const Slots<VPT, kInputs> slots(ring);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int sub = warp % s.R, N = (int)a.N;
    const int64_t step = (int64_t)gridDim.x * s.rows;
    const uint16_t *dy = reinterpret_cast<const uint16_t *>(a.dy), *h = reinterpret_cast<const uint16_t *>(a.h),
                   *in = reinterpret_cast<const uint16_t *>(a.dh_in);
    const auto column = [&](int k) { return ((k * s.R + sub) * 32 + lane) * kVec; };
    Eight dw[VPT];
#pragma unroll
    for (int k = 0; k < VPT; ++k)
#pragma unroll
        for (int u = 0; u < 4; ++u)
            dw[k].v[u] = pair_of(0.0f);
    int64_t row = (int64_t)blockIdx.x * s.rows + warp / s.R;
    const auto ahead = [&](int64_t at, int d) {
        if (at < a.M) {
            const uint16_t *yr = dy + at * a.lddy, *hr = h + at * a.ldh, *ir = IN ? in + at * a.lddhin : nullptr;
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int n = column(k);
                slots.template copy<WHOLE>(d, 0, k, yr, n, N - n);
                slots.template copy<WHOLE>(d, 1, k, hr, n, N - n);
                if (IN)
                    slots.template copy<WHOLE>(d, kInputs - 1, k, ir, n, N - n);
            }
        }
        copies_commit();
    };
    wait_dependencies();
    launch_dependents();
    Eight w[VPT];
#pragma unroll
    for (int k = 0; k < VPT; ++k)
        w[k] = load_weights<BF16>(a.weight, a.weight_f32, a.weight_vec, column(k), N - column(k));
    if constexpr (D > 1) {
        if (WHOLE)
            slots.clear(D);
#pragma unroll
        for (int d = 0; d < D - 1; ++d)
            ahead(row + d * step, d);
    }
    int turn = 0, slot = 0;
    for (int64_t row0 = (int64_t)blockIdx.x * s.rows; row0 < a.M; row0 += step, row += step, turn ^= 1) {
        const bool live = row < a.M;
        uint4 qy[VPT], qh[VPT], qi[VPT];
        float dot = 0.0f, rstd = 0.0f;
        if (live)
            rstd = a.rstd[row];
        if constexpr (D > 1) {
            ahead(row + (D - 1) * step, slot == 0 ? D - 1 : slot - 1);
            copies_wait<D - 1>();
        }
        if (live) {
            if constexpr (D == 1) {
                const uint16_t *yr = dy + row * a.lddy, *hr = h + row * a.ldh, *ir = IN ? in + row * a.lddhin : nullptr;
#pragma unroll
                for (int k = 0; k < VPT; ++k) {
                    const int n = column(k);
                    qy[k] = load8(yr + n, N - n);
                    qh[k] = load8(hr + n, N - n);
                    if (IN)
                        qi[k] = load8(ir + n, N - n);
                }
            }
            F2 part = pair_of(0.0f);
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const Eight y = eight_of<BF16>(D > 1 ? *slots.at(slot, 0, k) : qy[k]);
                const Eight v = eight_of<BF16>(D > 1 ? *slots.at(slot, 1, k) : qh[k]);
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const F2 t = mul2(v.v[u], pair_of(rstd));
                    part = fma2(mul2(y.v[u], w[k].v[u]), t, part);
                    dw[k].v[u] = fma2(y.v[u], t, dw[k].v[u]);
                }
            }
            const float2 both = halves_of(part);
            dot = both.x + both.y;
        }
        // dh = rstd (g - u c) + dh_in: g rstd, and u by -rstd c
        const float c = row_sum(dot, s, sums, turn) / (float)N;
        if (live && a.dh) {
            uint16_t *out = reinterpret_cast<uint16_t *>(a.dh) + row * a.lddh;
            const F2 r2 = pair_of(rstd), less = pair_of(-rstd * c);
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int n = column(k);
                const Eight y = eight_of<BF16>(D > 1 ? *slots.at(slot, 0, k) : qy[k]);
                Eight v = eight_of<BF16>(D > 1 ? *slots.at(slot, 1, k) : qh[k]);
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    v.v[u] = fma2(mul2(y.v[u], w[k].v[u]), r2, mul2(mul2(v.v[u], r2), less));
                if (IN) {
                    const Eight t = eight_of<BF16>(D > 1 ? *slots.at(slot, kInputs - 1, k) : qi[k]);
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        v.v[u] = add2(v.v[u], t.v[u]);
                }
                store_vector<WHOLE>(out + n, N - n, halves8<BF16>(v));
            }
        }
        if constexpr (D > 1)
            slot = slot + 1 == D ? 0 : slot + 1;
    }
    if (!a.partial)
        return;
    float *out = a.partial + (int64_t)blockIdx.x * a.N;
    float *columns = reinterpret_cast<float *>(ring);
    if (D > 1 && s.rows > 1) {
        copies_wait<0>();
        __syncthreads();  // the slots become the columns' sums
    }
    for (int g = 0; g < s.rows; ++g) {  // row group by row group, in order
        if (warp / s.R == g) {
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int n = column(k);
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    if (n + u < N) {
                        const float2 mine = halves_of(dw[k].v[u / 2]);
                        float t = u & 1 ? mine.y : mine.x;
                        if (g > 0)
                            t += columns[n + u];
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

// dw from the blocks' rows: 32 columns a block, 32 shares of the rows, added in order.  It begins while the
// launch before it ends, and waits for that.
__global__ void __launch_bounds__(1024) norm_join_kernel(const float *partial, int parts, int64_t N, void *out, int out_f32,
                                                         int is_bf16, int accumulate)
{
    __shared__ float share[32][33];
    const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
    const int64_t n = (int64_t)blockIdx.x * 32 + lane;
    wait_dependencies();
    launch_dependents();
    float t = 0.0f;
    if (n < N) {
        const int from = parts * g / 32, to = parts * (g + 1) / 32;
#pragma unroll 10
        for (int p = from; p < to; ++p)
            t += partial[p * N + n];
    }
    share[g][lane] = t;
    __syncthreads();
    if (g > 0 || n >= N)
        return;
    t = 0.0f;
#pragma unroll
    for (int k = 0; k < 32; ++k)
        t += share[k][lane];
    if (out_f32) {
        float *o = reinterpret_cast<float *>(out) + n;
        *o = accumulate ? *o + t : t;
    } else {
        store16(out, n, accumulate ? load16(out, n, is_bf16) + t : t, is_bf16);
    }
}

// ---- 8-bit activations by themselves --------------------------------------------------------
// Eight lanes a block of 128 elements, two vectors each; kAhead blocks' loads in flight.  A lane's place
// (row, block of the row) is stepped, not divided for: one division of a place costs as much as a
// quarter of the block's arithmetic.
constexpr int kAhead = 2;
template <bool BF16>
__global__ void __launch_bounds__(256) pack_kernel(const __grid_constant__ PackArgs a)
{
    const int units = (int)((a.N + kPackBlock - 1) / kPackBlock);  // blocks of a row
    const int lane = threadIdx.x & 7;
    const int64_t total = a.M * units, step = (int64_t)gridDim.x * 32;
    const int64_t first = (int64_t)blockIdx.x * 32 + (threadIdx.x >> 3);
    const int64_t step_rows = step / units;
    const int step_units = (int)(step - step_rows * units);
    int64_t row = first / units;
    int unit = (int)(first - row * units);
    wait_dependencies();
    launch_dependents();
    // a warp's four groups end together
    for (int64_t t0 = (int64_t)blockIdx.x * 32 + (threadIdx.x >> 5) * 4; t0 < total; t0 += step * kAhead) {
        uint4 q[kAhead][2];
        int64_t at[kAhead];
        int b[kAhead], left[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            at[k] = row;
            b[k] = unit;
            const int64_t n = (int64_t)unit * kPackBlock + lane * kVec;
            const int64_t l = row < a.M ? a.N - n : 0;
            left[k] = l > 127 ? 127 : (int)l;
            const uint16_t *p = reinterpret_cast<const uint16_t *>(a.x) + row * a.ldx + n;
            q[k][0] = load8(p, left[k]);
            q[k][1] = load8(p + 64, left[k] - 64);
            row += step_rows;
            unit += step_units;
            if (unit >= units) {
                unit -= units;
                ++row;
            }
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            int e;
            uint2 c[2];
            pack_block<BF16>(q[k], &e, c);
            if (left[k] > 0) {
                uint8_t *p = a.codes + at[k] * a.ldc + b[k] * kPackBlock + lane * kVec;
                store_codes8(p, left[k], c[0]);
                if (left[k] > 64)
                    store_codes8(p + 64, left[k] - 64, c[1]);
                if (lane == 0)
                    a.scales[at[k] * a.lds + b[k]] = power_of_two(e);
            }
        }
    }
}

template <bool BF16>
__global__ void __launch_bounds__(256) pack_any_kernel(const __grid_constant__ PackArgs a)
{
    const int64_t units = (a.N + kPackBlock - 1) / kPackBlock;
    const int64_t total = a.M * units;
    const int lane = threadIdx.x & 31;
    wait_dependencies();
    launch_dependents();
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

// V elements per thread and step (8 where rows of out are 16-byte and rows of codes 8-byte aligned), kSteps
// steps' loads in flight.  I: 32-bit indices where all vectors have one.
constexpr int kSteps = 4;
template <bool BF16, int V, typename I>
__global__ void __launch_bounds__(256) unpack_kernel(const __grid_constant__ UnpackArgs a)
{
    const I units = (I)((a.N + V - 1) / V);
    const I total = (I)a.M * units;
    wait_dependencies();
    launch_dependents();
    for (I t0 = (I)blockIdx.x * (256 * kSteps) + threadIdx.x; t0 < total; t0 += (I)gridDim.x * (256 * kSteps)) {
        uint2 c[kSteps];
        float scale[kSteps];
        uint16_t *out[kSteps];
        int left[kSteps];
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
            const I t = t0 + 256 * k;
            const I row = t / units;
            const int64_t n = (int64_t)(t - row * units) * V;
            left[k] = 0;
            if (t < total) {
                left[k] = V == 8 ? (a.N - n >= 8 ? 8 : (int)(a.N - n)) : 1;
                const uint8_t *p = a.codes + row * a.ldc + n;
                c[k] = V == 8 ? load_codes8(p, left[k]) : make_uint2(*p, 0u);
                scale[k] = a.scales[row * a.lds + n / kPackBlock];
                out[k] = reinterpret_cast<uint16_t *>(a.out) + row * a.ldo + n;
            }
        }
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
            if (left[k] == 0)
                break;
            float v[8];
            values8<BF16>(c[k], scale[k], v);
            if (a.act != GG_ACT_NONE)
                with_act(a.act, [&](auto f) { apply_act<decltype(f)::value>(v); });
            uint32_t w[4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
                w[u] = pair16_of<BF16>(v[2 * u], v[2 * u + 1]);
            if (V == 8)
                store8(out[k], left[k], make_uint4(w[0], w[1], w[2], w[3]));
            else
                *out[k] = (uint16_t)w[0];
            if (a.rest) {
                uint16_t *rest = reinterpret_cast<uint16_t *>(a.rest) + (out[k] - reinterpret_cast<uint16_t *>(a.out));
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const float2 f = pair16<BF16>(w[u]);
                    w[u] = pair16_of<BF16>(v[2 * u] - f.x, v[2 * u + 1] - f.y);
                }
                if (V == 8)
                    store8(rest, left[k], make_uint4(w[0], w[1], w[2], w[3]));
                else
                    *rest = (uint16_t)w[0];
            }
        }
    }
}

// ---- host ----------------------------------------------------------------------------------
bool on16(const void *p, int64_t ld) { return ((reinterpret_cast<uint64_t>(p) | (uint64_t)(ld * 2)) & 15) == 0; }
bool on8(const void *p, int64_t ld) { return ((reinterpret_cast<uint64_t>(p) | (uint64_t)ld) & 7) == 0; }

// Warps and vectors a thread for rows of N elements.  While the rows' vectors, one a thread, fit the GPU's
// threads about once, a row's own latency is the time, so it gets as many warps as it has vectors for;
// else up to 4 vectors a thread, so that more rows are in flight: 777 x 1523 takes 5 us with one and 8 with
// four, 16384 x 8192 (forward) 315 us with one, 209 to 225 with two and 180 with four.  `most`: vectors a thread that 1024 threads hold.
bool row_shape(int64_t M, int64_t N, int most, RowShape *s, int *vpt)
{
    const int64_t warps = (N + 32 * kVec - 1) / (32 * kVec);  // at one vector a thread
    if (warps > 32 * most)
        return false;
    int v = M * warps <= kSMs * 32 ? 1 : 4;
    while (v > 1 && warps < v)
        v /= 2;
    while ((warps + v - 1) / v > (v > most ? 16 : 32))
        v *= 2;
    s->R = (int)((warps + v - 1) / v);
    s->rows = s->R >= 8 ? 1 : 8 / s->R;
    // (the backward pass leaves a block's sums behind: fewer blocks, each with its rows side by side)
    while (most == 2 && v == 1 && s->R * s->rows <= 8 && M > (int64_t)kSMs * 2 * s->rows)
        s->rows *= 2;
    *vpt = v;
    return true;
}

// Blocks of a launch and how deep their rows' copies go: two blocks of up to 256 threads and 110 KB an SM,
// where that makes every block walk a few rows; else a block a row group.
struct RowPlan {
    int grid, threads, depth, smem;
};

template <int INPUTS>
constexpr int kDepth = INPUTS == 3 ? 2 : 3;  // 256 threads, 4 vectors: 96 KB

template <int INPUTS>
RowPlan row_plan(int64_t M, const RowShape &s, int vpt, int most_blocks)
{
    RowPlan p{};
    p.threads = 32 * s.R * s.rows;
    const int64_t groups = (M + s.rows - 1) / s.rows;
    const int slot = p.threads * vpt * INPUTS * 16;
    if (vpt == 4 && p.threads <= 256 && groups >= 4 * kSMs) {
        p.depth = kDepth<INPUTS>;
        p.smem = p.depth * slot;
        p.grid = 2 * kSMs;
    } else {
        p.depth = 1;
        p.grid = (int)gg_min64(gg_min64(groups, most_blocks), (int64_t)kSMs * (2048 / p.threads));
    }
    return p;
}

// Dynamic shared memory of a kernel, set once per device.
constexpr int kMaxDevices = 64;
template <typename K>
cudaError_t allow_smem(K kernel, std::once_flag *once, cudaError_t *result)
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices)
        dev = 0;
    std::call_once(once[dev], [&] {
        result[dev] = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 222 * 1024);
    });
    return result[dev];
}

template <bool BF16, bool RES, bool WHOLE>
cudaError_t norm_rows(const NormArgs &a, const RowShape &r, int vpt, cudaStream_t s)
{
    const unsigned grid = (unsigned)((a.M + r.rows - 1) / r.rows);
    const int threads = 32 * r.R * r.rows;
    return launch_early(vpt == 1 ? norm_kernel<BF16, 1, RES, WHOLE>
                                 : (vpt == 2 ? norm_kernel<BF16, 2, RES, WHOLE> : norm_kernel<BF16, 4, RES, WHOLE>),
                        dim3(grid), threads, 0, s, a, r);
}

template <bool BF16>
cudaError_t norm_of(const NormArgs &a, cudaStream_t s)
{
    RowShape r;
    int vpt;
    const bool wide = on16(a.x, a.ldx) && (!a.residual || on16(a.residual, a.ldr)) && (!a.h || on16(a.h, a.ldh)) &&
                      (!a.y || on16(a.y, a.ldy)) && (!a.codes || on8(a.codes, a.ldc));
    if (!wide || !row_shape(a.M, a.N, 4, &r, &vpt))
        return launch_early(norm_any_kernel<BF16>, dim3((unsigned)gg_min64(a.M, kSMs * 4)), 512, 0, s, a);
    if (a.N % kVec == 0)
        return a.residual ? norm_rows<BF16, true, true>(a, r, vpt, s) : norm_rows<BF16, false, true>(a, r, vpt, s);
    return a.residual ? norm_rows<BF16, true, false>(a, r, vpt, s) : norm_rows<BF16, false, false>(a, r, vpt, s);
}

template <bool BF16, int VPT, int D, bool IN, bool WHOLE = false>
cudaError_t launch_backward_kernel(const NormBackwardArgs &a, const RowShape &r, const RowPlan &p, cudaStream_t s)
{
    if constexpr (D > 1) {
        static std::once_flag once[kMaxDevices];
        static cudaError_t result[kMaxDevices];
        const cudaError_t e = allow_smem(norm_backward_kernel<BF16, VPT, D, IN, WHOLE>, once, result);
        if (e != cudaSuccess)
            return e;
    }
    const int columns = r.rows > 1 ? (int)a.N * 4 : 0;
    return launch_early(norm_backward_kernel<BF16, VPT, D, IN, WHOLE>, dim3((unsigned)p.grid), p.threads,
                        p.smem > columns ? p.smem : columns, s, a, r);
}

template <bool BF16, bool IN>
cudaError_t norm_backward_rows(const NormBackwardArgs &a, const RowShape &r, int vpt, int *parts, cudaStream_t s)
{
    const RowPlan p = row_plan<IN ? 3 : 2>(a.M, r, vpt, norm_backward_parts(a.M));
    *parts = p.grid;
    if (p.depth > 1)
        return a.N % kVec == 0 ? launch_backward_kernel<BF16, 4, kDepth<IN ? 3 : 2>, IN, true>(a, r, p, s)
                               : launch_backward_kernel<BF16, 4, kDepth<IN ? 3 : 2>, IN>(a, r, p, s);
    return vpt == 1 ? launch_backward_kernel<BF16, 1, 1, IN>(a, r, p, s)
                    : (vpt == 2 ? launch_backward_kernel<BF16, 2, 1, IN>(a, r, p, s)
                                : launch_backward_kernel<BF16, 4, 1, IN>(a, r, p, s));
}

template <bool BF16>
cudaError_t norm_backward_of(const NormBackwardArgs &a, cudaStream_t s)
{
    RowShape r;
    int vpt, parts = 0;
    cudaError_t e = cudaSuccess;
    const bool wide = on16(a.dy, a.lddy) && on16(a.h, a.ldh) && (!a.dh_in || on16(a.dh_in, a.lddhin)) &&
                      (!a.dh || on16(a.dh, a.lddh));
    if (a.M == 0) {
        // no rows: the sums are zero
    } else if (wide && row_shape(a.M, a.N, 2, &r, &vpt)) {
        e = a.dh_in ? norm_backward_rows<BF16, true>(a, r, vpt, &parts, s)
                    : norm_backward_rows<BF16, false>(a, r, vpt, &parts, s);
    } else {
        if (a.partial) {  // first: dh may lie over what it reads
            parts = norm_backward_parts(a.M);
            norm_columns_kernel<BF16><<<dim3((unsigned)((a.N + 255) / 256), (unsigned)parts), 256, 0, s>>>(a);
        }
        if (a.dh)
            norm_backward_any_kernel<BF16><<<(int)gg_min64(a.M, kSMs * 4), 512, 0, s>>>(a);
        e = cudaGetLastError();
    }
    if (e == cudaSuccess && a.dweight) {
        e = launch_early(norm_join_kernel, dim3((unsigned)((a.N + 31) / 32)), 1024, 0, s, (const float *)a.partial, parts,
                         a.N, a.dweight, a.grad_f32, (int)BF16, a.accumulate);
    }
    return e;
}

template <bool BF16>
cudaError_t unpack_of(const UnpackArgs &a, cudaStream_t s)
{
    const bool wide = on16(a.out, a.ldo) && on8(a.codes, a.ldc);
    const int64_t total = a.M * (wide ? (a.N + 7) / 8 : a.N);
    const int grid = (int)gg_min64((total + 256 * kSteps - 1) / (256 * kSteps), 1 << 17);
    const bool small = total < 1ll << 30;  // the last step does not overflow
    return launch_early(wide ? (small ? unpack_kernel<BF16, 8, int> : unpack_kernel<BF16, 8, int64_t>)
                             : unpack_kernel<BF16, 1, int64_t>,
                        dim3((unsigned)grid), 256, 0, s, a);
}

template <bool BF16>
cudaError_t pack_of(const PackArgs &a, cudaStream_t s)
{
    const int64_t blocks = a.M * ((a.N + kPackBlock - 1) / kPackBlock);
    if (on16(a.x, a.ldx) && on8(a.codes, a.ldc))
        return launch_early(pack_kernel<BF16>, dim3((unsigned)gg_min64((blocks + 31) / 32, kSMs * 8)), 256, 0, s, a);
    return launch_early(pack_any_kernel<BF16>, dim3((unsigned)gg_min64((blocks + 7) / 8, kSMs * 8)), 256, 0, s, a);
}

}  // namespace

// Rows of dw's sums that blocks leave, at most: four blocks an SM.
int norm_backward_parts(int64_t M) { return (int)gg_min64(M, 4 * kSMs); }

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
