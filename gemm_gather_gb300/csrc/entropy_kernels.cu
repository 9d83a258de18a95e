// Softmax cross entropy of a vocabulary's logits z = X W that are never stored, and its gradients, for
// sm_103a: what stands around the products (linear_kernels.cu).
//
//     lse = log sum exp z,  loss = lse - z[target],  stats = sums of weight loss and of weight
//     dZ = weight (softmax(z) - onehot(target)),  dX = dZ W^T,  dW = X^T dZ
//
// 1. tokens_kernel counts the tokens whose weight is not 0 and gathers their rows of X: a masked token
//    costs no multiplication, and what its row holds (NaN, say) meets nothing.
// 2. The product z = X W over the whole vocabulary, in 32-bit sums that stay on chip: its epilogue keeps
//    of every 128 entries (CTA pairs) or 32 (the split kernel, few tokens) the largest logit and the sum of
//    exponentials, 8 bytes.
// 3. join_kernel makes lse and loss of them, and for the gradient a token's largest logit, its weight over the sum
//    and the target's term.  The rounding of lse would be all that is left of a confident token's p - 1 (2e-6 of the
//    weight at lse = 20), and so would a logit's own that is summed differently in step 4 (one chunk: 2e-6 of it at
//    K = 3584).
// 4. For a piece of the vocabulary at a time, the last one first: the product again (but for the last piece where
//    CTA pairs computed step 2 and K >= 512: its exponentials were kept in the workspace, and kept_kernel finishes
//    them; a long contraction is one chunk here, dZ's 16 bits being far coarser), its epilogue turning the logits into
//    dZ in 16 bits; then dX += dZ W^T (float32, in memory) and the piece's dW = X^T dZ in one launch.
// 5. dx_kernel rounds dX once, in the tokens' own order, zeros for the masked ones.
//
// Logits are multiplied twice (8 T V K operations instead of 6) so that they need not be kept, nor rounded
// to 16 bits before the softmax.  dZ is the only 16-bit step: weights enter it relative to the largest, which
// counts 2^13, and dX and dW are taken back in float32.  That keeps probabilities down to 2^-27 at float16's
// full precision however large or small all weights are (of a token r times the largest: 2^-27 / r, and below
// 2^-38 / r nothing is left; a factor a token would help dX but not dW, whose terms have to have one scale); and
// where all weights are equal, as most often, the targets' terms,
// -8192 (1 - p), lose next to nothing (a weight of 1 / 10 would be off by 2^-10 in all of them alike).
//
// Bound: the tensor cores, under the power limit.
#include <cuda_runtime.h>

#include "act.cuh"
#include "gg_internal.h"
#include "gg_ops.h"
#include "launch.cuh"
#include "pack8.cuh"
#include "tc.cuh"

namespace gg {
namespace {

using namespace tc;

constexpr int kSMs = 152;
constexpr int kThreads = 1024;
constexpr int kEach = 16;                      // tokens of a thread at a time
constexpr int kChunkTokens = kThreads * kEach;
constexpr int kMaxRows = 128;                  // rows a block copies for one such chunk
constexpr int kPad = 64;                       // a k-block of the products

// What the blocks of a launch share out: at most kChunkTokens / kBlocks + 1 rows each.
constexpr int kBlocks = kSMs;  // 1024 threads of 64 registers: one an SM
static_assert(kChunkTokens / kBlocks + 2 <= kMaxRows, "a block's list of rows");

// Piece m of a row of K elements, kPiece of them: four vectors a lane.
constexpr int kPiece = 1024;
__device__ __forceinline__ void copy_piece(uint16_t *to, const uint16_t *from, int64_t K, int m, int lane)
{
    const int64_t n0 = (int64_t)m * kPiece + lane * 8;
    uint4 q[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
        q[u] = load8(from + n0 + u * 256, K - n0 - u * 256);
#pragma unroll
    for (int u = 0; u < 4; ++u)
        store8(to + n0 + u * 256, K - n0 - u * 256, q[u]);
}

// Every block counts all the tokens (so that none waits for another) and copies its share of rows.
__global__ void __launch_bounds__(kThreads) tokens_kernel(const __grid_constant__ EntropyArgs a)
{
    __shared__ int counts[kEach * 32], offsets[kEach * 32], sums[kEach];
    __shared__ int list_token[kMaxRows], list_place[kMaxRows], listed;
    __shared__ float tops[32];
    wait_dependencies();
    launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t blocks = gridDim.x, me = blockIdx.x;
    const int T = (int)a.T;
    int base = 0;
    float top = 0.0f;
    for (int64_t c0 = 0; c0 < T; c0 += kChunkTokens) {
        const int steps = T - c0 >= kChunkTokens ? kEach : (int)((T - c0 + kThreads - 1) / kThreads);
        const int64_t t0 = c0 + threadIdx.x;
        float w[kEach];
        int64_t tg[kEach];
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const bool in = t0 + k * kThreads < T;
            w[k] = in ? a.weight[t0 + k * kThreads] : 0.0f;
            tg[k] = in ? a.target[t0 + k * kThreads] : 0;
        }
        unsigned live[kEach];
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            if (k >= steps)
                break;
            bool counts_in = w[k] != 0.0f;
            if (counts_in && (tg[k] < 0 || tg[k] >= a.V)) {
                counts_in = false;
                if (me == 0)
                    report_status(a.status, GG_ERR_INVALID_ARG);
            }
            live[k] = __ballot_sync(0xffffffffu, counts_in);
            if (counts_in)
                top = pack_top(top, w[k]);
            if (lane == 0)
                counts[k * 32 + warp] = __popc(live[k]);
        }
        if (threadIdx.x == 0)
            listed = 0;
        __syncthreads();
        if (warp < steps) {  // warp k: the 32 warps of step k
            const int own = counts[warp * 32 + lane];
            int sum = own;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int other = __shfl_up_sync(0xffffffffu, sum, d);
                sum += lane >= d ? other : 0;
            }
            offsets[warp * 32 + lane] = sum - own;
            if (lane == 31)
                sums[warp] = sum;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            if (k >= steps)
                break;
            const uint32_t t = (uint32_t)c0 + k * kThreads + threadIdx.x;  // (passes 2^31 behind the last token)
            const bool on = live[k] >> lane & 1;
            const int p = base + offsets[k * 32 + warp] + __popc(live[k] & ((1u << lane) - 1u));
            base += sums[k];
            if (on && (uint32_t)p % blocks == me) {
                const int at = atomicAdd(&listed, 1);
                list_token[at] = (int)t;
                list_place[at] = p;
            }
            // the small per-token arrays: a warp's 32 tokens by one block
            if (t / 32 % blocks == me && t < (uint32_t)T) {
                a.place[t] = on ? p : -1;
                if (on) {
                    a.token[p] = (int)t;
                    a.tgt[p] = (int)tg[k];
                    a.wt[p] = w[k];
                } else {
                    a.loss[t] = 0.0f;
                    if (a.lse)
                        a.lse[t] = 0.0f;
                }
            }
        }
        __syncthreads();
        const int pieces = (int)((a.K + kPiece - 1) / kPiece);
        for (int it = warp; it < listed * pieces; it += 32) {
            const int r = it / pieces;
            copy_piece(reinterpret_cast<uint16_t *>(a.x) + (int64_t)list_place[r] * a.ldw,
                       reinterpret_cast<const uint16_t *>(a.X) + (int64_t)list_token[r] * a.ldx, a.K, it - r * pieces,
                       lane);
        }
        __syncthreads();  // the lists and counts are written again
    }
    const int n = base;
    const int64_t pad = gg_min64(a.T, ((int64_t)base + kPad - 1) / kPad * kPad);
    for (int64_t p = (int64_t)base + warp; p < pad; p += 32)
        if ((uint32_t)p % blocks == me) {
            uint16_t *row = reinterpret_cast<uint16_t *>(a.x) + p * a.ldw;
            for (int64_t c = lane; c < a.K; c += 32)
                row[c] = 0;
            if (lane == 0) {
                a.tgt[p] = -1;
                a.wt[p] = 0.0f;
            }
        }
    if (me != 0)
        return;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    if (lane == 0)
        tops[warp] = top;
    __syncthreads();
    if (warp > 0)
        return;
    top = tops[lane];
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    if (lane == 0) {
        top = top > 0x1p-100f ? top : (top > 0.0f ? 0x1p-100f : 1.0f);
        a.head->live = n;
        a.head->live_pad = (int)pad;
        // A tile of dX is to be at most a quarter of what a CTA pair has to do, but 16 k-blocks; dW's tiles are nine
        // k-blocks' time at least (their epilogue).  Microseconds of calls with gradients, tokens (that count) x V x K:
        //                      777 (544) x 32768 x 2011   2796 (280) x 63131 x 1309   300 x 2000 x 1000   60 x 4000 x 512
        //   as here                      258                        321                     40.1                33.0
        //   half, eighth              267, 259                   298, 320                40.1, 42.5          33.0, 33.0
        //   8, 32 k-blocks            258, 258                   321, 321                43.3, 44.4          35.9, 39.0
        //   one, 18 for dW            258, 254                   321, 321                40.1, 41.9          33.0, 33.0
        // at eight other sizes, of 16 to 4096 tokens and V of 8192 to 100003, within 4 % of one another (32 k-blocks 6 %).
        const int64_t dx = (int64_t)a.dx_tiles_i * ((n + a.dx_bt - 1) / a.dx_bt) * a.dx_kb;
        const int64_t all = dx + a.dw_tiles * ((n + kPad - 1) / kPad > 9 ? (n + kPad - 1) / kPad : 9);
        const int64_t want = gg_min64(a.dx_kb / 16, all > 0 ? (2 * kSMs * (int64_t)a.dx_kb + all - 1) / all : 1);
        a.head->shares = (int)(want < 1 ? 1 : gg_min64(want, a.most_shares));
        a.head->ticket = 0;
        a.head->scale = 8192.0f / top;
        a.head->alpha = a.grad_scale * (top * 0x1p-13f);
    }
}

__device__ __forceinline__ double warp_total(double v)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

// 32 tokens a block, 32 shares of the rows; the rows twice (the second time from L2), so that no
// exponential waits for another.  A sum of NaN stays NaN; rows of nothing but -inf have sum 0.
__global__ void __launch_bounds__(kThreads) join_kernel(const __grid_constant__ EntropyArgs a)
{
    __shared__ float part[32][33];
    __shared__ unsigned turn;
    wait_dependencies();
    launch_dependents();
    const int g = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int live = a.head->live, pad = a.head->live_pad;
    const int64_t p = (int64_t)blockIdx.x * 32 + lane;
    const float2 *rows = a.partial + p;
    const int64_t n = p < live ? a.rows : 0;
    float weight = 0.0f, target = 0.0f;
    int token = 0;
    if (g == 0 && p < pad) {
        weight = a.wt[p];
        if (p < live) {
            target = a.ztarget[p];
            token = a.token[p];
        }
    }
    constexpr int kHeld = 8;  // rows of a thread that stay in registers
    float2 held[kHeld];
    float m = -INFINITY;
#pragma unroll
    for (int k = 0; k < kHeld; ++k) {
        const int64_t r = g + 32 * k;
        held[k] = r < n ? rows[r * a.T] : make_float2(-INFINITY, 0.0f);
    }
#pragma unroll
    for (int k = 0; k < kHeld; ++k)
        m = fmaxf(m, held[k].x);
#pragma unroll 8
    for (int64_t r = g + 32 * kHeld; r < n; r += 32)
        m = fmaxf(m, rows[r * a.T].x);
    part[g][lane] = m;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 32; ++k)
        m = fmaxf(m, part[k][lane]);
    const float from = m == -INFINITY ? 0.0f : m;
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < kHeld; ++k)
        s += held[k].y * expf(held[k].x - from);
#pragma unroll 8
    for (int64_t r = g + 32 * kHeld; r < n; r += 32) {
        const float2 q = rows[r * a.T];
        s += q.y * expf(q.x - from);
    }
    __syncthreads();
    part[g][lane] = s;
    __syncthreads();
    if (g > 0)
        return;
    double sum = 0.0, total = 0.0;  // of the block's 32 tokens
    if (p < pad) {
        float inv = 0.0f, tgrad = 0.0f;
        if (p < live) {
            s = 0.0f;
#pragma unroll
            for (int k = 0; k < 32; ++k)
                s += part[k][lane];
            // (the loss from the logits' difference: lse is rounded to its own size, which a confident
            // token's loss is far below)
            const float rest = logf(s), loss = m - target + rest;
            a.loss[token] = loss;
            if (a.lse)
                a.lse[token] = m + rest;
            sum = (double)weight * (double)loss;
            total = (double)weight;
            const float coef = weight * a.head->scale;
            inv = coef / s;
            tgrad = inv * expf(target - m) - coef;
        }
        a.largest[p] = m;
        a.inv[p] = inv;
        a.tgrad[p] = tgrad;
    }
    if (!a.stats)
        return;
    sum = warp_total(sum);
    total = warp_total(total);
    // the last block to be done adds up the blocks' sums, in an order that does not depend on which it is
    if (gridDim.x > 1) {
        double2 *sums = reinterpret_cast<double2 *>(a.sums);
        if (lane == 0) {
            sums[blockIdx.x] = make_double2(sum, total);
            __threadfence();
            turn = atomicAdd(&a.head->ticket, 1u);
        }
        __syncwarp();
        if (turn + 1 != gridDim.x)
            return;
        __threadfence();
        sum = total = 0.0;
        for (unsigned b = lane; b < gridDim.x; b += 32) {
            const double2 q = __ldcg(sums + b);
            sum += q.x;
            total += q.y;
        }
        sum = warp_total(sum);
        total = warp_total(total);
    }
    if (lane == 0) {
        a.stats[0] = (float)sum;
        a.stats[1] = (float)total;
    }
}

// The kept exponentials exp(z - top) of a piece to the gradient of its logits, in place:
// inv exp(top - largest) of it, but at the target tgrad, from the 16 bits of kept_code to the layer's type.  A block takes 32 tokens and 1024
// entries, whose 32 x 32 factors it makes once.  Bound: a read and a write of the piece, from L2 as far as it
// stayed there.
template <bool BF16>
__global__ void __launch_bounds__(256, 4) kept_kernel(const __grid_constant__ EntropyArgs a)
{
    __shared__ float factor[32][33];
    wait_dependencies();
    launch_dependents();
    const int live = a.head->live, pad = a.head->live_pad;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t p0 = (int64_t)blockIdx.x * 32;
    if (p0 >= pad)
        return;
    for (int64_t c0 = (int64_t)blockIdx.y * 1024; c0 < a.kept_n; c0 += (int64_t)gridDim.y * 1024) {
        __syncthreads();  // the factors are made anew
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int g = warp + 8 * k;
            float f = 0.0f;
            if (p0 + lane < live && c0 + g * 32 < a.kept_n) {
                const float top = a.kept_top[(c0 / 32 + g) * a.T + p0 + lane];
                f = ex2_approx((top - a.largest[p0 + lane]) * 1.44269504f) * a.inv[p0 + lane];
            }
            factor[lane][g] = f;
        }
        __syncthreads();
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
            uint4 q[2][4];  // two rows of a warp, all loads in flight
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int64_t p = p0 + warp + 8 * (2 * half + k);
                const uint16_t *row = a.dz + p * a.piece + c0;
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const int c = (lane + 32 * m) * 8;
                    q[k][m] = p < live && c0 + c < a.kept_n ? *reinterpret_cast<const uint4 *>(row + c)
                                                            : make_uint4(0u, 0u, 0u, 0u);
                }
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int r = warp + 8 * (2 * half + k);
                const int64_t p = p0 + r;
                if (p >= pad)
                    continue;
                uint16_t *row = a.dz + p * a.piece + c0;
                const int64_t target = (int64_t)a.tgt[p] - a.kept0 - c0;  // behind the last token: none
                const float tgrad = a.tgrad[p];
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const int c = (lane + 32 * m) * 8;
                    if (c0 + c >= a.kept_n)
                        continue;
                    const float f = factor[r][c / 32];
                    uint32_t *w = reinterpret_cast<uint32_t *>(&q[k][m]);
                    const bool here = target >= c && target < c + 8;
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        float2 v = make_float2(kept_value(w[u] & 0xffffu) * f, kept_value(w[u] >> 16) * f);
                        if (here && target == c + 2 * u)
                            v.x = tgrad;
                        if (here && target == c + 2 * u + 1)
                            v.y = tgrad;
                        w[u] = pair16_of<BF16>(v.x, v.y);
                    }
                    *reinterpret_cast<uint4 *>(row + c) = q[k][m];
                }
            }
        }
    }
}

// V elements per thread and step (8 where dX's rows are 16-byte aligned).
template <bool BF16, int V>
__global__ void __launch_bounds__(256) dx_kernel(const __grid_constant__ EntropyArgs a)
{
    wait_dependencies();
    launch_dependents();
    const float alpha = a.head->alpha;
    const int shares = a.head->shares;
    const int64_t units = (a.K + V - 1) / V, total = a.T * units;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t t = i / units, n = (i - t * units) * V;
        const int p = a.place[t];
        uint16_t *out = reinterpret_cast<uint16_t *>(a.dX) + t * a.lddx + n;
        const float *from = a.dx32 + p * a.ldw + n;  // (rows of whole 8 elements)
        if constexpr (V == 8) {
            float v[8] = {};
            for (int s = 0; p >= 0 && s < shares; ++s, from += a.T * a.ldw) {
                const float4 x = *reinterpret_cast<const float4 *>(from), y = *reinterpret_cast<const float4 *>(from + 4);
                v[0] += x.x, v[1] += x.y, v[2] += x.z, v[3] += x.w;
                v[4] += y.x, v[5] += y.y, v[6] += y.z, v[7] += y.w;
            }
#pragma unroll
            for (int u = 0; u < 8; ++u)
                v[u] *= alpha;
            store8(out, a.K - n,
                   p >= 0 ? make_uint4(pair16_of<BF16>(v[0], v[1]), pair16_of<BF16>(v[2], v[3]),
                                       pair16_of<BF16>(v[4], v[5]), pair16_of<BF16>(v[6], v[7]))
                          : make_uint4(0u, 0u, 0u, 0u));
        } else {
            float v = 0.0f;
            for (int s = 0; p >= 0 && s < shares; ++s, from += a.T * a.ldw)
                v += *from;
            store16(out, 0, v * alpha, BF16);
        }
    }
}

}  // namespace

cudaError_t launch_entropy_tokens(const EntropyArgs &a, cudaStream_t s)
{
    return launch_early(tokens_kernel, dim3((unsigned)gg_min64(a.T, kBlocks)), kThreads, 0, s, a);
}

cudaError_t launch_entropy_join(const EntropyArgs &a, cudaStream_t s)
{
    return launch_early(join_kernel, dim3((unsigned)((a.T + 31) / 32)), kThreads, 0, s, a);
}

cudaError_t launch_entropy_kept(const EntropyArgs &a, cudaStream_t s)
{
    // (pieces have fewer than 2^21 times 1024 entries; token groups go down the grid's long side)
    const dim3 grid((unsigned)((a.T + 31) / 32), (unsigned)gg_min64((a.kept_n + 1023) / 1024, 65535));
    return launch_early(a.is_bf16 ? kept_kernel<true> : kept_kernel<false>, grid, 256, 0, s, a);
}

cudaError_t launch_entropy_dx(const EntropyArgs &a, cudaStream_t s)
{
    const bool wide = ((reinterpret_cast<uint64_t>(a.dX) | (uint64_t)(a.lddx * 2)) & 15) == 0;
    const int64_t total = a.T * (wide ? (a.K + 7) / 8 : a.K);
    const dim3 grid((unsigned)gg_min64((total + 255) / 256, kSMs * 8));
    if (wide)
        return launch_early(a.is_bf16 ? dx_kernel<true, 8> : dx_kernel<false, 8>, grid, 256, 0, s, a);
    return launch_early(a.is_bf16 ? dx_kernel<true, 1> : dx_kernel<false, 1>, grid, 256, 0, s, a);
}

}  // namespace gg
