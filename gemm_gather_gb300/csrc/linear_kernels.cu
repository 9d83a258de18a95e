// The linear layer for sm_103a: Y = act(X W + b) + R and its gradients.
//
// Every product of the layer is one form,
//     out[j, i] = epilogue( sum_k A[i, k] B[j, k] ),
// with i the contiguous index of the output (MMA rows, TMEM lanes) and j its
// row (MMA columns):
//     forward        i = out feature, j = token, k = in feature   A = W,  B = X
//     input gradient i = in feature,  j = token, k = out feature  A = W,  B = dZ
//     weight gradient, W K x N:  i = n, j = k, contraction over tokens  A = dZ, B = X
//                      W N x K:  i = k, j = n                           A = X,  B = dZ
// An operand whose contraction index is contiguous in memory is K-major, else
// MN-major; tcgen05 reads both from 128-byte swizzled shared memory, so no
// operand is ever transposed in memory.  One thread issues the MMAs, chosen by
// elect.sync: behind `lane == 0`, a condition the compiler takes for any
// thread's, the issue alone took 645 cycles a k-block of 512 tensor cycles, and
// the tensor pipes stood at 78%; elected, at 96% (256 x 256 tiles, K = 8192).
// Features on the MMA's 128 rows: a
// thread of the epilogue owns one feature, its warp 32 neighbouring ones, so
// the bias is one register, every global access of the epilogue is 32
// neighbouring elements at any alignment, and a product of a few tokens pads
// only the MMA's columns (16 at least) and not its 128 rows.
//
// Two kernels:
//  * pair_kernel: persistent CTA pairs on tiles of 256 features x 64 to 256
//    tokens (tcgen05 cta_group::2, 64-deep stages, 6 or 8 in a ring of 192 KB per
//    CTA, two accumulators in TMEM so that a tile's epilogue runs under the next
//    tile's MMAs).  Bound: the tensor pipes, under the power limit.  Measured:
//    16384 x 3584 x 8192 with gelu_tanh and Z stored in 503 to 594 us (1.62 to 1.91
//    PFLOP/s; cuBLAS's product alone on the same boxes 494 to 574), pipes 90 %
//    active at 4096 x 4864 x 8192 with gelu and Z.
//  * split_kernel: one CTA per tile of 128 features x {16, 32, 64} tokens and share
//    of the contraction; the CTAs of a cluster (up to 8) split one tile's
//    contraction and join their float32 partial tiles through distributed
//    shared memory in rank order (the same bits on every run, no workspace, no
//    second launch).  For few tokens, where the time is that of streaming W,
//    and for few tiles.  Bound: HBM, and below some 10 us the launch, the first
//    load and the join.  Measured: 1 x 3584 x 8192 in 12.2 us, of which the weights'
//    bytes take 8.6 (4.8 TB/s over all of it); the join takes 1.5, a launch 1.9.
//
// Sums.  tcgen05's float32 accumulator truncates when it adds: measured
// against float64 on normal operands, the relative error grows with the
// length of the contraction (4.7e-7 at 512, 4.4e-6 at 4096, 1.9e-5 at 16384,
// where a float32 sum rounded to nearest has 1.5e-6).  That is nothing to a
// 16-bit result, but weight gradients are kept in float32 over long sums of
// tokens, so the weight gradient accumulates kChunk k-blocks in TMEM and adds
// the chunks in registers with round-to-nearest.  Chunks of 896: 8.1e-7, near a
// float32 product's own 6.1e-7 at 4096 tokens, and 165 us for the gradient of an
// 8192 x 3584 weight over them (512: 4.7e-7 and 182 us; one chunk: 4.4e-6, 163 us).
//
// The vocabulary's products (entropy_kernels.cu) run on the same kernels: logits whose epilogue keeps sums of
// exponentials (kEpiLse), or the gradient of the logits (kEpiSoftGrad), and what that is multiplied into
// (kEpiVocab).  The tokens that count are known on the device only (kLive): a launch is laid out for all
// of them, and its walk ends at the last tile there is.
//
// Every mbarrier wait is bounded; one that gives up stores GG_ERR_TIMEOUT in
// the status word and raises the CTA's abort flag, and every role drains what
// it has in flight before TMEM is freed and the CTA exits.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <mutex>
#include <type_traits>

#include "act.cuh"
#include "f32x2.cuh"
#include "gg_internal.h"
#include "gg_ops.h"
#include "pack8.cuh"
#include "tc.cuh"

namespace gg {
namespace {

using namespace tc;

constexpr int kSMs = 152;
constexpr int kBK = 64;                    // k of one stage: a 128-byte swizzle row
constexpr int UK = 16;                     // k of one MMA
constexpr int kChunk = 14;                 // k-blocks per TMEM chunk of a weight gradient (896 k)
constexpr int kMnBox = kBK * 64 * 2;       // 8 KB: 64 k-rows x 64 columns of an MN-major operand
constexpr uint64_t kDrainLimitNs = 1000000000ull;
constexpr int kMaxStages = 8;

// The epilogue's staging (see below): tokens at a time, bytes of a warp, 16-byte
// accesses of a lane.
constexpr int kStageCols = 32;
constexpr int kWarpStage = kStageCols * 64;  // 32 tokens x 32 features x 2 bytes
constexpr int kRowSteps = kStageCols / 8;    // 16-byte accesses of a lane

// Epilogues that add the chunks of a long contraction in registers, and those of the vocabulary's
// products, whose number of tokens (their columns, or their contraction) is known on the device only.
template <int EPI>
constexpr bool kSums = EPI == kEpiGradW || EPI == kEpiVocab || EPI == kEpiLse;
template <int EPI>
constexpr bool kLogSum = EPI == kEpiLse || EPI == kEpiLseShort;
template <int EPI>
constexpr bool kLive = kLogSum<EPI> || EPI == kEpiSoftGrad || EPI == kEpiVocab || EPI == kEpiVocabShort;
// Results that may be float32, and may be added to what is there.  The short ones, of a contraction of
// one chunk, need no sums in registers; a zero is made positive as by the sums.
template <int EPI>
constexpr bool kShort = EPI == kEpiGradWShort || EPI == kEpiVocabShort;
template <int EPI>
constexpr bool kOwn = EPI == kEpiGradW || EPI == kEpiVocab || kShort<EPI>;
template <int EPI>
constexpr bool kScaled = EPI == kEpiVocab || EPI == kEpiVocabShort;
constexpr float kLog2e = 1.44269504f;

struct Shared {
    uint64_t full[kMaxStages];
    uint64_t empty[kMaxStages];
    uint64_t tmem_full[2];
    uint64_t tmem_empty[2];
    uint64_t mma_done;
    uint32_t tmem_base;
    int abort_flag;
};

// ---- epilogue arithmetic ---------------------------------------------------------
// An element of the tensor beside the sums.  One kept in 8 bits (its codes are at p) is taken in the
// layer's 16-bit type, which holds its four significant bits.
template <int EPI>
__device__ __forceinline__ float load_aux(const LinearArgs &a, const void *p, int64_t ld, int64_t j, int64_t i)
{
    if constexpr (EPI == kEpiGradIn8) {
        float x[4];
        unpack4(reinterpret_cast<const uint8_t *>(p)[j * ld + i], x);
        const float v = x[0] * a.scales[j * a.lds + i / kPackBlock];
        return a.is_bf16 ? held16<true>(v) : pair16<false>(pair16_of<false>(held16<false>(v), 0.0f)).x;
    }
    return load16(p, j * ld + i, a.is_bf16);
}

// ---- the vocabulary's softmax -----------------------------------------------------------
// The gradient over a logit z of token j, for vocabulary entry i of a piece:
// coef (exp(z - largest) / total - (i is the target)).  The difference first: it is small where it counts, however
// large the logits are.  From the largest and the sum, not from lse, whose rounding to its own size would be all that
// is left of a confident token's p - 1.  That term, the target's, is the join's (of the logits that the loss has): it
// is read where a target lies, once a token.
struct TokenTerms {
    float largest, inv;  // inv: coef / total
    int target;          // within the piece; any other number: not there
};

__device__ __forceinline__ float soft_grad(float z, float largest, float inv)
{
    // (what rows of zeros fill a k-block up with is 0, whatever W holds)
    return inv != 0.0f ? ex2_approx((z - largest) * kLog2e) * inv : 0.0f;
}

// exp of two logits less what they are taken from.
__device__ __forceinline__ float2 above(float z0, float z1, float from0, float from1)
{
    const float2 d = halves_of(mul2(add2(pair_of(z0, z1), pair_of(-from0, -from1)), pair_of(kLog2e)));
    return make_float2(ex2_approx(d.x), ex2_approx(d.y));
}

// (largest z, sum of exp(z - largest)) of a warp's 32 vocabulary entries, for each of n columns: a row of
// the partial results is the warp's, place j is token j.  Every lane calls it; where all of them are past
// the vocabulary's end there is no such row.
template <int C>
__device__ __forceinline__ void emit_lse(const LinearArgs &a, int64_t i, int64_t j0, int jstep, int n,
                                         const float (&v)[16])
{
    const int lane = threadIdx.x & 31;
    const bool in = i < a.I;
#pragma unroll
    for (int u = 0; u < C; ++u) {
        if (u >= n)
            break;
        const int64_t j = j0 + (int64_t)u * jstep;
        const float z = in ? v[u] : -INFINITY;
        float m = z;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1)
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
        float e = in ? ex2_approx((z - (m == -INFINITY ? 0.0f : m)) * kLog2e) : 0.0f;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1)
            e += __shfl_xor_sync(0xffffffffu, e, d);
        if (lane == 0 && in)
            a.partial[i / 32 * a.ldpartial + j] = make_float2(m, e);
        if (in && (int)i == a.target[j])
            a.ztarget[j] = z;
    }
}

// The same of 16 neighbouring columns in 2 KB of shared memory: a lane turns from a vocabulary entry
// to half a column's entries (the exclusive or spreads both over the banks).  target: lane c mod 16
// has column c's, and gets its result.  The difference comes first, as everywhere: log2 e times each of two
// large logits would be rounded apart, which costs a confident token's loss 2^-24 of the logit, and logits
// beyond 2^30 everything.
__device__ __forceinline__ float2 lse16(const LinearArgs &a, int64_t i0, int64_t j0, int n, int lane, int target,
                                        const float (&v)[16], uint8_t *stage)
{
    float *t = reinterpret_cast<float *>(stage);
    const bool in = i0 + lane < a.I;
#pragma unroll
    for (int u = 0; u < 16; ++u)
        t[u * 32 + (lane ^ u)] = in ? v[u] : -INFINITY;
    __syncwarp();
    const int c = lane & 15, half = lane & 16;
    float x[16], m = -INFINITY, s = 0.0f;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        x[k] = t[c * 32 + ((half + k) ^ c)];
        m = fmaxf(m, x[k]);
    }
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
    const float from = m == -INFINITY ? 0.0f : m;
#pragma unroll
    for (int k = 0; k < 16; k += 2) {
        const float2 e = above(x[k], x[k + 1], from, from);
        s += e.x;
        s += e.y;
    }
    s += __shfl_xor_sync(0xffffffffu, s, 16);
    if (c < n) {
        const int64_t at = (int64_t)target - i0;
        if (at >= half && at < half + 16 && at + i0 < a.I)
            a.ztarget[j0 + c] = t[c * 32 + ((int)at ^ c)];
    }
    __syncwarp();
    return make_float2(m, s);
}

// Whether all of 128 threads (the four warps of one group of columns) say yes; a barrier between them.
__device__ __forceinline__ bool group_agrees(int group, bool yes)
{
    int all;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\t"
                 "barrier.cta.red.and.pred q, %2, 128, p;\n\tselp.b32 %0, 1, 0, q;\n\t}"
                 : "=r"(all)
                 : "r"((int)yes), "r"(1 + group)
                 : "memory");
    return all != 0;
}

__device__ __forceinline__ void group_sync(int group)
{
    asm volatile("barrier.cta.sync %0, 128;" ::"r"(1 + group) : "memory");
}

// One feature's sums for columns j0, j0 + jstep, ... (n of them, at most C):
// the epilogue and the store.  A warp's 32 lanes hold 32 neighbouring
// features.  Loads of the columns are issued together, ahead of their use.
template <int EPI, int C = 16>
__device__ __forceinline__ void emit16(const LinearArgs &a, int64_t i, int64_t j0, int jstep, int n,
                                       float (&v)[16], float bias)
{
    if constexpr (kLogSum<EPI>) {
        emit_lse<C>(a, i, j0, jstep, n, v);
        return;
    }
    if (i >= a.I)
        return;
    if constexpr (kShort<EPI>) {
#pragma unroll
        for (int u = 0; u < C; ++u)
            v[u] += 0.0f;
    }
    if constexpr (kScaled<EPI>) {
        const float alpha = a.alpha ? *a.alpha : 1.0f;
#pragma unroll
        for (int u = 0; u < C; ++u)
            v[u] *= alpha;
    }
    if constexpr (kOwn<EPI>) {
        if (a.out_f32) {
            float *o = reinterpret_cast<float *>(a.out) + j0 * a.ldo + i;
            const int64_t step = (int64_t)jstep * a.ldo;
            // added where it lies (one addition to each element, rounded to nearest as
            // here; the memory's adder takes subnormals for zero): with loads instead,
            // a warp waited 8 times for memory while the next tile's MMAs ran out of
            // accumulators
            if (a.accumulate) {
#pragma unroll
                for (int u = 0; u < C; ++u)
                    if (u < n)
                        asm volatile("red.global.add.f32 [%0], %1;" ::"l"(o + u * step), "f"(v[u]) : "memory");
                return;
            }
#pragma unroll
            for (int u = 0; u < C; ++u)
                if (u < n)
                    o[u * step] = v[u];
            return;
        }
    }
    float x[C];
    const void *aux = kOwn<EPI> ? (a.accumulate ? a.out : nullptr) : (EPI == kEpiSoftGrad ? nullptr : a.aux);
    const int64_t ldaux = kOwn<EPI> ? a.ldo : a.ldaux;
    if (aux != nullptr) {
#pragma unroll
        for (int u = 0; u < C; ++u)
            x[u] = u < n ? load_aux<EPI>(a, aux, ldaux, j0 + (int64_t)u * jstep, i) : 0.0f;
    }
    if constexpr (EPI == kEpiForward) {
#pragma unroll
        for (int u = 0; u < C; ++u)
            v[u] += bias;
        if (a.zout != nullptr) {
#pragma unroll
            for (int u = 0; u < C; ++u)
                if (u < n)
                    store16(a.zout, (j0 + (int64_t)u * jstep) * a.ldz + i, v[u], a.is_bf16);
        }
        float y[C];
#pragma unroll
        for (int u = 0; u < C; ++u)
            y[u] = v[u];
        with_act(a.act, [&](auto k) { apply_act<decltype(k)::value>(y); });
#pragma unroll
        for (int u = 0; u < C; ++u)
            v[u] = y[u];
        if (aux != nullptr) {
#pragma unroll
            for (int u = 0; u < C; ++u)
                v[u] += x[u];
        }
    } else if constexpr (EPI == kEpiGradIn || EPI == kEpiGradIn8) {
        float y[C];
#pragma unroll
        for (int u = 0; u < C; ++u)
            y[u] = v[u];
        if (aux != nullptr)
            with_act(a.act, [&](auto k) { apply_slope<decltype(k)::value>(y, x); });
#pragma unroll
        for (int u = 0; u < C; ++u)
            v[u] = y[u];
    } else if constexpr (EPI == kEpiSoftGrad) {
#pragma unroll
        for (int u = 0; u < C; ++u)
            if (u < n) {
                const int64_t j = j0 + (int64_t)u * jstep;
                v[u] = (int)i == a.target[j] - a.v0 ? a.tgrad[j] : soft_grad(v[u], a.largest[j], a.inv[j]);
            }
    } else if (aux != nullptr) {
#pragma unroll
        for (int u = 0; u < C; ++u)
            v[u] += x[u];
    }
#pragma unroll
    for (int u = 0; u < C; ++u)
        if (u < n)
            store16(a.out, (j0 + (int64_t)u * jstep) * a.ldo + i, v[u], a.is_bf16);
}

__device__ __forceinline__ float load_bias(const LinearArgs &a, int64_t i)
{
    if (a.bias == nullptr || i >= a.I)
        return 0.0f;
    return a.bias_f32 ? reinterpret_cast<const float *>(a.bias)[i] : load16(a.bias, i, a.is_bf16);
}

// Valid columns of a staging's, or of 16, from j0.
__device__ __forceinline__ int valid_rows(int64_t J, int64_t j0)
{
    return J - j0 >= kStageCols ? kStageCols : (J > j0 ? (int)(J - j0) : 0);
}

__device__ __forceinline__ int valid16(int64_t J, int64_t j0)
{
    return J - j0 >= 16 ? 16 : (J > j0 ? (int)(J - j0) : 0);
}

// ---- staged epilogue -----------------------------------------------------------------
// A lane owns one feature (MMA row), so a warp that stored its values directly
// would write 64-byte pieces two bytes a lane: measured, 20 cycles of an SM for
// each such store, 40,000 for a 256 x 256 tile, as long as a contraction over
// 8192.  Instead a warp turns 32 features x 32 tokens around in 2 KB of its
// own shared memory, in words of two neighbouring tokens: a lane stores its
// feature's 16 words, then takes 8 features of a pair, which are 16 bytes of each
// of the two rows, so that a global access is 8 rows of 64 bytes, and half as many
// stores are made as of single elements.  Tensors read in the epilogue come the same
// way, loaded into registers ahead of the accumulator.
//
// Pair p's word of feature f lies in row p (128 bytes), its 16-byte pieces swapped in
// odd rows, which keeps the pieces of neighbouring rows in different banks.
__device__ __forceinline__ uint32_t low_halves(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x5410); }
__device__ __forceinline__ uint32_t high_halves(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x7632); }

// Piece `half` (0 or 1) of this lane's 8 features of pair (lane / 4) + 8 h.
__device__ __forceinline__ int piece_at(int lane, int h, int half)
{
    return ((lane >> 2) + 8 * h) * 128 + ((((lane & 3) * 2 + half) ^ (lane >> 2 & 1)) * 16);
}

// A lane's row of global access k: tokens of one pair are k and k + 1.
__device__ __forceinline__ int row_of(int lane, int k) { return (lane >> 2) * 2 + (k & 1) + 16 * (k >> 1); }

// One 16-bit M x N tensor of the epilogue; vec: 16-byte accesses are aligned.
struct Rows {
    uint16_t *p;
    int64_t ld;
    bool vec;
};

__device__ __forceinline__ Rows rows_of(const void *p, int64_t ld)
{
    Rows r;
    r.p = reinterpret_cast<uint16_t *>(const_cast<void *>(p));
    r.ld = ld;
    r.vec = ((reinterpret_cast<uint64_t>(p) | (uint64_t)(ld * 2)) & 15) == 0;
    return r;
}

// 32 features from i0 of `n` tokens from j0: lane l takes features 8 (l mod 4)
// on of tokens row_of(l, k).
__device__ __forceinline__ void read_rows(const Rows &t, int64_t I, int64_t i0, int64_t j0, int n, int lane,
                                          uint4 (&x)[kRowSteps])
{
    const int64_t i = i0 + (lane & 3) * 8;
    const uint16_t *p = t.p + (j0 + row_of(lane, 0)) * t.ld + i;
#pragma unroll
    for (int k = 0; k < kRowSteps; ++k) {
        x[k] = make_uint4(0u, 0u, 0u, 0u);
        if (row_of(lane, k) < n) {
            const uint16_t *q = p + (int64_t)row_of(0, k) * t.ld;
            if (t.vec && i + 8 <= I) {
                x[k] = *reinterpret_cast<const uint4 *>(q);
            } else {
                uint16_t h[8];
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    h[u] = i + u < I ? q[u] : (uint16_t)0;
                x[k] = *reinterpret_cast<uint4 *>(h);
            }
        }
    }
}

// The same of a tensor kept in 8 bits: a lane's eight features lie in one block of 128, under one
// scale.
template <bool BF16>
__device__ __forceinline__ void read_codes(const LinearArgs &a, int64_t i, int64_t j0, int n, int lane, bool vec,
                                           uint4 (&x)[kRowSteps])
{
    const uint8_t *p = reinterpret_cast<const uint8_t *>(a.aux) + (j0 + row_of(lane, 0)) * a.ldaux + i;
    const float *s = a.scales + (j0 + row_of(lane, 0)) * a.lds + i / kPackBlock;
#pragma unroll
    for (int k = 0; k < kRowSteps; ++k) {
        x[k] = make_uint4(0u, 0u, 0u, 0u);
        if (row_of(lane, k) < n && i < a.I) {
            const uint8_t *q = p + (int64_t)row_of(0, k) * a.ldaux;
            uint2 c = make_uint2(0u, 0u);
            if (vec && i + 8 <= a.I) {
                c = *reinterpret_cast<const uint2 *>(q);
            } else {
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    if (i + u < a.I)
                        (u < 4 ? c.x : c.y) |= (uint32_t)q[u] << (8 * (u & 3));
            }
            float v[8];
            values8<BF16>(c, s[(int64_t)row_of(0, k) * a.lds], v);
            x[k] = make_uint4(pair16_of<BF16>(v[0], v[1]), pair16_of<BF16>(v[2], v[3]), pair16_of<BF16>(v[4], v[5]),
                              pair16_of<BF16>(v[6], v[7]));
        }
    }
}

// The rows that an epilogue reads beside the sums.
template <int EPI>
__device__ __forceinline__ void read_aux(const LinearArgs &a, const Rows &t, int64_t i0, int64_t j0, int n, int lane,
                                         uint4 (&x)[kRowSteps])
{
    if constexpr (EPI == kEpiGradIn8) {
        if (a.is_bf16)
            read_codes<true>(a, i0 + (lane & 3) * 8, j0, n, lane, t.vec, x);
        else
            read_codes<false>(a, i0 + (lane & 3) * 8, j0, n, lane, t.vec, x);
    } else {
        read_rows(t, a.I, i0, j0, n, lane, x);
    }
}

__device__ __forceinline__ void stage_pair(uint8_t *stage, int lane, int h, const uint4 &a, const uint4 &b)
{
    *reinterpret_cast<uint4 *>(stage + piece_at(lane, h, 0)) =
        make_uint4(low_halves(a.x, b.x), high_halves(a.x, b.x), low_halves(a.y, b.y), high_halves(a.y, b.y));
    *reinterpret_cast<uint4 *>(stage + piece_at(lane, h, 1)) =
        make_uint4(low_halves(a.z, b.z), high_halves(a.z, b.z), low_halves(a.w, b.w), high_halves(a.w, b.w));
}

__device__ __forceinline__ void stage_rows(uint8_t *stage, int lane, const uint4 (&x)[kRowSteps])
{
#pragma unroll
    for (int h = 0; h < kRowSteps / 2; ++h)
        stage_pair(stage, lane, h, x[2 * h], x[2 * h + 1]);
    __syncwarp();
}

// read_rows and stage_rows, two rows of a lane at a time.
__device__ __forceinline__ void fetch_rows(const Rows &t, int64_t I, int64_t i0, int64_t j0, int n, int lane,
                                           uint8_t *stage)
{
    const int64_t i = i0 + (lane & 3) * 8;
#pragma unroll 1
    for (int h = 0; h < kRowSteps / 2; ++h) {
        uint4 x[2];
#pragma unroll
        for (int odd = 0; odd < 2; ++odd) {
            const int row = row_of(lane, 2 * h + odd);
            x[odd] = make_uint4(0u, 0u, 0u, 0u);
            if (row < n) {
                const uint16_t *q = t.p + (j0 + row) * t.ld + i;
                if (t.vec && i + 8 <= I) {
                    x[odd] = *reinterpret_cast<const uint4 *>(q);
                } else {
                    uint16_t e[8];
#pragma unroll
                    for (int u = 0; u < 8; ++u)
                        e[u] = i + u < I ? q[u] : (uint16_t)0;
                    x[odd] = *reinterpret_cast<uint4 *>(e);
                }
            }
        }
        stage_pair(stage, lane, h, x[0], x[1]);
    }
    __syncwarp();
}

// This lane's word of tokens col and col + 1 (col even).
__device__ __forceinline__ uint32_t *staged(uint8_t *stage, int lane, int col)
{
    const int p = col >> 1;
    return reinterpret_cast<uint32_t *>(stage + p * 128) + (p & 1 ? lane ^ 4 : lane);
}

__device__ __forceinline__ void write_rows(const Rows &t, int64_t I, int64_t i0, int64_t j0, int n, int lane,
                                           uint8_t *stage)
{
    __syncwarp();
    if (!t.vec) {  // a token at a time, its 32 features side by side (see above: 64-byte pieces)
        uint16_t *q = t.p + j0 * t.ld + i0 + lane;
        if (i0 + lane < I) {
#pragma unroll 4
            for (int r = 0; r < n; r += 2) {
                const uint32_t w = *staged(stage, lane, r);
                q[r * t.ld] = (uint16_t)w;
                if (r + 1 < n)
                    q[(r + 1) * t.ld] = (uint16_t)(w >> 16);
            }
        }
        __syncwarp();
        return;
    }
    const int64_t i = i0 + (lane & 3) * 8;
    uint16_t *p = t.p + (j0 + row_of(lane, 0)) * t.ld + i;
#pragma unroll
    for (int h = 0; h < kRowSteps / 2; ++h) {
        const uint4 a = *reinterpret_cast<const uint4 *>(stage + piece_at(lane, h, 0));
        const uint4 b = *reinterpret_cast<const uint4 *>(stage + piece_at(lane, h, 1));
#pragma unroll
        for (int odd = 0; odd < 2; ++odd) {
            if (row_of(lane, 2 * h + odd) >= n)
                continue;
            const uint4 x = odd ? make_uint4(high_halves(a.x, a.y), high_halves(a.z, a.w), high_halves(b.x, b.y),
                                             high_halves(b.z, b.w))
                                : make_uint4(low_halves(a.x, a.y), low_halves(a.z, a.w), low_halves(b.x, b.y),
                                             low_halves(b.z, b.w));
            uint16_t *q = p + (int64_t)row_of(0, 2 * h + odd) * t.ld;
            if (i + 8 <= I) {
                *reinterpret_cast<uint4 *>(q) = x;
            } else {
                const uint16_t *e = reinterpret_cast<const uint16_t *>(&x);
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    if (i + u < I)
                        q[u] = e[u];
            }
        }
    }
    __syncwarp();
}

// 16 tokens' values of this lane's feature from col on, rounded; and what is staged there.
__device__ __forceinline__ void stage16(const LinearArgs &a, const float (&v)[16], uint8_t *stage, int lane, int col)
{
#pragma unroll
    for (int u = 0; u < 16; u += 2)
        *staged(stage, lane, col + u) = a.is_bf16 ? pair16_of<true>(v[u], v[u + 1]) : pair16_of<false>(v[u], v[u + 1]);
}

__device__ __forceinline__ void unstage16(const LinearArgs &a, float (&x)[16], uint8_t *stage, int lane, int col)
{
#pragma unroll
    for (int u = 0; u < 16; u += 2) {
        const uint32_t w = *staged(stage, lane, col + u);
        const float2 f = a.is_bf16 ? pair16<true>(w) : pair16<false>(w);
        x[u] = f.x, x[u + 1] = f.y;
    }
}

// The tensor an epilogue reads beside the sums, or a null pointer.
template <int EPI>
__device__ __forceinline__ Rows aux_of(const LinearArgs &a)
{
    if constexpr (kLogSum<EPI> || EPI == kEpiSoftGrad)
        return rows_of(nullptr, 0);
    if constexpr (kOwn<EPI>)
        return rows_of(a.accumulate && !a.out_f32 ? a.out : nullptr, a.ldo);
    if constexpr (EPI == kEpiGradIn8) {  // codes: eight bytes a lane
        Rows r = rows_of(a.aux, 0);
        r.vec = ((reinterpret_cast<uint64_t>(a.aux) | (uint64_t)a.ldaux) & 7) == 0;
        return r;
    }
    return rows_of(a.aux, a.ldaux);
}

// The epilogue of a warp's 32 features (from i0) and up to 32 tokens (from j0, n
// of them).  sums(col, v) gives this lane's sums of columns col .. col + 15; it
// may be called twice.  aux: the rows read beside them (has_aux).
template <int EPI, bool REGISTERS = false, typename Sums>
__device__ __forceinline__ void emit_rows(const LinearArgs &a, int64_t i0, int64_t j0, int n, int lane,
                                       float bias, bool has_aux, const uint4 (&aux)[kRowSteps],
                                       uint8_t *stage, Sums sums, const TokenTerms &terms = TokenTerms{})
{
    // sums in registers need constant columns; the others keep the code small
    constexpr int kUnroll = REGISTERS ? kStageCols / 16 : 1;
    if constexpr (EPI == kEpiForward) {
        if (a.zout != nullptr) {
#pragma unroll 1
            for (int c = 0; c < n; c += 16) {
                float v[16];
                sums(c, v);
#pragma unroll
                for (int u = 0; u < 16; ++u)
                    v[u] += bias;
                stage16(a, v, stage, lane, c);
            }
            write_rows(rows_of(a.zout, a.ldz), a.I, i0, j0, n, lane, stage);
        }
    }
    if (has_aux && !REGISTERS)
        stage_rows(stage, lane, aux);
    if (has_aux && REGISTERS)  // beside the sums there is room for half of them
        fetch_rows(aux_of<EPI>(a), a.I, i0, j0, n, lane, stage);
    // columns whose target is one of the warp's features: few
    const uint32_t hits =
        EPI == kEpiSoftGrad ? __ballot_sync(0xffffffffu, terms.target >= i0 && terms.target < i0 + 32) : 0u;
#pragma unroll(kUnroll)
    for (int c = 0; c < kStageCols; c += 16) {
        if (c >= n)
            break;
        float v[16], x[16];
        sums(c, v);
        if constexpr (kShort<EPI>) {
#pragma unroll
            for (int u = 0; u < 16; ++u)
                v[u] += 0.0f;
        }
        if constexpr (kScaled<EPI>) {
            const float alpha = a.alpha ? *a.alpha : 1.0f;
#pragma unroll
            for (int u = 0; u < 16; ++u)
                v[u] *= alpha;
        }
        if (has_aux) {  // a lane reads its own elements before it writes over them
            unstage16(a, x, stage, lane, c);
        }
        if constexpr (EPI == kEpiForward) {
#pragma unroll
            for (int u = 0; u < 16; ++u)
                v[u] += bias;
            with_act(a.act, [&](auto k) { apply_act<decltype(k)::value>(v); });
            if (has_aux) {
#pragma unroll
                for (int u = 0; u < 16; ++u)
                    v[u] += x[u];
            }
        } else if constexpr (EPI == kEpiGradIn || EPI == kEpiGradIn8) {
            if (has_aux)
                with_act(a.act, [&](auto k) { apply_slope<decltype(k)::value>(v, x); });
        } else if constexpr (EPI == kEpiSoftGrad) {  // lane c has column c's terms
#pragma unroll
            for (int u = 0; u < 16; ++u)
                v[u] = soft_grad(v[u], __shfl_sync(0xffffffffu, terms.largest, c + u),
                                 __shfl_sync(0xffffffffu, terms.inv, c + u));
#pragma unroll 1
            for (uint32_t left = hits >> c & 0xffffu; left != 0; left &= left - 1) {
                const int at = __ffs((int)left) - 1;
                const bool mine = __shfl_sync(0xffffffffu, terms.target, c + at) == (int)i0 + lane;
                const float own = mine ? a.tgrad[j0 + c + at] : 0.0f;
#pragma unroll
                for (int u = 0; u < 16; ++u)
                    v[u] = mine && u == at ? own : v[u];
            }
        } else if (has_aux) {
#pragma unroll
            for (int u = 0; u < 16; ++u)
                v[u] += x[u];
        }
        stage16(a, v, stage, lane, c);
    }
    write_rows(rows_of(a.out, a.ldo), a.I, i0, j0, n, lane, stage);
}

// Column j0 + lane's terms, of n columns.
template <int EPI>
__device__ __forceinline__ TokenTerms terms_of(const LinearArgs &a, int64_t j0, int n, int lane)
{
    TokenTerms t{0.0f, 0.0f, -1};
    if constexpr (kLogSum<EPI>) {
        if (lane < n)
            t.target = a.target[j0 + lane];
    }
    if constexpr (EPI == kEpiSoftGrad) {
        if (lane < n)
            t = TokenTerms{a.largest[j0 + lane], a.inv[j0 + lane], a.target[j0 + lane] - a.v0};
    }
    return t;
}

// One stage's operand: `rows` rows (or columns) of 64 k.  K-major: one box of
// 64 k x rows.  MN-major: boxes of 64 columns x 64 k-rows.
template <int CG>
__device__ __forceinline__ void load_operand(uint32_t dst, const CUtensorMap *map, int mn, int rows, int row0,
                                             int k0, uint32_t bar, uint64_t policy)
{
    if (!mn) {
        tma_load_2d<CG>(dst, map, k0, row0, bar, policy);
    } else {
        for (int b = 0; b * 64 < rows; ++b)
            tma_load_2d<CG>(dst + b * kMnBox, map, row0 + b * 64, k0, bar, policy);
    }
}

// ---- pair kernel: 256 features x bt <= BT tokens per CTA pair ----------------------------
// Part `part`'s k-blocks of num_kb (below 2^26, the tensor map's limit).
__device__ __forceinline__ void share_of(int num_kb, int part, int parts, int &kb0, int &n)
{
    kb0 = (int)((uint32_t)num_kb * (uint32_t)part / (uint32_t)parts);
    n = (int)((uint32_t)num_kb * (uint32_t)(part + 1) / (uint32_t)parts) - kb0;
}

namespace pair {
constexpr int kTileI = 256;
constexpr int kA = 128 * kBK * 2;        // 16 KB: this CTA's 128 features of one k-block
constexpr int kEpiWarps = 16;            // four per TMEM lane quarter, a quarter of the columns each
constexpr int kProducer2 = 2 + kEpiWarps;  // the second producer's warp
constexpr int kThreads = 32 * (kProducer2 + 1);
template <int BT>
struct Geo {
    static constexpr int kB = BT / 2 * kBK * 2;  // this CTA's half of the tokens
    static constexpr int kStage = kA + kB;
    static constexpr int kStages = BT == 256 ? 6 : 8;  // 192 KB of ring
    static constexpr int kRing = kStages * kStage;
    static constexpr int kPartial = 128 * BT * 4;  // float32 partial tile, over the spent ring
    static constexpr int kOffStage = kRing;
    static constexpr int kOffShared = kOffStage + kEpiWarps * kWarpStage;
    static constexpr int kSmemBytes = kOffShared + (int)sizeof(Shared) + 1024;
    static_assert(kSmemBytes <= 232448 && kStages <= kMaxStages && kStages % 2 == 0 && kPartial <= kRing,
                  "shared memory of a CTA");
};

struct Tile {
    int ti, tj;
    // kLive: the share of the contraction that is this tile's, its first k-block and how many
    int share, kb0, num_kb;
};

// Tile order: feature tiles in groups of a.group; group by group, every token
// tile runs over the group's feature tiles.  The pairs running at one time
// then cover about as many feature tiles as token tiles, which keeps the
// slices of A and B that they read from DRAM and share through L2 few.
// Unsigned: a product has fewer than 2^31 tiles (launch_pair refuses more).
__device__ __forceinline__ Tile tile_at(const LinearArgs &a, uint32_t tiles_j, uint32_t t)
{
    const uint32_t full = (uint32_t)a.group * tiles_j;
    const uint32_t g = t / full;
    const uint32_t r = t - g * full;
    const uint32_t left = (uint32_t)a.tiles_i - g * (uint32_t)a.group;
    const uint32_t width = left < (uint32_t)a.group ? left : (uint32_t)a.group;
    Tile c = {};
    c.tj = (int)(r / width);
    c.ti = (int)(g * (uint32_t)a.group + r - (uint32_t)c.tj * width);
    return c;
}

// One product's tiles (this pair's: first, first + nunits, ...), and this pair's
// share of their contraction.
struct Product {
    int kb0, num_kb;
    uint32_t total, first;
    Tile tile;  // the first
    // kLive: the columns, their tiles and the shares of the contraction that the device knows
    int64_t J;
    uint32_t tiles_j, shares;
    __device__ __forceinline__ Product() : kb0(0), num_kb(0), total(0), first(0), tile{}, J(0), tiles_j(0), shares(1) {}
    __device__ __forceinline__ Product(const LinearArgs &a, int part, int parts, uint32_t first_)
        : kb0(0), num_kb(a.num_kb), total((uint32_t)a.tiles_i * (uint32_t)a.tiles_j), first(first_),
          tile(first_ < total ? tile_at(a, (uint32_t)a.tiles_j, first_) : Tile{})
    {
        if (parts > 1)  // 2 or 4
            share_of(a.num_kb, part, parts, kb0, num_kb);
    }
    // The same with the tokens that the device counted; the launches before have to be waited for.
    // Where there are shares, every tile comes that many times, with a share of the contraction each.
    __device__ __forceinline__ void count(const LinearArgs &a, int part, int parts)
    {
        const int live = *a.live;
        num_kb = a.live_k ? (live + kBK - 1) / kBK : a.num_kb;
        J = a.live_k ? a.J : (int64_t)live;
        tiles_j = (uint32_t)((J + a.bt - 1) / a.bt);
        shares = a.shares ? (uint32_t)*a.shares : 1u;
        total = (uint32_t)a.tiles_i * tiles_j * shares;
        if (parts > 1)
            share_of(num_kb, part, parts, kb0, num_kb);
    }
    __device__ __forceinline__ void start(const LinearArgs &a, uint32_t first_)
    {
        first = first_;
        if (first < total)
            tile = live_tile(a, first);
    }
    __device__ __forceinline__ Tile live_tile(const LinearArgs &a, uint32_t t) const
    {
        if (shares == 1) {
            Tile c = tile_at(a, tiles_j, t);
            c.kb0 = kb0;
            c.num_kb = num_kb;
            return c;
        }
        const uint32_t tiles = (uint32_t)a.tiles_i * tiles_j, share = t / tiles;
        Tile c = tile_at(a, tiles_j, t - share * tiles);
        c.share = (int)share;
        share_of(num_kb, (int)share, (int)shares, c.kb0, c.num_kb);
        return c;
    }
};

template <bool LIVE>
__device__ __forceinline__ Tile tile_of(const LinearArgs &a, const Product &p, uint32_t t)
{
    if constexpr (LIVE)
        return p.live_tile(a, t);
    return tile_at(a, (uint32_t)a.tiles_j, t);
}
template <int EPI>
__device__ __forceinline__ int64_t columns_of(const LinearArgs &a, const Product &p)
{
    if constexpr (kLive<EPI>)
        return p.J;
    return a.J;
}
// Where a thread block stands: the same for all its roles but the fields a role moves.
struct Place {
    uint32_t base;          // shared memory, 1024-aligned
    uint8_t *smem;
    Shared *sh;
    volatile int *abort_flag;
    uint32_t tmem, rank, lead;  // position in the CTA pair; cluster rank of its leader
    int part, parts;        // pairs that share a tile's contraction
    int lane, q, group;     // epilogue: TMEM lane quarter, which of every four groups of 32 columns
    uint8_t *stage_buf;
    // a role's progress
    int stage;
    uint32_t phase;
    uint32_t unit, nunits;  // this pair (or cluster) of the grid
    int64_t count;          // k-blocks (producers), chunks (MMA issuer, epilogue)
    int half;               // which producer
    int64_t issued;         // the k-blocks it has loaded
    int64_t stall_at;       // the k-block that is not loaded (a test's), or -1
};

// Producer `half`'s loads of a product's tiles, every second k-block; false when a
// wait gave up.  A k-block's wait, expectation and two loads take a thread 450
// cycles whatever their size (570 with a warp's votes around them), as long as the
// MMAs of a 256 x 224 tile and twice those of smaller ones; so two threads share
// them, of warps of their own.
template <int BT, bool LIVE>
__device__ __forceinline__ bool produce(const CUtensorMap &map_a, const CUtensorMap &map_b, const LinearArgs &a,
                                        const Product &p, Place &at)
{
    using G = Geo<BT>;
    const uint64_t pol = ptx::policy_evict_normal();
    const uint32_t stage_bytes = 2u * (uint32_t)(kA + a.bt / 2 * kBK * 2);  // both CTAs'
    const uint32_t empty0 = ptx::smem_addr(at.sh->empty), full0 = ptx::smem_addr(at.sh->full);
    const uint32_t bar0 = map_to_rank(full0, at.lead);  // both CTAs' loads
    Tile c = p.tile;
    for (uint32_t t = p.first; t < p.total;) {
        const int i0 = c.ti * kTileI + (int)at.rank * 128;
        const int j0 = c.tj * a.bt + (int)at.rank * (a.bt / 2);
        const int skip = (int)(at.count + at.half) & 1;  // the other producer's
        const int num_kb = LIVE ? c.num_kb : p.num_kb;
        int k0 = ((LIVE ? c.kb0 : p.kb0) + skip) * kBK;
        for (int kb = skip; kb < num_kb; kb += 2, k0 += 2 * kBK) {
            const uint32_t bar_at = (uint32_t)at.stage * 8;
            if (!role_wait(empty0 + bar_at, at.phase ^ 1u, a.wait_limit_ns, at.abort_flag))
                return false;
            if (at.count + kb != at.stall_at) {  // test hook: the first stage is never armed
                if (at.rank == 0)
                    mbar_expect(full0 + bar_at, stage_bytes);
                const uint32_t sa = at.base + at.stage * G::kStage;
                load_operand<2>(sa, &map_a, a.a_mn, 128, i0, k0, bar0 + bar_at, pol);
                load_operand<2>(sa + kA, &map_b, a.b_mn, a.bt / 2, j0, k0, bar0 + bar_at, pol);
            }
            ++at.issued;
            if ((at.stage += 2) >= G::kStages) {
                at.stage -= G::kStages;
                at.phase ^= 1u;
            }
        }
        at.count += num_kb;
        t += at.nunits;
        if (t < p.total)
            c = tile_of<LIVE>(a, p, t);
    }
    return true;
}

// The MMA issuer's share of the same.
template <int BT, bool LIVE>
__device__ __forceinline__ bool multiply(const LinearArgs &a, const Product &p, Place &at, bool *issued_any)
{
    using G = Geo<BT>;
    const uint32_t idesc = instr_desc(a.is_bf16, a.a_mn, a.b_mn, 256, a.bt);
    const uint32_t step_a = (a.a_mn ? UK * 128 : UK * 2) >> 4;  // 16 k further, in descriptors
    const uint32_t step_b = (a.b_mn ? UK * 128 : UK * 2) >> 4;
    const uint32_t lo_a = desc_lo(at.base, a.a_mn ? kMnBox : 16);
    const uint32_t lo_b = desc_lo(at.base + kA, a.b_mn ? kMnBox : 16);
    const uint32_t empty0 = ptx::smem_addr(at.sh->empty), full0 = ptx::smem_addr(at.sh->full);
    const uint16_t both = (uint16_t)(3u << at.lead);
    for (uint32_t t = p.first; t < p.total; t += at.nunits) {
        int in_chunk = 0;
        const int num_kb = LIVE ? p.live_tile(a, t).num_kb : p.num_kb;
        for (int kb = 0; kb < num_kb; ++kb) {
            const int acc = (int)(at.count & 1);  // chunks issued so far: accumulator count & 1
            if (in_chunk == 0 &&
                !role_wait(ptx::smem_addr(&at.sh->tmem_empty[acc]), (uint32_t)((at.count >> 1) & 1) ^ 1u,
                           a.wait_limit_ns, at.abort_flag))
                return false;
            if (!role_wait(full0 + (uint32_t)at.stage * 8, at.phase, a.wait_limit_ns, at.abort_flag))
                return false;
            fence_after();
            const uint32_t stage_at = (uint32_t)(at.stage * G::kStage) >> 4;
#pragma unroll
            for (int k = 0; k < kBK / UK; ++k)
                mma_f16<2>(at.tmem + (uint32_t)(acc * BT), lo_a + stage_at + k * step_a,
                           lo_b + stage_at + k * step_b, idesc, (uint32_t)(in_chunk | k));
            mma_commit_to(empty0 + (uint32_t)at.stage * 8, both);
            *issued_any = true;
            ++in_chunk;
            if (in_chunk == a.chunk || kb + 1 == num_kb) {
                mma_commit_to(ptx::smem_addr(&at.sh->tmem_full[acc]), both);
                ++at.count;
                in_chunk = 0;
            }
            if (++at.stage == G::kStages) {
                at.stage = 0;
                at.phase ^= 1u;
            }
        }
    }
    return true;
}

// The log-sum's epilogue of a tile: each warp its 32 entries, then the four of a group their 128, of this
// group's kCols columns (every fourth 32).  logits(col, v) gives columns col .. col + 15 of them; it is called
// twice where the piece's exponentials are kept.
template <int kCols, typename Logits>
__device__ __forceinline__ void log_sums(const LinearArgs &a, const Place &at, int64_t i0, int64_t j0, int64_t end,
                                         const TokenTerms *terms, Logits logits)
{
    const auto column = [](int u) { return u / kStageCols * 4 * kStageCols + u % kStageCols; };
    const int lane = at.lane;
    float2 own[kCols / 16];
#pragma unroll
    for (int col = 0; col < kCols; col += 16) {
        const int64_t jc = j0 + column(col);
        const int n = valid16(end, jc);
        if (n <= 0)
            continue;
        float v[16];
        logits(col, v);
        const int target = __shfl_sync(0xffffffffu, terms[col / kStageCols].target, (lane & 15) + col % kStageCols);
        own[col / 16] = lse16(a, i0, jc, n, lane, target, v, at.stage_buf);
    }
    if (a.kept && i0 >= a.kept0 && i0 < a.I) {
        // the last piece's exponentials, from the largest of each 32: the gradient of its logits needs no
        // second product
#pragma unroll
        for (int g = 0; g < kCols; g += kStageCols) {
            const int64_t jg = j0 + column(g);
            const int n = valid_rows(end, jg);
            if (n <= 0)
                continue;
#pragma unroll
            for (int c = 0; c < kStageCols; c += 16) {
                if (c >= n)
                    continue;
                const float m = own[(g + c) / 16].x;
                const float from = m == -INFINITY ? 0.0f : m;
                if (lane < 16 && c + lane < n)
                    a.kept_top[(i0 - a.kept0) / 32 * a.ldpartial + jg + c + lane] = m;
                float v[16];
                logits(g + c, v);
#pragma unroll
                for (int u = 0; u < 16; u += 2) {
                    const float2 e = above(v[u], v[u + 1], __shfl_sync(0xffffffffu, from, u),
                                           __shfl_sync(0xffffffffu, from, u + 1));
                    *staged(at.stage_buf, lane, c + u) = kept_code(e.x) | kept_code(e.y) << 16;
                }
            }
            write_rows(rows_of(a.kept, a.ldkept), a.I - a.kept0, i0 - a.kept0, jg, n, lane, at.stage_buf);
        }
    }
    float2 *mine = reinterpret_cast<float2 *>(at.stage_buf);
#pragma unroll
    for (int col = 0; col < kCols; col += 16)
        if (lane < 16)
            mine[col + lane] = own[col / 16];
    group_sync(at.group);
    // warp q finishes a quarter of the columns
    constexpr int kEach = kCols / 4;
    const int col = at.q * kEach + lane;
    const int64_t j = j0 + column(col);
    if (lane < kEach && j < end) {
        const uint8_t *first = at.stage_buf - ((at.q + 2) & 3) * kWarpStage;  // q = (2, 3, 0, 1)
        float2 x[4];
        float m = -INFINITY, s = 0.0f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            x[k] = reinterpret_cast<const float2 *>(first + k * kWarpStage)[col];
            m = fmaxf(m, x[k].x);
        }
        const float from = m == -INFINITY ? 0.0f : m;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            s += x[k].y * ex2_approx((x[k].x - from) * kLog2e);
        const int64_t row = (i0 - at.q * 32) / 128;
        if (row * 128 < a.I)
            a.partial[row * a.ldpartial + j] = make_float2(m, s);
    }
    group_sync(at.group);
}

// An epilogue warp's share of the same.
template <int EPI, int BT>
__device__ __forceinline__ bool finish(const LinearArgs &a, const Product &p, Place &at)
{
    // This warp's columns: every fourth group of 32, so that tiles of fewer tokens
    // leave no warp two groups while another has none.
    constexpr int kCols = BT / 4;
    constexpr int kGroups = kCols / kStageCols;
    constexpr int kStep = 4 * kStageCols;
    const int lane = at.lane;
    const uint32_t t_lane = at.tmem + ((uint32_t)(at.q * 32) << 16) + (uint32_t)(at.group * kStageCols);
    const uint32_t empty0 = map_to_rank(ptx::smem_addr(&at.sh->tmem_empty[0]), at.lead);
    float *partial = reinterpret_cast<float *>(at.smem) + at.group * kStageCols * 128 + at.q * 32 + lane;
    const Rows aux = aux_of<EPI>(a);
    const bool early = aux.p != nullptr && at.parts == 1;
    int chunks = kLive<EPI> ? 0 : (p.num_kb + a.chunk - 1) / a.chunk;
    const auto column = [](int u) { return u / kStageCols * kStep + u % kStageCols; };
    for (uint32_t t = p.first; t < p.total; t += at.nunits) {
        const Tile c = tile_of<kLive<EPI>>(a, p, t);
        if (kLive<EPI>)
            chunks = (c.num_kb + a.chunk - 1) / a.chunk;
        const int64_t i0 = (int64_t)c.ti * kTileI + (int)at.rank * 128 + at.q * 32;
        const int64_t j0 = (int64_t)c.tj * a.bt + at.group * kStageCols;
        // the first token that is not this tile's
        const int64_t end = gg_min64(columns_of<EPI>(a, p), (int64_t)(c.tj + 1) * a.bt);
        // each share has rows of its own
        const int64_t row0 = kScaled<EPI> ? c.share * a.J : 0;
        const float bias = EPI == kEpiForward ? load_bias(a, i0 + lane) : 0.0f;
        uint4 pre[kRowSteps];
        if (!kSums<EPI> && early)  // the first group's rows, while the MMAs run
            read_aux<EPI>(a, aux, i0, row0 + j0, valid_rows(end, j0), lane, pre);
        TokenTerms terms[kGroups];
        if constexpr (kLogSum<EPI> || EPI == kEpiSoftGrad) {
#pragma unroll
            for (int g = 0; g < kGroups; ++g)
                terms[g] = terms_of<EPI>(a, j0 + g * kStep, valid_rows(end, j0 + g * kStep), lane);
        }
        float sum[kSums<EPI> ? kCols : 1];
        if constexpr (kSums<EPI>) {
#pragma unroll
            for (int u = 0; u < kCols; ++u)
                sum[u] = 0.0f;
        }
        for (int h = 0; h < chunks; ++h, ++at.count) {
            const int acc = (int)(at.count & 1);
            const bool got = role_wait(ptx::smem_addr(&at.sh->tmem_full[acc]),
                                       (uint32_t)((at.count >> 1) & 1), a.wait_limit_ns, at.abort_flag);
            // (the warps of a group meet below: they give up together)
            if (kLogSum<EPI> ? !group_agrees(at.group, got) : !__all_sync(0xffffffffu, got))
                return false;
            fence_after();
            const uint32_t t_addr = t_lane + (uint32_t)(acc * BT);
            const auto from_tmem = [&](int col, float(&v)[16]) {
                uint32_t r[16];
                tmem_ld16(t_addr + (uint32_t)col, r);
                tmem_wait16(r);
#pragma unroll
                for (int u = 0; u < 16; ++u)
                    v[u] = __uint_as_float(r[u]);
            };
            if (EPI == kEpiLse && h + 1 == chunks) {  // the last chunk straight from TMEM
                log_sums<kCols>(a, at, i0, j0, end, terms, [&](int col, float(&v)[16]) {
                    from_tmem(column(col), v);
#pragma unroll
                    for (int u = 0; u < 16; ++u)
                        v[u] += sum[kSums<EPI> ? col + u : 0];
                });
            } else if constexpr (kSums<EPI>) {
#pragma unroll
                for (int col = 0; col < kCols; col += 16) {
                    if (valid_rows(end, j0 + column(col)) <= 0)
                        continue;
                    float v[16];
                    from_tmem(column(col), v);
#pragma unroll
                    for (int u = 0; u < 16; ++u)
                        sum[col + u] += v[u];
                }
            } else if (at.parts > 1) {  // every load and MMA of this CTA is done: the ring is free
#pragma unroll 1
                for (int col = 0; col < kCols; col += 16) {
                    float v[16];
                    from_tmem(column(col), v);
#pragma unroll
                    for (int u = 0; u < 16; ++u)
                        partial[(column(col) + u) * 128] = v[u];
                }
            } else if constexpr (EPI == kEpiLseShort) {
                log_sums<kCols>(a, at, i0, j0, end, terms, [&](int col, float(&v)[16]) { from_tmem(column(col), v); });
            } else if (kShort<EPI> && a.out_f32) {
#pragma unroll 1
                for (int col = 0; col < kCols; col += 16) {
                    const int64_t jc = j0 + column(col);
                    const int n = valid16(end, jc);
                    if (n <= 0)
                        continue;
                    float v[16];
                    from_tmem(column(col), v);
                    emit16<EPI>(a, i0 + lane, row0 + jc, 1, n, v, 0.0f);
                }
            } else {
#pragma unroll 1
                for (int g = 0; g < kGroups; ++g) {
                    const int64_t jg = j0 + g * kStep;
                    if (valid_rows(end, jg) <= 0)
                        break;
                    emit_rows<EPI>(a, i0, row0 + jg, valid_rows(end, jg), lane, bias, early, pre, at.stage_buf,
                                   [&](int col, float(&v)[16]) { from_tmem(g * kStep + col, v); },
                                   terms[kGroups > 1 && g > 0 ? kGroups - 1 : 0]);
                    if (early && g + 1 < kGroups)
                        read_aux<EPI>(a, aux, i0, row0 + jg + kStep, valid_rows(end, jg + kStep), lane, pre);
                }
            }
            // accumulator read: hand it back to the leader's MMA warp
            fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive_cluster(empty0 + (uint32_t)(acc * sizeof(uint64_t)));
        }
        if constexpr (EPI == kEpiVocabShort) {
            if (chunks == 0 && at.parts > 1) {  // no token counts, or none in this share: zeros
#pragma unroll 1
                for (int u = 0; u < kCols; ++u)
                    partial[column(u) * 128] = 0.0f;
            } else if (chunks == 0) {
#pragma unroll 1
                for (int col = 0; col < kCols; col += 16) {
                    float v[16] = {};
                    const int64_t jc = j0 + column(col);
                    emit16<EPI>(a, i0 + lane, row0 + jc, 1, valid16(end, jc), v, 0.0f);
                }
            }
        }
        if constexpr (kSums<EPI> && EPI != kEpiLse) {
            if (at.parts > 1) {
#pragma unroll
                for (int u = 0; u < kCols; ++u)
                    partial[column(u) * 128] = sum[u];
            } else if (a.out_f32) {
#pragma unroll
                for (int col = 0; col < kCols; col += 16) {
                    float v[16];
#pragma unroll
                    for (int u = 0; u < 16; ++u)
                        v[u] = sum[col + u];
                    const int64_t jc = j0 + column(col);
                    emit16<EPI>(a, i0 + lane, row0 + jc, 1, valid16(end, jc), v, 0.0f);
                }
            } else {
#pragma unroll
                for (int g = 0; g < kGroups; ++g) {
                    const int64_t jg = j0 + g * kStep;
                    emit_rows<EPI, true>(a, i0, row0 + jg, valid_rows(end, jg), lane, 0.0f, early, pre, at.stage_buf,
                                   [&](int col, float(&v)[16]) {
#pragma unroll
                                       for (int u = 0; u < 16; ++u)
                                           v[u] = sum[g * kStageCols + col + u];
                                   });
                }
            }
        }
        __syncwarp();
    }
    return true;
}

// The end of a split tile: the pairs' partial tiles, added in order.  Pair `part`
// finishes columns [part, part + 1) * BT / parts, its CTAs their own 128 features.
template <int EPI, int BT>
__device__ __forceinline__ void join_parts(const LinearArgs &a, const Product &p, Place &at)
{
    const int lane = at.lane, parts = at.parts;
    if (kLive<EPI> && at.unit >= p.total)
        return;
    const Tile c = tile_of<kLive<EPI>>(a, p, at.unit);
    // 16 columns a warp at least: with 32 left for a pair, half the warps finish them
    const int cols = BT / parts >= 64 ? BT / parts / 4 : 16;
    const int col0 = at.part * (BT / parts) + at.group * cols;
    const int64_t i0 = (int64_t)c.ti * kTileI + (int)at.rank * 128 + at.q * 32;
    const int64_t j0 = (int64_t)c.tj * BT + col0;
    const int64_t left = columns_of<EPI>(a, p) - j0;
    const int n = at.group * cols >= BT / parts ? 0 : (left > cols ? cols : (left > 0 ? (int)left : 0));
    const float bias = EPI == kEpiForward ? load_bias(a, i0 + lane) : 0.0f;
    const uint32_t mine = at.base + (uint32_t)((col0 * 128 + at.q * 32 + lane) * 4);
    const auto joined = [&](int col, float(&v)[16], int have = 16) {  // `have` columns are used
#pragma unroll
        for (int h = 0; h < 16; h += 8) {
            float x[4][8];  // every pair's sums, all loads in flight
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const uint32_t from = 2 * (uint32_t)(s < parts ? s : 0) + at.rank;
                const uint32_t src = map_to_rank(mine, from) + (uint32_t)(col + h) * 512;
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    x[s][u] = s < parts && h + u < have ? ld_cluster_f32(src + (uint32_t)u * 512) : 0.0f;
            }
#pragma unroll
            for (int u = 0; u < 8; ++u)
                v[h + u] = (x[0][u] + x[1][u]) + (x[2][u] + x[3][u]);
        }
    };
    if (kOwn<EPI> && a.out_f32) {
        // nothing is read past the last feature or token: reads that no store waits for
        // could outlive the CTA (the staged rows below store all that they read)
#pragma unroll 1
        for (int col = 0; col < n && i0 < a.I; col += 16) {
            float v[16];
            const int have = n - col < 16 ? n - col : 16;
            joined(col, v, have);
            emit16<EPI>(a, i0 + lane, j0 + col, 1, have, v, 0.0f);
        }
    } else if (n > 0) {
        const Rows aux = aux_of<EPI>(a);
        uint4 pre[kRowSteps];
        if (aux.p)
            read_aux<EPI>(a, aux, i0, j0, n, lane, pre);
        emit_rows<EPI>(a, i0, j0, n, lane, bias, aux.p != nullptr, pre, at.stage_buf, joined);
    }
}
}  // namespace pair

// A cluster is one CTA pair that walks its share of the tiles, or, when tiles
// are few, 2 or 4 pairs that split one tile's contraction.  With a second product
// (EPI1 >= 0: a layer's input and weight gradients, which both read dZ), its
// tiles follow the first one's in the same walk: one launch, one last wave, and
// small products side by side.
template <int EPI, int EPI1, int BT>
__global__ void __launch_bounds__(pair::kThreads, 1)
    pair_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                const __grid_constant__ LinearArgs a, const __grid_constant__ CUtensorMap map_a1,
                const __grid_constant__ CUtensorMap map_b1, const __grid_constant__ LinearArgs a1)
{
    using G = pair::Geo<BT>;
    constexpr bool kTwo = EPI1 >= 0;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_addr(smem_raw);
    pair::Place at;
    at.base = (raw + 1023u) & ~1023u;  // 1024-aligned for the 128B swizzle
    at.smem = smem_raw + (at.base - raw);
    at.sh = reinterpret_cast<Shared *>(at.smem + G::kOffShared);
    at.abort_flag = &at.sh->abort_flag;
    Shared &sh = *at.sh;

    const int warp = threadIdx.x >> 5;
    // Set-up first, the rest of the arithmetic under it: all of it is on the way of
    // every call (with 64-bit divisions ahead of it, the barriers stood after 1300
    // cycles and the first load went out 2600 cycles later).
    if (threadIdx.x == 0) {
        for (int s = 0; s < G::kStages; ++s) {
            ptx::mbar_init(ptx::smem_addr(&sh.full[s]), 1);
            ptx::mbar_init(ptx::smem_addr(&sh.empty[s]), 1);
        }
        for (int s = 0; s < 2; ++s) {
            ptx::mbar_init(ptx::smem_addr(&sh.tmem_full[s]), 1);
            ptx::mbar_init(ptx::smem_addr(&sh.tmem_empty[s]), 2 * pair::kEpiWarps);
        }
        ptx::mbar_init(ptx::smem_addr(&sh.mma_done), 1);
        sh.abort_flag = 0;
        ptx::fence_barrier_init();
    }
    if (threadIdx.x == 0) {
        prefetch_tensormap(&map_a);
        prefetch_tensormap(&map_b);
        if (kTwo) {
            prefetch_tensormap(&map_a1);
            prefetch_tensormap(&map_b1);
        }
    }
    if (warp == 1) {
        tmem_alloc<2>(ptx::smem_addr(&sh.tmem_base), 2 * BT);
        fence_before();
    }
    const uint32_t crank = cluster_ctarank();
    at.lane = threadIdx.x & 31;
    at.rank = crank & 1u;
    at.lead = crank & ~1u;
    at.parts = kTwo ? 1 : (int)cluster_size() / 2;
    at.part = kTwo ? 0 : (int)crank / 2;
    at.unit = cluster_id_x();
    at.nunits = ncluster_x();
    at.q = warp & 3;
    at.group = (warp - 2) >> 2;
    at.stage_buf = at.smem + G::kOffStage + (warp >= 2 ? warp - 2 : 0) * kWarpStage;  // of an epilogue warp
    at.half = warp == pair::kProducer2 ? 1 : 0;
    at.stage = at.half;
    at.phase = 0;
    at.count = 0;
    at.issued = 0;
    at.stall_at = a.inject_stall && at.unit == 0 && at.part == 0 ? 0 : -1;
    pair::Product p, p1;
    if constexpr (!kLive<EPI>) {
        p = pair::Product(a, at.part, at.parts, at.unit);
        // the second product's walk goes on where the first ended
        const uint32_t at1 = at.unit + (at.unit < (uint32_t)a1.skip ? at.nunits : 0u) - (uint32_t)a1.skip;
        p1 = pair::Product(kTwo ? a1 : a, at.part, at.parts, kTwo ? at1 : 0u);
    }
    __syncthreads();
    cluster_meet();  // the peer's barriers exist before anything signals them
    fence_after();
    at.tmem = sh.tmem_base;
    wait_dependencies();  // what earlier launches write is there from here on
    launch_dependents();
    if constexpr (kLive<EPI>) {
        p.count(a, at.part, at.parts);
        p.start(a, at.unit);
        if constexpr (kTwo) {
            const uint32_t skip = p.total % at.nunits;
            p1.count(a1, at.part, at.parts);
            p1.start(a1, at.unit + (at.unit < skip ? at.nunits : 0u) - skip);
        }
    }

    bool ok = true;
    if (warp == 0 || warp == pair::kProducer2) {
        // ===================== producers (a thread each) ====================
        if (ptx::elect_one_sync()) {
            ok = pair::produce<BT, kLive<EPI>>(map_a, map_b, a, p, at);
            if (kTwo && ok)
                ok = pair::produce<BT, kLive<EPI>>(map_a1, map_b1, a1, p1, at);
            if (!ok) {
                *at.abort_flag = 1;
                report_status(a.status, kStatusTimeout);
            }
            // drain: every load this thread issued has landed before the CTA may exit
            if (at.rank == 0) {
                for (int64_t d = 0; d < G::kStages / 2 && d < at.issued; ++d) {
                    const int64_t idx = at.half + 2 * (at.issued - 1 - d);
                    ptx::mbar_wait(ptx::smem_addr(&sh.full[idx % G::kStages]),
                                   (uint32_t)((idx / G::kStages) & 1), kDrainLimitNs);
                }
            }
            // The other CTA's loads complete on the leader's barriers, and where either gave up
            // the leader need not have armed them, nor waited for them: let them land.
            if (!ok)
                sleep_ns(200000);
        }
    } else if (warp == 1) {
        // ===================== MMA issuer (one thread of the leader CTA) ====
        if (at.rank == 0 && ptx::elect_one_sync()) {
            bool issued_any = false;
            ok = pair::multiply<BT, kLive<EPI>>(a, p, at, &issued_any);
            if (kTwo && ok)
                ok = pair::multiply<BT, kLive<EPI>>(a1, p1, at, &issued_any);
            if (!ok) {
                *at.abort_flag = 1;
                report_status(a.status, kStatusTimeout);
            }
            // drain: all its MMAs have completed before TMEM is freed
            if (issued_any) {
                mma_commit_local<2>(ptx::smem_addr(&sh.mma_done));
                ptx::mbar_wait(ptx::smem_addr(&sh.mma_done), 0, kDrainLimitNs);
            }
        }
    } else {
        // ===================== epilogue (warps 2-17) ========================
        ok = pair::finish<EPI, BT>(a, p, at);
        if constexpr (kTwo) {
            if (ok)
                ok = pair::finish<EPI1, BT>(a1, p1, at);
        }
        if (!ok) {
            *at.abort_flag = 1;
            report_status(a.status, kStatusTimeout);
        }
    }

    __syncwarp();
    if constexpr (!kTwo) {
        if (at.parts > 1) {
            cluster_sync();
            if constexpr (!kLogSum<EPI> && EPI != kEpiSoftGrad) {  // (these do not split tiles)
                if (warp >= 2 && warp < pair::kProducer2 && ok)
                    pair::join_parts<EPI, BT>(a, p, at);
            }
            __syncwarp();
        }
    }

    // ---- teardown ---------------------------------------------------------------
    fence_before();
    // The leader's MMAs into the peer's TMEM and smem are done, and partials read: each value
    // has gone into a store.
    cluster_meet();
    if (warp == 1) {
        fence_after();
        tmem_dealloc<2>(at.tmem, 2 * BT);
    }
}

// ---- split kernel: 128 features x BT tokens per cluster ------------------------------
namespace split {
constexpr int kProducer2 = 6;   // warps: producer, MMA, 4 epilogue, second producer
constexpr int kThreads = 224;
constexpr int kA = 128 * kBK * 2;
template <int BT>
struct Geo {
    static constexpr int kB = BT * kBK * 2;
    static constexpr int kStage = kA + kB;
    // about 100 KB of ring, so that two CTAs share an SM; even: a producer has its own stages
    static constexpr int kStages = BT == 16 ? 6 : 4;
    static constexpr int kRing = kStages * kStage;
    static constexpr int kPartial = 128 * BT * 4;  // float32 partial tile, over the spent ring
    static constexpr int kTmemCols = 2 * BT;       // two accumulators (a power of two >= 32)
    static constexpr int kSmemBytes = kRing + (int)sizeof(Shared) + 1024;
    static_assert(kPartial <= kRing && kStages <= kMaxStages && kStages % 2 == 0 && 2 * (kSmemBytes + 1024) <= 233472,
                  "shared memory of a CTA");
};
}  // namespace split

template <int EPI, int BT>
__global__ void __launch_bounds__(split::kThreads, 2)
    split_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                 const __grid_constant__ LinearArgs a)
{
    using G = split::Geo<BT>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (base - raw);
    Shared &sh = *reinterpret_cast<Shared *>(smem + G::kRing);
    volatile int *abort_flag = &sh.abort_flag;

    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int s = 0; s < G::kStages; ++s) {
            ptx::mbar_init(ptx::smem_addr(&sh.full[s]), 1);
            ptx::mbar_init(ptx::smem_addr(&sh.empty[s]), 1);
        }
        for (int s = 0; s < 2; ++s) {
            ptx::mbar_init(ptx::smem_addr(&sh.tmem_full[s]), 1);
            ptx::mbar_init(ptx::smem_addr(&sh.tmem_empty[s]), 4);
        }
        ptx::mbar_init(ptx::smem_addr(&sh.mma_done), 1);
        sh.abort_flag = 0;
        ptx::fence_barrier_init();
    }
    if (threadIdx.x == 0) {
        prefetch_tensormap(&map_a);
        prefetch_tensormap(&map_b);
    }
    if (warp == 1) {
        tmem_alloc<1>(ptx::smem_addr(&sh.tmem_base), G::kTmemCols);
        fence_before();
    }
    const int lane = threadIdx.x & 31;
    const int rank = (int)cluster_ctarank();
    const int parts = (int)cluster_size();
    const uint32_t tile = cluster_id_x();
    const int tj = (int)(tile / (uint32_t)a.tiles_i);
    const int ti = (int)(tile - (uint32_t)tj * (uint32_t)a.tiles_i);
    int kb0, kb1;
    int64_t J = a.J;
    if constexpr (!kLive<EPI>) {
        share_of(a.num_kb, rank, parts, kb0, kb1);
        kb1 += kb0;
    }
    __syncthreads();
    fence_after();
    const uint32_t tmem = sh.tmem_base;
    wait_dependencies();
    launch_dependents();
    if constexpr (kLive<EPI>) {  // (a tile past the last token multiplies zeros or stale rows, and writes nothing)
        const int live = *a.live;
        share_of(a.live_k ? (live + kBK - 1) / kBK : a.num_kb, rank, parts, kb0, kb1);
        kb1 += kb0;
        if (!a.live_k)
            J = live;
    }

    const int q = warp & 3;  // epilogue: TMEM lane quarter
    const int64_t i = (int64_t)ti * 128 + q * 32 + lane;
    const int64_t jt = (int64_t)tj * BT;
    const float bias = EPI == kEpiForward && warp >= 2 ? load_bias(a, i) : 0.0f;
    bool ok = true;

    if (warp == 0 || warp == split::kProducer2) {
        // ===================== producers (a thread each, see pair) ==========
        if (ptx::elect_one_sync()) {
            const uint64_t pol = ptx::policy_evict_normal();
            const uint32_t empty0 = ptx::smem_addr(sh.empty), full0 = ptx::smem_addr(sh.full);
            const int half = warp == 0 ? 0 : 1;
            const bool stall = a.inject_stall && tile == 0 && rank == 0 && half == 0;
            int stage = half;
            uint32_t phase = 0;
            int issued = 0;
            for (int kb = kb0 + half; kb < kb1; kb += 2) {
                const uint32_t bar = full0 + (uint32_t)stage * 8;
                if (!role_wait(empty0 + (uint32_t)stage * 8, phase ^ 1u, a.wait_limit_ns, abort_flag)) {
                    ok = false;
                    break;
                }
                if (!stall || issued > 0) {  // test hook: the first stage is never armed
                    mbar_expect(bar, G::kStage);
                    const uint32_t sa = base + stage * G::kStage;
                    load_operand<1>(sa, &map_a, a.a_mn, 128, ti * 128, kb * kBK, bar, pol);
                    load_operand<1>(sa + split::kA, &map_b, a.b_mn, BT, tj * BT, kb * kBK, bar, pol);
                }
                ++issued;
                if ((stage += 2) >= G::kStages) {
                    stage -= G::kStages;
                    phase ^= 1u;
                }
            }
            if (!ok) {
                *abort_flag = 1;
                report_status(a.status, kStatusTimeout);
            }
            for (int d = 0; d < G::kStages / 2 && d < issued; ++d) {
                const int idx = half + 2 * (issued - 1 - d);
                ptx::mbar_wait(ptx::smem_addr(&sh.full[idx % G::kStages]),
                               (uint32_t)((idx / G::kStages) & 1), kDrainLimitNs);
            }
        }
    } else if (warp == 1) {
        // ===================== MMA issuer (one thread) ======================
        if (ptx::elect_one_sync()) {
            const uint32_t idesc = instr_desc(a.is_bf16, a.a_mn, a.b_mn, 128, BT);
            const uint32_t step_a = (a.a_mn ? UK * 128 : UK * 2) >> 4;
            const uint32_t step_b = (a.b_mn ? UK * 128 : UK * 2) >> 4;
            const uint32_t lo_a = desc_lo(base, a.a_mn ? kMnBox : 16);
            const uint32_t lo_b = desc_lo(base + split::kA, a.b_mn ? kMnBox : 16);
            const uint32_t empty0 = ptx::smem_addr(sh.empty), full0 = ptx::smem_addr(sh.full);
            int stage = 0;
            uint32_t phase = 0;
            int nchunk = 0, in_chunk = 0;
            for (int kb = kb0; kb < kb1; ++kb) {
                const int acc = nchunk & 1;
                bool got = true;
                if (in_chunk == 0)
                    got = role_wait(ptx::smem_addr(&sh.tmem_empty[acc]), (uint32_t)((nchunk >> 1) & 1) ^ 1u,
                                    a.wait_limit_ns, abort_flag);
                got = got && role_wait(full0 + (uint32_t)stage * 8, phase, a.wait_limit_ns, abort_flag);
                if (!got) {
                    ok = false;
                    break;
                }
                fence_after();
                const uint32_t at = (uint32_t)(stage * G::kStage) >> 4;
#pragma unroll
                for (int k = 0; k < kBK / UK; ++k)
                    mma_f16<1>(tmem + (uint32_t)(acc * BT), lo_a + at + k * step_a,
                               lo_b + at + k * step_b, idesc, (uint32_t)(in_chunk | k));
                mma_commit_local<1>(empty0 + (uint32_t)stage * 8);
                ++in_chunk;
                if (in_chunk == a.chunk || kb + 1 == kb1) {
                    mma_commit_local<1>(ptx::smem_addr(&sh.tmem_full[acc]));
                    ++nchunk;
                    in_chunk = 0;
                }
                if (++stage == G::kStages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            if (!ok) {
                *abort_flag = 1;
                report_status(a.status, kStatusTimeout);
            }
            if (nchunk + in_chunk > 0) {
                mma_commit_local<1>(ptx::smem_addr(&sh.mma_done));
                ptx::mbar_wait(ptx::smem_addr(&sh.mma_done), 0, kDrainLimitNs);
            }
        }
    } else {
        // ===================== epilogue (warps 2-5) =========================
        const uint32_t t_lane = tmem + ((uint32_t)(q * 32) << 16);
        float *partial = reinterpret_cast<float *>(smem) + q * 32 + lane;  // [column][feature]
        uint8_t *stage_buf = smem + q * kWarpStage;  // over the spent ring, like partial
        const int64_t i0 = i - lane;
        const Rows aux = aux_of<EPI>(a);
        uint4 pre[kRowSteps];
        const int chunks = (kb1 - kb0 + a.chunk - 1) / a.chunk;
        float sum[kSums<EPI> ? BT : 1];
        if constexpr (kSums<EPI>) {
#pragma unroll
            for (int u = 0; u < BT; ++u)
                sum[u] = 0.0f;
        }
        for (int h = 0; h < chunks; ++h) {
            const int acc = h & 1;
            const bool got = role_wait(ptx::smem_addr(&sh.tmem_full[acc]), (uint32_t)((h >> 1) & 1),
                                       a.wait_limit_ns, abort_flag);
            if (!__all_sync(0xffffffffu, got)) {
                ok = false;
                break;
            }
            fence_after();
            if constexpr (kSums<EPI>) {
#pragma unroll
                for (int c16 = 0; c16 < BT / 16; ++c16) {
                    uint32_t r[16];
                    tmem_ld16(t_lane + (uint32_t)(acc * BT + c16 * 16), r);
                    tmem_wait16(r);
#pragma unroll
                    for (int u = 0; u < 16; ++u)
                        sum[c16 * 16 + u] += __uint_as_float(r[u]);
                }
            } else {  // one chunk: every load and MMA of this CTA is done, the ring is free
#pragma unroll 1
                for (int c16 = 0; c16 < BT / 16; ++c16) {
                    uint32_t r[16];
                    tmem_ld16(t_lane + (uint32_t)(acc * BT + c16 * 16), r);
                    tmem_wait16(r);
                    if (parts == 1)
                        break;
#pragma unroll
                    for (int u = 0; u < 16; ++u)
                        partial[(c16 * 16 + u) * 128] = __uint_as_float(r[u]);
                }
#pragma unroll 1
                for (int g = 0; parts == 1 && g < BT; g += kStageCols) {
                    const int n = valid_rows(J, jt + g) < BT - g ? valid_rows(J, jt + g) : BT - g;
                    if (aux.p)
                        read_aux<EPI>(a, aux, i0, jt + g, n, lane, pre);
                    emit_rows<EPI>(a, i0, jt + g, n, lane, bias, aux.p != nullptr, pre, stage_buf,
                                [&](int col, float(&v)[16]) {
                                    uint32_t r[16];
                                    tmem_ld16(t_lane + (uint32_t)(acc * BT + g + col), r);
                                    tmem_wait16(r);
#pragma unroll
                                    for (int u = 0; u < 16; ++u)
                                        v[u] = __uint_as_float(r[u]);
                                },
                                terms_of<EPI>(a, jt + g, n, lane));
                }
            }
            fence_before();
            __syncwarp();
            if (lane == 0)
                ptx::mbar_arrive(ptx::smem_addr(&sh.tmem_empty[acc]));
        }
        if constexpr (kSums<EPI>) {
            if (ok) {  // past the last chunk every load and MMA of this CTA is done
                if (parts > 1) {
#pragma unroll
                    for (int u = 0; u < BT; ++u)
                        partial[u * 128] = sum[u];
                } else if (EPI == kEpiLse || a.out_f32) {
#pragma unroll
                    for (int c16 = 0; c16 < BT / 16; ++c16) {
                        float v[16];
#pragma unroll
                        for (int u = 0; u < 16; ++u)
                            v[u] = sum[c16 * 16 + u];
                        emit16<EPI>(a, i, jt + c16 * 16, 1, valid16(J, jt + c16 * 16), v, 0.0f);
                    }
                } else {
#pragma unroll
                    for (int g = 0; g < BT; g += kStageCols) {
                        const int n = valid_rows(J, jt + g);
                        emit_rows<EPI, true>(a, i0, jt + g, n, lane, 0.0f, aux.p != nullptr, pre, stage_buf,
                                       [&](int col, float(&v)[16]) {
#pragma unroll
                                           for (int u = 0; u < 16; ++u)
                                               v[u] = sum[g + col + u];
                                       });
                    }
                }
            }
        }
        if (!ok) {
            *abort_flag = 1;
            report_status(a.status, kStatusTimeout);
        }
    }

    __syncwarp();
    if (parts > 1) {
        // the cluster's partial tiles, added in rank order; CTA `rank` takes
        // columns rank, rank + parts, ...
        cluster_sync();
        // A warp whose features all lie past the end reads nothing: it would use none of
        // it, and could leave, and let the others leave, with its reads in flight.
        if (warp >= 2 && warp < split::kProducer2 && ok && i - lane < a.I) {
            const uint32_t mine = base + (uint32_t)(q * 32 + lane) * 4;
            const int64_t left = J - jt;  // valid columns of the tile
            const int cols = left < BT ? (int)left : BT;
            // Columns at a time: as many as a CTA of a full cluster has, up to 4.  This is
            // code that runs once, and what it costs is mostly its fetching: with 4 instead
            // of 2 for 16-token tiles, one token took 12.6 us instead of 12.35, 27 tokens 5.35
            // instead of 5.1; with 1, 12.3 and 5.4.
            constexpr int C = BT == 16 ? 2 : 4;
#pragma unroll 1
            for (int c0 = rank; c0 < cols; c0 += C * parts) {
                const int n = (cols - c0 + parts - 1) / parts;
                float x[8][C];  // every CTA's sums of C columns, all loads in flight
#pragma unroll
                for (int s = 0; s < 8; ++s) {
                    const uint32_t src = map_to_rank(mine, (uint32_t)(s < parts ? s : 0));
#pragma unroll
                    for (int u = 0; u < C; ++u)
                        x[s][u] = s < parts && u < n
                                      ? ld_cluster_f32(src + (uint32_t)(c0 + u * parts) * 512)
                                      : 0.0f;
                }
                float v[16] = {};
#pragma unroll
                for (int s = 0; s < 8; ++s)
#pragma unroll
                    for (int u = 0; u < C; ++u)
                        v[u] += x[s][u];
                emit16<EPI, C>(a, i, jt + c0, parts, n < C ? n : C, v, bias);
            }
        }
        __syncwarp();
        // No CTA leaves while its partial tile may still be read: every value read above has
        // gone into a store (a barrier that orders the reads waits for those stores as well,
        // 0.15 to 0.3 us of a product).
        cluster_meet();
    }
    fence_before();
    __syncthreads();
    if (warp == 1) {
        fence_after();
        tmem_dealloc<1>(tmem, G::kTmemCols);
    }
}

// ---- an empty contraction: the epilogue of zero sums ------------------------------------
template <int EPI>
__global__ void __launch_bounds__(256) empty_kernel(const __grid_constant__ LinearArgs a)
{
    const int64_t blocks_i = (a.I + 31) / 32;
    const int64_t groups = blocks_i * ((a.J + 15) / 16);
    const int64_t step = (int64_t)gridDim.x * 8;
    for (int64_t g = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); g < groups; g += step) {
        const int64_t i = (g % blocks_i) * 32 + (threadIdx.x & 31);
        const int64_t j0 = g / blocks_i * 16;
        float v[16] = {};
        const int64_t J = kLive<EPI> && !a.live_k ? (int64_t)*a.live : a.J;
        emit16<EPI>(a, i, j0, 1, valid16(J, j0), v, load_bias(a, i));
    }
}

// ---- column sums (bias gradient) -----------------------------------------------------
// A cluster of kSumParts CTAs owns 64 columns; its CTAs split the rows and
// each reads whole 128-byte row pieces (4 columns per thread, 8 rows at a
// time), sums in registers, joins its 8 row groups by shuffles and in shared
// memory and the cluster's 8 sums through distributed shared memory, in a fixed
// order.  Bound: the read of dZ.
//
// After the products of the same call it runs beside them (a.beside): a CTA fits
// next to one of theirs (19 warps of 96 registers leave a quarter of an SM 1024
// registers, a warp's 32, and 225 KB of shared memory leave 0.8), and it need not
// wait for them.  It may start once every CTA of theirs has passed its own wait
// for the launches before, so what dZ and dbias hold is there; and one of its CTAs
// waits for them before it ends, so that whoever waits for this launch has waited
// for those.  All three gradients of 777 tokens, K = 1523, N = 1000: one after the
// other 17.5 us, side by side 14.7; of 4096 tokens, K = 8192, N = 3584: 289 us with
// 54 registers a thread, which do not fit, and 278 side by side.
constexpr int kSumParts = 8;
constexpr int kSumThreads = 128;
constexpr int kSumRows = kSumThreads / 16;  // rows at a time

template <bool BF16>
__global__ void __launch_bounds__(kSumThreads, 16)
    colsum_kernel(const __grid_constant__ ColSumArgs a)
{
    __shared__ float part[2][64];
    if (!a.beside) {
        wait_dependencies();
        launch_dependents();
    }
    const int rank = (int)cluster_ctarank();
    const int64_t i0 = (int64_t)cluster_id_x() * 64;
    const int c = threadIdx.x & 15, warp = threadIdx.x >> 5;
    const int64_t col = i0 + c * 4;
    float s[4] = {};
    if (col < a.I) {
        const int64_t row0 = a.J * rank / kSumParts + threadIdx.x / 16;
        int64_t n = (a.J * (rank + 1) / kSumParts - row0 + kSumRows - 1) / kSumRows;
        const int64_t step = kSumRows * a.ldx;
        const uint16_t *x = reinterpret_cast<const uint16_t *>(a.x) + row0 * a.ldx + col;
        if (col + 4 > a.I) {  // nothing is read past a row's end: behind the last there may be none
            for (; n > 0; --n, x += step)
                for (int u = 0; u < 3; ++u)
                    s[u] += col + u < a.I ? load16(x, u, BF16) : 0.0f;
        }
#pragma unroll 4
        for (; n > 0; --n, x += step) {
            const uint2 w = __ldcg(reinterpret_cast<const uint2 *>(x));
            if (BF16) {
                s[0] += __uint_as_float(w.x << 16);
                s[1] += __uint_as_float(w.x & 0xffff0000u);
                s[2] += __uint_as_float(w.y << 16);
                s[3] += __uint_as_float(w.y & 0xffff0000u);
            } else {
                const float2 f0 = __half22float2(*reinterpret_cast<const __half2 *>(&w.x));
                const float2 f1 = __half22float2(*reinterpret_cast<const __half2 *>(&w.y));
                s[0] += f0.x;
                s[1] += f0.y;
                s[2] += f1.x;
                s[3] += f1.y;
            }
        }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)  // the warp's two rows
        s[u] += __shfl_xor_sync(~0u, s[u], 16);
    if (warp >= 2 && (threadIdx.x & 16) == 0) {
#pragma unroll
        for (int u = 0; u < 4; ++u)
            part[warp - 2][c * 4 + u] = s[u];
    }
    __syncthreads();
    if (warp < 2 && (threadIdx.x & 16) == 0) {
#pragma unroll
        for (int u = 0; u < 4; ++u)
            part[warp][c * 4 + u] += s[u];
    }
    __syncwarp();
    cluster_sync();
    const int64_t i = i0 + threadIdx.x;
    if (rank == 0 && threadIdx.x < 64 && i < a.I) {
        float t = 0.0f;
        for (int p = 0; p < kSumParts; ++p) {
            t += ld_cluster_f32(map_to_rank(ptx::smem_addr(&part[0][threadIdx.x]), (uint32_t)p));
            t += ld_cluster_f32(map_to_rank(ptx::smem_addr(&part[1][threadIdx.x]), (uint32_t)p));
        }
        if (a.out_f32) {
            float *o = reinterpret_cast<float *>(a.out) + i;
            *o = a.accumulate ? *o + t : t;
        } else {
            store16(a.out, i, a.accumulate ? load16(a.out, i, BF16) + t : t, BF16);
        }
    }
    __syncwarp();
    cluster_sync();
    if (a.beside && i0 == 0 && rank == 0)
        wait_dependencies();
}

// ---- activation backward: dz = dy * act'(z) --------------------------------------------
// V elements per thread and step (8: 16-byte accesses when every pointer and
// pitch allows them, else 1).  Bound: two reads and a write of HBM.
template <int V>
__global__ void __launch_bounds__(256) act_backward_kernel(const __grid_constant__ ActBackwardArgs a)
{
    const int64_t units = (a.N + V - 1) / V;
    const int64_t total = a.M * units;
    const int64_t step = (int64_t)gridDim.x * blockDim.x;
    for (int64_t t = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; t < total; t += step) {
        const int64_t m = t / units, n = (t - m * units) * V;
        const uint16_t *dy = reinterpret_cast<const uint16_t *>(a.dy) + m * a.lddy + n;
        const uint16_t *z = reinterpret_cast<const uint16_t *>(a.z) + m * a.ldz + n;
        uint16_t *dz = reinterpret_cast<uint16_t *>(a.dz) + m * a.lddz + n;
        uint16_t hy[V], hz[V];
        const bool whole = n + V <= a.N;
        if (V == 8 && whole) {
            *reinterpret_cast<uint4 *>(hy) = *reinterpret_cast<const uint4 *>(dy);
            *reinterpret_cast<uint4 *>(hz) = *reinterpret_cast<const uint4 *>(z);
        } else {
#pragma unroll
            for (int u = 0; u < V; ++u) {
                hy[u] = n + u < a.N ? dy[u] : (uint16_t)0;
                hz[u] = n + u < a.N ? z[u] : (uint16_t)0;
            }
        }
        constexpr int C = V < 2 ? 2 : V;
        float v[C] = {}, x[C] = {};
#pragma unroll
        for (int u = 0; u < V; ++u) {
            v[u] = load16(hy, u, a.is_bf16);
            x[u] = load16(hz, u, a.is_bf16);
        }
        with_act(a.act, [&](auto k) { apply_slope<decltype(k)::value>(v, x); });
#pragma unroll
        for (int u = 0; u < V; ++u)
            store16(hy, u, v[u], a.is_bf16);
        if (V == 8 && whole) {
            *reinterpret_cast<uint4 *>(dz) = *reinterpret_cast<const uint4 *>(hy);
        } else {
#pragma unroll
            for (int u = 0; u < V; ++u)
                if (n + u < a.N)
                    dz[u] = hy[u];
        }
    }
}

// ---- host ----------------------------------------------------------------------------
constexpr int kMaxDevices = 64;

int current_device()
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices)
        dev = 0;
    return dev;
}

// Dynamic shared memory of a kernel, set once per device.
template <typename K>
cudaError_t allow_smem(K kernel, int bytes, std::once_flag *once, cudaError_t *result)
{
    const int dev = current_device();
    std::call_once(once[dev], [&] {
        result[dev] = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    });
    return result[dev];
}

bool operand_map(CUtensorMap *map, const LinearArgs &a, const void *p, int64_t rows, int64_t ld, int mn,
                 uint32_t box_rows)
{
    const CUtensorMapDataType dt =
        a.is_bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    const uint64_t strides[1] = {(uint64_t)ld * 2};
    if (mn) {
        const uint64_t dims[2] = {(uint64_t)rows, (uint64_t)a.K};
        const uint32_t box[2] = {64, kBK};
        return encode_map(map, dt, 2, p, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
    }
    const uint64_t dims[2] = {(uint64_t)a.K, (uint64_t)rows};
    const uint32_t box[2] = {kBK, box_rows};
    return encode_map(map, dt, 2, p, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

// A launch in clusters of `size`, allowed to start while the launch before it on
// the stream finishes (the kernels wait for it after their own set-up).
struct ClusterLaunch {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    ClusterLaunch(int size, int64_t grid, int threads, int smem, cudaStream_t s)
    {
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = (unsigned)size;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[1].val.programmaticStreamSerializationAllowed = 1;
        cfg.gridDim = dim3((unsigned)grid, 1, 1);
        cfg.blockDim = dim3((unsigned)threads, 1, 1);
        cfg.dynamicSmemBytes = (size_t)smem;
        cfg.stream = s;
        cfg.attrs = attr;
        cfg.numAttrs = 2;
    }
};

// One product, or two (args1, with bt1) in one walk.
template <int EPI, int EPI1, int BT>
cudaError_t launch_pair(const LinearArgs &args, int bt, int parts, const LinearArgs *args1, int bt1, cudaStream_t s,
                        const char **why)
{
    using G = pair::Geo<BT>;
    static std::once_flag once[kMaxDevices], once_res[kMaxDevices];
    static cudaError_t result[kMaxDevices];
    static int resident_by_dev[kMaxDevices];
    cudaError_t e = allow_smem(pair_kernel<EPI, EPI1, BT>, G::kSmemBytes, once, result);
    if (e != cudaSuccess) {
        *why = "setting the shared-memory size of the linear kernel";
        return e;
    }
    const int dev = current_device();
    std::call_once(once_res[dev], [&] {
        int resident = 0;
        ClusterLaunch l(2, 2, pair::kThreads, G::kSmemBytes, nullptr);
        l.cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&resident, pair_kernel<EPI, EPI1, BT>, &l.cfg) != cudaSuccess)
            resident = 0;
        (void)cudaGetLastError();
        resident_by_dev[dev] = resident;
    });
    CUtensorMap maps[4];
    LinearArgs a[2] = {args, args1 ? *args1 : args};
    a[0].bt = bt;
    a[1].bt = args1 ? bt1 : bt;
    int64_t tiles = 0;
    for (int k = 0; k < (args1 ? 2 : 1); ++k) {
        LinearArgs &x = a[k];
        if (!operand_map(&maps[2 * k], x, x.a, x.I, x.lda, x.a_mn, 128) ||
            !operand_map(&maps[2 * k + 1], x, x.b, x.J, x.ldb, x.b_mn, (uint32_t)x.bt / 2)) {
            *why = "encoding the operands' tensor maps";
            return cudaErrorInvalidValue;
        }
        const int64_t tiles_i = (x.I + pair::kTileI - 1) / pair::kTileI, tiles_j = (x.J + x.bt - 1) / x.bt;
        // feature tiles in equal groups of at most 8: 76 pairs cover about 8 x 9 tiles
        const int64_t groups = (tiles_i + 7) / 8;
        x.group = (int)((tiles_i + groups - 1) / groups);
        x.tiles_i = (int)tiles_i;
        x.tiles_j = (int)tiles_j;
        x.num_kb = (int)((x.K + kBK - 1) / kBK);
        tiles += tiles_i * tiles_j * (x.shares ? x.most_shares : 1);
    }
    if (tiles >= 1ll << 31) {
        *why = "more than 2^31 tiles";
        return cudaErrorInvalidValue;
    }
    if (!args1) {
        maps[2] = maps[0];
        maps[3] = maps[1];
    }
    const int resident = resident_by_dev[dev] > 0 ? resident_by_dev[dev] : kSMs / 2;
    // split tiles: one cluster each; whole ones: the pairs that fit walk them
    const int64_t clusters = parts > 1 ? tiles : gg_min64(resident, tiles);
    a[1].skip = (int)((int64_t)a[0].tiles_i * a[0].tiles_j % clusters);
    ClusterLaunch l(2 * parts, 2 * parts * clusters, pair::kThreads, G::kSmemBytes, s);
    return cudaLaunchKernelEx(&l.cfg, pair_kernel<EPI, EPI1, BT>, maps[0], maps[1], a[0], maps[2], maps[3], a[1]);
}

template <int EPI, int BT>
cudaError_t launch_split(const LinearArgs &args, int parts, cudaStream_t s, const char **why)
{
    using G = split::Geo<BT>;
    static std::once_flag once[kMaxDevices];
    static cudaError_t result[kMaxDevices];
    cudaError_t e = allow_smem(split_kernel<EPI, BT>, G::kSmemBytes, once, result);
    if (e != cudaSuccess) {
        *why = "setting the shared-memory size of the linear kernel";
        return e;
    }
    CUtensorMap map_a, map_b;
    LinearArgs a = args;
    if (!operand_map(&map_a, a, a.a, a.I, a.lda, a.a_mn, 128) ||
        !operand_map(&map_b, a, a.b, a.J, a.ldb, a.b_mn, BT)) {
        *why = "encoding the operands' tensor maps";
        return cudaErrorInvalidValue;
    }
    a.tiles_i = (int)((a.I + 127) / 128);
    a.tiles_j = (int)((a.J + BT - 1) / BT);
    a.num_kb = (int)((a.K + kBK - 1) / kBK);
    const int64_t tiles = (int64_t)a.tiles_i * a.tiles_j;
    ClusterLaunch l(parts, tiles * parts, split::kThreads, G::kSmemBytes, s);
    return cudaLaunchKernelEx(&l.cfg, split_kernel<EPI, BT>, map_a, map_b, a);
}

// Logits of longer contractions than kPlainLse are summed in chunks for lse, which holds all tokens' losses
// together within 1.2e-6 of their size.  Measured against float64 (600 tokens, V = 4000, logits of deviation 2.5;
// bfloat16, float16): in one chunk 5.3e-7, 6.4e-7 at 1024, 8.1e-7, 9.7e-7 at 1536, 9.8e-7, 1.14e-6 at kPlainLse, and on
// with the length; in chunks of 1024 4.7e-7 to 6.3e-7 at 1800 to 8192; a float32 product 1e-7 to 4e-7.  In registers the sums of chunks
// spill, which only tiles of long contractions hide: 4096 tokens, 100003 entries, K = 1024 take 570 us with and 460
// without, the product of 777 tokens, 32768 entries, K = 2011 90 and 65.
constexpr int64_t kPlainLse = 1792;
constexpr int kLseChunk = 16;  // k-blocks

// Whether a gradient's sum over tokens stays in one chunk: where it is no longer, and where a vocabulary's
// weight gradient is rounded to 16 bits at the end (truncation costs 2e-5 of it at kPlainTokens, float16's
// half step is 2.4e-4).  64 sums a thread leave the epilogue too few registers, which the products of a long
// contraction hide and those of a short one do not: the 32768 x 2048 gradient of 64 tokens takes 59 us with
// them and 35 without, of 576, 76 and 57.
constexpr int64_t kPlainTokens = 16384;
bool one_chunk(int epi, const LinearArgs &a)
{
    return a.K <= kChunk * kBK || (epi == kEpiVocab && a.live_k && !a.out_f32 && a.K <= kPlainTokens);
}

template <int EPI>
cudaError_t launch_epi(const LinearArgs &a, const LinearPlan &p, cudaStream_t s, const char **why)
{
    if constexpr (EPI != kEpiSoftGrad && EPI != kEpiVocab) {  // (these are called for a contraction only)
        if (a.K == 0) {
            const int64_t groups = ((a.I + 31) / 32) * ((a.J + 15) / 16);
            empty_kernel<EPI><<<(int)gg_min64((groups + 7) / 8, kSMs * 8), 256, 0, s>>>(a);
            return cudaGetLastError();
        }
    }
    if (p.kernel == GG_LINEAR_PAIR) {
        if constexpr (EPI == kEpiGradW || EPI == kEpiVocab || EPI == kEpiLse) {
            constexpr int kBrief =
                EPI == kEpiGradW ? kEpiGradWShort : (EPI == kEpiVocab ? kEpiVocabShort : kEpiLseShort);
            if (EPI == kEpiLse ? a.K <= kPlainLse : one_chunk(EPI, a))
                return p.bt > 128 ? launch_pair<kBrief, -1, 256>(a, p.bt, p.split, nullptr, 0, s, why)
                                  : launch_pair<kBrief, -1, 128>(a, p.bt, p.split, nullptr, 0, s, why);
        }
        return p.bt > 128 ? launch_pair<EPI, -1, 256>(a, p.bt, p.split, nullptr, 0, s, why)
                          : launch_pair<EPI, -1, 128>(a, p.bt, p.split, nullptr, 0, s, why);
    }
    switch (p.bt) {
    case 16:
        if constexpr (EPI != kEpiGradW && EPI != kEpiVocab)
            return launch_split<EPI, 16>(a, p.split, s, why);
        break;
    case 32:
        if constexpr (EPI != kEpiGradW && EPI != kEpiVocab)
            return launch_split<EPI, 32>(a, p.split, s, why);
        break;
    case 64: return launch_split<EPI, 64>(a, p.split, s, why);
    }
    *why = "no such tile";
    return cudaErrorInvalidValue;
}

}  // namespace

// Everybody's operands of a k-block through the L2 cache, in nanoseconds.
static double l2_ns(bool lines, double ctas, double bytes)
{
    return ctas * bytes / (lines ? 15950.0 : 9950.0);
}

// A k-block of a pair's 256 x bt tile, `ctas` at work: its operands through the SM's
// port (its MMAs take as long at 256 tokens, less below), the ring's latency, or L2.
static double pair_kb_ns(int bt, bool lines, double ctas)
{
    const double bytes = (128 + bt / 2) * kBK * 2;
    const double port = bytes / 117.8, l2 = l2_ns(lines, ctas, bytes);
    const double kb = port > l2 ? port : l2;
    return kb > 110.7 ? kb : 110.7;
}

// Launch, set-up and first load of a pair, and its epilogue.
static double pair_ns(int bt) { return 1724.0 + 23.2 * bt; }

// Whether the operands' pitches keep their rows on 128-byte lines.  Where they do not,
// each row of a tile touches two lines: with pitches of 1008 and 1024 elements, 768
// tokens, 1536 features and K = 1000 take 8.6 and 6.4 us.  The addresses stay out of it:
// the same values elsewhere have to be summed in the same order.
static bool on_lines(const LinearArgs &a) { return ((a.lda | a.ldb) * 2 & 127) == 0; }

// Which kernel, tile and split: the one of least estimated time, in nanoseconds.
// The estimate is a launch and its set-up, then waves x k-blocks x the time of a
// k-block, then the epilogue.  Its constants were fitted to 2300 timings of both
// kernels (weights of 512 x 512 to 8192 x 3584, 1 to 4096 tokens, pitches on and off
// 128-byte lines, every tile and split, forward and both gradients): the choice is
// on average 1.4 % slower than the best of them, 15 % at most.
LinearPlan plan_linear(int epi, const LinearArgs &a, int path)
{
    LinearPlan best{GG_LINEAR_NONE, 0, 0, 0.0};
    const int64_t I = a.I, J = a.J, K = a.K;
    if (I <= 0 || J <= 0 || K <= 0)
        return best;
    const bool lines = on_lines(a);
    const int64_t num_kb = (K + kBK - 1) / kBK;
    const auto offer = [&](int kernel, int bt, int parts, double ns) {
        if (best.kernel == GG_LINEAR_NONE || ns < best.ns)
            best = LinearPlan{kernel, bt, parts, ns};
    };
    for (int bt = epi == kEpiGradW || epi == kEpiVocab ? 64 : 16; path != GG_LINEAR_PAIR && bt <= 64; bt *= 2) {
        const int64_t tiles = ((I + 127) / 128) * ((J + bt - 1) / bt);
        for (int parts = 1; parts <= 8 && parts <= num_kb; ++parts) {
            const int64_t ctas = tiles * parts;
            if (parts > 1 && ctas > 2 * kSMs)
                break;
            const double here = ctas < 2 * kSMs ? (double)ctas : 2.0 * kSMs;
            const double per_sm = here <= kSMs ? 1.0 : here / kSMs;
            const double waves = (double)((ctas + 2 * kSMs - 1) / (2 * kSMs));
            const double bytes = (128 + bt) * kBK * 2;
            const double latency = 122.3 + 0.867 * bt, port = per_sm * bytes / 91.5, l2 = l2_ns(lines, here, bytes);
            double kb = latency > port ? latency : port;
            kb = kb > l2 ? kb : l2;
            offer(GG_LINEAR_SPLIT, bt, parts,
                  2360.0 + (parts > 1 ? 912.0 : 0.0) + waves * (double)((num_kb + parts - 1) / parts) * kb +
                      (waves - 1.0) * 1328.0 + bt * 40.4);
        }
    }
    // an MN-major operand is loaded 64 columns at a time by each CTA of a pair
    const int step = a.b_mn ? 128 : 32;
    for (int bt = a.b_mn ? 128 : 64; path != GG_LINEAR_SPLIT && bt <= 256; bt += step) {
        const int64_t tiles = ((I + 255) / 256) * ((J + bt - 1) / bt);
        const int most = epi == kEpiLse || epi == kEpiSoftGrad ? 1 : 4;  // they join no partial tiles
        for (int parts = 1; parts <= most && parts <= num_kb; parts *= 2) {
            // pairs, and clusters of 4 and 8 CTAs, that are resident at once
            const int64_t room = parts == 1 ? 76 : (parts == 2 ? 36 : 14);
            if (parts > 1 && (tiles > room || (bt != 128 && bt != 256)))
                break;
            const double waves = (double)((tiles + room - 1) / room);
            const double ctas = 2.0 * parts * (double)(tiles < room ? tiles : room);
            offer(GG_LINEAR_PAIR, bt, parts,
                  pair_ns(bt / parts) + (parts > 1 ? 3021.0 : 0.0) +
                      waves * (double)((num_kb + parts - 1) / parts) * pair_kb_ns(bt, lines, ctas) +
                      (waves - 1.0) * 272.0);
        }
    }
    return best;
}

// The tiles of both gradients of a layer in one walk of the pairs, where that is
// estimated to end before the two products one after the other: side by side when
// all tiles fit one wave, else with one launch and one last wave less (apart and
// together: 19.0 and 14.2 us for 777 tokens, K = 1523, N = 1000; 298 and 289 us for
// 4096 tokens, K = 8192, N = 3584).
bool plan_both(const LinearArgs &dx, const LinearArgs &dw, const LinearPlan &plan_dx, const LinearPlan &plan_dw,
               int path, int *bt_dx, int *bt_dw)
{
    if (path == GG_LINEAR_SPLIT || dx.K <= 0 || dw.K <= 0)
        return false;
    const auto tiles = [](const LinearArgs &x, int bt) { return ((x.I + 255) / 256) * ((x.J + bt - 1) / bt); };
    const auto kbs = [](const LinearArgs &x) { return (double)((x.K + kBK - 1) / kBK); };
    const bool lines_dx = on_lines(dx), lines_dw = on_lines(dw);
    double least = path == GG_LINEAR_PAIR ? 1e300 : plan_dx.ns + plan_dw.ns;
    bool found = false;
    for (int b0 = 64; b0 <= 256; b0 += 32)
        for (int b1 = 128; b1 <= 256; b1 += 128) {
            const int64_t t0 = tiles(dx, b0), t1 = tiles(dw, b1);
            const double ctas = 2.0 * (double)(t0 + t1 < 76 ? t0 + t1 : 76);
            const double w0 = kbs(dx) * pair_kb_ns(b0, lines_dx, ctas) + 196.0;
            const double w1 = kbs(dw) * pair_kb_ns(b1, lines_dw, ctas) + 196.0;
            // waves of tiles; a walk of both kinds ends with either
            double ns = 0.0;
            if (t0 + t1 <= 76)
                ns = w0 > w1 ? w0 : w1;
            else
                ns = ((double)t0 * w0 + (double)t1 * w1) / 76.0 + 0.695 * (w0 < w1 ? w0 : w1);
            ns += pair_ns(b0 > b1 ? b0 : b1);
            if (ns < least) {
                least = ns;
                *bt_dx = b0;
                *bt_dw = b1;
                found = true;
            }
        }
    return found;
}

template <int EPI, int EPI1>
static cudaError_t launch_both_of(const LinearArgs &x, int bt_dx, const LinearArgs &w, int bt_dw, cudaStream_t s,
                                  const char **why)
{
    return bt_dx > 128 || bt_dw > 128 ? launch_pair<EPI, EPI1, 256>(x, bt_dx, 1, &w, bt_dw, s, why)
                                      : launch_pair<EPI, EPI1, 128>(x, bt_dx, 1, &w, bt_dw, s, why);
}

// The products that the gradient of a piece's logits goes into, in one walk of the pairs: dX's tiles are few
// and long (its contraction is the piece), dW's many and short.  A pair with one long tile more than the others
// would end long after them, so a long contraction is dealt out in shares (up to most_shares; how many, the
// device decides when it has counted the tokens), each into float32 rows of its own; the walk deals tiles in
// turn, so three pairs show the last to end.  Tiles whose contraction is shorter than their epilogue take the
// epilogue's time.  777 tokens, 544 of which count, V = 32768, K = 2011: 160 us in one share, 123 in four.
bool plan_vocab(const LinearArgs &dx, const LinearArgs &dw, double other_ns, int most_shares, int *bt_dx, int *bt_dw)
{
    const auto tiles = [](const LinearArgs &x, int bt) { return ((x.I + 255) / 256) * ((x.J + bt - 1) / bt); };
    const auto tile_ns = [](double kbs, double kb_ns, int bt) {
        const double ns = kbs * kb_ns, epilogue = 23.2 * bt;
        return (ns > epilogue ? ns : epilogue) + 196.0;
    };
    const int64_t kb0 = (dx.K + kBK - 1) / kBK, kb1 = (dw.K + kBK - 1) / kBK;
    const bool lines_dx = on_lines(dx), lines_dw = on_lines(dw);
    double least = other_ns;
    bool found = false;
    for (int b0 = 64; b0 <= 256; b0 += 32)
        for (int b1 = 128; b1 <= 256; b1 += 128)
            for (int s = 1; s <= most_shares && s <= kb0; s += s < 4 ? 1 : 2) {
                const int64_t n0 = tiles(dx, b0) * s, n1 = tiles(dw, b1);
                const double ctas = 2.0 * (double)(n0 + n1 < 76 ? n0 + n1 : 76);
                const double w0 = tile_ns((double)((kb0 + s - 1) / s), pair_kb_ns(b0, lines_dx, ctas), b0);
                const double w1 = tile_ns((double)kb1, pair_kb_ns(b1, lines_dw, ctas), b1);
                double ns = 0.0;
                for (const int64_t u : {(int64_t)0, n0 % 76, (n0 + 75) % 76}) {
                    const int64_t c0 = u < n0 ? (n0 - u + 75) / 76 : 0;
                    const int64_t all = u < n0 + n1 ? (n0 + n1 - u + 75) / 76 : 0;
                    const double here = (double)c0 * w0 + (double)(all - c0) * w1;
                    ns = here > ns ? here : ns;
                }
                ns += pair_ns(b0 > b1 ? b0 : b1);
                if (ns < least) {
                    least = ns;
                    *bt_dx = b0;
                    *bt_dw = b1;
                    found = true;
                }
            }
    return found;
}

cudaError_t launch_both(int epi, const LinearArgs &dx, int bt_dx, const LinearArgs &dw, int bt_dw, cudaStream_t s,
                        const char **why)
{
    if (!tensor_maps_available()) {
        *why = "cuTensorMapEncodeTiled is not available";
        return cudaErrorNotSupported;
    }
    LinearArgs x = dx, w = dw;
    const bool brief = one_chunk(epi == kEpiVocab ? kEpiVocab : kEpiGradW, w);
    x.chunk = epi == kEpiVocab ? kChunk : 1 << 30;
    w.chunk = brief ? 1 << 30 : kChunk;
    switch (epi) {
    case kEpiVocab:
        return brief ? launch_both_of<kEpiVocab, kEpiVocabShort>(x, bt_dx, w, bt_dw, s, why)
                     : launch_both_of<kEpiVocab, kEpiVocab>(x, bt_dx, w, bt_dw, s, why);
    case kEpiGradIn8:
        return brief ? launch_both_of<kEpiGradIn8, kEpiGradWShort>(x, bt_dx, w, bt_dw, s, why)
                     : launch_both_of<kEpiGradIn8, kEpiGradW>(x, bt_dx, w, bt_dw, s, why);
    default:
        return brief ? launch_both_of<kEpiGradIn, kEpiGradWShort>(x, bt_dx, w, bt_dw, s, why)
                     : launch_both_of<kEpiGradIn, kEpiGradW>(x, bt_dx, w, bt_dw, s, why);
    }
}

cudaError_t launch_linear(int epi, const LinearArgs &args, const LinearPlan &p, cudaStream_t s,
                          const char **why)
{
    if (args.I == 0 || args.J == 0)
        return cudaSuccess;
    if (args.K > 0 && !tensor_maps_available()) {
        *why = "cuTensorMapEncodeTiled is not available";
        return cudaErrorNotSupported;
    }
    LinearArgs a = args;
    a.chunk = (epi == kEpiGradW || epi == kEpiVocab) && !one_chunk(epi, a) ? kChunk : 1 << 30;
    if (epi == kEpiLse && a.K > kPlainLse)
        a.chunk = kLseChunk;
    switch (epi) {
    case kEpiForward: return launch_epi<kEpiForward>(a, p, s, why);
    case kEpiGradIn: return launch_epi<kEpiGradIn>(a, p, s, why);
    case kEpiGradIn8: return launch_epi<kEpiGradIn8>(a, p, s, why);
    case kEpiLse: return launch_epi<kEpiLse>(a, p, s, why);
    case kEpiSoftGrad: return launch_epi<kEpiSoftGrad>(a, p, s, why);
    case kEpiVocab: return launch_epi<kEpiVocab>(a, p, s, why);
    default: return launch_epi<kEpiGradW>(a, p, s, why);
    }
}

cudaError_t launch_colsum(const ColSumArgs &a, cudaStream_t s)
{
    ClusterLaunch l(kSumParts, (a.I + 63) / 64 * kSumParts, kSumThreads, 0, s);
    return cudaLaunchKernelEx(&l.cfg, a.is_bf16 ? colsum_kernel<true> : colsum_kernel<false>, a);
}

cudaError_t launch_act_backward(const ActBackwardArgs &a, cudaStream_t s)
{
    const uint64_t bits = reinterpret_cast<uint64_t>(a.dy) | reinterpret_cast<uint64_t>(a.z) |
                          reinterpret_cast<uint64_t>(a.dz) |
                          (uint64_t)((a.lddy | a.ldz | a.lddz) * 2);
    const bool wide = bits % 16 == 0;
    const int64_t total = a.M * (wide ? (a.N + 7) / 8 : a.N);
    const int grid = (int)gg_min64((total + 255) / 256, kSMs * 8);
    if (wide)
        act_backward_kernel<8><<<grid, 256, 0, s>>>(a);
    else
        act_backward_kernel<1><<<grid, 256, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace gg
