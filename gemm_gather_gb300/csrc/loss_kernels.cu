// The clipped policy loss with its gradient, from the logits, for sm_103a.
//
// A row of logits x (scaled by the inverse temperature) becomes
//     logp = x[a] - log sum exp x,     dlogits = k (onehot(a) - softmax(x)),
// with k = weight * grad_scale * inv_temperature * dloss/dlogp known as soon as
// logp is: so one launch reads a row, reduces it to its maximum and sum of
// exponentials in one pass (each thread rescales its running sum when its
// maximum grows), and writes the gradient.  Powers of two: exp(x - max) =
// 2^((x - max) c), c = inv_temperature * log2(e); the difference comes first, so
// a large common offset of a row's logits, up to the type's lowest value in
// every place, costs no precision (x c - max c would lose 2^-24 |max| c).  Sums
// are float32.
//
// A cluster of CTAs owns a row, each CTA a slice, and the CTAs exchange
// (maximum, sum) through distributed shared memory.
// Bound: HBM, one read and one write of the logits.  Measured: 8191 x 32768
// float32 with a tenth of the tokens masked in 310 us (97 % of the copy rate),
// 4096 x 100003 bfloat16 with a quarter masked in 250 us (85 %; twice the powers a
// byte, instructions issue in 57 % of the cycles, and the passes' ends are not all
// covered by the SM's other CTA); 16 x 8192 in 5.4 us, which is two launches.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <mutex>

#include "f32x2.cuh"
#include "gg_internal.h"
#include "gg_ops.h"
#include "tc.cuh"

namespace gg {
namespace {

constexpr int kSMs = 152;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kInvalidArg = GG_ERR_INVALID_ARG;
constexpr uint64_t kDrainLimitNs = 1000000000ull;

// An element type: elements of a 16-byte vector, and pairs of them in (a pair of)
// its four words.
template <typename E>
struct Elem;
template <>
struct Elem<float> {
    static constexpr int kVec = 4;
    static constexpr uint32_t kMinusInf = 0xff800000u;
    static __device__ __forceinline__ float get(float x) { return x; }
    static __device__ __forceinline__ float put(float x) { return x; }
    static __device__ __forceinline__ F2 pair(const uint32_t (&w)[4], int i)
    {
        return pair_of(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    }
    static __device__ __forceinline__ void set(uint32_t (&w)[4], int i, F2 x)
    {
        const float2 f = halves_of(x);
        w[2 * i] = __float_as_uint(f.x);
        w[2 * i + 1] = __float_as_uint(f.y);
    }
};
template <>
struct Elem<__half> {
    static constexpr int kVec = 8;
    static constexpr uint32_t kMinusInf = 0xfc00fc00u;
    static __device__ __forceinline__ float get(__half x) { return __half2float(x); }
    static __device__ __forceinline__ __half put(float x) { return __float2half_rn(x); }
    static __device__ __forceinline__ F2 pair(const uint32_t (&w)[4], int i)
    {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
        return pair_of(f.x, f.y);
    }
    static __device__ __forceinline__ void set(uint32_t (&w)[4], int i, F2 x)
    {
        const __half2 h = __float22half2_rn(halves_of(x));
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
};
template <>
struct Elem<__nv_bfloat16> {
    static constexpr int kVec = 8;
    static constexpr uint32_t kMinusInf = 0xff80ff80u;
    static __device__ __forceinline__ float get(__nv_bfloat16 x) { return __bfloat162float(x); }
    static __device__ __forceinline__ __nv_bfloat16 put(float x) { return __float2bfloat16_rn(x); }
    static __device__ __forceinline__ F2 pair(const uint32_t (&w)[4], int i)
    {
        return pair_of(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    }
    static __device__ __forceinline__ void set(uint32_t (&w)[4], int i, F2 x)
    {
        const __nv_bfloat162 h = __float22bfloat162_rn(halves_of(x));
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
};

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Maximum (of raw logits) and sum of 2^((x - max) c).  An empty sum has maximum
// -inf; -inf logits are probability 0 and never meet inf - inf.
struct Sum {
    float m, s;
};

// What is subtracted from a logit: the maximum, or 0 where there is none.
__device__ __forceinline__ float base_of(float m) { return m == -INFINITY ? 0.0f : m; }

// The factor that takes a sum from maximum `from` to a maximum no smaller
// (1 for two empty sums, whose difference is NaN).
__device__ __forceinline__ float rescale(float from, float to, float c)
{
    return ex2(fminf((from - to) * c, 0.0f));
}

__device__ __forceinline__ Sum join(Sum a, Sum b, float c)
{
    Sum r;
    r.m = fmaxf(a.m, b.m);
    r.s = a.s * rescale(a.m, r.m, c) + b.s * rescale(b.m, r.m, c);
    return r;
}

// A vector is kept as its four words: as 16-bit elements the compiler splits it
// into eight registers and packs and unpacks it at every use.
template <typename E>
struct alignas(16) Vec {
    uint32_t w[4];
    __device__ __forceinline__ void fill(uint32_t x) { w[0] = w[1] = w[2] = w[3] = x; }
};

// Keeps the compiler from carrying a vector's unpacked values from one pass over
// it to the next (twice the registers of the packed ones).
template <typename E>
__device__ __forceinline__ void stay_packed(Vec<E> &v)
{
    asm volatile("" : "+r"(v.w[0]), "+r"(v.w[1]), "+r"(v.w[2]), "+r"(v.w[3]));
}

// The larger of top and a vector's elements (NaN is passed over, and shows in the sum).
__device__ __forceinline__ float top_of(const Vec<float> &v, float top)
{
    return fmaxf(fmaxf(fmaxf(__uint_as_float(v.w[0]), __uint_as_float(v.w[1])),
                       fmaxf(__uint_as_float(v.w[2]), __uint_as_float(v.w[3]))), top);
}
__device__ __forceinline__ float top_of(const Vec<__half> &v, float top)
{
    const __half2 *h = reinterpret_cast<const __half2 *>(v.w);
    const __half2 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
    return fmaxf(fmaxf(__low2float(m), __high2float(m)), top);
}
__device__ __forceinline__ float top_of(const Vec<__nv_bfloat16> &v, float top)
{
    const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(v.w);
    const __nv_bfloat162 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
    const uint32_t b = *reinterpret_cast<const uint32_t *>(&m);
    return fmaxf(fmaxf(__uint_as_float(b << 16), __uint_as_float(b & 0xffff0000u)), top);
}

// 2^((x - m) c) of the i-th pair of a vector.
template <typename E>
__device__ __forceinline__ F2 power_of(const Vec<E> &v, int i, F2 minus_m, F2 cc)
{
    const float2 y = halves_of(mul2(add2(Elem<E>::pair(v.w, i), minus_m), cc));
    return pair_of(ex2(y.x), ex2(y.y));
}

// The sum of a vector's powers, added to `part`.
template <typename E>
__device__ __forceinline__ void add_powers(const Vec<E> &v, float m, float c, F2 (&part)[2])
{
    const F2 minus_m = pair_of(-m), cc = pair_of(c);
#pragma unroll
    for (int u = 0; u < Elem<E>::kVec / 2; ++u)
        part[u & 1] = add2(part[u & 1], power_of(v, u, minus_m, cc));
}

// One CTA's slice of a token's row, whole vectors from the input's first 16-byte
// boundary on (V is below 2^31: indices are int).
template <typename E>
struct Slice {
    const E *row;
    E *out;  // or null
    int lo, hi, v0, v1, nvec;
    bool wide;  // the output's vectors are aligned as the input's
    // The bounds of CTA `rank` of `parts`, the same for every row.
    __device__ __forceinline__ Slice(const LossArgs &a, int rank, int parts)
    {
        constexpr int VEC = Elem<E>::kVec;
        const uint32_t units = ((uint32_t)a.V + VEC - 1) / VEC;
        uint32_t each = units, more = 0;  // the first `more` have one unit more
        if (parts > 1) {
            each = units / (uint32_t)parts;
            more = units - each * (uint32_t)parts;
        }
        const uint32_t r = (uint32_t)rank, from = each * r + (r < more ? r : more);
        const uint32_t to = (from + each + (r < more ? 1u : 0u)) * VEC;
        lo = (int)(from * VEC);
        hi = to < (uint32_t)a.V ? (int)to : (int)a.V;
    }
    __device__ __forceinline__ void at(const LossArgs &a, int64_t t)
    {
        constexpr int VEC = Elem<E>::kVec;
        row = reinterpret_cast<const E *>(a.logits) + t * a.ld;
        out = a.dlogits ? reinterpret_cast<E *>(a.dlogits) + t * a.ldd : nullptr;
        const int head = (int)((16 - (reinterpret_cast<uint64_t>(row + lo) & 15)) & 15) / (int)sizeof(E);
        v0 = lo + head < hi ? lo + head : hi;
        nvec = (hi - v0) / VEC;
        v1 = v0 + nvec * VEC;
        wide = out && (reinterpret_cast<uint64_t>(out + v0) & 15) == 0;
    }
    // The ragged ends hold fewer than VEC elements each: one of either per thread.
    __device__ __forceinline__ bool has_head(int tid) const { return tid < v0 - lo; }
    __device__ __forceinline__ bool has_tail(int tid) const { return tid < hi - v1; }
    __device__ __forceinline__ const Vec<E> *vec() const { return reinterpret_cast<const Vec<E> *>(row + v0); }

    __device__ __forceinline__ void zero(int tid, int threads) const
    {
        if (!out)
            return;
        if (wide) {
            for (int i = tid; i < nvec; i += threads)
                reinterpret_cast<uint4 *>(out + v0)[i] = make_uint4(0, 0, 0, 0);
        } else {
            for (int i = v0 + tid; i < v1; i += threads)
                out[i] = Elem<E>::put(0.0f);
        }
        if (has_head(tid))
            out[lo + tid] = Elem<E>::put(0.0f);
        if (has_tail(tid))
            out[v1 + tid] = Elem<E>::put(0.0f);
    }
};

// What a token brings beside its logits.
struct Token {
    float weight, advantage, old_logp, ref_logp;
    int64_t target;
    __device__ __forceinline__ Token(const LossArgs &a, int64_t t)
    {
        const bool there = t < a.T;
        weight = there ? a.weight[t] : 0.0f;
        advantage = there ? a.advantage[t] : 0.0f;
        old_logp = there && a.old_logp ? a.old_logp[t] : 0.0f;
        ref_logp = there && a.ref_logp ? a.ref_logp[t] : 0.0f;
        target = there ? a.target[t] : -1;
    }
    __device__ __forceinline__ bool in_range(const LossArgs &a) const { return target >= 0 && target < a.V; }
    __device__ __forceinline__ bool live(const LossArgs &a) const { return weight != 0.0f && in_range(a); }
};

// What a token's logp gives: the loss terms and dloss/dlogp.
struct Terms {
    float loss, kl, clipped, ratio, slope;
};

__device__ __forceinline__ Terms terms_of(const LossArgs &a, const Token &t, float logp)
{
    Terms r;
    const float adv = t.advantage;
    r.ratio = expf(logp - (a.old_logp ? t.old_logp : logp));  // NaN for a row without a logp
    const bool over = (adv > 0.0f && r.ratio > 1.0f + a.clip_high) ||
                      (adv < 0.0f && r.ratio < 1.0f - a.clip_low);
    r.clipped = over ? 1.0f : 0.0f;
    const float held = fminf(fmaxf(r.ratio, 1.0f - a.clip_low), 1.0f + a.clip_high);
    r.loss = -(over ? held : r.ratio) * adv;
    r.slope = over ? 0.0f : -adv * r.ratio;
    r.kl = 0.0f;
    if (a.ref_logp && a.kl_coef != 0.0f) {
        const float d = t.ref_logp - logp;
        const float e = expm1f(d);  // exp(d) - d - 1 without losing it for small d
        r.kl = e - d;
        r.loss += a.kl_coef * r.kl;
        r.slope -= a.kl_coef * e;
    }
    return r;
}

// A token's gradient, from its row's sum: dlogits = coef (onehot - e / sum).
template <typename E>
struct Gradient {
    float m, c, k, coef;
    int target;
    __device__ __forceinline__ Gradient(const LossArgs &a, const Token &t, const Sum &all, float logp, float c_)
    {
        m = base_of(all.m);
        c = c_;
        coef = t.weight * terms_of(a, t, logp).slope * a.inv_temperature * a.grad_scale;
        k = -coef / all.s;
        target = (int)t.target;
    }
    // -coef softmax of an element, and of a vector in place; the target's element
    // has coef added.
    __device__ __forceinline__ E one(float x) const { return Elem<E>::put(k * ex2((x - m) * c)); }
    __device__ __forceinline__ E target_one(float x) const { return Elem<E>::put(fmaf(k, ex2((x - m) * c), coef)); }
    __device__ __forceinline__ void softmax(Vec<E> &v) const
    {
        const F2 minus_m = pair_of(-m), cc = pair_of(c), kk = pair_of(k);
#pragma unroll
        for (int u = 0; u < Elem<E>::kVec / 2; ++u)
            Elem<E>::set(v.w, u, mul2(power_of(v, u, minus_m, cc), kk));
    }
};

__device__ __forceinline__ float warp_max(float x)
{
    float y;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float warp_add(float x)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        x += __shfl_xor_sync(~0u, x, d);
    return x;
}

// Lanes' sums as one.
__device__ __forceinline__ Sum warp_join(Sum x, float c)
{
    Sum r;
    r.m = warp_max(x.m);
    r.s = warp_add(x.s * ex2((x.m - base_of(r.m)) * c));
    return r;
}

// The warps' sums of all the cluster's CTAs, from `sums` (one per warp) of each, as they
// lie in distributed shared memory: lane i takes the i-th, the (i + 32)th and so on.
__device__ __forceinline__ Sum cluster_join(const Sum *sums, int warps, int parts, int lane, float c)
{
    Sum x{-INFINITY, 0.0f};
#pragma unroll 1
    for (int i = lane; i < warps * parts; i += 32) {
        const int p = i / warps;
        const uint32_t at = tc::map_to_rank(ptx::smem_addr(sums + (i - p * warps)), (uint32_t)p);
        Sum y;
        asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(y.m), "=f"(y.s) : "r"(at) : "memory");
        x = join(x, y, c);
    }
    return warp_join(x, c);
}

__device__ __forceinline__ float logp_of(const LossArgs &a, const Sum &all, float picked)
{
    return (picked - base_of(all.m)) * a.inv_temperature - logf(all.s);
}

// Clusters walk the tokens, each CTA with its slice of the row in shared memory,
// so that a row is read from memory once.  Two passes: a running maximum and sum
// of powers over the slice; then the gradient, where each vector that has been
// used is at once replaced by the next row's (its copy runs under the rest of
// this pass and the start of the next, which waits for it batch by batch).
// A warp owns NV x 32 consecutive 16-byte vectors, a lane every 32nd of them: no
// thread waits for another's copies, and all addresses of a lane are constants
// apart.  What the kernel costs besides memory is instructions, 8 an element for
// the powers: with a test and an address computed for each vector it was 24, and
// the passes took longer than the memory; whole warps take a path without.
constexpr int kBatch = 4;  // vectors of a lane that are waited for together

// Wait for all but the newest `left` groups of this thread's copies.
__device__ __forceinline__ void wait_groups(int left)
{
    switch (left) {
    case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
    case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
    case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
    default: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
    }
}

__device__ __forceinline__ void commit_group() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// How much of a row a lane has: `have` vectors; of batches, `whole` that every lane
// of the warp has in full, `some` that any has of (the warp's vectors are dealt out
// in turn: lane 31 has the fewest, lane 0 the most).
struct Share {
    int have, whole, some;
    // a warp's vectors from `base` on, of nvec, at most NV a lane
    template <int NV>
    static __device__ __forceinline__ Share of(int nvec, int base, int lane)
    {
        const int left = nvec > base ? nvec - base : 0;
        const int least = left / 32, most = (left + 31) / 32;
        Share r;
        r.have = least + (lane < left % 32 ? 1 : 0);
        r.have = r.have < NV ? r.have : NV;
        r.whole = (least < NV ? least : NV) / kBatch;
        r.some = ((most < NV ? most : NV) + kBatch - 1) / kBatch;
        return r;
    }
};

// A lane's NB * kBatch vectors: `slot` in shared memory, in steps of 512 bytes;
// `have` of them exist (all, where FULL).  A warp skips the batches that it has none
// of: when the last warp of a row took the tests for all 16 of its vectors, the
// others waited for it (8000 x 8192 float16: 86 us, then 64).
template <typename E, int NB>
struct Lane {
    static constexpr int NV = NB * kBatch;
    uint8_t *slot;
    uint32_t slot_at;

    template <bool FULL>
    __device__ __forceinline__ void fetch(const uint8_t *from, int q, int have) const
    {
        if (FULL || q < have)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(slot_at + q * 512), "l"(from + q * 512)
                         : "memory");
    }
    __device__ __forceinline__ void fetch_all(const uint8_t *from, int have) const
    {
#pragma unroll
        for (int q = 0; q < NV; ++q) {
            fetch<false>(from, q, have);
            if (q % kBatch == kBatch - 1)
                commit_group();
        }
    }
    template <bool FULL>
    __device__ __forceinline__ void take(int q, int have, Vec<E> &v) const
    {
        if (!FULL)
            v.fill(Elem<E>::kMinusInf);
        if (FULL || q < have)
            v = *reinterpret_cast<const Vec<E> *>(slot + q * 512);
    }

    // The running maximum and sum over batch `b`.
    template <bool FULL>
    __device__ __forceinline__ void sum_batch(int b, Sum &acc, int have, float c) const
    {
        Vec<E> v[kBatch];
        float top = acc.m;
#pragma unroll
        for (int q = 0; q < kBatch; ++q) {
            take<FULL>(b * kBatch + q, have, v[q]);
            top = top_of(v[q], top);
            stay_packed(v[q]);
        }
        if (top > acc.m) {
            acc.s *= rescale(acc.m, top, c);
            acc.m = top;
        }
        F2 part[2] = {pair_of(0.0f), pair_of(0.0f)};
#pragma unroll
        for (int q = 0; q < kBatch; ++q)
            add_powers(v[q], base_of(acc.m), c, part);
        const float2 sum2 = halves_of(add2(part[0], part[1]));
        acc.s += sum2.x + sum2.y;
    }

    // All batches: those that every lane has whole without tests, none that no lane has.
    __device__ __forceinline__ void sum_up(Sum &acc, const Share &now, float c) const
    {
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            wait_groups(NB - 1 - b);
            if (b < now.whole)
                sum_batch<true>(b, acc, NV, c);
            else if (b < now.some)
                sum_batch<false>(b, acc, now.have, c);
        }
    }

    // Batch `b` of the gradient to `to`, the next row's vectors (FETCH) in its place.
    template <bool FULL, bool FETCH>
    __device__ __forceinline__ void write_batch(int b, const Gradient<E> &g, uint8_t *to, int have,
                                                const uint8_t *from, int have_next) const
    {
        Vec<E> v[kBatch];
#pragma unroll
        for (int q = 0; q < kBatch; ++q)
            take<FULL>(b * kBatch + q, have, v[q]);
#pragma unroll
        for (int q = 0; q < kBatch; ++q) {
            g.softmax(v[q]);  // uses the vector: its place is free
            if (FULL || b * kBatch + q < have)
                *reinterpret_cast<Vec<E> *>(to + (b * kBatch + q) * 512) = v[q];
            if (FETCH)
                fetch<FULL>(from, b * kBatch + q, have_next);
        }
    }

    __device__ __forceinline__ void write(const Gradient<E> &g, uint8_t *to, const Share &now, const uint8_t *from,
                                          const Share &next) const
    {
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            if (b < now.whole && b < next.whole)
                write_batch<true, true>(b, g, to, NV, from, NV);
            else if (b < now.whole && b >= next.some)
                write_batch<true, false>(b, g, to, NV, from, 0);
            else if (b < now.some || b < next.some)
                write_batch<false, true>(b, g, to, now.have, from, next.have);
            commit_group();
        }
    }
};

// What a warp sends to every CTA of the cluster: its maximum and sum; the first
// warp of the first CTA also the target's logit.
struct alignas(16) Message {
    float m, s, logit, unused;
};

// One asynchronous store of 16 bytes into CTA `to`'s shared memory, counted on its
// barrier.  Nobody waits for a fence: with a cluster barrier (release, acquire) in
// its place, each row also waited for the stores of the row before, and a quarter
// of the stall cycles were those.
__device__ __forceinline__ void send(uint32_t dst, uint32_t bar, uint32_t to, const Message &x)
{
    asm volatile(
        "st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(
            tc::map_to_rank(dst, to)),
        "r"(__float_as_uint(x.m)), "r"(__float_as_uint(x.s)), "r"(__float_as_uint(x.logit)), "r"(0),
        "r"(tc::map_to_rank(bar, to))
        : "memory");
}

template <typename E, int NB>
__global__ void __launch_bounds__(NB == 4 ? 896 : 512) policy_loss_kernel(const __grid_constant__ LossArgs a)
{
    constexpr int VEC = Elem<E>::kVec, NV = NB * kBatch;
    extern __shared__ __align__(16) uint8_t smem[];  // [warp][vector of a lane][lane], then the messages
    __shared__ uint64_t arrived[2];
    tc::launch_dependents();  // the statistics' launch
    const int parts = (int)tc::cluster_size(), rank = (int)tc::cluster_ctarank();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x / 32;
    const int64_t step = tc::ncluster_x();
    const float c = a.inv_temperature * kLog2e;
    const int first = warp * NV * 32 + lane;  // this lane's first vector of the slice
    const int count = warps * parts;
    Message *const messages = reinterpret_cast<Message *>(smem + blockDim.x * NV * 16);  // [2][count]
    Lane<E, NB> mine;
    mine.slot = smem + first * 16;
    mine.slot_at = ptx::smem_addr(mine.slot);
    if (tid < 2)
        ptx::mbar_init(ptx::smem_addr(&arrived[tid]), 1);
    ptx::fence_barrier_init();
    __syncthreads();
    tc::cluster_meet();  // every CTA's barriers are there

    // The next row: its slice, how many vectors this lane has in it (none where the
    // token is masked), its ragged ends and, in one thread of the cluster, its
    // target's logit.
    Slice<E> s(a, rank, parts), n = s;
    const uint8_t *from = nullptr;
    Share share_next{0, 0, 0};
    float xh = 0.0f, xt = 0.0f, picked = 0.0f;
    const auto look = [&](int64_t t, const Token &k) {
        n.at(a, t);
        share_next = Share{0, 0, 0};
        if (!k.live(a))
            return;
        from = reinterpret_cast<const uint8_t *>(n.vec() + first);
        share_next = Share::of<NV>(n.nvec, warp * NV * 32, lane);
        if (rank == 0 && tid == 0)
            picked = Elem<E>::get(n.row[k.target]);
        xh = n.has_head(tid) ? Elem<E>::get(n.row[n.lo + tid]) : -INFINITY;
        xt = n.has_tail(tid) ? Elem<E>::get(n.row[n.v1 + tid]) : -INFINITY;
    };

    int64_t t = tc::cluster_id_x();
    Token now(a, t), next(a, t + step);
    look(t, now);
    mine.fetch_all(from, share_next.have);
    uint32_t turn = 0, phase = 0;  // of the messages: two buffers in turn
    for (; t < a.T; t += step) {
        const Token later(a, t + 2 * step);
        s = n;
        const bool live = now.live(a);  // the same for the whole cluster
        const Share share = share_next;
        const float head = xh, tail = xt, logit = picked;
        look(t + step, next);
        if (live) {
            const uint32_t bar = ptx::smem_addr(&arrived[turn]);
            Message *const box = messages + turn * count;
            if (tid == 0 && count > 1)
                ptx::mbar_arrive_expect_tx(bar, (uint32_t)(count * (int)sizeof(Message)));
            Sum acc{fmaxf(head, tail), 0.0f};
            const float m = base_of(acc.m);
            acc.s = ex2((head - m) * c) + ex2((tail - m) * c);  // -inf where there is none
            mine.sum_up(acc, share, c);
            Sum all = warp_join(acc, c);
            float target_logit = __shfl_sync(~0u, logit, 0);
            if (count > 1) {
                // The warps' sums, to every CTA.  The target's logit travels with one of
                // them, so that no gradient is written over it before it has been read.  A
                // buffer is filled again two rows on: by then every warp of the cluster has
                // sent the next row's sum, after it had read this one's.
                const Message said{all.m, all.s, target_logit, 0.0f};
                // test hook: one warp's message is never sent
                const bool stall = a.inject_stall && t == 0 && rank == 0 && warp == 0;
                if (lane < parts && !stall)
                    send(ptx::smem_addr(box + rank * warps + warp), bar, (uint32_t)lane, said);
                if (!__all_sync(~0u, tc::bounded_wait(bar, phase, a.wait_limit_ns))) {
                    if (lane == 0)
                        report_status(a.status, kStatusTimeout);
                    // Messages that are only late still come: they have to find this CTA.  Later
                    // rows' cannot be missed: their senders wait as long for this warp's.
                    ptx::mbar_wait(bar, phase, kDrainLimitNs);
                    break;
                }
                all = Sum{-INFINITY, 0.0f};
                for (int i = lane; i < count; i += 32)
                    all = join(all, Sum{box[i].m, box[i].s}, c);
                all = warp_join(all, c);
                target_logit = box[0].logit;
                __syncwarp();
                phase ^= turn;
                turn ^= 1;
            }
            const float logp = logp_of(a, all, target_logit);
            if (rank == 0 && tid == 0)
                a.logp_out[t] = logp;
            const Gradient<E> g(a, now, all, logp, c);
            if (s.wide) {
                uint8_t *to = reinterpret_cast<uint8_t *>(s.out + s.v0) + first * 16;
                mine.write(g, to, share, from, share_next);
            } else {  // an output of another alignment, or none
#pragma unroll 1
                for (int q = 0; q < share.have && s.out; ++q) {
                    Vec<E> v = *reinterpret_cast<const Vec<E> *>(mine.slot + q * 512);
                    g.softmax(v);
#pragma unroll
                    for (int u = 0; u < VEC; ++u)
                        s.out[s.v0 + (first + q * 32) * VEC + u] = reinterpret_cast<const E *>(v.w)[u];
                }
                mine.fetch_all(from, share_next.have);
            }
            if (s.out) {
                if (s.has_head(tid))
                    s.out[s.lo + tid] = g.one(head);
                if (s.has_tail(tid))
                    s.out[s.v1 + tid] = g.one(tail);
                // the target's element, by the thread that has just written it
                const int at = g.target - s.v0, vi = at / VEC;
                const bool in_vectors = at >= 0 && g.target < s.v1 && vi % 32 == lane && vi / (NV * 32) == warp;
                if (in_vectors || (s.has_head(tid) && g.target == s.lo + tid) ||
                    (s.has_tail(tid) && g.target == s.v1 + tid))
                    s.out[g.target] = g.target_one(target_logit);
            }
        } else {
            mine.fetch_all(from, share_next.have);
            if (rank == 0 && tid == 0) {
                a.logp_out[t] = 0.0f;
                if (now.weight != 0.0f)
                    report_status(a.status, kInvalidArg);
            }
            s.zero(tid, blockDim.x);
        }
        now = next;
        next = later;
    }
    wait_groups(0);
    __syncwarp();
    tc::cluster_meet();  // no CTA leaves while a message may still be on its way to it
}

// Rows beyond what a cluster's shared memory holds: the second pass reads memory
// again.  One cluster per token.
template <typename E>
__global__ void __launch_bounds__(1024) policy_loss_long_kernel(const __grid_constant__ LossArgs a)
{
    constexpr int VEC = Elem<E>::kVec;
    __shared__ Sum sums[32];
    tc::launch_dependents();
    const int64_t t = tc::cluster_id_x();
    const int parts = (int)tc::cluster_size(), rank = (int)tc::cluster_ctarank();
    const int tid = threadIdx.x, threads = blockDim.x, lane = tid & 31;
    Slice<E> s(a, rank, parts);
    s.at(a, t);
    const Token now(a, t);
    if (!now.live(a)) {  // the same for the whole cluster
        if (rank == 0 && tid == 0) {
            a.logp_out[t] = 0.0f;
            if (now.weight != 0.0f)
                report_status(a.status, kInvalidArg);
        }
        s.zero(tid, threads);
        return;
    }
    const float c = a.inv_temperature * kLog2e;
    const float picked = Elem<E>::get(s.row[now.target]);  // before any CTA may write over it
    const float head = s.has_head(tid) ? Elem<E>::get(s.row[s.lo + tid]) : -INFINITY;
    const float tail = s.has_tail(tid) ? Elem<E>::get(s.row[s.v1 + tid]) : -INFINITY;
    Sum acc{-INFINITY, 0.0f};
#pragma unroll 4
    for (int i = tid; i < s.nvec; i += threads) {
        const Vec<E> v = s.vec()[i];
        const float top = top_of(v, -INFINITY);
        if (top > acc.m) {
            acc.s *= rescale(acc.m, top, c);
            acc.m = top;
        }
        F2 part[2] = {pair_of(0.0f), pair_of(0.0f)};
        add_powers(v, base_of(acc.m), c, part);
        const float2 sum2 = halves_of(add2(part[0], part[1]));
        acc.s += sum2.x + sum2.y;
    }
    if (s.has_head(tid))
        acc = join(acc, Sum{head, ex2((head - base_of(head)) * c)}, c);
    if (s.has_tail(tid))
        acc = join(acc, Sum{tail, ex2((tail - base_of(tail)) * c)}, c);
    acc = warp_join(acc, c);
    if (lane == 0)
        sums[tid >> 5] = acc;
    __syncwarp();
    tc::cluster_sync();  // every warp's sum is there, every read of the target's logit done
    const Sum all = cluster_join(sums, threads / 32, parts, lane, c);
    const float logp = logp_of(a, all, picked);
    if (rank == 0 && tid == 0)
        a.logp_out[t] = logp;
    if (s.out) {
        const Gradient<E> g(a, now, all, logp, c);
#pragma unroll 4
        for (int i = tid; i < s.nvec; i += threads) {
            Vec<E> v = s.vec()[i];
            g.softmax(v);
            if (s.wide) {
                reinterpret_cast<Vec<E> *>(s.out + s.v0)[i] = v;
            } else {
#pragma unroll
                for (int u = 0; u < VEC; ++u)
                    s.out[s.v0 + i * VEC + u] = reinterpret_cast<const E *>(v.w)[u];
            }
        }
        if (s.has_head(tid))
            s.out[s.lo + tid] = g.one(head);
        if (s.has_tail(tid))
            s.out[s.v1 + tid] = g.one(tail);
        __syncthreads();  // the target's element after the others
        if (tid == 0 && g.target >= s.lo && g.target < s.hi)
            s.out[g.target] = g.target_one(picked);
    }
    __syncwarp();
    tc::cluster_sync();  // no CTA leaves while its sums may still be read
}

// An unevaluated sum of two floats (Knuth's two-sum): the statistics' terms of
// either sign may cancel, and double additions are slow here (8 us for 16 tokens).
struct Two {
    float hi, lo;
};

__device__ __forceinline__ Two add_two(Two a, Two b)
{
    const float s = __fadd_rn(a.hi, b.hi), t = __fsub_rn(s, a.hi);
    const float e = __fadd_rn(__fsub_rn(a.hi, __fsub_rn(s, t)), __fsub_rn(b.hi, t));
    const float lo = __fadd_rn(e, __fadd_rn(a.lo, b.lo));
    Two r;
    r.hi = __fadd_rn(s, lo);
    r.lo = __fsub_rn(lo, __fsub_rn(r.hi, s));
    return r;
}

// weight x, with the product's rounding error in lo.
__device__ __forceinline__ Two product_two(float w, float x)
{
    const float p = __fmul_rn(w, x);
    return Two{p, __fmaf_rn(w, x, -p)};
}

// The four statistics from the tokens' logp, in one CTA and a fixed order.
__global__ void __launch_bounds__(1024) loss_stats_kernel(const __grid_constant__ LossArgs a)
{
    __shared__ Two part[4][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x / 32;
    Two s[4] = {};
    Token token(a, threadIdx.x);  // what the rows' kernel does not write: ahead of the wait
    tc::wait_dependencies();      // the rows' kernel is done
    for (int64_t t = threadIdx.x; t < a.T; t += blockDim.x) {
        const Token next(a, t + blockDim.x);
        if (token.live(a)) {
            const Terms r = terms_of(a, token, a.logp_out[t]);
            s[0] = add_two(s[0], product_two(token.weight, r.loss));
            s[1] = add_two(s[1], product_two(token.weight, r.kl));
            s[2] = add_two(s[2], product_two(token.weight, r.clipped));
            s[3] = add_two(s[3], product_two(token.weight, r.ratio));
        }
        token = next;
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
#pragma unroll
        for (int d = 16; d > 0; d >>= 1)
            s[q] = add_two(s[q], Two{__shfl_xor_sync(~0u, s[q].hi, d), __shfl_xor_sync(~0u, s[q].lo, d)});
        if (lane == 0)
            part[q][warp] = s[q];
    }
    __syncthreads();
    if (warp < 4) {
        Two t = lane < warps ? part[warp][lane] : Two{0.0f, 0.0f};
#pragma unroll
        for (int d = 16; d > 0; d >>= 1)
            t = add_two(t, Two{__shfl_xor_sync(~0u, t.hi, d), __shfl_xor_sync(~0u, t.lo, d)});
        if (lane == 0)
            a.stats[warp] = t.hi;
    }
}

constexpr int kMaxDevices = 64;
constexpr int kSliceVecs = 6400;             // 100 KB: two CTAs on an SM
constexpr int kMaxSliceBytes = 216 * 1024;
constexpr int kMaxMessageBytes = 2 * 8 * (kMaxSliceBytes / 8192) * 16;  // of 8 CTAs

template <typename E, int NB>
cudaError_t launch_held(cudaLaunchConfig_t &cfg, const LossArgs &a)
{
    static std::once_flag once[kMaxDevices];
    static cudaError_t result[kMaxDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices)
        dev = 0;
    std::call_once(once[dev], [&] {
        result[dev] = cudaFuncSetAttribute(policy_loss_kernel<E, NB>,
                                           cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           kMaxSliceBytes + kMaxMessageBytes);
    });
    if (result[dev] != cudaSuccess)
        return result[dev];
    return cudaLaunchKernelEx(&cfg, policy_loss_kernel<E, NB>, a);
}

template <typename E>
cudaError_t launch_rows(const LossArgs &a, cudaStream_t s)
{
    // A row's vectors are shared by as few CTAs as hold 100 KB each, two on an
    // SM; by up to 8 (a portable cluster) of up to 216 KB where that is not enough.
    // (Of up to 67 KB each: 283 us where this took 262, at 4096 x 100003 bfloat16; of
    // up to 52 KB 294, of up to 200 KB, one on an SM, 293, at 8191 x 32768 float32
    // then 332 and 390 for 320.)
    // When the rows are few, more and smaller CTAs share a row, down to 128 vectors
    // each.  Threads have up to 16 vectors.
    const int64_t vecs = (a.V + Elem<E>::kVec - 1) / Elem<E>::kVec;
    int64_t parts = (vecs + kSliceVecs - 1) / kSliceVecs;
    parts = parts > 8 ? 8 : parts;
    while (parts <= 4 && a.T * parts * 2 <= 2 * kSMs && vecs / (parts * 2) >= 128)
        parts *= 2;
    const int64_t slice = (vecs + parts - 1) / parts;  // a row that starts between two 16-byte boundaries has no more
    const int nb = slice <= 4 * 128 ? 1 : (slice <= 8 * 128 ? 2 : 4);
    int64_t threads = (slice + nb * kBatch * 32 - 1) / (nb * kBatch * 32) * 32;
    const int64_t bytes = threads * nb * kBatch * 16;
    const bool held = bytes <= kMaxSliceBytes;
    threads = held ? threads : 1024;
    // Clusters: one for every 3 rows, as far as there are more rows than clusters
    // resident at once.  Masked rows cost half: with fixed shares for all rows
    // (resident clusters only) the unluckiest ended a quarter late.  4096 x 100003
    // bfloat16: 2 rows 267 us, 3 rows 263, 4 rows 262, 6 rows 264; with the slower
    // exchange of an earlier build 12 rows 315, all rows 297, 1 row (no copy ahead) 305, 3 rows 284.
    const int64_t fit = kMaxSliceBytes / bytes;
    const int64_t per_sm = fit < 1 ? 1 : gg_min64(fit, gg_min64(32, 896 / threads > 0 ? 896 / threads : 1));
    const int64_t resident = per_sm * kSMs / parts;
    const int64_t thirds = (a.T + 2) / 3;
    const int64_t clusters = !held || a.T <= resident ? a.T : (thirds > resident ? thirds : resident);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)parts;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)(clusters * parts), 1, 1);
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.dynamicSmemBytes = held ? (size_t)(bytes + 2 * parts * (threads / 32) * (int64_t)sizeof(Message)) : 0;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (!held)
        return cudaLaunchKernelEx(&cfg, policy_loss_long_kernel<E>, a);
    switch (nb) {
    case 1: return launch_held<E, 1>(cfg, a);
    case 2: return launch_held<E, 2>(cfg, a);
    default: return launch_held<E, 4>(cfg, a);
    }
}

}  // namespace

cudaError_t launch_policy_loss(const LossArgs &a, cudaStream_t s)
{
    cudaError_t e = cudaSuccess;
    if (a.T > 0 && a.V > 0) {
        if (a.dtype == GG_F32)
            e = launch_rows<float>(a, s);
        else if (a.dtype == GG_F16)
            e = launch_rows<__half>(a, s);
        else
            e = launch_rows<__nv_bfloat16>(a, s);
    }
    if (e == cudaSuccess && a.stats) {
        // may be launched while the rows' kernel still runs; it waits for it
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.gridDim = dim3(1, 1, 1);
        cfg.blockDim = dim3(a.T <= 128 ? 128 : 1024, 1, 1);
        cfg.stream = s;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        e = cudaLaunchKernelEx(&cfg, loss_stats_kernel, a);
    }
    return e;
}

}  // namespace gg
