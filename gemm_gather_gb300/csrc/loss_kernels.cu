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
// Bound: HBM, one read and one write of the logits.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "f32x2.cuh"
#include "gg_internal.h"
#include "gg_ops.h"
#include "tc.cuh"

namespace gg {
namespace {

constexpr int kSMs = 152;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kInvalidArg = GG_ERR_INVALID_ARG;

template <typename E>
struct Elem;
template <>
struct Elem<float> {
    static constexpr int kVec = 4;
    static __device__ __forceinline__ float get(float x) { return x; }
    static __device__ __forceinline__ float put(float x) { return x; }
    static __device__ __forceinline__ void put2(float *e, float2 x) { e[0] = x.x, e[1] = x.y; }
};
template <>
struct Elem<__half> {
    static constexpr int kVec = 8;
    static __device__ __forceinline__ float get(__half x) { return __half2float(x); }
    static __device__ __forceinline__ __half put(float x) { return __float2half_rn(x); }
    static __device__ __forceinline__ void put2(__half *e, float2 x)
    {
        *reinterpret_cast<__half2 *>(e) = __float22half2_rn(x);
    }
};
template <>
struct Elem<__nv_bfloat16> {
    static constexpr int kVec = 8;
    static __device__ __forceinline__ float get(__nv_bfloat16 x) { return __bfloat162float(x); }
    static __device__ __forceinline__ __nv_bfloat16 put(float x) { return __float2bfloat16_rn(x); }
    static __device__ __forceinline__ void put2(__nv_bfloat16 *e, float2 x)
    {
        *reinterpret_cast<__nv_bfloat162 *>(e) = __float22bfloat162_rn(x);
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

// What a token's logp gives: the loss terms and dloss/dlogp.
struct Terms {
    float loss, kl, clipped, ratio, slope;
};

__device__ __forceinline__ Terms terms_of(const LossArgs &a, int64_t t, float logp)
{
    Terms r;
    const float adv = a.advantage[t];
    r.ratio = expf(logp - (a.old_logp ? a.old_logp[t] : logp));  // NaN for a row without a logp
    const bool over = (adv > 0.0f && r.ratio > 1.0f + a.clip_high) ||
                      (adv < 0.0f && r.ratio < 1.0f - a.clip_low);
    r.clipped = over ? 1.0f : 0.0f;
    const float held = fminf(fmaxf(r.ratio, 1.0f - a.clip_low), 1.0f + a.clip_high);
    r.loss = -(over ? held : r.ratio) * adv;
    r.slope = over ? 0.0f : -adv * r.ratio;
    r.kl = 0.0f;
    if (a.ref_logp && a.kl_coef != 0.0f) {
        const float d = a.ref_logp[t] - logp;
        const float e = expm1f(d);  // exp(d) - d - 1 without losing it for small d
        r.kl = e - d;
        r.loss += a.kl_coef * r.kl;
        r.slope -= a.kl_coef * e;
    }
    return r;
}

template <typename E>
struct alignas(16) Vec {
    union {
        E e[Elem<E>::kVec];
        uint32_t w[4];
    };
    __device__ __forceinline__ Vec() {}
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
    return fmaxf(fmaxf(fmaxf(v.e[0], v.e[1]), fmaxf(v.e[2], v.e[3])), top);
}
__device__ __forceinline__ float top_of(const Vec<__half> &v, float top)
{
    const __half2 *h = reinterpret_cast<const __half2 *>(v.e);
    const __half2 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
    return fmaxf(fmaxf(__low2float(m), __high2float(m)), top);
}
__device__ __forceinline__ float top_of(const Vec<__nv_bfloat16> &v, float top)
{
    const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(v.e);
    const __nv_bfloat162 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
    return fmaxf(fmaxf(__low2float(m), __high2float(m)), top);
}

// 2^((x - m) c) of a vector's elements, in pairs.
template <typename E>
__device__ __forceinline__ void powers_of(const Vec<E> &v, float m, float c,
                                          float2 (&e)[Elem<E>::kVec / 2])
{
    const F2 minus_m = pair_of(-m, -m), cc = pair_of(c, c);
#pragma unroll
    for (int u = 0; u < Elem<E>::kVec / 2; ++u) {
        const F2 x = pair_of(Elem<E>::get(v.e[2 * u]), Elem<E>::get(v.e[2 * u + 1]));
        const float2 y = halves_of(mul2(add2(x, minus_m), cc));
        e[u] = make_float2(ex2(y.x), ex2(y.y));
    }
}

// One cluster per token.  NV > 0: each thread keeps its NV 16-byte vectors of
// the row in registers, so the row is read from memory once; all NV loads are
// in flight together, and the sum needs no rescaling (a thread's maximum is
// known before its first exponential).  NV == 0, for rows beyond what a
// cluster's registers hold: a running maximum and sum, and a second read.
template <typename E, int NV>
__global__ void __launch_bounds__(1024) policy_loss_kernel(const __grid_constant__ LossArgs a)
{
    constexpr int VEC = Elem<E>::kVec;
    __shared__ Sum warps[32];
    __shared__ Sum mine;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the statistics' launch
    const int64_t t = tc::cluster_id_x();
    const int parts = (int)tc::cluster_size(), rank = (int)tc::cluster_ctarank();
    const int tid = threadIdx.x, threads = blockDim.x;
    const E *row = reinterpret_cast<const E *>(a.logits) + t * a.ld;
    E *out = a.dlogits ? reinterpret_cast<E *>(a.dlogits) + t * a.ldd : nullptr;
    // this CTA's slice, in units of VEC elements (V is below 2^31: row indices are int)
    const int64_t units = (a.V + VEC - 1) / VEC;
    const int lo = (int)(units * rank / parts * VEC);
    const int hi = (int)gg_min64(units * (rank + 1) / parts * VEC, a.V);
    // whole vectors from the first 16-byte boundary of the input on
    const int head = (int)((16 - (reinterpret_cast<uint64_t>(row + lo) & 15)) & 15) / (int)sizeof(E);
    const int v0 = lo + head < hi ? lo + head : hi;
    const int nvec = (hi - v0) / VEC;
    const int v1 = v0 + nvec * VEC;
    const bool wide = out && (reinterpret_cast<uint64_t>(out + v0) & 15) == 0;

    const float w = a.weight[t];
    int target = 0;
    bool live = w != 0.0f;
    if (live) {
        const int64_t id = a.target[t];
        target = (int)id;
        if (id < 0 || id >= a.V) {
            live = false;
            if (rank == 0 && tid == 0)
                report_status(a.status, kInvalidArg);
        }
    }
    if (!live) {  // the same for the whole cluster
        if (rank == 0 && tid == 0)
            a.logp_out[t] = 0.0f;
        if (out) {
            for (int i = lo + tid; i < v0; i += threads)
                out[i] = Elem<E>::put(0.0f);
            if (wide) {
                for (int i = tid; i < nvec; i += threads)
                    reinterpret_cast<uint4 *>(out + v0)[i] = make_uint4(0, 0, 0, 0);
            } else {
                for (int i = v0 + tid; i < v1; i += threads)
                    out[i] = Elem<E>::put(0.0f);
            }
            for (int i = v1 + tid; i < hi; i += threads)
                out[i] = Elem<E>::put(0.0f);
        }
        return;
    }

    const float c = a.inv_temperature * kLog2e;
    const Vec<E> *vec = reinterpret_cast<const Vec<E> *>(row + v0);
    Vec<E> held[NV > 0 ? NV : 1];
    if constexpr (NV > 0) {
#pragma unroll
        for (int k = 0; k < NV; ++k)
            if (tid + k * threads < nvec)
                held[k] = vec[tid + k * threads];
    }
    const float picked = Elem<E>::get(row[target]);  // before any CTA may write over it
    // the ragged ends, fewer than VEC elements each: one of either per thread
    const bool has_head = tid < v0 - lo, has_tail = tid < hi - v1;
    const float xh = has_head ? Elem<E>::get(row[lo + tid]) : -INFINITY;
    const float xt = has_tail ? Elem<E>::get(row[v1 + tid]) : -INFINITY;
    Sum acc{-INFINITY, 0.0f};
    if constexpr (NV > 0) {
        float top = fmaxf(xh, xt);
#pragma unroll
        for (int k = 0; k < NV; ++k)
            if (tid + k * threads < nvec) {
                top = top_of(held[k], top);
                stay_packed(held[k]);
            }
        const float m = base_of(top);
        F2 part[2] = {pair_of(0.0f, 0.0f), pair_of(0.0f, 0.0f)};
#pragma unroll
        for (int k = 0; k < NV; ++k)
            if (tid + k * threads < nvec) {
                float2 e[VEC / 2];
                powers_of<E>(held[k], m, c, e);
#pragma unroll
                for (int u = 0; u < VEC / 2; ++u)
                    part[u & 1] = add2(part[u & 1], pair_of(e[u].x, e[u].y));
                stay_packed(held[k]);
            }
        const float2 p0 = halves_of(part[0]), p1 = halves_of(part[1]);
        acc.m = top;
        acc.s = (p0.x + p0.y) + (p1.x + p1.y);
        if (has_head)
            acc.s += ex2((xh - m) * c);
        if (has_tail)
            acc.s += ex2((xt - m) * c);
    } else {
#pragma unroll 4
        for (int i = tid; i < nvec; i += threads) {
            const Vec<E> v = vec[i];
            const float top = top_of(v, -INFINITY);
            if (top > acc.m) {
                acc.s *= rescale(acc.m, top, c);
                acc.m = top;
            }
            float2 e[VEC / 2];
            powers_of<E>(v, base_of(acc.m), c, e);
#pragma unroll
            for (int u = 0; u < VEC / 2; ++u)
                acc.s += e[u].x + e[u].y;
        }
        if (has_head)
            acc = join(acc, Sum{xh, ex2((xh - base_of(xh)) * c)}, c);
        if (has_tail)
            acc = join(acc, Sum{xt, ex2((xt - base_of(xt)) * c)}, c);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        acc = join(acc, Sum{__shfl_xor_sync(~0u, acc.m, d), __shfl_xor_sync(~0u, acc.s, d)}, c);
    if ((tid & 31) == 0)
        warps[tid >> 5] = acc;
    __syncthreads();
    if (tid < 32) {
        acc = tid < threads / 32 ? warps[tid] : Sum{-INFINITY, 0.0f};
#pragma unroll
        for (int d = 16; d > 0; d >>= 1)
            acc = join(acc, Sum{__shfl_xor_sync(~0u, acc.m, d), __shfl_xor_sync(~0u, acc.s, d)}, c);
        if (tid == 0)
            mine = acc;
    }
    __syncthreads();
    tc::cluster_sync();  // every CTA's sum is there, and every read of row[target] is done
    Sum all{-INFINITY, 0.0f};
    for (int p = 0; p < parts; ++p) {
        const uint32_t at = tc::map_to_rank(ptx::smem_addr(&mine), (uint32_t)p);
        all = join(all, Sum{tc::ld_cluster_f32(at), tc::ld_cluster_f32(at + 4)}, c);
    }
    tc::cluster_arrive();  // its sum read, this CTA lets the others go
    const float m = base_of(all.m);
    const float logp = (picked - m) * a.inv_temperature - logf(all.s);
    if (rank == 0 && tid == 0)
        a.logp_out[t] = logp;
    if (out) {
        const float coef = w * terms_of(a, t, logp).slope * a.inv_temperature * a.grad_scale;
        const float k = -coef / all.s;
        // the gradient at element i, whose logit is x
        const auto grad = [&](int i, float x) {
            return fmaf(k, ex2((x - m) * c), i == target ? coef : 0.0f);
        };
        if (wide) {
            // the vector that holds the target, and the target's place in it
            const int tv = target >= v0 && target < v1 ? (target - v0) / VEC : -1;
            const int tu = target - v0 - tv * VEC;
            const auto put = [&](int i, Vec<E> v) {
                float2 y[VEC / 2];
                powers_of<E>(v, m, c, y);
#pragma unroll
                for (int u = 0; u < VEC / 2; ++u)
                    y[u] = halves_of(mul2(pair_of(y[u].x, y[u].y), pair_of(k, k)));
                if (i == tv) {
#pragma unroll
                    for (int u = 0; u < VEC / 2; ++u) {
                        y[u].x += 2 * u == tu ? coef : 0.0f;
                        y[u].y += 2 * u + 1 == tu ? coef : 0.0f;
                    }
                }
#pragma unroll
                for (int u = 0; u < VEC / 2; ++u)
                    Elem<E>::put2(v.e + 2 * u, y[u]);
                reinterpret_cast<Vec<E> *>(out + v0)[i] = v;
            };
            if constexpr (NV > 0) {
#pragma unroll
                for (int q = 0; q < NV; ++q)
                    if (tid + q * threads < nvec)
                        put(tid + q * threads, held[q]);
            } else {
                for (int i = tid; i < nvec; i += threads)
                    put(i, vec[i]);
            }
        } else if constexpr (NV > 0) {
#pragma unroll
            for (int q = 0; q < NV; ++q)
                if (tid + q * threads < nvec) {
                    const int i = v0 + (tid + q * threads) * VEC;
#pragma unroll
                    for (int u = 0; u < VEC; ++u)
                        out[i + u] = Elem<E>::put(grad(i + u, Elem<E>::get(held[q].e[u])));
                }
        } else {
            for (int i = v0 + tid; i < v1; i += threads)
                out[i] = Elem<E>::put(grad(i, Elem<E>::get(row[i])));
        }
        if (has_head)
            out[lo + tid] = Elem<E>::put(grad(lo + tid, xh));
        if (has_tail)
            out[v1 + tid] = Elem<E>::put(grad(v1 + tid, xt));
    }
    tc::cluster_wait();  // no CTA leaves while its sum may still be read
}

// The four statistics from the tokens' logp, in one CTA and a fixed order (in
// double: the float32 terms of either sign may cancel).
__global__ void __launch_bounds__(1024) loss_stats_kernel(const __grid_constant__ LossArgs a)
{
    __shared__ double part[32][4];
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the rows' kernel is done
    double s[4] = {0, 0, 0, 0};
    for (int64_t t = threadIdx.x; t < a.T; t += 1024) {
        const float w = a.weight[t];
        if (w == 0.0f)
            continue;
        const int64_t target = a.target[t];
        if (target < 0 || target >= a.V)
            continue;
        const Terms r = terms_of(a, t, a.logp_out[t]);
        s[0] += (double)w * r.loss;
        s[1] += (double)w * r.kl;
        s[2] += (double)w * r.clipped;
        s[3] += (double)w * r.ratio;
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
#pragma unroll
        for (int d = 16; d > 0; d >>= 1)
            s[q] += __shfl_xor_sync(~0u, s[q], d);
        if ((threadIdx.x & 31) == 0)
            part[threadIdx.x >> 5][q] = s[q];
    }
    __syncthreads();
    if (threadIdx.x < 4) {
        double t = 0;
        for (int i = 0; i < 32; ++i)
            t += part[i][threadIdx.x];
        a.stats[threadIdx.x] = (float)t;
    }
}

constexpr int kHeld = 8;          // vectors a thread keeps at most (32 registers)
constexpr int kRowThreads = 256;  // threads of a CTA, unless the row asks for more

template <typename E>
cudaError_t launch_rows(const LossArgs &a, cudaStream_t s)
{
    // A row's vectors (one more than V needs: a row may start between two
    // 16-byte boundaries) go to CTAs of 256 threads with 8 vectors each, so that
    // four CTAs of 64 registers a thread share an SM; to larger CTAs when 8 CTAs
    // (a portable cluster) of 256 do not hold them.  When the rows are few, more
    // and smaller CTAs share a row, down to 128 vectors each.
    const int64_t vecs = (a.V + Elem<E>::kVec - 1) / Elem<E>::kVec + 1;
    int64_t parts = (vecs + kHeld * kRowThreads - 1) / (kHeld * kRowThreads);
    parts = parts > 8 ? 8 : parts;
    while (parts <= 4 && a.T * parts * 2 <= 2 * kSMs && vecs / (parts * 2) >= 128)
        parts *= 2;
    const int64_t slice = (vecs + parts - 1) / parts + 1;
    const bool held = slice <= kHeld * 1024;
    int nv = 1;
    while (nv < kHeld && slice > (int64_t)nv * kRowThreads)
        nv *= 2;
    int64_t threads = held ? ((slice + nv - 1) / nv + 31) / 32 * 32 : 1024;
    threads = threads < 64 ? 64 : threads;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)parts;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)(a.T * parts), 1, 1);
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (!held)
        return cudaLaunchKernelEx(&cfg, policy_loss_kernel<E, 0>, a);
    switch (nv) {
    case 1: return cudaLaunchKernelEx(&cfg, policy_loss_kernel<E, 1>, a);
    case 2: return cudaLaunchKernelEx(&cfg, policy_loss_kernel<E, 2>, a);
    case 4: return cudaLaunchKernelEx(&cfg, policy_loss_kernel<E, 4>, a);
    default: return cudaLaunchKernelEx(&cfg, policy_loss_kernel<E, 8>, a);
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
        cfg.blockDim = dim3(1024, 1, 1);
        cfg.stream = s;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        e = cudaLaunchKernelEx(&cfg, loss_stats_kernel, a);
    }
    return e;
}

}  // namespace gg
