// The clipped policy loss with its gradient, from the logits, for sm_103a.
//
// A row of logits x (scaled by the inverse temperature) becomes
//     logp = x[a] - log sum exp x,     dlogits = k (onehot(a) - softmax(x)),
// with k = weight * grad_scale * inv_temperature * dloss/dlogp known as soon as
// logp is: so one launch reads a row, reduces it to its maximum and sum of
// exponentials in one pass (each thread rescales its running sum when its
// maximum grows), and writes the gradient.  Powers of two: exp(x - max) =
// 2^(x c - max c), c = inv_temperature * log2(e), one fused multiply-add and
// one ex2 an element; sums are float32.
//
// A cluster of CTAs owns a row, each CTA a slice, and the CTAs exchange
// (maximum, sum) through distributed shared memory.
// Bound: HBM, one read and one write of the logits.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

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
};
template <>
struct Elem<__half> {
    static constexpr int kVec = 8;
    static __device__ __forceinline__ float get(__half x) { return __half2float(x); }
    static __device__ __forceinline__ __half put(float x) { return __float2half_rn(x); }
};
template <>
struct Elem<__nv_bfloat16> {
    static constexpr int kVec = 8;
    static __device__ __forceinline__ float get(__nv_bfloat16 x) { return __bfloat162float(x); }
    static __device__ __forceinline__ __nv_bfloat16 put(float x) { return __float2bfloat16_rn(x); }
};

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Running maximum (of raw logits) and sum of 2^((x - max) c).  An empty sum has
// maximum -inf; -inf logits are probability 0 and never meet inf - inf.
struct Sum {
    float m, s;
};

__device__ __forceinline__ float shift_of(float m, float c) { return m == -INFINITY ? 0.0f : m * c; }

__device__ __forceinline__ Sum join(Sum a, Sum b, float c)
{
    Sum r;
    r.m = fmaxf(a.m, b.m);
    const float k = shift_of(r.m, c);
    r.s = a.s * ex2(shift_of(a.m, c) - k) + b.s * ex2(shift_of(b.m, c) - k);
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
    E e[Elem<E>::kVec];
};

template <typename E>
__device__ __forceinline__ void add_to(Sum &acc, const float (&x)[Elem<E>::kVec], float c)
{
    float top = x[0];
#pragma unroll
    for (int u = 1; u < Elem<E>::kVec; ++u)
        top = fmaxf(top, x[u]);
    if (top > acc.m) {
        acc.s *= ex2(shift_of(acc.m, c) - top * c);
        acc.m = top;
    }
    const float k = shift_of(acc.m, c);
#pragma unroll
    for (int u = 0; u < Elem<E>::kVec; ++u)
        acc.s += ex2(fmaf(x[u], c, -k));
}

// One cluster per token.
template <typename E>
__global__ void __launch_bounds__(1024) policy_loss_kernel(const __grid_constant__ LossArgs a)
{
    constexpr int VEC = Elem<E>::kVec;
    __shared__ Sum warps[32];
    __shared__ Sum mine;
    const int64_t t = tc::cluster_id_x();
    const int parts = (int)tc::cluster_size(), rank = (int)tc::cluster_ctarank();
    const int tid = threadIdx.x, threads = blockDim.x;
    const E *row = reinterpret_cast<const E *>(a.logits) + t * a.ld;
    E *out = a.dlogits ? reinterpret_cast<E *>(a.dlogits) + t * a.ldd : nullptr;
    // this CTA's slice, in units of VEC elements
    const int64_t units = (a.V + VEC - 1) / VEC;
    const int64_t lo = units * rank / parts * VEC;
    const int64_t end = units * (rank + 1) / parts * VEC;
    const int64_t hi = end < a.V ? end : a.V;
    // whole vectors from the first 16-byte boundary of the input on
    const int64_t head = ((16 - (reinterpret_cast<uint64_t>(row + lo) & 15)) & 15) / sizeof(E);
    const int64_t v0 = lo + head < hi ? lo + head : hi;
    const int64_t nvec = (hi - v0) / VEC;
    const int64_t v1 = v0 + nvec * VEC;
    const bool wide = out && (reinterpret_cast<uint64_t>(out + v0) & 15) == 0;

    const float w = a.weight[t];
    int64_t target = 0;
    bool live = w != 0.0f;
    if (live) {
        target = a.target[t];
        if (target < 0 || target >= a.V) {
            live = false;
            if (rank == 0 && tid == 0)
                report_status(a.status, kInvalidArg);
        }
    }
    if (!live) {  // the same for the whole cluster
        if (rank == 0 && tid == 0)
            a.logp_out[t] = 0.0f;
        if (out) {
            for (int64_t i = lo + tid; i < v0; i += threads)
                out[i] = Elem<E>::put(0.0f);
            if (wide) {
                for (int64_t i = tid; i < nvec; i += threads)
                    reinterpret_cast<uint4 *>(out + v0)[i] = make_uint4(0, 0, 0, 0);
            } else {
                for (int64_t i = v0 + tid; i < v1; i += threads)
                    out[i] = Elem<E>::put(0.0f);
            }
            for (int64_t i = v1 + tid; i < hi; i += threads)
                out[i] = Elem<E>::put(0.0f);
        }
        return;
    }

    const float c = a.inv_temperature * kLog2e;
    const float picked = Elem<E>::get(row[target]);  // before any CTA may write over it
    Sum acc{-INFINITY, 0.0f};
    const Vec<E> *vec = reinterpret_cast<const Vec<E> *>(row + v0);
#pragma unroll 4
    for (int64_t i = tid; i < nvec; i += threads) {
        const Vec<E> v = vec[i];
        float x[VEC];
#pragma unroll
        for (int u = 0; u < VEC; ++u)
            x[u] = Elem<E>::get(v.e[u]);
        add_to<E>(acc, x, c);
    }
    for (int part = 0; part < 2; ++part) {  // the ragged ends, fewer than VEC elements each
        const int64_t i = (part == 0 ? lo : v1) + tid;
        if (i < (part == 0 ? v0 : hi)) {
            const float x = Elem<E>::get(row[i]);
            acc = join(acc, Sum{x, x == -INFINITY ? 0.0f : ex2(x * c - shift_of(x, c))}, c);
        }
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
    const float logp = (picked - (all.m == -INFINITY ? 0.0f : all.m)) * a.inv_temperature - logf(all.s);
    if (rank == 0 && tid == 0)
        a.logp_out[t] = logp;
    if (out) {
        const float coef = w * terms_of(a, t, logp).slope * a.inv_temperature * a.grad_scale;
        const float k = -coef / all.s;
        const float shift = shift_of(all.m, c);
        if (wide) {
#pragma unroll 4
            for (int64_t i = tid; i < nvec; i += threads) {
                Vec<E> v = vec[i];
#pragma unroll
                for (int u = 0; u < VEC; ++u)
                    v.e[u] = Elem<E>::put(k * ex2(fmaf(Elem<E>::get(v.e[u]), c, -shift)));
                reinterpret_cast<Vec<E> *>(out + v0)[i] = v;
            }
        } else {
            for (int64_t i = v0 + tid; i < v1; i += threads)
                out[i] = Elem<E>::put(k * ex2(fmaf(Elem<E>::get(row[i]), c, -shift)));
        }
        for (int part = 0; part < 2; ++part) {
            const int64_t i = (part == 0 ? lo : v1) + tid;
            if (i < (part == 0 ? v0 : hi))
                out[i] = Elem<E>::put(k * ex2(fmaf(Elem<E>::get(row[i]), c, -shift)));
        }
        __syncthreads();  // the target's element after the others
        if (tid == 0 && target >= lo && target < hi)
            out[target] = Elem<E>::put(coef + k * ex2(fmaf(picked, c, -shift)));
    }
    tc::cluster_sync();  // no CTA leaves while its sum may still be read
}

// The four statistics from the tokens' logp, in one CTA and a fixed order (in
// double: the float32 terms of either sign may cancel).
__global__ void __launch_bounds__(1024) loss_stats_kernel(const __grid_constant__ LossArgs a)
{
    __shared__ double part[32][4];
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

template <typename E>
cudaError_t launch_rows(const LossArgs &a, cudaStream_t s)
{
    // CTAs per row: one when the rows alone fill the GPU, else up to 8, while a
    // slice keeps 2048 elements; threads: 16 elements each at most, 1024 at most
    int parts = 1;
    while (parts < 8 && a.T * parts * 2 <= kSMs * 2 && a.V / (parts * 2) >= 2048)
        parts *= 2;
    const int64_t slice = (a.V + parts - 1) / parts;
    int threads = 128;
    while (threads < 1024 && threads * 16 < slice)
        threads *= 2;
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
    return cudaLaunchKernelEx(&cfg, policy_loss_kernel<E>, a);
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
        loss_stats_kernel<<<1, 1024, 0, s>>>(a);
        e = cudaGetLastError();
    }
    return e;
}

}  // namespace gg
