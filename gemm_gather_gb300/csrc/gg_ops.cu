// C entry points of the operators: argument validation and launches.
// Declared in include/gemm_gather.h.
#include <cuda_runtime.h>

#include <cmath>

#include "gg_ops.h"

namespace {

using gg::op_cuda_fail;
using gg::op_fail;
using gg::op_ok;

constexpr int64_t kMaxSize = ((int64_t)1 << 31) - 1;

// A rows x cols matrix argument of a call (element size es, pitch in elements).
struct Mat {
    const char *name;
    const void *p;
    int64_t rows, cols, ld, es;

    uint64_t begin() const { return reinterpret_cast<uint64_t>(p); }
    uint64_t bytes() const
    {
        return rows > 0 && cols > 0 ? (uint64_t)((rows - 1) * ld + cols) * (uint64_t)es : 0;
    }
};

// Whether two matrices share an element's bytes.  Matrices of one pitch may
// interleave (column ranges of one buffer): their rows are compared then.
bool share(const Mat &a, const Mat &b)
{
    if (!a.p || !b.p || a.bytes() == 0 || b.bytes() == 0)
        return false;
    if (a.begin() + a.bytes() <= b.begin() || b.begin() + b.bytes() <= a.begin())
        return false;
    const uint64_t pa = (uint64_t)(a.ld * a.es), pb = (uint64_t)(b.ld * b.es);
    if (pa != pb || a.rows < 2 || b.rows < 2)
        return true;
    const Mat &lo = a.begin() <= b.begin() ? a : b, &hi = a.begin() <= b.begin() ? b : a;
    const uint64_t shift = (hi.begin() - lo.begin()) % pa;  // hi's first column within lo's row
    const uint64_t wl = (uint64_t)(lo.cols * lo.es), wh = (uint64_t)(hi.cols * hi.es);
    return !(shift >= wl && shift + wh <= pa);
}

bool same(const Mat &a, const Mat &b) { return a.p == b.p && a.ld == b.ld; }

gg_status check_mat(const Mat &m, bool needed)
{
    if (m.rows == 0 || m.cols == 0)
        return GG_OK;
    if (!m.p)
        return needed ? op_fail(GG_ERR_INVALID_ARG, "%s must be non-NULL", m.name) : GG_OK;
    if (m.ld < m.cols)
        return op_fail(GG_ERR_INVALID_ARG, "%s: the pitch %lld is below the row length %lld", m.name,
                       (long long)m.ld, (long long)m.cols);
    if (m.ld > INT64_MAX / 16 / (m.rows > 0 ? m.rows : 1))
        return op_fail(GG_ERR_UNSUPPORTED, "%s: its extent passes 2^59 bytes", m.name);
    if (m.begin() % (uint64_t)m.es != 0)
        return op_fail(GG_ERR_ALIGNMENT, "%s must be aligned to its %lld-byte elements", m.name,
                       (long long)m.es);
    return GG_OK;
}

// Matrices that tensor maps (or 16-byte loads) read.
gg_status check_tma(const Mat &m)
{
    if (m.rows == 0 || m.cols == 0)
        return GG_OK;
    if (m.begin() % 16 != 0 || m.ld % 8 != 0)
        return op_fail(GG_ERR_ALIGNMENT, "%s must be 16-byte aligned with a pitch that is a multiple "
                                         "of 8", m.name);
    if (m.ld >= (int64_t)1 << 39)  // a tensor map's strides are below 2^40 bytes
        return op_fail(GG_ERR_UNSUPPORTED, "%s: its pitch must be below 2^39 elements", m.name);
    return GG_OK;
}

gg_status check_apart(const Mat &out, const Mat &other)
{
    return share(out, other) ? op_fail(GG_ERR_INVALID_ARG, "%s overlaps %s", out.name, other.name)
                             : GG_OK;
}

gg_status check_sizes(int64_t M, int64_t N, int64_t K)
{
    if (M < 0 || N < 0 || K < 0)
        return op_fail(GG_ERR_INVALID_ARG, "sizes must be >= 0");
    if (M > kMaxSize || N > kMaxSize || K > kMaxSize)
        return op_fail(GG_ERR_UNSUPPORTED, "sizes must be below 2^31");
    return GG_OK;
}

gg_status check_types(gg_dtype dtype, gg_activation act, const char *what)
{
    if (dtype != GG_F16 && dtype != GG_BF16)
        return op_fail(GG_ERR_UNSUPPORTED, "%s takes GG_F16 or GG_BF16", what);
    if (act < GG_ACT_NONE || act > GG_ACT_SILU)
        return op_fail(GG_ERR_INVALID_ARG, "unknown activation %d", (int)act);
    return GG_OK;
}

gg_status check_route(gg_weight_layout layout, gg_linear_path path)
{
    if (layout != GG_WEIGHT_KN && layout != GG_WEIGHT_NK)
        return op_fail(GG_ERR_INVALID_ARG, "unknown weight layout %d", (int)layout);
    if (path != GG_LINEAR_AUTO && path != GG_LINEAR_SPLIT && path != GG_LINEAR_PAIR)
        return op_fail(GG_ERR_INVALID_ARG, "unknown linear path %d", (int)path);
    return GG_OK;
}

#define GG_TRY(x)                  \
    do {                           \
        const gg_status st_ = (x); \
        if (st_ != GG_OK)          \
            return st_;            \
    } while (0)

// Validation of gg_linear; *a and *plan describe the launch.
gg_status prepare_linear(const void *X, int64_t ldx, const void *W, int64_t ldw,
                         gg_weight_layout layout, const void *bias, gg_dtype bias_dtype,
                         gg_activation act, const void *residual, int64_t ldr, const void *Y,
                         int64_t ldy, const void *z, int64_t ldz, int64_t M, int64_t N, int64_t K,
                         gg_dtype dtype, gg_linear_path path, gg::LinearArgs *a, gg::LinearPlan *plan)
{
    *plan = gg::LinearPlan{};
    GG_TRY(check_types(dtype, act, "linear"));
    GG_TRY(check_route(layout, path));
    GG_TRY(check_sizes(M, N, K));
    if (bias && bias_dtype != dtype && bias_dtype != GG_F32)
        return op_fail(GG_ERR_UNSUPPORTED, "the bias is of the layer's type or GG_F32");
    const bool kn = layout == GG_WEIGHT_KN;
    const int64_t k = M > 0 && N > 0 ? K : 0;  // nothing is multiplied for an empty output
    const Mat x{"X", X, M, k, ldx, 2}, w{"W", W, kn ? k : N, kn ? N : k, ldw, 2};
    const Mat r{"residual", residual, M, N, ldr, 2}, y{"Y", Y, M, N, ldy, 2}, zz{"z", z, M, N, ldz, 2};
    const Mat b{"bias", bias, M > 0 ? 1 : 0, N, N, bias_dtype == GG_F32 ? 4 : 2};
    GG_TRY(check_mat(x, true));
    GG_TRY(check_mat(w, true));
    GG_TRY(check_mat(b, false));
    GG_TRY(check_mat(r, false));
    GG_TRY(check_mat(y, true));
    GG_TRY(check_mat(zz, false));
    GG_TRY(check_tma(x));
    GG_TRY(check_tma(w));
    for (const Mat *in : {&x, &w, &b, &r}) {
        if (!(in == &r && same(r, y)))
            GG_TRY(check_apart(y, *in));
        GG_TRY(check_apart(zz, *in));
    }
    GG_TRY(check_apart(zz, y));
    gg::LinearArgs l{};
    l.I = N;
    l.J = M;
    l.K = K;
    l.a = W;
    l.lda = ldw;
    l.a_mn = kn;
    l.b = X;
    l.ldb = ldx;
    l.b_mn = 0;
    l.is_bf16 = dtype == GG_BF16;
    l.out = const_cast<void *>(Y);
    l.ldo = ldy;
    l.bias = bias;
    l.bias_f32 = bias_dtype == GG_F32;
    l.act = act;
    l.aux = residual;
    l.ldaux = ldr;
    l.zout = const_cast<void *>(z);
    l.ldz = ldz;
    *a = l;
    *plan = gg::plan_linear(gg::kEpiForward, l, path);
    return op_ok();
}

// What a launch takes from the library's settings and the caller's status word.
gg_status fill_in(gg::LinearArgs *a, int *dev_status)
{
    a->status = dev_status;
    GG_TRY(gg::op_status_word(&a->status));
    a->wait_limit_ns = gg::op_wait_limit_ns();
    a->inject_stall = gg::op_inject_stall();
    return GG_OK;
}

gg_status run_product(int epi, gg::LinearArgs *a, const gg::LinearPlan &plan, int *dev_status,
                      gg_stream_t stream)
{
    if (a->I == 0 || a->J == 0)
        return op_ok();
    GG_TRY(fill_in(a, dev_status));
    const char *why = nullptr;
    const cudaError_t e =
        gg::launch_linear(epi, *a, plan, reinterpret_cast<cudaStream_t>(stream), &why);
    if (e != cudaSuccess)
        return op_cuda_fail(e, why ? why : "launching the linear kernel");
    return op_ok();
}

// What a validated gg_linear_backward call launches.
struct Backward {
    gg::LinearArgs dx, dw;
    gg::LinearPlan plan_dx, plan_dw;
    gg::ColSumArgs sum;
    bool run_dx, run_dw, run_sum;
    bool both;  // dX and dW in one launch, with these tiles
    int bt_dx, bt_dw;
};

gg_status prepare_backward(const void *dZ, int64_t lddz, const void *X, int64_t ldx, const void *W,
                           int64_t ldw, gg_weight_layout layout, const void *z_in, int64_t ldzin,
                           gg_activation act_in, const void *dX, int64_t lddx, const void *dW,
                           int64_t lddw, const void *dbias, gg_dtype grad_dtype, int accumulate,
                           int64_t M, int64_t N, int64_t K, gg_dtype dtype, gg_linear_path path,
                           Backward *out)
{
    Backward r{};
    GG_TRY(check_types(dtype, act_in, "linear_backward"));
    GG_TRY(check_route(layout, path));
    GG_TRY(check_sizes(M, N, K));
    if ((dW || dbias) && grad_dtype != dtype && grad_dtype != GG_F32)
        return op_fail(GG_ERR_UNSUPPORTED, "dW and dbias are of the layer's type or GG_F32");
    const bool kn = layout == GG_WEIGHT_KN;
    const int64_t ge = grad_dtype == GG_F32 ? 4 : 2;
    r.run_dx = dX && M > 0 && K > 0;
    r.run_dw = dW && K > 0 && N > 0;
    r.run_sum = dbias && N > 0;
    const bool any = r.run_dx || r.run_dw || r.run_sum;
    const Mat dz{"dZ", dZ, any ? M : 0, N, lddz, 2};
    const Mat x{"X", X, r.run_dw ? M : 0, K, ldx, 2};
    const int64_t wn = r.run_dx ? N : 0;
    const Mat w{"W", W, kn ? K : wn, kn ? wn : K, ldw, 2};
    const Mat zi{"z_in", z_in, r.run_dx ? M : 0, K, ldzin, 2};
    const Mat gx{"dX", dX, M, K, lddx, 2};
    const Mat gw{"dW", dW, kn ? K : N, kn ? N : K, lddw, ge}, gb{"dbias", dbias, 1, N, N, ge};
    GG_TRY(check_mat(dz, true));
    GG_TRY(check_mat(x, true));
    GG_TRY(check_mat(w, true));
    GG_TRY(check_mat(zi, false));
    GG_TRY(check_mat(gx, false));
    GG_TRY(check_mat(gw, false));
    GG_TRY(check_mat(gb, false));
    GG_TRY(check_tma(dz));
    GG_TRY(check_tma(x));
    GG_TRY(check_tma(w));
    const Mat *outs[] = {&gx, &gw, &gb};
    for (const Mat *o : outs) {
        for (const Mat *in : {&dz, &x, &w, &zi})
            if (!(o == &gx && in == &zi && same(gx, zi)))
                GG_TRY(check_apart(*o, *in));
        for (const Mat *p : outs)
            if (o < p)
                GG_TRY(check_apart(*o, *p));
    }
    gg::LinearArgs l{};
    l.is_bf16 = dtype == GG_BF16;
    r.dx = l;
    r.dx.I = K;
    r.dx.J = M;
    r.dx.K = N;
    r.dx.a = W;
    r.dx.lda = ldw;
    r.dx.a_mn = !kn;
    r.dx.b = dZ;
    r.dx.ldb = lddz;
    r.dx.out = const_cast<void *>(dX);
    r.dx.ldo = lddx;
    r.dx.act = act_in;
    r.dx.aux = z_in;
    r.dx.ldaux = ldzin;
    r.dw = l;
    r.dw.I = kn ? N : K;
    r.dw.J = kn ? K : N;
    r.dw.K = M;
    r.dw.a = kn ? dZ : X;
    r.dw.lda = kn ? lddz : ldx;
    r.dw.b = kn ? X : dZ;
    r.dw.ldb = kn ? ldx : lddz;
    r.dw.a_mn = r.dw.b_mn = 1;
    r.dw.out = const_cast<void *>(dW);
    r.dw.ldo = lddw;
    r.dw.out_f32 = grad_dtype == GG_F32;
    r.dw.accumulate = accumulate != 0;
    r.sum.x = dZ;
    r.sum.ldx = lddz;
    r.sum.J = M;
    r.sum.I = N;
    r.sum.is_bf16 = l.is_bf16;
    r.sum.out = const_cast<void *>(dbias);
    r.sum.out_f32 = grad_dtype == GG_F32;
    r.sum.accumulate = accumulate != 0;
    r.plan_dx = r.run_dx ? gg::plan_linear(gg::kEpiGradIn, r.dx, path)
                         : gg::LinearPlan{};
    r.plan_dw = r.run_dw ? gg::plan_linear(gg::kEpiGradW, r.dw, path)
                         : gg::LinearPlan{};
    r.both = r.run_dx && r.run_dw &&
             gg::plan_both(r.dx, r.dw, r.plan_dx, r.plan_dw, path, &r.bt_dx, &r.bt_dw);
    if (r.both)
        r.plan_dx.kernel = r.plan_dw.kernel = GG_LINEAR_PAIR;
    *out = r;
    return op_ok();
}

gg_status prepare_loss(const void *logits, int64_t ld, const int64_t *target, const float *old_logp,
                       const float *ref_logp, const float *advantage, const float *weight, int64_t T,
                       int64_t V, gg_dtype dtype, float inv_temperature, float clip_low,
                       float clip_high, float kl_coef, float grad_scale, const float *stats,
                       const float *logp_out, const void *dlogits, int64_t ldd, gg::LossArgs *out)
{
    if (dtype != GG_F16 && dtype != GG_BF16 && dtype != GG_F32)
        return op_fail(GG_ERR_INVALID_ARG, "unknown dtype %d", (int)dtype);
    GG_TRY(check_sizes(T, V, 0));
    if (T > 0 && V == 0)
        return op_fail(GG_ERR_INVALID_ARG, "a token needs a vocabulary: V must be >= 1");
    if (T > kMaxSize / 8)  // rows x CTAs of a cluster
        return op_fail(GG_ERR_UNSUPPORTED, "T must be below 2^28");
    if (!(inv_temperature > 0.0f) || !std::isfinite(inv_temperature))
        return op_fail(GG_ERR_INVALID_ARG, "inv_temperature must be positive and finite");
    if (!(clip_low >= 0.0f) || !(clip_high >= 0.0f))
        return op_fail(GG_ERR_INVALID_ARG, "clip_low and clip_high must be >= 0");
    if (!std::isfinite(kl_coef) || !std::isfinite(grad_scale))
        return op_fail(GG_ERR_INVALID_ARG, "kl_coef and grad_scale must be finite");
    const int64_t es = dtype == GG_F32 ? 4 : 2;
    const Mat x{"logits", logits, T, V, ld, es}, d{"dlogits", dlogits, T, V, ldd, es};
    const Mat tg{"target", target, 1, T, T, 8}, ol{"old_logp", old_logp, 1, T, T, 4},
        rl{"ref_logp", ref_logp, 1, T, T, 4}, ad{"advantage", advantage, 1, T, T, 4},
        we{"weight", weight, 1, T, T, 4}, lo{"logp_out", logp_out, 1, T, T, 4},
        st{"stats", stats, 1, 4, 4, 4};
    GG_TRY(check_mat(x, true));
    GG_TRY(check_mat(tg, true));
    GG_TRY(check_mat(ol, false));
    GG_TRY(check_mat(rl, false));
    GG_TRY(check_mat(ad, true));
    GG_TRY(check_mat(we, true));
    GG_TRY(check_mat(lo, true));
    GG_TRY(check_mat(st, false));
    GG_TRY(check_mat(d, false));
    const Mat *outs[] = {&d, &lo, &st};
    for (const Mat *o : outs) {
        for (const Mat *in : {&x, &tg, &ol, &rl, &ad, &we})
            if (!(o == &d && in == &x && same(d, x)))
                GG_TRY(check_apart(*o, *in));
        for (const Mat *p : outs)
            if (o < p)
                GG_TRY(check_apart(*o, *p));
    }
    *out = gg::LossArgs{logits,    ld,        target,  old_logp, ref_logp,
                        advantage, weight,    T,       V,        (int)dtype,
                        inv_temperature, clip_low, clip_high, kl_coef, grad_scale,
                        const_cast<float *>(stats), const_cast<float *>(logp_out),
                        const_cast<void *>(dlogits), ldd, nullptr, gg::op_wait_limit_ns(),
                        gg::op_inject_stall()};
    return op_ok();
}

gg_status prepare_adamw(const gg_adamw_tensor *tensors, int count, int64_t step, double lr,
                        double beta1, double beta2, double eps, double weight_decay,
                        const float *grad_scale, gg::AdamwStep *out)
{
    if (count < 0 || (count > 0 && !tensors))
        return op_fail(GG_ERR_INVALID_ARG, "count must be >= 0 and tensors non-NULL");
    if (step < 1)
        return op_fail(GG_ERR_INVALID_ARG, "step %lld: steps count from 1", (long long)step);
    if (!(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0))
        return op_fail(GG_ERR_INVALID_ARG, "beta1 and beta2 must be in [0, 1)");
    if (!std::isfinite(lr) || !(eps >= 0.0) || !std::isfinite(eps) || !std::isfinite(weight_decay))
        return op_fail(GG_ERR_INVALID_ARG, "lr, eps and weight_decay must be finite, eps >= 0");
    if (reinterpret_cast<uint64_t>(grad_scale) % 4)
        return op_fail(GG_ERR_ALIGNMENT, "grad_scale must be 4-byte aligned");
    for (int i = 0; i < count; ++i) {
        const gg_adamw_tensor &t = tensors[i];
        if (t.n < 0)
            return op_fail(GG_ERR_INVALID_ARG, "tensor %d: n must be >= 0", i);
        if (t.n > (int64_t)1 << 40)
            return op_fail(GG_ERR_UNSUPPORTED, "tensor %d: n must be at most 2^40", i);
        const auto known = [](gg_dtype d) { return d == GG_F16 || d == GG_BF16 || d == GG_F32; };
        if (!known(t.param_dtype) || !known(t.grad_dtype))
            return op_fail(GG_ERR_INVALID_ARG, "tensor %d: unknown dtype", i);
        if (t.state_bits != 32 && t.state_bits != 8)
            return op_fail(GG_ERR_UNSUPPORTED, "tensor %d: states have 32 or 8 bits", i);
        if (t.copy && t.copy_dtype != GG_F16 && t.copy_dtype != GG_BF16)
            return op_fail(GG_ERR_UNSUPPORTED, "tensor %d: the copy is GG_F16 or GG_BF16", i);
        const bool eight = t.state_bits == 8;
        if (t.n > 0 && (!t.param || !t.grad || !t.m || !t.v || (eight && (!t.m_scale || !t.v_scale))))
            return op_fail(GG_ERR_INVALID_ARG, "tensor %d: param, grad and states must be non-NULL", i);
        const int64_t pe = t.param_dtype == GG_F32 ? 4 : 2, ge = t.grad_dtype == GG_F32 ? 4 : 2;
        const int64_t blocks = eight ? (t.n + GG_ADAMW_BLOCK - 1) / GG_ADAMW_BLOCK : 0;
        // a few hundred tensors a step: plain comparisons, the names only for an error
        struct Span {
            uint64_t lo, hi;
            const char *name;
        } spans[7];
        int used = 0;
        const char *odd = nullptr;
        const auto add = [&](const void *p, int64_t n, int64_t es, const char *name) {
            const uint64_t lo = reinterpret_cast<uint64_t>(p);
            if (!p || n == 0)
                return;
            if (lo & (uint64_t)(es - 1))
                odd = name;
            spans[used++] = Span{lo, lo + (uint64_t)(n * es), name};
        };
        add(t.grad, t.n, ge, "grad");
        add(t.param, t.n, pe, "param");
        add(t.m, t.n, eight ? 1 : 4, "m");
        add(t.v, t.n, eight ? 1 : 4, "v");
        add(t.copy, t.n, 2, "copy");
        if (eight) {
            add(t.m_scale, blocks, 4, "m_scale");
            add(t.v_scale, blocks, 4, "v_scale");
        }
        if (odd)
            return op_fail(GG_ERR_ALIGNMENT, "tensor %d: %s must be aligned to its elements", i, odd);
        for (int x = 1; x < used; ++x)
            for (int y = 0; y < x; ++y)
                if (spans[x].lo < spans[y].hi && spans[y].lo < spans[x].hi)
                    return op_fail(GG_ERR_INVALID_ARG, "tensor %d: %s overlaps %s", i, spans[x].name,
                                   spans[y].name);
    }
    gg::AdamwStep h{};
    h.beta1 = (float)beta1;
    h.one_minus_beta1 = (float)(1.0 - beta1);
    h.beta2 = (float)beta2;
    h.one_minus_beta2 = (float)(1.0 - beta2);
    h.step_size = (float)(lr / (1.0 - std::pow(beta1, (double)step)));
    h.inv_sqrt_c2 = (float)(1.0 / std::sqrt(1.0 - std::pow(beta2, (double)step)));
    h.eps = (float)eps;
    h.decay = (float)(1.0 - lr * weight_decay);
    h.grad_scale = grad_scale;
    h.step = (uint32_t)step;
    *out = h;
    return op_ok();
}

}  // namespace

extern "C" {

gg_status gg_policy_loss(const void *logits, int64_t ld, const int64_t *target,
                         const float *old_logp, const float *ref_logp, const float *advantage,
                         const float *weight, int64_t T, int64_t V, gg_dtype dtype,
                         float inv_temperature, float clip_low, float clip_high, float kl_coef,
                         float grad_scale, float *stats, float *logp_out, void *dlogits,
                         int64_t ldd, int *dev_status, gg_stream_t stream)
{
    gg::LossArgs a;
    GG_TRY(prepare_loss(logits, ld, target, old_logp, ref_logp, advantage, weight, T, V, dtype,
                        inv_temperature, clip_low, clip_high, kl_coef, grad_scale, stats, logp_out,
                        dlogits, ldd, &a));
    if (T == 0 && !stats)
        return op_ok();
    a.status = dev_status;
    GG_TRY(gg::op_status_word(&a.status));
    const cudaError_t e = gg::launch_policy_loss(a, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? op_ok() : op_cuda_fail(e, "launching the policy loss");
}

gg_status gg_policy_loss_check(const void *logits, int64_t ld, const int64_t *target,
                               const float *old_logp, const float *ref_logp,
                               const float *advantage, const float *weight, int64_t T, int64_t V,
                               gg_dtype dtype, float inv_temperature, float clip_low,
                               float clip_high, float kl_coef, float grad_scale,
                               const float *stats, const float *logp_out, const void *dlogits,
                               int64_t ldd)
{
    gg::LossArgs a;
    return prepare_loss(logits, ld, target, old_logp, ref_logp, advantage, weight, T, V, dtype,
                        inv_temperature, clip_low, clip_high, kl_coef, grad_scale, stats, logp_out,
                        dlogits, ldd, &a);
}

gg_status gg_adamw(const gg_adamw_tensor *tensors, int count, int64_t step, double lr, double beta1,
                   double beta2, double eps, double weight_decay, const float *grad_scale,
                   uint64_t seed, gg_stream_t stream)
{
    gg::AdamwStep h;
    GG_TRY(prepare_adamw(tensors, count, step, lr, beta1, beta2, eps, weight_decay, grad_scale, &h));
    h.seed = seed;
    const cudaError_t e =
        gg::launch_adamw(tensors, count, h, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? op_ok() : op_cuda_fail(e, "launching AdamW");
}

gg_status gg_adamw_check(const gg_adamw_tensor *tensors, int count, int64_t step, double lr,
                         double beta1, double beta2, double eps, double weight_decay,
                         const float *grad_scale)
{
    gg::AdamwStep h;
    return prepare_adamw(tensors, count, step, lr, beta1, beta2, eps, weight_decay, grad_scale, &h);
}

gg_status gg_linear(const void *X, int64_t ldx, const void *W, int64_t ldw, gg_weight_layout layout,
                    const void *bias, gg_dtype bias_dtype, gg_activation act, const void *residual,
                    int64_t ldr, void *Y, int64_t ldy, void *z, int64_t ldz, int64_t M, int64_t N,
                    int64_t K, gg_dtype dtype, int *dev_status, gg_stream_t stream,
                    gg_linear_path path)
{
    gg::LinearArgs a;
    gg::LinearPlan plan;
    GG_TRY(prepare_linear(X, ldx, W, ldw, layout, bias, bias_dtype, act, residual, ldr, Y, ldy, z, ldz,
                          M, N, K, dtype, path, &a, &plan));
    return run_product(gg::kEpiForward, &a, plan, dev_status, stream);
}

gg_status gg_linear_check(const void *X, int64_t ldx, const void *W, int64_t ldw,
                          gg_weight_layout layout, const void *bias, gg_dtype bias_dtype,
                          gg_activation act, const void *residual, int64_t ldr, const void *Y,
                          int64_t ldy, const void *z, int64_t ldz, int64_t M, int64_t N, int64_t K,
                          gg_dtype dtype, gg_linear_path path, int *chosen)
{
    gg::LinearArgs a;
    gg::LinearPlan plan;
    const gg_status st = prepare_linear(X, ldx, W, ldw, layout, bias, bias_dtype, act, residual, ldr, Y,
                                        ldy, z, ldz, M, N, K, dtype, path, &a, &plan);
    if (chosen)
        *chosen = plan.kernel;
    return st;
}

gg_status gg_linear_backward(const void *dZ, int64_t lddz, const void *X, int64_t ldx, const void *W,
                             int64_t ldw, gg_weight_layout layout, const void *z_in, int64_t ldzin,
                             gg_activation act_in, void *dX, int64_t lddx, void *dW, int64_t lddw,
                             void *dbias, gg_dtype grad_dtype, int accumulate, int64_t M, int64_t N,
                             int64_t K, gg_dtype dtype, int *dev_status, gg_stream_t stream,
                             gg_linear_path path)
{
    Backward b;
    GG_TRY(prepare_backward(dZ, lddz, X, ldx, W, ldw, layout, z_in, ldzin, act_in, dX, lddx, dW, lddw,
                            dbias, grad_dtype, accumulate, M, N, K, dtype, path, &b));
    if (b.both) {
        GG_TRY(fill_in(&b.dx, dev_status));
        GG_TRY(fill_in(&b.dw, dev_status));
        const char *why = nullptr;
        const cudaError_t e = gg::launch_both(b.dx, b.bt_dx, b.dw, b.bt_dw,
                                              reinterpret_cast<cudaStream_t>(stream), &why);
        if (e != cudaSuccess)
            return op_cuda_fail(e, why ? why : "launching the gradients");
    } else {
        if (b.run_dx)
            GG_TRY(run_product(gg::kEpiGradIn, &b.dx, b.plan_dx, dev_status, stream));
        if (b.run_dw)
            GG_TRY(run_product(gg::kEpiGradW, &b.dw, b.plan_dw, dev_status, stream));
    }
    if (b.run_sum) {
        b.sum.beside = b.both || (b.run_dx && b.dx.I > 0 && b.dx.J > 0) || (b.run_dw && b.dw.I > 0 && b.dw.J > 0);
        const cudaError_t e = gg::launch_colsum(b.sum, reinterpret_cast<cudaStream_t>(stream));
        if (e != cudaSuccess)
            return op_cuda_fail(e, "launching the bias gradient");
    }
    return op_ok();
}

gg_status gg_linear_backward_check(const void *dZ, int64_t lddz, const void *X, int64_t ldx,
                                   const void *W, int64_t ldw, gg_weight_layout layout,
                                   const void *z_in, int64_t ldzin, gg_activation act_in,
                                   const void *dX, int64_t lddx, const void *dW, int64_t lddw,
                                   const void *dbias, gg_dtype grad_dtype, int accumulate, int64_t M,
                                   int64_t N, int64_t K, gg_dtype dtype, gg_linear_path path,
                                   int *chosen_dx, int *chosen_dw)
{
    Backward b{};
    const gg_status st =
        prepare_backward(dZ, lddz, X, ldx, W, ldw, layout, z_in, ldzin, act_in, dX, lddx, dW, lddw,
                         dbias, grad_dtype, accumulate, M, N, K, dtype, path, &b);
    if (chosen_dx)
        *chosen_dx = b.plan_dx.kernel;
    if (chosen_dw)
        *chosen_dw = b.plan_dw.kernel;
    return st;
}

gg_status gg_act_backward(const void *dy, int64_t lddy, const void *z, int64_t ldz, void *dz,
                          int64_t lddz, gg_activation act, int64_t M, int64_t N, gg_dtype dtype,
                          gg_stream_t stream)
{
    GG_TRY(check_types(dtype, act, "act_backward"));
    GG_TRY(check_sizes(M, N, 0));
    const Mat my{"dy", dy, M, N, lddy, 2}, mz{"z", z, M, N, ldz, 2}, out{"dz", dz, M, N, lddz, 2};
    GG_TRY(check_mat(my, true));
    GG_TRY(check_mat(mz, true));
    GG_TRY(check_mat(out, true));
    for (const Mat *in : {&my, &mz})
        if (!same(*in, out))
            GG_TRY(check_apart(out, *in));
    if (M == 0 || N == 0)
        return op_ok();
    gg::ActBackwardArgs a{dy, z, dz, lddy, ldz, lddz, M, N, dtype == GG_BF16, (int)act};
    const cudaError_t e = gg::launch_act_backward(a, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? op_ok() : op_cuda_fail(e, "launching the activation's backward pass");
}

}  // extern "C"
