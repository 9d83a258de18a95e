// C entry points of the operators: argument validation and launches.
// Declared in include/gemm_gather.h.
#include <cuda_runtime.h>

#include <cmath>

#include "gg_ops.h"
#include "op_args.h"

namespace {

using namespace gg;

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
    int epi_dx; // kEpiGradIn, or kEpiGradIn8 where z_in is kept in 8 bits
};

gg_status prepare_backward(const void *dZ, int64_t lddz, const void *X, int64_t ldx, const void *W,
                           int64_t ldw, gg_weight_layout layout, const void *z_in, int64_t ldzin,
                           gg_activation act_in, const void *dX, int64_t lddx, const void *dW,
                           int64_t lddw, const void *dbias, gg_dtype grad_dtype, int accumulate,
                           int64_t M, int64_t N, int64_t K, gg_dtype dtype, gg_linear_path path,
                           Backward *out)
{
    Backward r{};
    r.epi_dx = gg::kEpiGradIn;
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

gg_status run_backward(Backward *b, int *dev_status, gg_stream_t stream)
{
    if (b->both) {
        GG_TRY(fill_in(&b->dx, dev_status));
        GG_TRY(fill_in(&b->dw, dev_status));
        const char *why = nullptr;
        const cudaError_t e = gg::launch_both(b->epi_dx, b->dx, b->bt_dx, b->dw, b->bt_dw,
                                              reinterpret_cast<cudaStream_t>(stream), &why);
        if (e != cudaSuccess)
            return op_cuda_fail(e, why ? why : "launching the gradients");
    } else {
        if (b->run_dx)
            GG_TRY(run_product(b->epi_dx, &b->dx, b->plan_dx, dev_status, stream));
        if (b->run_dw)
            GG_TRY(run_product(gg::kEpiGradW, &b->dw, b->plan_dw, dev_status, stream));
    }
    if (b->run_sum) {
        b->sum.beside = b->both || (b->run_dx && b->dx.I > 0 && b->dx.J > 0) || (b->run_dw && b->dw.I > 0 && b->dw.J > 0);
        const cudaError_t e = gg::launch_colsum(b->sum, reinterpret_cast<cudaStream_t>(stream));
        if (e != cudaSuccess)
            return op_cuda_fail(e, "launching the bias gradient");
    }
    return op_ok();
}

// Device bytes of gg_linear_backward8: `parts` matrices of 16 bits, X and (2) what that rounding left of it, rows
// on 16-byte boundaries.
int64_t unpacked_pitch(int64_t K) { return (K + 7) / 8 * 8; }
uint64_t unpacked_bytes(int64_t M, int64_t K, int parts)
{
    return (uint64_t)parts * (uint64_t)M * (uint64_t)unpacked_pitch(K) * 2;
}

// Whether act(P) needs more than 16 bits where float32 is to come of it: P itself and max(P, 0) do not.  (A gradient in
// 16 bits takes X in 16 bits, as the forward product read it: bfloat16, 777 tokens, silu, 2.4e-3 from the gradient of an
// unrounded X, of which 1.7e-3 is the output's own rounding.)
bool smooth(gg_activation act) { return act != GG_ACT_NONE && act != GG_ACT_RELU; }

// Validation of gg_linear_backward8: the plan of gg_linear_backward on the unpacked X, with z_in read
// from the codes.  *u: what unpacks X (M == 0 where nothing reads it); *rest: the product that adds what X's
// rounding to 16 bits left (J == 0: none).
gg_status prepare_backward8(const void *dZ, int64_t lddz, const void *codes, int64_t ldc, const float *scales,
                            int64_t lds, gg_activation act, const void *W, int64_t ldw, gg_weight_layout layout,
                            const void *dX, int64_t lddx, const void *dW, int64_t lddw, const void *dbias,
                            gg_dtype grad_dtype, int accumulate, const void *workspace, uint64_t workspace_bytes,
                            int64_t M, int64_t N, int64_t K, gg_dtype dtype, gg_linear_path path, Backward *out,
                            gg::UnpackArgs *u, gg::LinearArgs *rest)
{
    GG_TRY(check_types(dtype, act, "linear_backward8"));
    GG_TRY(check_sizes(M, N, K));
    const bool x = dW && N > 0, z = dX && act != GG_ACT_NONE;  // what the codes are read for
    const bool unpacks = x && M > 0 && K > 0;
    const int64_t rows = x || z ? M : 0;
    const Mat c{"codes", codes, rows, K, ldc, 1},
        sc{"scales", scales, rows, (K + GG_PACK_BLOCK - 1) / GG_PACK_BLOCK, lds, 4};
    GG_TRY(check_mat(c, true));
    GG_TRY(check_mat(sc, true));
    // Float32 gradients are those of act(P), not of its rounding: X goes through the product in two parts
    const bool two = unpacks && grad_dtype == GG_F32 && smooth(act);
    const int64_t ldx = unpacked_pitch(K);
    const Mat ws{"workspace", workspace, unpacks ? (two ? 2 * M : M) : 0, ldx, ldx, 2};
    const uint64_t need = unpacks ? unpacked_bytes(M, K, two ? 2 : 1) : 0;
    if (need && (!workspace || workspace_bytes < need))
        return op_fail(GG_ERR_INVALID_ARG, "workspace: %llu bytes are needed", (unsigned long long)need);
    Backward r;
    // the workspace is checked as X is: 16-byte aligned, apart from the outputs
    GG_TRY(prepare_backward(dZ, lddz, unpacks ? workspace : nullptr, ldx, W, ldw, layout, nullptr, 0, act, dX, lddx,
                            dW, lddw, dbias, grad_dtype, accumulate, M, N, K, dtype, path, &r));
    const bool kn = layout == GG_WEIGHT_KN;
    const int64_t ge = grad_dtype == GG_F32 ? 4 : 2;
    const Mat gx{"dX", dX, M, K, lddx, 2}, gw{"dW", dW, kn ? K : N, kn ? N : K, lddw, ge}, gb{"dbias", dbias, 1, N, N, ge};
    for (const Mat *in : {&c, &sc}) {
        for (const Mat *o : {&gx, &gw, &gb})
            GG_TRY(check_apart(*o, *in));
        GG_TRY(check_apart(ws, *in));
    }
    for (const Mat *o : {&gx, &gw, &gb})
        GG_TRY(check_apart(*o, ws));
    const Mat dz{"dZ", dZ, M, N, lddz, 2}, w{"W", W, r.run_dx ? (kn ? K : N) : 0, kn ? N : K, ldw, 2};
    GG_TRY(check_apart(ws, dz));
    GG_TRY(check_apart(ws, w));
    r.epi_dx = gg::kEpiGradIn8;
    r.dx.aux = act != GG_ACT_NONE ? codes : nullptr;
    r.dx.ldaux = ldc;
    r.dx.scales = scales;
    r.dx.lds = lds;
    *out = r;
    uint16_t *const x16 = reinterpret_cast<uint16_t *>(const_cast<void *>(workspace));
    *rest = gg::LinearArgs{};
    if (two) {
        *rest = r.dw;
        (kn ? rest->b : rest->a) = x16 + M * ldx;
        rest->accumulate = 1;
    }
    *u = gg::UnpackArgs{reinterpret_cast<const uint8_t *>(codes), ldc, scales, lds, (int)act, x16, ldx,
                        unpacks ? M : 0, K, dtype == GG_BF16, two ? x16 + M * ldx : nullptr};
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
    return run_backward(&b, dev_status, stream);
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

gg_status gg_linear_backward8(const void *dZ, int64_t lddz, const void *codes, int64_t ldc, const float *scales,
                              int64_t lds, gg_activation act, const void *W, int64_t ldw, gg_weight_layout layout,
                              void *dX, int64_t lddx, void *dW, int64_t lddw, void *dbias, gg_dtype grad_dtype,
                              int accumulate, void *workspace, uint64_t workspace_bytes, int64_t M, int64_t N,
                              int64_t K, gg_dtype dtype, int *dev_status, gg_stream_t stream, gg_linear_path path)
{
    Backward b;
    gg::UnpackArgs u;
    gg::LinearArgs rest;
    GG_TRY(prepare_backward8(dZ, lddz, codes, ldc, scales, lds, act, W, ldw, layout, dX, lddx, dW, lddw, dbias,
                             grad_dtype, accumulate, workspace, workspace_bytes, M, N, K, dtype, path, &b, &u, &rest));
    if (u.M > 0) {
        const cudaError_t e = gg::launch_unpack(u, reinterpret_cast<cudaStream_t>(stream));
        if (e != cudaSuccess)
            return op_cuda_fail(e, "unpacking the activations");
    }
    GG_TRY(run_backward(&b, dev_status, stream));
    return run_product(gg::kEpiGradW, &rest, gg::plan_linear(gg::kEpiGradW, rest, path), dev_status, stream);
}

gg_status gg_linear_backward8_check(const void *dZ, int64_t lddz, const void *codes, int64_t ldc,
                                    const float *scales, int64_t lds, gg_activation act, const void *W,
                                    int64_t ldw, gg_weight_layout layout, const void *dX, int64_t lddx,
                                    const void *dW, int64_t lddw, const void *dbias, gg_dtype grad_dtype,
                                    int accumulate, const void *workspace, uint64_t workspace_bytes, int64_t M,
                                    int64_t N, int64_t K, gg_dtype dtype, gg_linear_path path, int *chosen_dx,
                                    int *chosen_dw)
{
    Backward b{};
    gg::UnpackArgs u;
    gg::LinearArgs rest;
    const gg_status st = prepare_backward8(dZ, lddz, codes, ldc, scales, lds, act, W, ldw, layout, dX, lddx, dW,
                                           lddw, dbias, grad_dtype, accumulate, workspace, workspace_bytes, M, N,
                                           K, dtype, path, &b, &u, &rest);
    if (chosen_dx)
        *chosen_dx = b.plan_dx.kernel;
    if (chosen_dw)
        *chosen_dw = b.plan_dw.kernel;
    return st;
}

uint64_t gg_linear_backward8_workspace(int64_t M, int64_t K)
{
    return M > 0 && K > 0 && M <= kMaxSize && K <= kMaxSize ? unpacked_bytes(M, K, 2) : 0;
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
