// C entry points of the norm, of activations in 8 bits and of the vocabulary's cross entropy: argument
// validation and launches.
// Declared in include/gemm_gather.h.
#include <cuda_runtime.h>

#include <cmath>

#include "gg_ops.h"
#include "op_args.h"

namespace {

using namespace gg;

bool vectors(const void *p) { return reinterpret_cast<uint64_t>(p) % 16 == 0; }

int64_t blocks_of(int64_t N) { return (N + GG_PACK_BLOCK - 1) / GG_PACK_BLOCK; }

gg_status check_16bit(gg_dtype dtype, const char *what)
{
    return dtype == GG_F16 || dtype == GG_BF16 ? GG_OK
                                               : op_fail(GG_ERR_UNSUPPORTED, "%s takes GG_F16 or GG_BF16", what);
}

gg_status check_weight_type(gg_dtype type, gg_dtype dtype, const char *what)
{
    return type == dtype || type == GG_F32 ? GG_OK
                                           : op_fail(GG_ERR_UNSUPPORTED, "%s of the norm's type or GG_F32", what);
}

// Codes and scales of M x N elements, both or neither.
gg_status check_packed(const Mat &codes, const Mat &scales, bool needed)
{
    if (codes.rows > 0 && codes.cols > 0 && (codes.p == nullptr) != (scales.p == nullptr))
        return op_fail(GG_ERR_INVALID_ARG, "codes and scales go together");
    GG_TRY(check_mat(codes, needed));
    return check_mat(scales, needed);
}

gg_status prepare_norm(const void *x, int64_t ldx, const void *residual, int64_t ldr, const void *weight,
                       gg_dtype weight_dtype, float eps, const void *h, int64_t ldh, const void *y, int64_t ldy,
                       const void *codes, int64_t ldc, const float *scales, int64_t lds, const float *rstd,
                       int64_t M, int64_t N, gg_dtype dtype, NormArgs *out)
{
    GG_TRY(check_16bit(dtype, "rms_norm"));
    GG_TRY(check_weight_type(weight_dtype, dtype, "the weight is"));
    GG_TRY(check_sizes(M, N, 0));
    if (!(eps >= 0.0f) || !std::isfinite(eps))
        return op_fail(GG_ERR_INVALID_ARG, "eps must be finite and >= 0");
    const Mat mx{"x", x, M, N, ldx, 2}, mr{"residual", residual, M, N, ldr, 2}, mh{"h", h, M, N, ldh, 2},
        my{"y", y, M, N, ldy, 2}, mc{"codes", codes, M, N, ldc, 1}, ms{"scales", scales, M, blocks_of(N), lds, 4};
    const Mat mw{"weight", weight, M > 0 ? 1 : 0, N, N, weight_dtype == GG_F32 ? 4 : 2},
        mi{"rstd", rstd, N > 0 ? 1 : 0, M, M, 4};
    GG_TRY(check_mat(mx, true));
    GG_TRY(check_mat(mr, false));
    GG_TRY(check_mat(mw, true));
    GG_TRY(check_mat(mh, false));
    GG_TRY(check_mat(my, codes == nullptr));
    GG_TRY(check_packed(mc, ms, false));
    GG_TRY(check_mat(mi, false));
    const Mat *outs[] = {&mh, &my, &mc, &ms, &mi};
    for (const Mat *o : outs) {
        for (const Mat *in : {&mx, &mr, &mw})
            if (!((o == &mh || o == &my) && in != &mw && same(*o, *in)))
                GG_TRY(check_apart(*o, *in));
        for (const Mat *p : outs)
            if (o < p)
                GG_TRY(check_apart(*o, *p));
    }
    *out = NormArgs{x, residual, weight, ldx, ldr, weight_dtype == GG_F32, vectors(weight), eps,
                    const_cast<void *>(h), const_cast<void *>(y), ldh, ldy,
                    reinterpret_cast<uint8_t *>(const_cast<void *>(codes)), ldc, const_cast<float *>(scales), lds,
                    const_cast<float *>(rstd), M, N, dtype == GG_BF16};
    return op_ok();
}

gg_status prepare_norm_backward(const void *dy, int64_t lddy, const void *h, int64_t ldh, const float *rstd,
                                const void *weight, gg_dtype weight_dtype, const void *dh_in, int64_t lddhin,
                                const void *dh, int64_t lddh, const void *dweight, gg_dtype grad_dtype,
                                int accumulate, const void *workspace, uint64_t workspace_bytes, int64_t M, int64_t N,
                                gg_dtype dtype, NormBackwardArgs *out)
{
    GG_TRY(check_16bit(dtype, "rms_norm_backward"));
    GG_TRY(check_weight_type(weight_dtype, dtype, "the weight is"));
    if (dweight)
        GG_TRY(check_weight_type(grad_dtype, dtype, "dweight is"));
    GG_TRY(check_sizes(M, N, 0));
    const Mat my{"dy", dy, M, N, lddy, 2}, mh{"h", h, M, N, ldh, 2}, min{"dh_in", dh ? dh_in : nullptr, M, N, lddhin, 2},
        mo{"dh", dh, M, N, lddh, 2}, mi{"rstd", rstd, N > 0 ? 1 : 0, M, M, 4},
        mw{"weight", weight, M > 0 ? 1 : 0, N, N, weight_dtype == GG_F32 ? 4 : 2},
        mg{"dweight", dweight, 1, N, N, grad_dtype == GG_F32 ? 4 : 2};
    GG_TRY(check_mat(my, true));
    GG_TRY(check_mat(mh, true));
    GG_TRY(check_mat(mi, true));
    GG_TRY(check_mat(mw, true));
    GG_TRY(check_mat(min, false));
    GG_TRY(check_mat(mo, false));
    GG_TRY(check_mat(mg, false));
    const uint64_t need = dweight ? gg_rms_norm_backward_workspace(M, N) : 0;
    if (workspace_bytes < need || (need && !workspace))
        return op_fail(GG_ERR_INVALID_ARG, "workspace: %llu bytes are needed", (unsigned long long)need);
    const int64_t parts = need ? norm_backward_parts(M) : 0;
    const Mat ws{"workspace", workspace, parts, N, N, 4};
    GG_TRY(check_mat(ws, false));
    const Mat *outs[] = {&mo, &mg, &ws};
    for (const Mat *o : outs) {
        for (const Mat *in : {&my, &mh, &min, &mi, &mw})
            if (!(o == &mo && (in == &my || in == &mh || in == &min) && same(*o, *in)))
                GG_TRY(check_apart(*o, *in));
        for (const Mat *p : outs)
            if (o < p)
                GG_TRY(check_apart(*o, *p));
    }
    *out = NormBackwardArgs{dy, h, weight, dh ? dh_in : nullptr, lddy, ldh, lddhin, rstd, weight_dtype == GG_F32,
                            vectors(weight), const_cast<void *>(dh), const_cast<void *>(dweight), lddh,
                            grad_dtype == GG_F32, accumulate != 0,
                            need ? reinterpret_cast<float *>(const_cast<void *>(workspace)) : nullptr, M, N,
                            dtype == GG_BF16};
    return op_ok();
}

// ---- cross entropy --------------------------------------------------------------------------
// A piece of the vocabulary: as many columns as make the float32 additions of dX a small part of
// its products (8 bytes against 2 piece operations for an element of dX), so that the gradient of
// its logits is what takes memory; equal pieces, in whole 128.
constexpr int64_t kPiece = 32768;

// From which length of a logit's contraction the loss's product keeps the last piece's exponentials for the
// gradient, in place of a second product: 4096 tokens, V = 32768, with gradients: K = 256 375 us without and 401
// with, 512 464 and 477, 1024 674 and 639; 600 tokens: 101 and 94, 128 and 121, 175 and 160.
constexpr int64_t kKeepFrom = 512;

int64_t piece_of(int64_t V, int64_t piece)
{
    if (piece == 0) {
        const int64_t n = (V + kPiece - 1) / kPiece;
        piece = n > 0 ? (V + n - 1) / n : 0;
    }
    piece = (piece + 127) / 128 * 128;
    const int64_t most = (V + 127) / 128 * 128;
    return piece < most ? piece : most;
}

// The loss's product leaves a partial result of every 128 entries where CTA pairs compute it, else of
// every 32.  Beyond a few hundred tokens the pairs always do (the others would be slower, and the
// partial results an eighth of the 16-bit logits).
bool pairs_only(int64_t T, int64_t K) { return T > 512 && K > 0; }

int64_t partial_rows(int64_t V, bool pairs) { return pairs ? (V + 127) / 128 : (V + 31) / 32; }

// Shares of dX's contraction that there is room for (plan_vocab): few tokens that count leave most CTA pairs
// without a tile of dX otherwise.  A share is dX in float32; they may take a quarter of a gigabyte.
int most_shares(int64_t T, int64_t K)
{
    const uint64_t one = (uint64_t)T * (uint64_t)((K + 7) / 8 * 8) * 4;
    for (int s = 8; s > 1; s /= 2)
        if (one <= ((uint64_t)1 << 28) / (uint64_t)s)
            return s;
    return 1;
}

// The workspace's parts, one behind the other on 256-byte boundaries.
struct EntropyPlaces {
    uint64_t x, place, token, tgt, wt, sums, largest, inv, tgrad, ztarget, partial, dx32, dz, top, end;
};

EntropyPlaces entropy_places(int64_t T, int64_t V, int64_t K, int64_t piece, bool gradients)
{
    EntropyPlaces w{};
    uint64_t at = 256;  // EntropyHead
    const auto take = [&](uint64_t bytes) {
        const uint64_t here = at;
        at += (bytes + 255) / 256 * 256;
        return here;
    };
    const uint64_t t = (uint64_t)T, kp = (uint64_t)((K + 7) / 8 * 8);
    w.x = take(t * kp * 2);
    for (uint64_t *p : {&w.place, &w.token, &w.tgt, &w.wt, &w.largest, &w.inv, &w.tgrad, &w.ztarget})
        *p = take(t * 4);
    w.sums = take((t + 31) / 32 * 16);
    w.partial = take(t * (uint64_t)partial_rows(V, pairs_only(T, K)) * 8);
    if (gradients) {
        w.dx32 = take(t * kp * 4 * (uint64_t)most_shares(T, K));
        w.dz = take(t * (uint64_t)piece_of(V, piece) * 2);
        w.top = take(t * (uint64_t)(piece_of(V, piece) / 32) * 4);
    }
    w.end = at;
    return w;
}

struct Entropy {
    EntropyArgs a;
    const void *W;
    int64_t ldw;
    bool kn;
    void *dW;
    int64_t lddw;
    int grad_f32, accumulate;
};

gg_status prepare_entropy(const void *X, int64_t ldx, const void *W, int64_t ldw, gg_weight_layout layout,
                          const int64_t *target, const float *weight, const float *stats, const float *loss,
                          const float *lse, const void *dX, int64_t lddx, const void *dW, int64_t lddw,
                          gg_dtype grad_dtype, int accumulate, const void *workspace, uint64_t workspace_bytes,
                          int64_t T, int64_t V, int64_t K, gg_dtype dtype, int64_t piece, float grad_scale,
                          Entropy *out)
{
    GG_TRY(check_16bit(dtype, "linear_cross_entropy"));
    GG_TRY(check_route(layout, GG_LINEAR_AUTO));
    GG_TRY(check_sizes(T, V, K));
    if (T > 0 && V == 0)
        return op_fail(GG_ERR_INVALID_ARG, "a token needs a vocabulary: V must be >= 1");
    if (piece < 0 || piece % 128 != 0)
        return op_fail(GG_ERR_INVALID_ARG, "piece must be 0 or a positive multiple of 128");
    if (!std::isfinite(grad_scale))
        return op_fail(GG_ERR_INVALID_ARG, "grad_scale must be finite");
    if (dW && grad_dtype != dtype && grad_dtype != GG_F32)
        return op_fail(GG_ERR_UNSUPPORTED, "dW is of the layer's type or GG_F32");
    const bool kn = layout == GG_WEIGHT_KN;
    const int64_t used = T > 0 ? V : 0;  // entries that W is read for
    const Mat x{"X", X, T, K, ldx, 2}, w{"W", W, kn ? (T > 0 ? K : 0) : used, kn ? used : K, ldw, 2};
    const Mat tg{"target", target, 1, T, T, 8}, we{"weight", weight, 1, T, T, 4};
    const Mat st{"stats", stats, 1, 2, 2, 4}, lo{"loss", loss, 1, T, T, 4}, ls{"lse", lse, 1, T, T, 4};
    const Mat gx{"dX", dX, T, K, lddx, 2},
        gw{"dW", dW, kn ? K : V, kn ? V : K, lddw, grad_dtype == GG_F32 ? 4 : 2};
    GG_TRY(check_mat(x, true));
    GG_TRY(check_mat(w, true));
    GG_TRY(check_tma(x));
    GG_TRY(check_tma(w));
    GG_TRY(check_mat(tg, true));
    GG_TRY(check_mat(we, true));
    GG_TRY(check_mat(st, false));
    GG_TRY(check_mat(lo, true));
    GG_TRY(check_mat(ls, false));
    GG_TRY(check_mat(gx, false));
    GG_TRY(check_mat(gw, false));
    const bool gradients = dX || dW;
    const uint64_t need = T > 0 ? entropy_places(T, V, K, piece, gradients).end : 0;
    if (need >= (uint64_t)1 << 59)
        return op_fail(GG_ERR_UNSUPPORTED, "the workspace passes 2^59 bytes");
    if (workspace_bytes < need || (need && !workspace))
        return op_fail(GG_ERR_INVALID_ARG, "workspace: %llu bytes are needed", (unsigned long long)need);
    if (need && reinterpret_cast<uint64_t>(workspace) % 16 != 0)
        return op_fail(GG_ERR_ALIGNMENT, "workspace must be 16-byte aligned");
    const Mat ws{"workspace", workspace, need ? 1 : 0, (int64_t)need, (int64_t)need, 1};
    const Mat *outs[] = {&st, &lo, &ls, &gx, &gw, &ws};
    for (const Mat *o : outs) {
        for (const Mat *in : {&x, &w, &tg, &we})
            if (!(o == &gx && in == &x && same(gx, x)))
                GG_TRY(check_apart(*o, *in));
        for (const Mat *p : outs)
            if (o < p)
                GG_TRY(check_apart(*o, *p));
    }
    const EntropyPlaces at = entropy_places(T, V, K, piece, gradients);
    uint8_t *const base = reinterpret_cast<uint8_t *>(const_cast<void *>(workspace));
    const auto floats = [&](uint64_t o) { return reinterpret_cast<float *>(base + o); };
    const auto ints = [&](uint64_t o) { return reinterpret_cast<int *>(base + o); };
    Entropy e{};
    if (need) {
        e.a.head = reinterpret_cast<EntropyHead *>(base);
        e.a.x = base + at.x;
        e.a.place = ints(at.place);
        e.a.token = ints(at.token);
        e.a.tgt = ints(at.tgt);
        e.a.wt = floats(at.wt);
        e.a.sums = base + at.sums;
        e.a.largest = floats(at.largest);
        e.a.inv = floats(at.inv);
        e.a.tgrad = floats(at.tgrad);
        e.a.ztarget = floats(at.ztarget);
        e.a.partial = reinterpret_cast<float2 *>(base + at.partial);
        e.a.dx32 = gradients ? floats(at.dx32) : nullptr;
        e.a.dz = gradients ? reinterpret_cast<uint16_t *>(base + at.dz) : nullptr;
        e.a.kept_top = gradients ? floats(at.top) : nullptr;
    }
    e.a.X = X;
    e.a.ldx = ldx;
    e.a.target = target;
    e.a.weight = weight;
    e.a.T = T;
    e.a.V = V;
    e.a.K = K;
    e.a.is_bf16 = dtype == GG_BF16;
    e.a.grad_scale = grad_scale;
    e.a.stats = const_cast<float *>(stats);
    e.a.loss = const_cast<float *>(loss);
    e.a.lse = const_cast<float *>(lse);
    e.a.dX = const_cast<void *>(dX);
    e.a.lddx = lddx;
    e.a.ldw = (K + 7) / 8 * 8;
    e.W = W;
    e.ldw = ldw;
    e.kn = kn;
    e.dW = const_cast<void *>(dW);
    e.lddw = lddw;
    e.grad_f32 = grad_dtype == GG_F32;
    e.accumulate = accumulate != 0;
    e.a.piece = piece_of(V, piece);
    *out = e;
    return op_ok();
}

gg_status launched(cudaError_t e, const char *what) { return e == cudaSuccess ? GG_OK : op_cuda_fail(e, what); }

gg_status product(int epi, const LinearArgs &a, const LinearPlan &plan, cudaStream_t s)
{
    const char *why = nullptr;
    const cudaError_t e = launch_linear(epi, a, plan, s, &why);
    return launched(e, why ? why : "launching a product of the vocabulary");
}

gg_status product(int epi, const LinearArgs &a, cudaStream_t s)
{
    return product(epi, a, plan_linear(epi, a, GG_LINEAR_AUTO), s);
}

gg_status run_entropy(const Entropy &e, cudaStream_t s)
{
    EntropyArgs a = e.a;
    LinearArgs l{};
    l.is_bf16 = a.is_bf16;
    l.status = a.status;
    l.wait_limit_ns = op_wait_limit_ns();
    l.inject_stall = op_inject_stall();
    if (a.T == 0) {
        if (a.stats)
            GG_TRY(launched(cudaMemsetAsync(a.stats, 0, 8, s), "clearing the statistics"));
        if (e.dW && !e.accumulate) {  // the sum over no tokens
            l.I = e.kn ? a.V : a.K;
            l.J = e.kn ? a.K : a.V;
            l.out = e.dW;
            l.ldo = e.lddw;
            l.out_f32 = e.grad_f32;
            GG_TRY(product(kEpiGradW, l, s));
        }
        return op_ok();
    }
    const int64_t es = 2;
    const auto entries = [&](int64_t v0) {  // W from entry v0 on
        return reinterpret_cast<const uint8_t *>(e.W) + v0 * (e.kn ? 1 : e.ldw) * es;
    };
    // logits of entries v0 on: features are entries, columns are tokens
    const auto logits = [&](int64_t v0, int64_t n, const int *live) {
        LinearArgs z = l;
        z.I = n;
        z.J = a.T;
        z.K = a.K;
        z.a = entries(v0);
        z.lda = e.ldw;
        z.a_mn = e.kn;
        z.b = a.x;
        z.ldb = a.ldw;
        z.live = live;
        z.target = a.tgt;
        z.v0 = (int)v0;
        return z;
    };
    const bool gradients = (a.dX || e.dW) && a.K > 0;
    const int64_t last = (a.V - 1) / a.piece * a.piece;  // the last piece's first entry
    // dX and dW of a piece
    const auto gradient_of = [&](int64_t v0, LinearArgs *dx, LinearArgs *dw) {
        const int64_t n = a.V - v0 < a.piece ? a.V - v0 : a.piece;
        LinearArgs x = l, w = l;
        x.I = a.K;
        x.J = a.T;
        x.K = n;
        x.a = entries(v0);
        x.lda = e.ldw;
        x.a_mn = !e.kn;
        x.b = a.dz;
        x.ldb = a.piece;
        x.out = a.dx32;
        x.ldo = a.ldw;
        x.out_f32 = 1;
        x.accumulate = v0 != last;
        x.live = &a.head->live;
        w.I = e.kn ? n : a.K;
        w.J = e.kn ? a.K : n;
        w.K = a.T;
        w.a = e.kn ? (const void *)a.dz : a.x;
        w.lda = e.kn ? a.piece : a.ldw;
        w.b = e.kn ? a.x : (const void *)a.dz;
        w.ldb = e.kn ? a.ldw : a.piece;
        w.a_mn = w.b_mn = 1;
        w.out = reinterpret_cast<uint8_t *>(e.dW) + v0 * (e.kn ? 1 : e.lddw) * (e.grad_f32 ? 4 : 2);
        w.ldo = e.lddw;
        w.out_f32 = e.grad_f32;
        w.accumulate = e.accumulate;
        w.live = &a.head->live_pad;
        w.live_k = 1;
        w.alpha = &a.head->alpha;
        *dx = x;
        *dw = w;
    };
    // both in one walk of the pairs, or apart: chosen once, since the pieces are alike and share dX's rows
    LinearArgs x, w;
    bool both = false;
    int bt_dx = 0, bt_dw = 0;
    a.most_shares = 1;
    a.dx_bt = 1;
    if (gradients && a.dX && e.dW) {
        gradient_of(last > 0 ? 0 : last, &x, &w);  // (a whole piece)
        const double apart = plan_linear(kEpiVocab, x, GG_LINEAR_AUTO).ns + plan_linear(kEpiVocab, w, GG_LINEAR_AUTO).ns;
        both = plan_vocab(x, w, apart, most_shares(a.T, a.K), &bt_dx, &bt_dw);
    }
    if (both) {
        a.dx_tiles_i = (int)((x.I + 255) / 256);
        a.dx_bt = bt_dx;
        a.dx_kb = (int)((x.K + 63) / 64);
        const int room = most_shares(a.T, a.K), all = a.dx_kb / 16 > 1 ? a.dx_kb / 16 : 1;  // (tokens_kernel)
        a.most_shares = room < all ? room : all;
        a.dw_tiles = ((w.I + 255) / 256) * ((w.J + bt_dw - 1) / bt_dw);
    }
    GG_TRY(launched(launch_entropy_tokens(a, s), "gathering the tokens"));
    LinearArgs z = logits(0, a.V, &a.head->live);
    z.partial = a.partial;
    z.ldpartial = a.T;
    z.ztarget = a.ztarget;
    const LinearPlan plan = plan_linear(kEpiLse, z, pairs_only(a.T, a.K) ? GG_LINEAR_PAIR : GG_LINEAR_AUTO);
    a.rows = partial_rows(a.V, plan.kernel == GG_LINEAR_PAIR);
    const bool keeps = gradients && plan.kernel == GG_LINEAR_PAIR && a.K >= kKeepFrom;
    if (keeps) {
        a.kept0 = last;
        a.kept_n = a.V - last;
        z.kept = a.dz;
        z.ldkept = a.piece;
        z.kept0 = last;
        z.kept_top = const_cast<float *>(a.kept_top);
    }
    GG_TRY(product(kEpiLse, z, plan, s));
    GG_TRY(launched(launch_entropy_join(a, s), "joining the vocabulary's sums"));
    if (!gradients)
        return op_ok();
    // the last piece first: its logits may still be there
    for (int64_t v0 = last; v0 >= 0; v0 -= a.piece) {
        const int64_t n = a.V - v0 < a.piece ? a.V - v0 : a.piece;
        if (v0 == last && keeps) {
            GG_TRY(launched(launch_entropy_kept(a, s), "the gradient of the kept logits"));
        } else {
            z = logits(v0, n, &a.head->live_pad);
            z.largest = a.largest;
            z.inv = a.inv;
            z.tgrad = a.tgrad;
            z.out = a.dz;
            z.ldo = a.piece;
            GG_TRY(product(kEpiSoftGrad, z, s));
        }
        gradient_of(v0, &x, &w);
        if (both) {
            x.shares = &a.head->shares;
            x.most_shares = a.most_shares;
            const char *why = nullptr;
            const cudaError_t err = launch_both(kEpiVocab, x, bt_dx, w, bt_dw, s, &why);
            GG_TRY(launched(err, why ? why : "launching the gradients of a piece"));
        } else {
            if (a.dX)
                GG_TRY(product(kEpiVocab, x, s));
            if (e.dW)
                GG_TRY(product(kEpiVocab, w, s));
        }
    }
    if (a.dX)
        GG_TRY(launched(launch_entropy_dx(a, s), "rounding dX"));
    return op_ok();
}

}  // namespace

extern "C" {

uint64_t gg_linear_cross_entropy_workspace(int64_t T, int64_t V, int64_t K, int64_t piece, int gradients)
{
    if (T <= 0 || V <= 0 || K < 0 || T > kMaxSize || V > kMaxSize || K > kMaxSize || piece < 0 || piece > kMaxSize)
        return 0;
    return entropy_places(T, V, K, piece, gradients != 0).end;
}

gg_status gg_linear_cross_entropy(const void *X, int64_t ldx, const void *W, int64_t ldw, gg_weight_layout layout,
                                  const int64_t *target, const float *weight, float *stats, float *loss,
                                  float *lse, void *dX, int64_t lddx, void *dW, int64_t lddw, gg_dtype grad_dtype,
                                  int accumulate, void *workspace, uint64_t workspace_bytes, int64_t T, int64_t V,
                                  int64_t K, gg_dtype dtype, int64_t piece, float grad_scale, int *dev_status,
                                  gg_stream_t stream)
{
    Entropy e;
    GG_TRY(prepare_entropy(X, ldx, W, ldw, layout, target, weight, stats, loss, lse, dX, lddx, dW, lddw, grad_dtype,
                           accumulate, workspace, workspace_bytes, T, V, K, dtype, piece, grad_scale, &e));
    e.a.status = dev_status;
    GG_TRY(op_status_word(&e.a.status));
    return run_entropy(e, reinterpret_cast<cudaStream_t>(stream));
}

gg_status gg_linear_cross_entropy_check(const void *X, int64_t ldx, const void *W, int64_t ldw,
                                        gg_weight_layout layout, const int64_t *target, const float *weight,
                                        const float *stats, const float *loss, const float *lse, const void *dX,
                                        int64_t lddx, const void *dW, int64_t lddw, gg_dtype grad_dtype,
                                        int accumulate, const void *workspace, uint64_t workspace_bytes, int64_t T,
                                        int64_t V, int64_t K, gg_dtype dtype, int64_t piece, float grad_scale)
{
    Entropy e;
    return prepare_entropy(X, ldx, W, ldw, layout, target, weight, stats, loss, lse, dX, lddx, dW, lddw, grad_dtype,
                           accumulate, workspace, workspace_bytes, T, V, K, dtype, piece, grad_scale, &e);
}

gg_status gg_rms_norm(const void *x, int64_t ldx, const void *residual, int64_t ldr, const void *weight,
                      gg_dtype weight_dtype, float eps, void *h, int64_t ldh, void *y, int64_t ldy, void *codes,
                      int64_t ldc, float *scales, int64_t lds, float *rstd, int64_t M, int64_t N, gg_dtype dtype,
                      gg_stream_t stream)
{
    NormArgs a;
    GG_TRY(prepare_norm(x, ldx, residual, ldr, weight, weight_dtype, eps, h, ldh, y, ldy, codes, ldc, scales, lds,
                        rstd, M, N, dtype, &a));
    if (M == 0 || N == 0)
        return op_ok();
    const cudaError_t e = launch_norm(a, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? op_ok() : op_cuda_fail(e, "launching the norm");
}

gg_status gg_rms_norm_check(const void *x, int64_t ldx, const void *residual, int64_t ldr, const void *weight,
                            gg_dtype weight_dtype, float eps, const void *h, int64_t ldh, const void *y,
                            int64_t ldy, const void *codes, int64_t ldc, const float *scales, int64_t lds,
                            const float *rstd, int64_t M, int64_t N, gg_dtype dtype)
{
    NormArgs a;
    return prepare_norm(x, ldx, residual, ldr, weight, weight_dtype, eps, h, ldh, y, ldy, codes, ldc, scales, lds,
                        rstd, M, N, dtype, &a);
}

uint64_t gg_rms_norm_backward_workspace(int64_t M, int64_t N)
{
    if (M <= 0 || N <= 0 || M > kMaxSize || N > kMaxSize)
        return 0;
    return (uint64_t)norm_backward_parts(M) * (uint64_t)N * 4;
}

gg_status gg_rms_norm_backward(const void *dy, int64_t lddy, const void *h, int64_t ldh, const float *rstd,
                               const void *weight, gg_dtype weight_dtype, const void *dh_in, int64_t lddhin,
                               void *dh, int64_t lddh, void *dweight, gg_dtype grad_dtype, int accumulate,
                               void *workspace, uint64_t workspace_bytes, int64_t M, int64_t N, gg_dtype dtype,
                               gg_stream_t stream)
{
    NormBackwardArgs a;
    GG_TRY(prepare_norm_backward(dy, lddy, h, ldh, rstd, weight, weight_dtype, dh_in, lddhin, dh, lddh, dweight,
                                 grad_dtype, accumulate, workspace, workspace_bytes, M, N, dtype, &a));
    if (N == 0 || (!a.dweight && (M == 0 || !a.dh)))
        return op_ok();
    const cudaError_t e = launch_norm_backward(a, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? op_ok() : op_cuda_fail(e, "launching the norm's backward pass");
}

gg_status gg_rms_norm_backward_check(const void *dy, int64_t lddy, const void *h, int64_t ldh, const float *rstd,
                                     const void *weight, gg_dtype weight_dtype, const void *dh_in, int64_t lddhin,
                                     const void *dh, int64_t lddh, const void *dweight, gg_dtype grad_dtype,
                                     int accumulate, const void *workspace, uint64_t workspace_bytes, int64_t M,
                                     int64_t N, gg_dtype dtype)
{
    NormBackwardArgs a;
    return prepare_norm_backward(dy, lddy, h, ldh, rstd, weight, weight_dtype, dh_in, lddhin, dh, lddh, dweight,
                                 grad_dtype, accumulate, workspace, workspace_bytes, M, N, dtype, &a);
}

gg_status gg_pack8(const void *x, int64_t ldx, void *codes, int64_t ldc, float *scales, int64_t lds, int64_t M,
                   int64_t N, gg_dtype dtype, gg_stream_t stream)
{
    GG_TRY(check_16bit(dtype, "pack8"));
    GG_TRY(check_sizes(M, N, 0));
    const Mat mx{"x", x, M, N, ldx, 2}, mc{"codes", codes, M, N, ldc, 1}, ms{"scales", scales, M, blocks_of(N), lds, 4};
    GG_TRY(check_mat(mx, true));
    GG_TRY(check_packed(mc, ms, true));
    GG_TRY(check_apart(mc, mx));
    GG_TRY(check_apart(ms, mx));
    GG_TRY(check_apart(ms, mc));
    if (M == 0 || N == 0)
        return op_ok();
    const PackArgs a{x, ldx, reinterpret_cast<uint8_t *>(codes), ldc, scales, lds, M, N, dtype == GG_BF16};
    const cudaError_t e = launch_pack(a, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? op_ok() : op_cuda_fail(e, "packing activations");
}

gg_status gg_unpack8(const void *codes, int64_t ldc, const float *scales, int64_t lds, gg_activation act, void *out,
                     int64_t ldo, int64_t M, int64_t N, gg_dtype dtype, gg_stream_t stream)
{
    GG_TRY(check_types(dtype, act, "unpack8"));
    GG_TRY(check_sizes(M, N, 0));
    const Mat mo{"out", out, M, N, ldo, 2}, mc{"codes", codes, M, N, ldc, 1}, ms{"scales", scales, M, blocks_of(N), lds, 4};
    GG_TRY(check_packed(mc, ms, true));
    GG_TRY(check_mat(mo, true));
    GG_TRY(check_apart(mo, mc));
    GG_TRY(check_apart(mo, ms));
    if (M == 0 || N == 0)
        return op_ok();
    const UnpackArgs a{reinterpret_cast<const uint8_t *>(codes), ldc, scales, lds, (int)act, out, ldo, M, N,
                       dtype == GG_BF16, nullptr};
    const cudaError_t e = launch_unpack(a, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? op_ok() : op_cuda_fail(e, "unpacking activations");
}

}  // extern "C"
