// C entry points of the norm and of activations in 8 bits: argument validation and launches.
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
                                int accumulate, const void *workspace, size_t workspace_bytes, int64_t M, int64_t N,
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
    const size_t need = dweight ? gg_rms_norm_backward_workspace(M, N) : 0;
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

}  // namespace

extern "C" {

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
    return (size_t)norm_backward_parts(M) * (size_t)N * 4;
}

gg_status gg_rms_norm_backward(const void *dy, int64_t lddy, const void *h, int64_t ldh, const float *rstd,
                               const void *weight, gg_dtype weight_dtype, const void *dh_in, int64_t lddhin,
                               void *dh, int64_t lddh, void *dweight, gg_dtype grad_dtype, int accumulate,
                               void *workspace, size_t workspace_bytes, int64_t M, int64_t N, gg_dtype dtype,
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
                                     int accumulate, const void *workspace, size_t workspace_bytes, int64_t M,
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
                       dtype == GG_BF16};
    const cudaError_t e = launch_unpack(a, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? op_ok() : op_cuda_fail(e, "unpacking activations");
}

}  // extern "C"
