// Declarations shared by the operators' translation units (host side): the
// linear layer (linear_kernels.cu), the policy loss (loss_kernels.cu) and
// AdamW (adamw_kernels.cu), whose C entry points are in gg_ops.cu.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/gemm_gather.h"

namespace gg {

// ---- what gg_api.cu shares with the operators' entry points --------------------
gg_status op_fail(gg_status s, const char *fmt, ...);  // sets gg_last_error
gg_status op_ok();
gg_status op_cuda_fail(cudaError_t e, const char *what);
gg_status op_status_word(int **status);  // the caller's word, else the library's
uint64_t op_wait_limit_ns();
int op_inject_stall();

// ---- linear ----------------------------------------------------------------------
// out[j*ldo + i] = epilogue( sum_k A[i, k] B[j, k] ), i < I, j < J.  i is the
// contiguous index of the output (features), j its row (tokens); A and B are
// stored K-major (k contiguous) or MN-major (i or j contiguous).
constexpr int kEpiForward = 0;  // act(acc + bias) + aux, zout = acc + bias
constexpr int kEpiGradIn = 1;   // acc * act'(aux)
constexpr int kEpiGradW = 2;    // acc (+ out)

struct LinearArgs {
    int64_t I, J, K;
    const void *a, *b;
    int64_t lda, ldb;      // row pitches in elements
    int a_mn, b_mn;        // MN-major operands
    int is_bf16;           // operands (and 16-bit outputs): bfloat16, else binary16
    void *out;
    int64_t ldo;
    int out_f32, accumulate;  // kEpiGradW
    const void *bias;
    int bias_f32, act;
    const void *aux;       // residual (forward) or Z_in (input gradient); may be null
    int64_t ldaux;
    void *zout;
    int64_t ldz;
    int chunk;             // k-blocks accumulated in TMEM before they are added in registers
    int group;             // feature tiles per group of the tile order (pair kernel)
    int bt;                // tokens of a tile (pair kernel)
    int tiles_i, tiles_j, num_kb;  // feature and token tiles, k-blocks
    int skip;              // pairs of the grid past the end of the first product's walk
    int *status;
    uint64_t wait_limit_ns;
    int inject_stall;
};

// Which kernel a product runs, with its tile and split (see plan_linear).
struct LinearPlan {
    int kernel;  // GG_LINEAR_NONE / GG_LINEAR_SPLIT / GG_LINEAR_PAIR
    int bt;      // tokens per tile
    int split;   // CTAs (split kernel) or CTA pairs that share one tile's contraction
    double ns;   // the estimate it was chosen by
};
LinearPlan plan_linear(int epi, const LinearArgs &a, int path);
cudaError_t launch_linear(int epi, const LinearArgs &a, const LinearPlan &p, cudaStream_t s,
                          const char **why);

// Both gradients of a layer in one launch (plan_both: whether, and their tiles).
bool plan_both(const LinearArgs &dx, const LinearArgs &dw, const LinearPlan &plan_dx, const LinearPlan &plan_dw,
               int path, int *bt_dx, int *bt_dw);
cudaError_t launch_both(const LinearArgs &dx, int bt_dx, const LinearArgs &dw, int bt_dw, cudaStream_t s,
                        const char **why);

struct ColSumArgs {  // out[i] (+)= sum_j x[j*ldx + i]
    const void *x;
    int64_t ldx, J, I;
    int is_bf16;
    void *out;
    int out_f32, accumulate;
    int beside;  // launched after the products of the same call, which do not write what it reads
};
cudaError_t launch_colsum(const ColSumArgs &a, cudaStream_t s);

struct ActBackwardArgs {  // dz = dy * act'(z)
    const void *dy, *z;
    void *dz;
    int64_t lddy, ldz, lddz, M, N;
    int is_bf16, act;
};
cudaError_t launch_act_backward(const ActBackwardArgs &a, cudaStream_t s);

// ---- policy loss -------------------------------------------------------------------
struct LossArgs {
    const void *logits;
    int64_t ld;
    const int64_t *target;
    const float *old_logp, *ref_logp, *advantage, *weight;
    int64_t T, V;
    int dtype;  // GG_F16 / GG_BF16 / GG_F32
    float inv_temperature, clip_low, clip_high, kl_coef, grad_scale;
    float *stats, *logp_out;
    void *dlogits;
    int64_t ldd;
    int *status;
    uint64_t wait_limit_ns;
    int inject_stall;
};
cudaError_t launch_policy_loss(const LossArgs &a, cudaStream_t s);

// ---- AdamW ---------------------------------------------------------------------------
struct AdamwStep {  // one step's constants, rounded once from double
    float beta1, one_minus_beta1, beta2, one_minus_beta2;
    float step_size;   // lr / (1 - beta1^step)
    float inv_sqrt_c2; // 1 / sqrt(1 - beta2^step)
    float eps, decay;  // decay = 1 - lr * weight_decay
    const float *grad_scale;
    uint64_t seed;
    uint32_t step;
};
cudaError_t launch_adamw(const gg_adamw_tensor *tensors, int count, const AdamwStep &h,
                         cudaStream_t s);

}  // namespace gg
