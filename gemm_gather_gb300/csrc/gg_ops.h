// Declarations shared by the operators' translation units (host side): the
// linear layer (linear_kernels.cu), the policy loss (loss_kernels.cu), AdamW
// (adamw_kernels.cu), the norm and 8-bit activations (norm_kernels.cu) and the
// vocabulary's cross entropy (entropy_kernels.cu, its products in linear_kernels.cu),
// whose C entry points are in gg_ops.cu and gg_block_ops.cu.
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
constexpr int kEpiGradIn8 = 3;  // acc * act'(aux), aux kept in 8 bits (codes, with scales)
// The vocabulary's products (entropy_kernels.cu): i is a vocabulary entry of a piece, j a token.
constexpr int kEpiLse = 4;       // (largest, sum of exponentials) of 32 or 128 entries, and the target's logit
constexpr int kEpiSoftGrad = 5;  // coef (softmax - (i is the target)), in 16 bits
constexpr int kEpiVocab = 6;     // alpha acc (+ out): what the gradient of the logits is multiplied into
// kEpiGradW, kEpiVocab and kEpiLse of a contraction that is one chunk (linear_kernels.cu chooses them).
constexpr int kEpiGradWShort = 7, kEpiVocabShort = 8, kEpiLseShort = 9;

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
    const float *scales;   // kEpiGradIn8: aux's, one for GG_PACK_BLOCK features of a token
    int64_t lds;
    void *zout;
    int64_t ldz;
    int chunk;             // k-blocks accumulated in TMEM before they are added in registers
    int group;             // feature tiles per group of the tile order (pair kernel)
    int bt;                // tokens of a tile (pair kernel)
    int tiles_i, tiles_j, num_kb;  // feature and token tiles, k-blocks
    // The vocabulary's products.  live: the tokens there are, counted on the device (J or, with
    // live_k, K is the most there can be).
    const int *live;
    int live_k;
    const int *shares;     // kEpiVocab: of the contraction, share s into rows s J of out (null: 1)
    int most_shares;       // what *shares is at most: the grid has pairs for that many
    const int *target;     // a token's, within the vocabulary
    int v0;                // the piece's first entry
    float2 *partial;       // kEpiLse: a row for every 128 entries (split kernel: 32), a place per token
    int64_t ldpartial;
    float *ztarget;
    void *kept;            // kEpiLse on pairs: exp(acc - top) of entries kept0 on, in 16 bits, or null;
    float *kept_top;       // top, of every 32 entries: rows of ldpartial tokens
    int64_t ldkept, kept0;
    const float *largest, *inv, *tgrad;  // kEpiSoftGrad: a token's largest logit, coef / sum of exponentials, and
                                         // what comes out at its target
    const float *alpha;    // kEpiVocab; null: 1
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
// The same for what the gradient of a piece of logits is multiplied into (kEpiVocab), where it takes less
// than other_ns.
bool plan_vocab(const LinearArgs &dx, const LinearArgs &dw, double other_ns, int most_shares, int *bt_dx, int *bt_dw);
cudaError_t launch_both(int epi, const LinearArgs &dx, int bt_dx, const LinearArgs &dw, int bt_dw, cudaStream_t s,
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

// ---- norm, 8-bit activations (norm_kernels.cu) -------------------------------------
struct NormArgs {
    const void *x, *residual, *weight;
    int64_t ldx, ldr;
    int weight_f32, weight_vec;  // weight_vec: 16-byte loads of weights are aligned
    float eps;
    void *h, *y;
    int64_t ldh, ldy;
    uint8_t *codes;
    int64_t ldc;
    float *scales;
    int64_t lds;
    float *rstd;
    int64_t M, N;
    int is_bf16;
};
cudaError_t launch_norm(const NormArgs &a, cudaStream_t s);

struct NormBackwardArgs {
    const void *dy, *h, *weight, *dh_in;
    int64_t lddy, ldh, lddhin;
    const float *rstd;
    int weight_f32, weight_vec;
    void *dh, *dweight;
    int64_t lddh;
    int grad_f32, accumulate;
    float *partial;  // norm_backward_parts(M) rows of N sums, or null
    int64_t M, N;
    int is_bf16;
};
int norm_backward_parts(int64_t M);
cudaError_t launch_norm_backward(const NormBackwardArgs &a, cudaStream_t s);

struct PackArgs {
    const void *x;
    int64_t ldx;
    uint8_t *codes;
    int64_t ldc;
    float *scales;
    int64_t lds, M, N;
    int is_bf16;
};
cudaError_t launch_pack(const PackArgs &a, cudaStream_t s);

struct UnpackArgs {
    const uint8_t *codes;
    int64_t ldc;
    const float *scales;
    int64_t lds;
    int act;
    void *out;
    int64_t ldo, M, N;
    int is_bf16;
    void *rest;  // or null: what out's rounding left, rounded (pitch ldo)
};
cudaError_t launch_unpack(const UnpackArgs &a, cudaStream_t s);

// ---- cross entropy over a vocabulary (entropy_kernels.cu) ------------------------------
// What the device knows of a call, at the start of its workspace.
struct EntropyHead {
    int live, live_pad;  // tokens that count; the same in whole k-blocks of 64, at most T
    int shares;          // of dX's contraction
    unsigned ticket;     // blocks of the join that are done
    float scale;         // takes the largest |weight| to 2^13
    float alpha;         // grad_scale / scale
};

struct EntropyArgs {
    const void *X;
    int64_t ldx;
    const int64_t *target;  // per token, as the caller has them
    const float *weight;
    int64_t T, V, K;
    int is_bf16;
    float grad_scale;
    float *stats, *loss, *lse;
    void *dX;
    int64_t lddx;
    // workspace; "compact": the tokens that count, in their order
    EntropyHead *head;
    void *x;             // compact X, pitch ldw
    int64_t ldw;
    int *place;          // a token's compact place, or -1
    int *token;          // compact: its token
    int *tgt;            // compact targets (-1 behind the last)
    float *wt, *largest, *inv, *tgrad, *ztarget;  // (coef: weight scale; inv: coef / sum of exponentials; tgrad: the
                                                  // gradient of the target's logit, inv exp(ztarget - largest) - coef)
    void *sums;          // two doubles for every 32 tokens
    float2 *partial;     // rows x T
    int64_t rows;
    uint16_t *dz;        // compact gradient of a piece's logits, pitch piece
    int64_t piece;
    const float *kept_top;  // of the piece whose exponentials lie in dz (launch_entropy_kept)
    int64_t kept0, kept_n;
    float *dx32;         // compact dX before its rounding, pitch ldw, a share's T rows behind another's
    // What the shares are chosen by: those there is room for; dX's feature tiles, tokens of its tiles and
    // k-blocks of its contraction; dW's tiles.
    int most_shares, dx_tiles_i, dx_bt, dx_kb;
    int64_t dw_tiles;
    int *status;
};
cudaError_t launch_entropy_tokens(const EntropyArgs &a, cudaStream_t s);  // counts and gathers the tokens
cudaError_t launch_entropy_join(const EntropyArgs &a, cudaStream_t s);    // partial sums to losses
cudaError_t launch_entropy_kept(const EntropyArgs &a, cudaStream_t s);    // the kept exponentials to the gradient
cudaError_t launch_entropy_dx(const EntropyArgs &a, cudaStream_t s);      // dX, rounded, in the tokens' order

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
