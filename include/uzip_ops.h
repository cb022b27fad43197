/*
 * uzip -- matrix products over the tensors that the codec stores (C ABI).
 *
 * A decompressed weight is multiplied, and the gradients that are compressed
 * come out of the same products.  Three operators, with their gradients:
 *   uzip_linear          y = act(x W^T + b) + r
 *   uzip_grouped_linear  the same product grouped by expert: rows
 *                        [offsets[e], offsets[e+1]) of x use W[e] and b[e]
 *   uzip_cross_entropy   loss_i = log(sum_j exp(s_ij)) - s_{i,t_i} with
 *                        s = h W^T, whose logits s are never stored
 *
 * Common rules.
 *   - Values are bf16 or fp16 (UZIP_BF16, UZIP_FP16), products are summed in
 *     32 bits and every result is rounded once; losses are fp32.  (The tensor
 *     cores cut their additions toward zero: a sum of one sign comes out short
 *     by 1e-4 of itself at 16384 terms and by 1.3e-4 at 2^20.)  Another dtype
 *     is UZIP_ERR_UNSUPPORTED_DTYPE.
 *   - Matrices are row-major with a row stride `ld` in elements, at least the
 *     row's length (a matrix of at most one row may give any).  Any element
 *     alignment and any stride are accepted; operands whose rows do not start
 *     on 16-byte boundaries are first copied into the workspace.
 *   - The library allocates nothing: the caller gives a workspace of
 *     uzip_*_workspace_size(args) bytes, 256-byte aligned (NULL where that is
 *     0), used until the call's work on the stream ends.  Calls that share no
 *     output and no workspace may overlap.
 *   - m, n, k below 2^31, at most 1024 groups.  Lengths of zero are fine.
 *   - Outputs must not overlap inputs or each other.
 *   - d_status (device i32, nullable) receives 0, or a uzip_status found on
 *     the device: UZIP_ERR_INVALID_ARG for bad offsets or targets (see
 *     there), UZIP_ERR_TIMEOUT when a bounded wait ran out (what was to be
 *     computed there is then NaN).
 *   - The same inputs give the same bits: no sum depends on the order in
 *     which blocks run.
 */
#ifndef UZIP_OPS_H
#define UZIP_OPS_H

#include "uzip.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    UZIP_ACT_NONE = 0,
    UZIP_ACT_RELU = 1,
    UZIP_ACT_GELU = 2, /* z Phi(z), with the error function */
    UZIP_ACT_SILU = 3  /* z / (1 + exp(-z)) */
} uzip_act;

#define UZIP_MAX_GROUPS 1024

/* Arguments of a product and of its gradient.  Dense: groups = 0 and
 * offsets = NULL.  Grouped: w is [groups, n, k] with w_group elements from one
 * expert to the next (at least what one extends over), bias [groups, n] contiguous, offsets groups + 1 device
 * int64 values that start at 0, never decrease and end at m.  Offsets that do
 * not are reported in d_status and every output is filled with NaN. */
typedef struct {
    int32_t dtype; /* uzip_dtype of every value */
    int32_t act;   /* uzip_act */
    int64_t m, n, k;
    int64_t groups;
    const int64_t* offsets;
    const void* x; /* [m, k] */
    int64_t ldx;
    const void* w; /* [n, k] or [groups, n, k] */
    int64_t ldw, w_group;
    const void* bias;     /* [n] or [groups, n], nullable */
    const void* residual; /* [m, n], nullable; added after the activation */
    int64_t ldr;
    void* y; /* [m, n] */
    int64_t ldy;
    void* z; /* [m, n], nullable: x W^T + b before the activation, for the gradient */
    int64_t ldz;
} uzip_linear_args;

uint64_t uzip_linear_workspace_size(const uzip_linear_args* a);
uzip_status uzip_linear(const uzip_linear_args* a, void* d_workspace, uint64_t workspace_bytes, int32_t* d_status,
                        cudaStream_t s);
uint64_t uzip_grouped_linear_workspace_size(const uzip_linear_args* a);
uzip_status uzip_grouped_linear(const uzip_linear_args* a, void* d_workspace, uint64_t workspace_bytes,
                                int32_t* d_status, cudaStream_t s);

/* Gradients, with dz = dy act'(z): dx = dz W, dw = dz^T x (for each expert
 * over its own rows; zero for one without rows), db = column sums of dz.  The
 * residual's gradient is dy itself.  Each of dx, dw, db may be NULL.  dz is
 * rounded to the dtype for the two products (tensor cores take 16-bit
 * operands); db sums it unrounded.  z is what uzip_linear stored: values that
 * relu's slope turns on were summed again there where the tensor core's sum
 * came within its own error of zero, and a positive one that the dtype cannot
 * hold is stored as its smallest value. */
typedef struct {
    int32_t dtype;
    int32_t act;
    int64_t m, n, k;
    int64_t groups;
    const int64_t* offsets;
    const void* dy; /* [m, n] */
    int64_t lddy;
    const void* x; /* [m, k], needed for dw */
    int64_t ldx;
    const void* w; /* [n, k] or [groups, n, k], needed for dx */
    int64_t ldw, w_group;
    const void* z; /* [m, n], needed when act is not UZIP_ACT_NONE */
    int64_t ldz;
    void* dx; /* [m, k], nullable */
    int64_t lddx;
    void* dw; /* [n, k] or [groups, n, k], nullable */
    int64_t lddw, dw_group;
    void* db; /* [n] or [groups, n], contiguous, nullable */
} uzip_linear_grad_args;

uint64_t uzip_linear_backward_workspace_size(const uzip_linear_grad_args* a);
uzip_status uzip_linear_backward(const uzip_linear_grad_args* a, void* d_workspace, uint64_t workspace_bytes,
                                 int32_t* d_status, cudaStream_t s);
uint64_t uzip_grouped_linear_backward_workspace_size(const uzip_linear_grad_args* a);
uzip_status uzip_grouped_linear_backward(const uzip_linear_grad_args* a, void* d_workspace, uint64_t workspace_bytes,
                                         int32_t* d_status, cudaStream_t s);

/* Softmax cross entropy of t tokens over v classes.  targets are int64; a
 * target equal to ignore_index drops its token: its loss and lse are 0, its
 * dh row is 0 and it adds nothing to dw, whatever its h row holds (NaN and
 * infinities included).  A target outside [0, v) that is not ignore_index is
 * reported in d_status and gives a NaN loss; its gradients are NaN too. */
typedef struct {
    int32_t dtype;
    int32_t reserved; /* 0 */
    int64_t t, v, d;
    const void* h; /* [t, d] */
    int64_t ldh;
    const void* w; /* [v, d] */
    int64_t ldw;
    const int64_t* targets;
    int64_t ignore_index;
    float* loss; /* [t] */
    float* lse;  /* [t]: log of the sum of exponentials, for the gradient */
} uzip_cross_entropy_args;

uint64_t uzip_cross_entropy_workspace_size(const uzip_cross_entropy_args* a);
uzip_status uzip_cross_entropy(const uzip_cross_entropy_args* a, void* d_workspace, uint64_t workspace_bytes,
                               int32_t* d_status, cudaStream_t s);

/* Gradients for the upstream gradient dloss of each token's loss:
 *   dh_i = dloss_i (sum_j p_ij w_j - w_{t_i}),  dw_j = sum_i dloss_i (p_ij - [j = t_i]) h_i.
 * The tokens that are not ignored are moved together in the workspace (t x d
 * values), so that ignored ones cost nothing.  The vocabulary is taken `piece`
 * classes at a time: their logits are computed again, with the same sums as
 * the loss's (p - 1 at a target that has nearly all of the probability is then
 * off by no more than the rounding of lse, half a unit in its last place), and
 * dloss (p - [j = t]), scaled so that the largest dloss is 2^10, is rounded to
 * the dtype in the workspace (t x piece values); dh is summed over the pieces
 * in fp32.  fp16 has no steps below 2^-24 there: a token whose dloss is far
 * below the largest loses what is under 2^-35 of the largest (a thousandth of
 * it keeps p down to 2^-25; bf16 has the range for any).  piece 0 takes the
 * default: as many classes as 512 MiB hold, at most 32768. */
typedef struct {
    int32_t dtype;
    int32_t reserved; /* 0 */
    int64_t t, v, d;
    int64_t piece;
    const void* h;
    int64_t ldh;
    const void* w;
    int64_t ldw;
    const int64_t* targets;
    int64_t ignore_index;
    const float* lse;   /* [t], from uzip_cross_entropy */
    const float* dloss; /* [t] */
    void* dh;           /* [t, d], nullable */
    int64_t lddh;
    void* dw; /* [v, d], nullable */
    int64_t lddw;
} uzip_cross_entropy_grad_args;

uint64_t uzip_cross_entropy_backward_workspace_size(const uzip_cross_entropy_grad_args* a);
uzip_status uzip_cross_entropy_backward(const uzip_cross_entropy_grad_args* a, void* d_workspace,
                                        uint64_t workspace_bytes, int32_t* d_status, cudaStream_t s);

#ifdef __cplusplus
}
#endif
#endif /* UZIP_OPS_H */
