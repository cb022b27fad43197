// Definitions shared by the matrix-product sources: the description of one
// product C = A B^T (sums in 32 bits) with its epilogue, and the element-wise
// arithmetic of the epilogues.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/uzip_ops.h"
#include "uzip_internal.cuh"

namespace uzip {

// ---- launches one after another ---------------------------------------------

// Every kernel of the products is launched so that its blocks may be set up
// while the blocks of the launch before it end, and calls this before it reads
// or writes memory: the launch before has then ended and its results are there.
// That launch waited in the same way for the one before itself, so the order is
// the stream's.  48 x 128256 x 4096 loss: 171 us, 166; 1001 x 32003 x 1000 loss
// and gradient: 271 us, 248; 1531 rows in 37 experts with gradients, in a graph:
// 75.6 us, 73.9.  Setting up earlier, as soon as the launch before has begun
// (griddepcontrol.launch_dependents), was slower: 168, 251 and 76.2 us.
__device__ __forceinline__ void wait_for_launch_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// ---- one product ------------------------------------------------------------

// An operand of `rows` x `depth` values (depth is the summed dimension).
// depth_major: a row's values are contiguous and rows are ld apart; else the
// rows of one depth index are contiguous and depths are ld apart.  Group g
// starts group * g elements further.
struct Operand {
    const void* p;
    uint64_t ld, group;
    uint32_t depth_major;
};

enum Schedule : uint32_t {
    kDense = 0,  // one product
    kRows = 1,   // the rows of A and C are cut by the offsets, B belongs to the group
    kDepth = 2,  // the depth is cut by the offsets, C[group] = A_g B_g^T
    // kRows with the operands exchanged, C^T = B A^T: the columns are cut by the
    // offsets, A belongs to the group, and the results are stored transposed
    kColumns = 3
};

enum EpilogueKind : uint32_t {
    kStore = 0,      // C = act(alpha acc + bias) + residual + sum so far, 16- or 32-bit
    kLossStats = 1,  // running maximum and sum of exponentials of each row, target logits
    kLossGrad = 2    // C = g (softmax - [target])
};

struct StoreEpilogue {
    void* out;
    uint64_t ldo, out_group;
    const void* bias;  // dtype, [groups, n]
    const void* residual;
    uint64_t ldr;
    void* z;
    uint64_t ldz;
    const float* sum_in;  // fp32 partial results to add, nullable
    uint64_t ld_sum;
    const float* alpha;  // device scalar on the products' sum, nullable
    uint32_t act;
    uint32_t out_fp32;
};

struct LossEpilogue {
    const int64_t* targets;
    int64_t ignore;
    uint64_t col0;     // class of column 0
    float2* part;      // kLossStats: [rows][tiles] maximum, sum of exponentials
    uint32_t tiles;    // of kStatsCols columns
    float* hit;        // kLossStats: [rows] logit of the target
    const float* lse;  // kLossGrad
    const float* g;    // kLossGrad: [rows], scaled
    void* out;         // kLossGrad: dtype [rows, ldo]
    uint64_t ldo;
};

struct Product {
    Operand a, b;
    uint64_t m, n, depth;  // kRows: m over all groups; kDepth: depth over all groups; kColumns: n over all groups
    uint32_t schedule, epilogue;
    uint32_t groups;  // 1 for kDense
    const int64_t* offsets;
    // kDense: how many of the rows, or of the depths, there are, where only the device knows (nullable; m and depth are
    // the most there may be, and what the operands hold beyond counts for nothing)
    const uint32_t *live_rows, *live_depth;
    StoreEpilogue st;
    LossEpilogue ls;
    int dtype;
    int32_t* status;
};

constexpr uint32_t kStatsCols = 128;  // columns of one kLossStats partial result
cudaError_t launch_product(const Product& p, int sms, cudaStream_t s);

// ---- steps around the products (product_steps.cu) ---------------------------

// matrices whose rows are copied to rows ld_to apart
struct PackJob {
    const void* from;
    void* to;
    uint64_t ld, group, ld_to, rows, cols, groups;
};
struct PackJobs {
    PackJob job[3];
    uint32_t count;
};
cudaError_t launch_pack(const PackJobs& jobs, cudaStream_t s);

// dz = dy act'(z) into dz (nullable) and its column sums into db (nullable); db
// is NaN where the offsets do not cut [0, m)
struct ActGrad {
    const void* dy;
    uint64_t lddy;
    const void* z;
    uint64_t ldz;
    void* dz;
    uint64_t lddz;
    void* db;
    float* part;  // [groups][splits][n] where splits > 1
    uint64_t m, n;
    uint32_t groups, splits;
    const int64_t* offsets;  // nullable: one group of all rows
    uint32_t act;
    int dtype;
    int32_t* status;
};
uint32_t act_grad_splits(uint64_t m, uint64_t n, uint64_t groups);
cudaError_t launch_act_grad(const ActGrad& a, cudaStream_t s);

// status only, for offsets that do not cut [0, m)
cudaError_t launch_offset_check(const int64_t* offsets, uint64_t groups, uint64_t m, int32_t* status, cudaStream_t s);

// The tokens that count, moved together in their order: their h rows, targets
// and (for the gradient) lse and scaled weights, their number, and where each
// is from and went.  Ignored tokens get loss and lse 0.
struct LossRows {
    const void* h;
    uint64_t ldh;
    const int64_t* targets;
    int64_t ignore;
    uint64_t t, v, d;
    int dtype;
    const float *dloss, *lse;  // nullable: the forward call has none
    void* out_h;
    uint64_t ld_out;
    int64_t* out_targets;
    float *out_lse, *out_g;
    float* scale;  // what undoes the weights' scale, which brings the largest |dloss| to 2^10
    uint32_t *token, *place, *count;  // compact row -> token, token -> compact row or ~0, rows
    float *loss, *zero_lse;           // forward: 0 for ignored tokens
    int32_t* status;
};
cudaError_t launch_loss_rows(const LossRows& a, cudaStream_t s);
// token and count are nullable: the rows are the tokens
cudaError_t launch_loss_join(const LossEpilogue& e, const uint32_t* token, const uint32_t* count, uint64_t t, uint64_t v,
                             float* loss, float* lse, int32_t* status, cudaStream_t s);
// to[i] = from[place[i]], or zeros where place[i] is ~0
cudaError_t launch_spread_rows(const void* from, uint64_t ld, const uint32_t* place, void* to, uint64_t ld_to, uint64_t rows,
                               uint64_t cols, cudaStream_t s);
// 16-bit zeros
cudaError_t launch_clear(void* p, uint64_t ld, uint64_t rows, uint64_t cols, cudaStream_t s);

// ---- arithmetic ---------------------------------------------------------------

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSqrtHalf = 0.70710678118654752f;
constexpr float kInvSqrt2Pi = 0.39894228040143268f;

__device__ __forceinline__ float from16(uint16_t b, int dtype) {
    return dtype == UZIP_BF16 ? __uint_as_float(uint32_t(b) << 16) : __half2float(__ushort_as_half(b));
}
__device__ __forceinline__ uint16_t to16(float v, int dtype) {
    return dtype == UZIP_BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(v)) : __half_as_ushort(__float2half_rn(v));
}
// two values in one word, the first in the low half; both types are computed
// and one is taken, which costs less than a branch for every word
__device__ __forceinline__ float2 from16x2(uint32_t w, int dtype) {
    const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&w));
    const bool bf = dtype == UZIP_BF16;
    return make_float2(bf ? __uint_as_float(w << 16) : h.x, bf ? __uint_as_float(w & 0xFFFF0000u) : h.y);
}
__device__ __forceinline__ uint32_t to16x2(float lo, float hi, int dtype) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    const __half2 h = __floats2half2_rn(lo, hi);
    return dtype == UZIP_BF16 ? *reinterpret_cast<const uint32_t*>(&b) : *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ float fast_exp2(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float fast_reciprocal(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// (1 - Phi(a)) exp(a^2 / 2) for a >= 0, as t P(t) with t = 1 / (1 + 0.305 a): t
// takes [0, inf) to (0, 1], where the function over t is smooth.  P is of degree
// 7, fitted to erfcx in 64 bits for the smallest relative error over [0, 14]
// (least squares, reweighted until the extremes are level): 9.4e-8, and 4e-7 as
// computed here, so gelu's negative tail keeps the type's precision however
// small it gets (to 9e-6 of itself at z = -12, from the exponential's argument).
__device__ __forceinline__ float gauss_tail(float a) {
    const float t = fast_reciprocal(fmaf(0.305000007f, a, 1.f));
    float s = fmaf(0.0366987698f, t, -0.152986616f);
    s = fmaf(s, t, 0.185714051f);
    s = fmaf(s, t, -0.0379742719f);
    s = fmaf(s, t, 0.121020354f);
    s = fmaf(s, t, 0.103421263f);
    s = fmaf(s, t, 0.122466758f);
    s = fmaf(s, t, 0.121639736f);
    return s * t;
}

__device__ __forceinline__ float act_value(float z, uint32_t act) {
    switch (act) {
        case UZIP_ACT_RELU: return z <= 0.f ? 0.f : z;
        case UZIP_ACT_GELU: {  // z Phi(z) = max(z, 0) - |z| (1 - Phi(|z|)); past 40 the tail is zero
            const float a = fminf(fabsf(z), 40.f), e = fast_exp2(a * (a * (-0.5f * kLog2e)));
            return (z <= 0.f ? 0.f : z) - a * (gauss_tail(a) * e);
        }
        case UZIP_ACT_SILU: return z * fast_reciprocal(1.f + fast_exp2(-z * kLog2e));
        default: return z;
    }
}
__device__ __forceinline__ float act_slope(float z, uint32_t act) {
    switch (act) {
        case UZIP_ACT_RELU: return z <= 0.f ? 0.f : (z > 0.f ? 1.f : z);
        case UZIP_ACT_GELU: {  // Phi(z) + z phi(z)
            const float a = fminf(fabsf(z), 40.f), e = fast_exp2(a * (a * (-0.5f * kLog2e)));
            const float tail = gauss_tail(a) * e, odd = a * e * kInvSqrt2Pi;
            return z <= 0.f ? tail - odd : (z > 0.f ? 1.f - tail + odd : z);
        }
        case UZIP_ACT_SILU: {
            const float q = fast_reciprocal(1.f + fast_exp2(-z * kLog2e));
            return fabsf(z) > 200.f ? q : q * (1.f + z * (1.f - q));  // (0 or 1 out there, where a kept z may be infinite)
        }
        default: return 1.f;
    }
}

}  // namespace uzip
