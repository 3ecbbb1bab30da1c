/*
 * gemm_experts.h -- C ABI of the block-scaled 8-bit products and of the experts built
 * on them (a companion of gemm.h: the same library, status codes, gemm_last_error,
 * streams and ownership rules).
 *
 * Block-scaled matrices
 * ---------------------
 *  A matrix of R x K numbers is held as 8-bit floating point codes (OCP e4m3 or e5m2)
 *  and one fp32 scale for each block of `block_rows` x 128 elements (block_rows 1 or
 *  128; the last block of a row or column may be partial). The number that element
 *  (i, k) stands for is
 *      data[i*ld + k] * scale[(i / block_rows)*scale_row + (k / 128)*scale_block]
 *  with op = GEMM_OP_N; with op = GEMM_OP_T the codes lie transposed, at data[k*ld + i] (a
 *  matrix of 128 x 128 blocks serves as its own transpose so: swap rows and cols, swap the
 *  scale's strides and set op).
 *
 * Plans
 * -----
 *  T tokens choose k experts each. gemm_experts_dispatch sorts the T*k (token, slot)
 *  pairs by expert, keeping their order within an expert, into P rows: expert e owns
 *  rows offsets[e] .. offsets[e+1]-1, of which the first counts[e] hold pairs and the
 *  rest (up to the next multiple of `align`) are padding, as are the rows from
 *  offsets[E] to P. rows[p] is the token of row p (-1: padding), position[t*k + j] the
 *  row of token t's slot j (-1: none, its expert lies outside 0 .. E-1).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - Pointers are DEVICE pointers (structs themselves are host memory, read during the
 *    call only). Work is enqueued on `stream`; the call returns without synchronizing,
 *    allocates nothing and can be captured into a HIP graph.
 *  - Codes, 16-bit and 32-bit values need no alignment beyond their element's.
 *  - Sizes are below 2^31 per dimension (GEMM_ERR_UNSUPPORTED otherwise); addresses are
 *    64 bits. Empty outputs are successful no-ops.
 *  - Index arrays come from the device and are not read by the host: kernels treat an
 *    index out of range as padding and never read or write outside the given arrays.
 *  - Every argument is validated before anything is enqueued. Outputs must not overlap
 *    inputs.
 */
#ifndef DENSE_GEMM_06_AMD_GEMM_EXPERTS_H
#define DENSE_GEMM_06_AMD_GEMM_EXPERTS_H

#include "gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* 8-bit element types, beside gemm_dtype's */
typedef enum { GEMM_E4M3 = 3, GEMM_E5M2 = 4 } gemm_code_type;

typedef struct gemm_block_matrix {
    void* data;           /* codes; read as an operand, written by gemm_block_quantize */
    float* scale;
    int64_t rows, cols;   /* R, K */
    int64_t ld;           /* >= max(1, cols); GEMM_OP_T: >= max(1, rows) */
    int64_t scale_row, scale_block;   /* strides of the scale in elements, >= 0 */
    int64_t stride, scale_stride;     /* between the matrices of a batch (one for each expert) */
    int32_t dtype;        /* GEMM_E4M3 or GEMM_E5M2 */
    int32_t block_rows;   /* 1 or 128 */
    int32_t op;           /* GEMM_OP_N or GEMM_OP_T (operands of products only) */
    int32_t reserved;     /* 0 */
} gemm_block_matrix;

/*
 * gemm_block_quantize -- X (GEMM_F32, GEMM_F16 or GEMM_BF16, row-major, leading
 * dimension ldx) into codes and block scales: for each block, in fp32,
 *     amax = max(max |x|, 2^-100),  scale = amax / qmax,  code = round(x * (qmax / amax))
 * with qmax the type's largest finite number (448, 57344) and rounding to nearest
 * even; a block that holds a NaN gets NaN codes and scale.
 * gather (or NULL): row i of the quantized matrix is row gather[i] of X, a row of zeros
 * where gather[i] lies outside 0 .. x_rows-1; rows is the number of rows quantized
 * (x_rows when gather is NULL). natural (or NULL) receives the rows x cols matrix,
 * transposed (or NULL) its cols x rows transpose, whose blocks of `block_rows` x 128 run
 * along the rows of X: one read of X gives both. At least one of the two is given; their
 * rows and cols have to match; both may differ in type and block_rows.
 */
int gemm_block_quantize(const void* X, int64_t x_rows, int64_t cols, int64_t ldx, int dtype, const int32_t* gather,
                        int64_t rows, const gemm_block_matrix* natural, const gemm_block_matrix* transposed,
                        void* stream);

/*
 * gemm_block_product -- C[i][j] = sum_k A(i,k) B(j,k) for block-scaled A (M x K) and
 * B (N x K, i.e. column-major as gemm_ex's GEMM_OP_T), any pair of types and block_rows.
 * Products of codes are exact, their sum over a block of 128 k is in fp32, and each block's
 * sum is multiplied by A's scale and then by B's and added in fp32, whatever C's type (the
 * scales' own product may lie outside fp32's normal numbers); the experts' products below do
 * the same. C is stored in out_dtype (GEMM_F32, GEMM_F16 or GEMM_BF16,
 * round to nearest even), leading dimension ldc.
 * K == 0 writes zeros. With a workspace (16-byte aligned; gemm_block_product_workspace
 * tells the bytes that help, 0 when none do) K may be split over workgroups, the parts
 * added in a fixed order; without one (NULL, 0) it is not split.
 */
int gemm_block_product(const gemm_block_matrix* A, const gemm_block_matrix* B, void* C, int64_t ldc, int out_dtype,
                       void* workspace, int64_t workspace_bytes, void* stream);
int64_t gemm_block_product_workspace(int64_t M, int64_t N, int64_t K);

/*
 * Routing. Scores are softmax or sigmoid of the logits, computed in fp64 (0 below e^-708).
 * Each token's choice value is its score plus bias (fp32, NULL: none). With groups > 1 the
 * experts are cut into `groups` equal runs; a run's value is the sum of its group_top largest
 * choice values, and only the top_groups best runs stay. The top_k experts of largest choice
 * value are taken in descending order, ties to the lowest index (a NaN counts as
 * largest). Their weights are the scores, divided by their sum with renorm, times factor.
 */
typedef enum { GEMM_SCORE_SOFTMAX = 0, GEMM_SCORE_SIGMOID = 1 } gemm_score;

typedef struct gemm_router {
    int32_t top_k;                          /* 1 .. min(32, experts) */
    int32_t score;                          /* gemm_score */
    int32_t groups, top_groups, group_top;  /* 1, 1, 1 without groups; group_top at most 4 */
    int32_t renorm;
    float factor;
} gemm_router;

/* logits: tokens x experts (at most 1024), fp32, fp16 or bf16; index, weight: tokens x top_k. */
int gemm_experts_route(const void* logits, int64_t tokens, int64_t experts, int64_t ld, int dtype,
                       const gemm_router* router, const float* bias, int32_t* index, float* weight, void* stream);

/* The logits' gradient (logits' type, tokens x experts, leading dimension ldg) from the
 * gradient of the weights (tokens x top_k, fp32), with the choice held fixed. */
int gemm_experts_route_backward(const void* logits, int64_t tokens, int64_t experts, int64_t ld, int dtype,
                                const gemm_router* router, const int32_t* index, const float* weight_grad, void* grad,
                                int64_t ldg, void* stream);

typedef struct gemm_expert_plan {
    int32_t* offsets;   /* experts + 1 */
    int32_t* counts;    /* experts */
    int32_t* rows;      /* capacity */
    int32_t* position;  /* tokens * top_k */
    int64_t experts, tokens, top_k;
    int64_t capacity;   /* P */
} gemm_expert_plan;

/* Rows that hold every expert's rows, each expert's first row at a multiple of align. */
int64_t gemm_experts_capacity(int64_t tokens, int64_t top_k, int64_t experts, int64_t align);

/* Fills the plan's arrays from index (tokens x top_k). capacity must be at least
 * gemm_experts_capacity; the workspace at least gemm_experts_dispatch_workspace bytes. */
int gemm_experts_dispatch(const int32_t* index, int64_t align, const gemm_expert_plan* plan, void* workspace,
                          int64_t workspace_bytes, void* stream);
int64_t gemm_experts_dispatch_workspace(int64_t tokens, int64_t top_k, int64_t experts);

/*
 * gemm_experts_product -- C[p][j] = sum_k A(r,k) B_e(j,k) for every row p of expert e,
 * r = rows[p] with gather (A holds the tokens' rows) or p without (A holds the sorted
 * rows); padding rows of C are zeros. B is a batch of `experts` matrices N x K; A has op
 * GEMM_OP_N.
 */
int gemm_experts_product(const gemm_block_matrix* A, const gemm_block_matrix* B, const gemm_expert_plan* plan,
                         int gather, void* C, int64_t ldc, int out_dtype, void* stream);

/*
 * gemm_experts_gradient -- C_e[i][j] = sum over the rows p of expert e, its padding
 * included, of A(i,p) B(j,p): A (M x P) and B (N x P) hold the sorted rows transposed, so
 * their blocks run along p and every offset has to be a multiple of 128 (the results of an
 * expert whose rows start elsewhere, or end inside 16, are NaN). Padding has to hold zeros, as
 * gemm_block_quantize makes of gathered rows. C is experts x M x N, stride_c elements
 * between matrices; experts without rows get zeros.
 */
int gemm_experts_gradient(const gemm_block_matrix* A, const gemm_block_matrix* B, const gemm_expert_plan* plan,
                          void* C, int64_t ldc, int64_t stride_c, int out_dtype, void* stream);

/* out[t] = sum_j weight[t*k + j] Y[position[t*k + j]], summed in fp32 in the slots' order; Y is
 * capacity x cols, out tokens x cols, both of type dtype. A slot without a row adds nothing. */
int gemm_experts_combine(const void* Y, int64_t cols, int64_t ldy, int dtype, const gemm_expert_plan* plan,
                         const float* weight, void* out, int64_t ldo, void* stream);

/* Its gradients from G (tokens x cols, type dtype): y_grad[p] = weight G[t] (zeros in padding
 * rows), weight_grad[t*k + j] = G[t] . Y[position[t*k + j]] in fp32 (0 without a row). */
int gemm_experts_combine_backward(const void* Y, int64_t cols, int64_t ldy, int dtype, const gemm_expert_plan* plan,
                                  const float* weight, const void* G, int64_t ldg, void* y_grad, int64_t ldyg,
                                  float* weight_grad, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* DENSE_GEMM_06_AMD_GEMM_EXPERTS_H */
