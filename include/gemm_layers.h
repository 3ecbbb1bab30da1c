/*
 * gemm_layers.h -- C ABI of the operators around a layer's dense products (a companion of
 * gemm.h and gemm_experts.h: the same library, status codes, gemm_last_error, streams and
 * ownership rules): low-rank adapters beside a shared projection, the loss over a
 * vocabulary, and activations whose input is kept in 8 bits.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - Matrices are row-major with unit stride along their rows and a leading dimension in
 *    elements; dtype (GEMM_F32, GEMM_F16 or GEMM_BF16) is the type of every matrix of the
 *    call unless said otherwise. No alignment beyond the element's is needed.
 *  - Pointers are DEVICE pointers (structs themselves are host memory, read during the
 *    call only). Work is enqueued on `stream`; the call returns without synchronizing,
 *    allocates nothing and can be captured into a HIP graph. Calls that share a workspace
 *    must be ordered.
 *  - Sizes are below 2^30 per dimension (2^31 for the activations), and the leading
 *    dimensions of what enters a product below 2^23, as everywhere in this library
 *    (GEMM_ERR_UNSUPPORTED otherwise, as where a launch would need 2^32 threads); addresses are
 *    64 bits. Empty outputs are successful no-ops.
 *  - Index arrays come from the device and are not read by the host: an index out of range
 *    stands for none, and nothing outside the given arrays is read or written.
 *  - Every argument is validated before anything is enqueued. Outputs must not overlap
 *    inputs, the workspace or each other. A workspace is 16-byte aligned; the call that
 *    tells its size gives the bytes that the call needs (0 for sizes that the call refuses).
 */
#ifndef DENSE_GEMM_06_AMD_GEMM_LAYERS_H
#define DENSE_GEMM_06_AMD_GEMM_LAYERS_H

#include "gemm_experts.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Low-rank adapters. Row t of x uses adapter i = index[t], or none where index[t] lies
 * outside 0 .. adapters-1:
 *     u[t] = a_i x[t],    y[t] = w x[t] + scale_i b_i u[t]
 * with w N x K, a_i rank x K, b_i N x rank. Ranks that differ are padded with zeros.
 */
typedef struct gemm_adapter_set {
    const void* a;            /* adapters x rank x K */
    const void* b;            /* adapters x N x rank */
    const float* scale;       /* adapters values, or NULL: all 1 */
    int64_t adapters, rank;   /* at most 32768; rank 1 .. 128 (0 without adapters) */
    int64_t lda, stride_a;    /* >= max(1, K); between adapters, >= 0 */
    int64_t ldb, stride_b;    /* >= max(1, rank) */
} gemm_adapter_set;

/*
 * gemm_adapters_product -- y (tokens x N) and u (tokens x rank, contiguous, fp32; zeros in
 * rows without an adapter), which the backward pass takes. Products are summed in fp32;
 * u enters the second product in fp32, or with 16-bit matrices as the sum of two numbers of
 * their type (fp16 after a power of two for each row, so that any size of scale * u will do).
 */
int gemm_adapters_product(const void* x, int64_t tokens, int64_t K, int64_t ldx, const void* w, int64_t N, int64_t ldw,
                          int dtype, const gemm_adapter_set* set, const int32_t* index, void* y, int64_t ldy, float* u,
                          void* workspace, int64_t workspace_bytes, void* stream);
int64_t gemm_adapters_workspace(int64_t tokens, int64_t N, int64_t K, int64_t rank, int dtype);

/*
 * gemm_adapters_backward -- from grad (tokens x N), the gradient of y, and u:
 *     v[t] = scale_i b_i^T grad[t]
 *     x_grad[t] = w^T grad[t] + a_i^T v[t]                  (tokens x K; NULL: not wanted)
 *     a_grad_i = sum over the rows t of adapter i of v[t] x[t]^T           (as a, contiguous)
 *     b_grad_i = sum over them of scale_i grad[t] u[t]^T                   (as b, contiguous)
 * v enters its products as u does. plan is gemm_experts_dispatch's of index as tokens x 1 (top_k 1,
 * align 1; for up to 1024 adapters, and with 16-bit matrices 2^25 tokens less 512 for each adapter);
 * an adapter without rows gets zeros. a_grad and b_grad come together or are both NULL (an empty
 * one may be NULL by itself). Sums are fp32 in a fixed order.
 */
int gemm_adapters_backward(const void* grad, int64_t tokens, int64_t N, int64_t ldg, const void* x, int64_t K,
                           int64_t ldx, const float* u, const void* w, int64_t ldw, int dtype,
                           const gemm_adapter_set* set, const int32_t* index, const gemm_expert_plan* plan, void* x_grad,
                           int64_t ldxg, void* a_grad, void* b_grad, void* workspace, int64_t workspace_bytes,
                           void* stream);
int64_t gemm_adapters_backward_workspace(int64_t tokens, int64_t N, int64_t K, int64_t adapters, int64_t rank,
                                         int dtype);

/*
 * Loss over a vocabulary: softmax cross entropy of the logits l[t] = w x[t] (x tokens x K,
 * w vocabulary x K), which are never held as a whole.
 *     lse[t] = log sum_v exp(l[t][v]),   loss[t] = lse[t] - l[t][target[t]]
 * (fp32; loss 0 where target[t], 64 bits, lies outside 0 .. vocabulary-1). Logits and sums
 * are fp32.
 */
int gemm_loss(const void* x, int64_t tokens, int64_t K, int64_t ldx, const void* w, int64_t vocabulary, int64_t ldw,
              int dtype, const int64_t* target, float* loss, float* lse, void* workspace, int64_t workspace_bytes,
              void* stream);
int64_t gemm_loss_workspace(int64_t tokens, int64_t vocabulary, int64_t K, int dtype);

/*
 * gemm_loss_backward -- with grad[t] (fp32) the gradient of loss[t] and lse of gemm_loss,
 *     d[t][v] = grad[t] (exp(l[t][v] - lse[t]) - [v = target[t]])
 * (zeros where the target lies outside), x_grad = d w and w_grad = d^T x, in the matrices'
 * type; either may be NULL. The vocabulary is taken `piece` columns at a time (0: the
 * library's choice), whose d are held in the workspace in the matrices' type (fp16: times a power
 * of two that brings the largest |grad| near 2^14, so that d of tokens whose |grad| is below 2^-20 of
 * it has fewer digits) and summed in fp32; smaller pieces need less workspace. w_grad takes up to
 * 2^23 - 32 tokens.
 */
int gemm_loss_backward(const float* grad, const void* x, int64_t tokens, int64_t K, int64_t ldx, const void* w,
                       int64_t vocabulary, int64_t ldw, int dtype, const int64_t* target, const float* lse, void* x_grad,
                       int64_t ldxg, void* w_grad, int64_t ldwg, int64_t piece, void* workspace,
                       int64_t workspace_bytes, void* stream);
int64_t gemm_loss_backward_workspace(int64_t tokens, int64_t vocabulary, int64_t K, int dtype, int want_x_grad,
                                     int want_w_grad, int64_t piece);

/* Activations beside gemm_activation's GEMM_ACT_RELU and GEMM_ACT_GELU_TANH: x / (1 + e^-x) */
enum { GEMM_ACT_SILU = 3 };

/*
 * gemm_activation_forward -- y = f(z) (rows x cols), or with gated y = f(z1) * z2 for z =
 * [z1 | z2] (rows x 2 cols), f one of GEMM_ACT_RELU, GEMM_ACT_GELU_TANH and GEMM_ACT_SILU in
 * fp32, and z itself as codes (NULL: not wanted), exactly gemm_block_quantize's natural
 * result with block_rows 1: what the backward pass keeps of z. A NaN in z is one in y, relu's too
 * (gemm_activation's gives 0).
 */
int gemm_activation_forward(const void* z, int64_t rows, int64_t cols, int64_t ldz, int dtype, int activation,
                            int gated, void* y, int64_t ldy, const gemm_block_matrix* codes, void* stream);

/*
 * gemm_activation_backward -- from grad (rows x cols, type dtype), the gradient of y, and the
 * codes of z: z_grad = grad f'(z), or gated [grad z2 f'(z1) | grad f(z1)], and y computed again
 * (NULL: not wanted) for the gradient of the weight that reads it, both of type dtype. grad and
 * z_grad are NULL together where y alone is wanted: it may be needed before grad is known.
 */
int gemm_activation_backward(const gemm_block_matrix* codes, const void* grad, int64_t rows, int64_t cols, int64_t ldg,
                             int dtype, int activation, int gated, void* z_grad, int64_t ldzg, void* y, int64_t ldy,
                             void* stream);

#ifdef __cplusplus
}
#endif

#endif /* DENSE_GEMM_06_AMD_GEMM_LAYERS_H */
