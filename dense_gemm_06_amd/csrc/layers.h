// layers.h -- arguments and launchers of the operators around a layer's dense products
// (declared for callers in include/gemm_layers.h). Launchers return 0 or the hipError_t of
// the launch.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/gemm_layers.h"
#include "experts.h"

namespace dg {

// A launcher of each 16-bit type.
#define DG_16BIT(name, params)                                    \
    int name##_f16 params;                                             \
    int name##_bf16 params;

constexpr int kMaxRank = 128;
constexpr int kMaxAdapters = 32768;  // of a grid's second direction, with room for the chunks of their rows

// ---------------------------------------------------------------- activations
struct ActArgs {
    const void* z;       // forward: rows x zcols
    int64_t ldz;
    QuantOut codes;      // of z (q == NULL: forward without); backward reads them
    int rows, cols;      // of y; zcols = cols, or 2 cols with a gate
    int act, gated;
    int passing;         // results leave past the caches
    void* y;             // NULL: not wanted (backward)
    int64_t ldy;
    const void* grad;    // backward
    int64_t ldg;
    void* z_grad;
    int64_t ldzg;
};

int launch_activation(const ActArgs& a, int dtype, hipStream_t s);
int launch_activation_backward(const ActArgs& a, int dtype, hipStream_t s);

// ---------------------------------------------------------------- loss over a vocabulary
// One piece of the vocabulary: columns v0 .. v0 + n - 1 of the logits.
struct LossArgs {
    const float* logits;    // tokens x n, leading dimension ld
    int64_t ld;
    int tokens, v0, n, vocabulary;
    const int64_t* target;
    float* top;             // running maximum, sum of exp(l - maximum) and target's logit
    float* sum;
    float* picked;
    int first, last;
    float* loss;
    float* lse;
    // backward: d in the matrices' type, as it is (tokens x n) and transposed (n x tokens)
    const float* lse_in;
    const float* grad;
    const float* factor;    // device: [0] what grad is multiplied with, [1] its inverse
    void* d;
    float* apart;           // 16 bits: 1 where d leaves the target's -1 to x's gradient
    int64_t ldd;
    void* dt;
    float* rest;            // 16 bits: what rounding took from the targets' d in dt
    int64_t lddt;
};

// Fused forms for 16-bit matrices: x tokens x K, w (its rows from v0 on) n x K. `direct`: rows of
// whole 16-byte pieces, 16-byte aligned.
struct LossProduct {
    const void* x;
    const void* w;
    int64_t ldx, ldw;
    int tokens, n, K, group_m, direct;
    int strip;              // columns of a part: 256 and 128 (tiles), 16 (few rows)
};
struct LossPart;            // a row's maximum and sum over a strip of columns
constexpr int64_t kLossPartBytes = 8;
DG_16BIT(launch_loss_skinny, (const LossProduct& p, const int64_t* target, void* part, float* picked, hipStream_t s))
DG_16BIT(launch_loss_tiles, (const LossProduct& p, int v0, const int64_t* target, void* part, float* picked, hipStream_t s))
DG_16BIT(launch_loss_grad_tiles, (const LossProduct& p, const LossArgs& a, hipStream_t s))
// out (n x cols, 16 bits) = factor[1] (dt x + the targets' rests), dt n x lddt (a multiple of 32), through
// `copy`: x as lddt x cols or, turned, cols x lddt, with rows of whole, aligned 16-byte pieces
DG_16BIT(launch_loss_w, (const LossArgs& a, const void* x, int64_t ldx, const void* copy, int64_t ld_copy, int turned, int cols, int group_m, void* out, int64_t ldo, hipStream_t s))
// out (cols x ld) = x^T, zeros from column `tokens` on
int launch_loss_turn(const void* x, int64_t ldx, int tokens, int cols, void* out, int64_t ld, hipStream_t s);
int launch_loss_finish(const void* part, int strips, int tokens, const int64_t* target, int vocabulary,
                       const float* picked, float* loss, float* lse, hipStream_t s);

int launch_loss_stats(const LossArgs& a, hipStream_t s);
int launch_loss_grad(const LossArgs& a, int dtype, hipStream_t s);
// factor[0], factor[1]: powers of two that bring the largest finite |grad| near 2^14, and back
int launch_loss_factor(const float* grad, int tokens, float* factor, hipStream_t s);
// out (rows x cols, 16 bits) = in (fp32) * factor[1], less apart[t] grad[t] w[target[t]] in row t where w is given
int launch_scaled_cast(const float* in, int64_t ldi, int rows, int cols, const float* factor, void* out, int64_t ldo,
                       const void* w, int64_t ldw, const int64_t* target, int vocabulary, const float* grad,
                       const float* apart, int dtype, hipStream_t s);

// ---------------------------------------------------------------- adapters
struct AdapterArgs {
    const void* x;          // rows that are multiplied: tokens x cols
    int64_t ldx;
    const void* m;          // adapters' matrices: turned 0: rank x cols, 1: cols x rank
    int64_t ldm, stride_m;
    int turned;
    int rank_m;             // numbers in a row of a turned m (zeros past the rank)
    int tokens, cols, rank, adapters;
    const int* index;
    const float* scale;     // NULL: 1
    float* u;               // tokens x rank
    uint16_t* us;           // scale u as hi and lo (tokens x 2 x rank_p)
    float* unit;            // fp16: the power of two of each token that us leaves out
    int rank_p;             // 16, 32, 64 or 128
    int fold;               // u holds scale u
    // expand: out = base + scale u m
    const float* base;
    int64_t ld_base;
    int slices;             // of base, tokens rows apart
    void* out;
    int64_t ldo;
    // gradient: plan
    const int* offsets;
    const int* counts;
    const int* rows;
    int capacity;
    int chunk;              // rows of the plan that a workgroup of the gradient takes
    float* work;            // their sums
};

// What the 16-bit kernels for a shared product x w^T (turned 1: x w) with adapters take.
struct AdapterProduct {
    const void* x;
    const void* w;
    int64_t ldx, ldw;
    int N, K;               // columns of the result, length of the sum
    int opb;                // GEMM_OP_T: w is N x K, GEMM_OP_N: K x N
    int direct;             // rows of whole 16-byte pieces, 16-byte aligned
};

// The adapters' transposes: in is rows x cols, out cols x out_ld.
struct TurnArgs {
    const void* in;
    int64_t ld, stride;
    int rows, cols;
    void* out;              // each matrix cols x out_ld, contiguous
    int out_ld;
    int tiles_r, tiles_c;
};

// 16-bit matrices, on the matrix instructions, one function for each type:
// out = x w + scale u m in one kernel, for up to 64 tokens (x w^T only) or in 256 x 256 tiles
DG_16BIT(launch_adapter_skinny, (const AdapterProduct& p, const AdapterArgs& a, hipStream_t s))
// the same through `slices` of k (direct rows): u and part (slices x tokens x cols rounded up to 4)
DG_16BIT(launch_adapter_decode, (const AdapterProduct& p, const AdapterArgs& u, const AdapterArgs& a, int slices, int slice_k, float* part, hipStream_t s))
DG_16BIT(launch_adapter_tiles, (const AdapterProduct& p, const AdapterArgs& a, int group_m, hipStream_t s))
// part (slices x tokens x N rounded up to 4) = x w^T over slices of k, in 128 x 128 tiles (direct rows)
DG_16BIT(launch_mid_part, (const AdapterProduct& p, int tokens, int group_m, int slices, int slice_k, float* part, hipStream_t s))
// the operators below, m with its long direction along memory in shrink and across it in expand
DG_16BIT(launch_adapter_shrink_row, (const AdapterArgs& a, hipStream_t s))
// through part (slices x tokens x rank_p): u, us. direct: 16-byte rows
DG_16BIT(launch_adapter_shrink16, (const AdapterArgs& a, int direct, int slices, int slice_k, float* part, hipStream_t s))
DG_16BIT(launch_adapter_expand16, (const AdapterArgs& a, hipStream_t s))
// both gradients from us: a's of v and x, b's of u and grad
DG_16BIT(launch_adapter_gradient16, (const AdapterArgs& a, const AdapterArgs& b, int slots, hipStream_t s))
// the adapters' transposes, and a.us from the forward pass's u (tokens x rank; a.tokens 0: none)
DG_16BIT(launch_adapter_prepare, (const TurnArgs& p, const TurnArgs& q, int adapters, const AdapterArgs& a, const float* u, hipStream_t s))

// u[t][j] = scale sum_k x[t][k] m(j,k)
int launch_adapter_shrink(const AdapterArgs& a, hipStream_t s);
// out[t][k] = base[t][k] + sum_j scale u[t][j] m(j,k)
int launch_adapter_expand(const AdapterArgs& a, hipStream_t s);
// out_i(j,k) = sum over the rows t of adapter i of scale u[t][j] x[t][k], laid out as m; two at once
int launch_adapter_gradient(const AdapterArgs& a, const AdapterArgs& b, hipStream_t s);

}  // namespace dg
