// layers.h -- arguments and launchers of the operators around a layer's dense products
// (declared for callers in include/gemm_layers.h). Launchers return 0 or the hipError_t of
// the launch.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/gemm_layers.h"
#include "experts.h"

namespace dg {

constexpr int kMaxRank = 128;

// ---------------------------------------------------------------- activations
struct ActArgs {
    const void* z;       // forward: rows x zcols
    int64_t ldz;
    QuantOut codes;      // of z (q == NULL: forward without); backward reads them
    int rows, cols;      // of y; zcols = cols, or 2 cols with a gate
    int act, gated;
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
    int64_t ldd;
    void* dt;
    int64_t lddt;
};

int launch_loss_stats(const LossArgs& a, hipStream_t s);
int launch_loss_grad(const LossArgs& a, int dtype, hipStream_t s);
// factor[0], factor[1]: powers of two that bring the largest finite |grad| near 2^14, and back
int launch_loss_factor(const float* grad, int tokens, float* factor, hipStream_t s);
// out (rows x cols, dtype) = in (fp32) * factor[1]
int launch_scaled_cast(const float* in, int64_t ldi, int rows, int cols, const float* factor, void* out, int64_t ldo,
                       int dtype, hipStream_t s);

// ---------------------------------------------------------------- adapters
struct AdapterArgs {
    const void* x;          // rows that are multiplied: tokens x cols
    int64_t ldx;
    const void* m;          // adapters' matrices: turned 0: rank x cols, 1: cols x rank
    int64_t ldm, stride_m;
    int turned;
    int tokens, cols, rank, adapters;
    const int* index;
    const float* scale;     // NULL: 1
    float* u;               // tokens x rank
    // expand: out = base + scale u m
    const float* base;
    int64_t ld_base;
    void* out;
    int64_t ldo;
    // gradient: plan
    const int* offsets;
    const int* counts;
    const int* rows;
    int capacity;
};

// u[t][j] = scale sum_k x[t][k] m(j,k)
int launch_adapter_shrink(const AdapterArgs& a, int dtype, hipStream_t s);
// out[t][k] = base[t][k] + sum_j scale u[t][j] m(j,k)
int launch_adapter_expand(const AdapterArgs& a, int dtype, hipStream_t s);
// out_i(j,k) = sum over the rows t of adapter i of scale u[t][j] x[t][k], laid out as m
int launch_adapter_gradient(const AdapterArgs& a, int dtype, hipStream_t s);

}  // namespace dg
