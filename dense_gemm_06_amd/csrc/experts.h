// experts.h -- arguments and launchers of the block-scaled products, the quantizer, and
// the experts' routing and combining (declared for callers in include/gemm_experts.h).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/gemm_experts.h"
#include "block_plan.h"

namespace dg {

constexpr int kMaxExperts = 1024;    // routing: 16 experts for each lane of a wave
constexpr int kMaxTopK = 32;
constexpr int kDispatchChunk = 4096; // (token, slot) pairs per workgroup of the dispatch

struct BlockArgs {
    const uint8_t* A;
    const uint8_t* B;
    const float* SA;
    const float* SB;
    int64_t lda, ldb;
    int64_t sa_row, sa_blk, sb_row, sb_blk;
    int64_t stride_b, stride_sb;  // between the experts' B
    void* C;
    int64_t ldc, stride_c;
    int M, N, K;                  // M: rows of C (experts: P); K: columns of A (gradient: P)
    int out_dt;
    int a_shift, b_shift;         // log2 of block_rows
    int tiles_m, tiles_n, group_m;
    int mode;                     // BlockMode
    int E;
    const int* offsets;
    const int* counts;
    const int* rows;              // NULL: row p of C is row p of A
    int a_rows;
    int k_split, kb_chunk;        // slices on grid y, and the blocks of 128 in each
    float* work;
    int64_t work_slice;
    int work_ld;
};

// Launchers return 0 or the hipError_t of the launch. ta, tb: 0 e4m3, 1 e5m2.
int launch_block_e4m3_e4m3(const BlockPlan& p, const BlockArgs& a, dim3 grid, hipStream_t s);
int launch_block_e4m3_e5m2(const BlockPlan& p, const BlockArgs& a, dim3 grid, hipStream_t s);
int launch_block_e5m2_e4m3(const BlockPlan& p, const BlockArgs& a, dim3 grid, hipStream_t s);
int launch_block_e5m2_e5m2(const BlockPlan& p, const BlockArgs& a, dim3 grid, hipStream_t s);

struct QuantOut {
    uint8_t* q;
    float* s;
    int64_t ld, s_row, s_blk;
    int type;        // 0 e4m3, 1 e5m2
    int block_rows;  // 1 or 128
};

struct QuantArgs {
    const void* X;
    int64_t ldx;
    const int* gather;
    int x_rows, rows, cols;
    QuantOut nat, tr;  // q == NULL: not wanted
};

int launch_block_quantize(const QuantArgs& a, int dtype, hipStream_t s);

struct RouteArgs {
    const void* logits;
    int64_t ld;
    int tokens, experts, top_k;
    int score, groups, top_groups, group_top, renorm;
    float factor;
    int group_lanes;           // lanes that hold a group, 0 where groups cut lanes (set by the launcher)
    const float* bias;
    int* index;
    float* weight;
    const int* index_in;       // backward
    const float* weight_grad;
    void* grad;
    int64_t ldg;
};

int launch_route(const RouteArgs& a, int dtype, bool backward, hipStream_t s);

struct DispatchArgs {
    const int* index;
    int n, top_k, experts, capacity;   // n = tokens * top_k
    int64_t align;
    int* offsets;
    int* counts;
    int* rows;
    int* position;
    int* work;                          // chunks x experts counts (more than one chunk)
    int chunks;
};

int launch_dispatch(const DispatchArgs& a, hipStream_t s);

struct CombineArgs {
    const void* Y;
    int64_t ldy;
    int cols, tokens, top_k, capacity;
    const int* position;
    const int* rows;
    const float* weight;
    void* out;
    int64_t ldo;
    const void* G;                      // backward
    int64_t ldg;
    void* y_grad;
    int64_t ldyg;
    float* weight_grad;
};

int launch_combine(const CombineArgs& a, int dtype, hipStream_t s);
int launch_combine_backward(const CombineArgs& a, int dtype, hipStream_t s);

}  // namespace dg
