// block_api.cpp -- the C ABI declared in include/gemm_experts.h: validation, the choice of
// kernel, and the launches. Everything is validated before the first launch.
#include <hip/hip_runtime.h>
#include <string.h>

#include <algorithm>

#include "checks.h"
#include "experts.h"
#include "launch.h"
#include "plan.h"
#include "product.h"

namespace {

using dg::block_plan;

// ---------------------------------------------------------------- the products' kernels
// Rows that start at multiples of 16 bytes and hold whole 16-byte chunks.
bool direct_rows(const gemm_block_matrix& m, int64_t batch) {
    const int64_t across = m.op == GEMM_OP_T ? m.rows : m.cols;
    return ((uintptr_t)m.data & 15) == 0 && m.ld % 16 == 0 && across % 16 == 0 && (batch <= 1 || m.stride % 16 == 0);
}

// BlockPlan::tr of two operands.
int tr_of(const gemm_block_matrix& A, const gemm_block_matrix& B) {
    return (A.op == GEMM_OP_T ? 2 : 0) | (B.op == GEMM_OP_T ? 1 : 0);
}

// Whether byte offsets within an operand fit 32 bits.
bool small_call(const gemm_block_matrix& A, const gemm_block_matrix& B) {
    auto bytes = [](const gemm_block_matrix& m) { return (m.op == GEMM_OP_T ? m.cols : m.rows) * m.ld; };
    return bytes(A) < ((int64_t)1 << 32) && bytes(B) < ((int64_t)1 << 32);
}

int64_t split_bytes(int split, int64_t M, int64_t N) { return split <= 1 ? 0 : split * M * ceil_div(N, 4) * 16; }

dg::BlockArgs block_args(const gemm_block_matrix& A, const gemm_block_matrix& B, void* C, int64_t ldc, int out_dtype) {
    dg::BlockArgs a;
    memset(&a, 0, sizeof a);
    a.A = static_cast<const uint8_t*>(A.data);
    a.B = static_cast<const uint8_t*>(B.data);
    a.SA = A.scale;
    a.SB = B.scale;
    a.lda = A.ld;
    a.ldb = B.ld;
    a.sa_row = A.scale_row;
    a.sa_blk = A.scale_block;
    a.sb_row = B.scale_row;
    a.sb_blk = B.scale_block;
    a.stride_b = B.stride;
    a.stride_sb = B.scale_stride;
    a.C = C;
    a.ldc = ldc;
    a.M = (int)A.rows;
    a.N = (int)B.rows;
    a.K = (int)A.cols;
    a.a_rows = (int)A.rows;
    a.out_dt = out_dtype;
    a.a_shift = A.block_rows == 1 ? 0 : 7;
    a.b_shift = B.block_rows == 1 ? 0 : 7;
    a.k_split = 1;
    return a;
}

int launch(const dg::BlockPlan& p, dg::BlockArgs& a, int64_t tiles, int type_a, int type_b, hipStream_t s) {
    const int64_t threads = p.kernel == dg::BLOCK_DIRECT || p.kernel == dg::BLOCK_STAGED ? 256 : 512;
    if (tiles * threads > kMaxThreads) {
        set_error("the product needs %lld workgroups, more than a launch holds", (long long)tiles);
        return GEMM_ERR_UNSUPPORTED;
    }
    if (a.group_m == 0) a.group_m = std::max(1, std::min(dg::default_group_m(a.tiles_m, a.tiles_n), a.tiles_m));
    const dim3 grid((unsigned)tiles, (unsigned)a.k_split);
    const int rc = type_a == GEMM_E4M3 ? (type_b == GEMM_E4M3 ? dg::launch_block_e4m3_e4m3(p, a, grid, s)
                                                              : dg::launch_block_e4m3_e5m2(p, a, grid, s))
                                       : (type_b == GEMM_E4M3 ? dg::launch_block_e5m2_e4m3(p, a, grid, s)
                                                              : dg::launch_block_e5m2_e5m2(p, a, grid, s));
    return launched(rc, "block product");
}

// Rows 0 .. M-1 of a product (checked).
int run_block(const gemm_block_matrix& A, const gemm_block_matrix& B, int64_t M, void* C, int64_t ldc, int out_dtype,
              void* workspace, int64_t workspace_bytes, hipStream_t stream) {
    const int64_t N = B.rows, K = A.cols;
    const int tr = tr_of(A, B);
    const bool direct = direct_rows(A, 1) && direct_rows(B, 1), small = small_call(A, B);
    dg::BlockPlan p = block_plan(dg::BLOCK_PLAIN, M, 1, N, K, direct, small, tr, true);
    if (split_bytes(p.split, M, N) > workspace_bytes) p = block_plan(dg::BLOCK_PLAIN, M, 1, N, K, direct, small, tr, false);
    dg::BlockArgs a = block_args(A, B, C, ldc, out_dtype);
    a.mode = dg::BLOCK_PLAIN;
    a.M = (int)M;
    a.tiles_m = (int)ceil_div(M, p.bm);
    a.tiles_n = (int)ceil_div(N, p.bn);
    if (p.split > 1) {
        a.k_split = p.split;
        a.kb_chunk = (int)ceil_div(ceil_div(K, dg::kBlock), p.split);
        a.work = static_cast<float*>(workspace);
        a.work_ld = (int)(ceil_div(N, 4) * 4);
        a.work_slice = M * (int64_t)a.work_ld;
    }
    DG_TRY(launch(p, a, (int64_t)a.tiles_m * a.tiles_n, A.dtype, B.dtype, stream));
    if (p.split > 1) {
        dg::Epilogue ep = dg::plain_epilogue();
        ep.kind = out_dtype != GEMM_F32;
        ep.out_dt = out_dtype;
        return launched(dg::launch_splitk_reduce(a.work, p.split, a.work_slice, a.work_ld, (int)M, (int)N, C, ldc, ep, stream),
                        "block product's reduction");
    }
    return GEMM_OK;
}

int check_c(void* C, int64_t ldc, int64_t N, int out_dtype) {
    DG_TRY(check_dtype("out_dtype", out_dtype));
    DG_TRY(check_ld("ldc", ldc, N));
    return check_pointer("C", C);
}

int check_router(const gemm_router* r, int64_t tokens, int64_t experts) {
    DG_TRY(check_pointer("router", r));
    DG_TRY(check_size("tokens", tokens));
    DG_TRY(check_size("experts", experts));
    if (experts < 1 || experts > dg::kMaxExperts) {
        set_error("experts = %lld must be 1 .. %d", (long long)experts, dg::kMaxExperts);
        return experts < 1 ? GEMM_ERR_INVALID_VALUE : GEMM_ERR_UNSUPPORTED;
    }
    if (r->top_k < 1 || r->top_k > experts || r->top_k > dg::kMaxTopK) {
        set_error("router.top_k = %d must be 1 .. min(%d, %lld experts)", r->top_k, dg::kMaxTopK, (long long)experts);
        return GEMM_ERR_INVALID_VALUE;
    }
    if (r->score != GEMM_SCORE_SOFTMAX && r->score != GEMM_SCORE_SIGMOID) {
        set_error("router.score = %d is not a gemm_score", r->score);
        return GEMM_ERR_INVALID_VALUE;
    }
    if (r->groups < 1 || experts % r->groups != 0 || r->top_groups < 1 || r->top_groups > r->groups ||
        r->group_top < 1 || r->group_top > 4 || (r->groups > 1 && r->group_top > experts / r->groups)) {
        set_error("router: groups = %d must divide %lld experts, top_groups = %d be 1 .. groups, group_top = %d be "
                  "1 .. min(4, experts of a group)", r->groups, (long long)experts, r->top_groups, r->group_top);
        return GEMM_ERR_INVALID_VALUE;
    }
    if (r->groups > 1 && r->top_k > r->top_groups * (experts / r->groups)) {
        set_error("router.top_k = %d exceeds the %lld experts of top_groups = %d groups", r->top_k,
                  (long long)(r->top_groups * (experts / r->groups)), r->top_groups);
        return GEMM_ERR_INVALID_VALUE;
    }
    return GEMM_OK;
}

dg::RouteArgs route_args(const void* logits, int64_t tokens, int64_t experts, int64_t ld, const gemm_router& r) {
    dg::RouteArgs a;
    memset(&a, 0, sizeof a);
    a.logits = logits;
    a.ld = ld;
    a.tokens = (int)tokens;
    a.experts = (int)experts;
    a.top_k = r.top_k;
    a.score = r.score;
    a.groups = r.groups;
    a.top_groups = r.top_groups;
    a.group_top = r.group_top;
    a.renorm = r.renorm;
    a.factor = r.factor;
    return a;
}

}  // namespace

extern "C" {

int gemm_block_quantize(const void* X, int64_t x_rows, int64_t cols, int64_t ldx, int dtype, const int32_t* gather,
                        int64_t rows, const gemm_block_matrix* natural, const gemm_block_matrix* transposed,
                        void* stream) {
    dg::clear_error();
    DG_TRY(check_dtype("dtype", dtype));
    DG_TRY(check_size("x_rows", x_rows));
    DG_TRY(check_size("cols", cols));
    DG_TRY(check_size("rows", rows));
    DG_TRY(check_ld("ldx", ldx, cols));
    if (natural == nullptr && transposed == nullptr) {
        set_error("natural and transposed are both NULL");
        return GEMM_ERR_NULL_POINTER;
    }
    if (gather == nullptr && rows != x_rows) {
        set_error("rows = %lld must be x_rows = %lld without gather", (long long)rows, (long long)x_rows);
        return GEMM_ERR_INVALID_VALUE;
    }
    if (natural) {
        DG_TRY(check_block("natural", natural));
        DG_TRY(check_op_n("natural", *natural));
        if (natural->rows != rows || natural->cols != cols) {
            set_error("natural is %lld x %lld, not %lld x %lld", (long long)natural->rows, (long long)natural->cols,
                      (long long)rows, (long long)cols);
            return GEMM_ERR_INVALID_VALUE;
        }
    }
    if (transposed) {
        DG_TRY(check_block("transposed", transposed));
        DG_TRY(check_op_n("transposed", *transposed));
        if (transposed->rows != cols || transposed->cols != rows) {
            set_error("transposed is %lld x %lld, not %lld x %lld", (long long)transposed->rows,
                      (long long)transposed->cols, (long long)cols, (long long)rows);
            return GEMM_ERR_INVALID_VALUE;
        }
    }
    if (rows == 0 || cols == 0) return GEMM_OK;
    if (x_rows > 0) DG_TRY(check_pointer("X", X));
    const Range none = range("", nullptr, 0);
    DG_TRY(check_overlap({natural ? data_range("natural.data", *natural) : none,
                          natural ? scale_range("natural.scale", *natural) : none,
                          transposed ? data_range("transposed.data", *transposed) : none,
                          transposed ? scale_range("transposed.scale", *transposed) : none},
                         {range("X", X, span(x_rows, cols, ldx, elem_size(dtype))),
                          range("gather", gather, (uint64_t)rows * 4)}));
    if (ceil_div(rows, 128) * ceil_div(cols, 128) * 256 > kMaxThreads) {
        set_error("%lld x %lld has more blocks than a launch holds", (long long)rows, (long long)cols);
        return GEMM_ERR_UNSUPPORTED;
    }
    DG_TRY(check_device());
    dg::QuantArgs a;
    memset(&a, 0, sizeof a);
    a.X = X;
    a.ldx = ldx;
    a.gather = gather;
    a.x_rows = (int)x_rows;
    a.rows = (int)rows;
    a.cols = (int)cols;
    auto out = [](dg::QuantOut& o, const gemm_block_matrix* m) {
        if (m == nullptr) return;
        o.q = static_cast<uint8_t*>(m->data);
        o.s = m->scale;
        o.ld = m->ld;
        o.s_row = m->scale_row;
        o.s_blk = m->scale_block;
        o.type = m->dtype == GEMM_E4M3 ? 0 : 1;
        o.block_rows = m->block_rows;
    };
    out(a.nat, natural);
    out(a.tr, transposed);
    return launched(dg::launch_block_quantize(a, dtype, (hipStream_t)stream), "block quantize");
}

int64_t gemm_block_product_workspace(int64_t M, int64_t N, int64_t K) {
    if (M <= 0 || N <= 0 || K <= 0 || M > kMaxDim || N > kMaxDim || K > kMaxDim) return 0;
    int64_t bytes = 0;
    // every plan that the call may make, for all rows or for whole tiles of them
    for (int64_t rows : {M, M - M % 128})
        for (bool direct : {false, true})
            for (int tr : {0, 1})
                if (rows > 0)
                    bytes = std::max(bytes, split_bytes(block_plan(dg::BLOCK_PLAIN, rows, 1, N, K, direct, direct, tr, true).split, rows, N));
    return bytes;
}

int gemm_block_product(const gemm_block_matrix* A, const gemm_block_matrix* B, void* C, int64_t ldc, int out_dtype,
                       void* workspace, int64_t workspace_bytes, void* stream) {
    dg::clear_error();
    DG_TRY(check_block("A", A));
    DG_TRY(check_block("B", B));
    if (A->cols != B->cols) {
        set_error("A has %lld columns, B %lld", (long long)A->cols, (long long)B->cols);
        return GEMM_ERR_INVALID_VALUE;
    }
    const int64_t M = A->rows, N = B->rows, K = A->cols;
    if (workspace_bytes < 0 || (workspace_bytes > 0 && ((uintptr_t)workspace & 15) != 0)) {
        set_error("the workspace must be 16-byte aligned and its size non-negative");
        return GEMM_ERR_INVALID_VALUE;
    }
    if (workspace_bytes > 0) DG_TRY(check_pointer("workspace", workspace));
    if (M == 0 || N == 0) {
        DG_TRY(check_dtype("out_dtype", out_dtype));
        return check_ld("ldc", ldc, N);
    }
    DG_TRY(check_c(C, ldc, N, out_dtype));
    DG_TRY(check_overlap({range("C", C, span(M, N, ldc, elem_size(out_dtype))),
                          range("the workspace", workspace, (uint64_t)workspace_bytes)},
                         {data_range("A.data", *A), scale_range("A.scale", *A), data_range("B.data", *B),
                          scale_range("B.scale", *B)}));
    DG_TRY(check_device());
    const bool direct = direct_rows(*A, 1) && direct_rows(*B, 1);
    const dg::BlockPlan whole = block_plan(dg::BLOCK_PLAIN, M, 1, N, K, direct, small_call(*A, *B), tr_of(*A, *B), true);
    const int64_t rest = dg::rest_rows(whole, M, N, K);
    DG_TRY(run_block(*A, *B, M - rest, C, ldc, out_dtype, workspace, workspace_bytes, (hipStream_t)stream));
    if (rest == 0) return GEMM_OK;
    gemm_block_matrix last = *A;
    last.rows = rest;
    last.data = static_cast<char*>(A->data) + (M - rest) * A->ld;
    last.scale = A->scale + (M - rest) / A->block_rows * A->scale_row;
    return run_block(last, *B, rest, static_cast<char*>(C) + (M - rest) * ldc * elem_size(out_dtype), ldc, out_dtype, nullptr,
                     0, (hipStream_t)stream);
}

int gemm_experts_route(const void* logits, int64_t tokens, int64_t experts, int64_t ld, int dtype,
                       const gemm_router* router, const float* bias, int32_t* index, float* weight, void* stream) {
    dg::clear_error();
    DG_TRY(check_dtype("dtype", dtype));
    DG_TRY(check_router(router, tokens, experts));
    DG_TRY(check_ld("ld", ld, experts));
    if (tokens == 0) return GEMM_OK;
    DG_TRY(check_pointer("logits", logits));
    DG_TRY(check_pointer("index", index));
    DG_TRY(check_pointer("weight", weight));
    const uint64_t pairs = (uint64_t)tokens * (uint64_t)router->top_k * 4;
    DG_TRY(check_overlap({range("index", index, pairs), range("weight", weight, pairs)},
                         {range("logits", logits, span(tokens, experts, ld, elem_size(dtype))),
                          range("bias", bias, (uint64_t)experts * 4)}));
    DG_TRY(check_device());
    dg::RouteArgs a = route_args(logits, tokens, experts, ld, *router);
    a.bias = bias;
    a.index = index;
    a.weight = weight;
    return launched(dg::launch_route(a, dtype, false, (hipStream_t)stream), "experts route");
}

int gemm_experts_route_backward(const void* logits, int64_t tokens, int64_t experts, int64_t ld, int dtype,
                                const gemm_router* router, const int32_t* index, const float* weight_grad, void* grad,
                                int64_t ldg, void* stream) {
    dg::clear_error();
    DG_TRY(check_dtype("dtype", dtype));
    DG_TRY(check_router(router, tokens, experts));
    DG_TRY(check_ld("ld", ld, experts));
    DG_TRY(check_ld("ldg", ldg, experts));
    if (tokens == 0) return GEMM_OK;
    DG_TRY(check_pointer("logits", logits));
    DG_TRY(check_pointer("index", index));
    DG_TRY(check_pointer("weight_grad", weight_grad));
    DG_TRY(check_pointer("grad", grad));
    const uint64_t pairs = (uint64_t)tokens * (uint64_t)router->top_k * 4;
    DG_TRY(check_overlap({range("grad", grad, span(tokens, experts, ldg, elem_size(dtype)))},
                         {range("logits", logits, span(tokens, experts, ld, elem_size(dtype))),
                          range("index", index, pairs), range("weight_grad", weight_grad, pairs)}));
    DG_TRY(check_device());
    dg::RouteArgs a = route_args(logits, tokens, experts, ld, *router);
    a.index_in = index;
    a.weight_grad = weight_grad;
    a.grad = grad;
    a.ldg = ldg;
    return launched(dg::launch_route(a, dtype, true, (hipStream_t)stream), "experts route's gradient");
}

int64_t gemm_experts_capacity(int64_t tokens, int64_t top_k, int64_t experts, int64_t align) {
    if (tokens <= 0 || top_k <= 0 || experts <= 0 || align <= 0 || tokens > kMaxDim || top_k > kMaxDim ||
        experts > kMaxDim || align > kMaxDim)
        return 0;
    const int64_t n = tokens * top_k;
    return ceil_div(n + std::min(experts, n) * (align - 1), align) * align;
}

int64_t gemm_experts_dispatch_workspace(int64_t tokens, int64_t top_k, int64_t experts) {
    if (tokens <= 0 || top_k <= 0 || experts <= 0 || tokens > kMaxDim || top_k > kMaxDim || experts > kMaxDim) return 0;
    const int64_t chunks = ceil_div(tokens * top_k, dg::kDispatchChunk);
    return chunks > 1 ? chunks * experts * 4 : 0;
}

int gemm_experts_dispatch(const int32_t* index, int64_t align, const gemm_expert_plan* plan, void* workspace,
                          int64_t workspace_bytes, void* stream) {
    dg::clear_error();
    DG_TRY(check_plan(plan));
    if (plan->experts < 1 || plan->experts > dg::kMaxExperts) {
        set_error("plan.experts = %lld must be 1 .. %d", (long long)plan->experts, dg::kMaxExperts);
        return plan->experts < 1 ? GEMM_ERR_INVALID_VALUE : GEMM_ERR_UNSUPPORTED;
    }
    if (align < 1 || align > ((int64_t)1 << 20)) {
        set_error("align = %lld must be 1 .. 2^20", (long long)align);
        return GEMM_ERR_INVALID_VALUE;
    }
    const int64_t n = plan->tokens * plan->top_k;
    const int64_t need = gemm_experts_capacity(plan->tokens, plan->top_k, plan->experts, align);
    if (need > kMaxDim) {
        set_error("the plan needs %lld rows, more than 2^31 - 1", (long long)need);
        return GEMM_ERR_UNSUPPORTED;
    }
    if (plan->capacity < need) {
        set_error("plan.capacity = %lld must be at least %lld", (long long)plan->capacity, (long long)need);
        return GEMM_ERR_INVALID_VALUE;
    }
    const int64_t ws = gemm_experts_dispatch_workspace(plan->tokens, plan->top_k, plan->experts);
    if (workspace_bytes < ws || ((uintptr_t)workspace & 3) != 0) {
        set_error("the workspace must be 4-byte aligned and hold %lld bytes, not %lld", (long long)ws,
                  (long long)workspace_bytes);
        return GEMM_ERR_INVALID_VALUE;
    }
    DG_TRY(check_pointer("plan.offsets", plan->offsets));
    DG_TRY(check_pointer("plan.counts", plan->counts));
    if (plan->capacity > 0) DG_TRY(check_pointer("plan.rows", plan->rows));
    if (n > 0) {
        DG_TRY(check_pointer("index", index));
        DG_TRY(check_pointer("plan.position", plan->position));
    }
    if (ws > 0) DG_TRY(check_pointer("workspace", workspace));
    DG_TRY(check_overlap({range("plan.offsets", plan->offsets, (uint64_t)(plan->experts + 1) * 4),
                          range("plan.counts", plan->counts, (uint64_t)plan->experts * 4),
                          range("plan.rows", plan->rows, (uint64_t)plan->capacity * 4),
                          range("plan.position", plan->position, (uint64_t)n * 4),
                          range("the workspace", workspace, (uint64_t)ws)},
                         {range("index", index, (uint64_t)n * 4)}));
    DG_TRY(check_device());
    dg::DispatchArgs a;
    memset(&a, 0, sizeof a);
    a.index = index;
    a.n = (int)n;
    a.top_k = (int)std::max<int64_t>(plan->top_k, 1);
    a.experts = (int)plan->experts;
    a.capacity = (int)plan->capacity;
    a.align = align;
    a.offsets = plan->offsets;
    a.counts = plan->counts;
    a.rows = plan->rows;
    a.position = plan->position;
    a.work = static_cast<int*>(workspace);
    a.chunks = (int)std::max<int64_t>(1, ceil_div(n, dg::kDispatchChunk));
    return launched(dg::launch_dispatch(a, (hipStream_t)stream), "experts dispatch");
}

int gemm_experts_product(const gemm_block_matrix* A, const gemm_block_matrix* B, const gemm_expert_plan* plan,
                         int gather, void* C, int64_t ldc, int out_dtype, void* stream) {
    dg::clear_error();
    DG_TRY(check_plan(plan));
    DG_TRY(check_block("A", A));
    DG_TRY(check_block("B", B, plan->experts));
    DG_TRY(check_op_n("A", *A));
    if (A->cols != B->cols) {
        set_error("A has %lld columns, B %lld", (long long)A->cols, (long long)B->cols);
        return GEMM_ERR_INVALID_VALUE;
    }
    const int64_t want = gather ? plan->tokens : plan->capacity;
    if (A->rows != want) {
        set_error("A has %lld rows, the plan %lld %s", (long long)A->rows, (long long)want, gather ? "tokens" : "rows");
        return GEMM_ERR_INVALID_VALUE;
    }
    const int64_t P = plan->capacity, N = B->rows, E = plan->experts;
    if (P == 0 || N == 0) {
        DG_TRY(check_dtype("out_dtype", out_dtype));
        return check_ld("ldc", ldc, N);
    }
    DG_TRY(check_c(C, ldc, N, out_dtype));
    DG_TRY(check_pointer("plan.offsets", plan->offsets));
    if (E > 0) DG_TRY(check_pointer("plan.counts", plan->counts));
    if (gather) DG_TRY(check_pointer("plan.rows", plan->rows));
    DG_TRY(check_overlap({range("C", C, span(P, N, ldc, elem_size(out_dtype)))},
                         {data_range("A.data", *A), scale_range("A.scale", *A), data_range("B.data", *B, E),
                          scale_range("B.scale", *B, E), range("plan.offsets", plan->offsets, (uint64_t)(E + 1) * 4),
                          range("plan.counts", plan->counts, (uint64_t)E * 4),
                          range("plan.rows", plan->rows, gather ? (uint64_t)P * 4 : 0)}));
    DG_TRY(check_device());
    const bool direct = direct_rows(*A, 1) && direct_rows(*B, E), small = small_call(*A, *B);
    const int64_t pairs = plan->tokens * plan->top_k, active = std::max<int64_t>(1, std::min(E, pairs));
    const dg::BlockPlan p = block_plan(dg::BLOCK_EXPERTS, std::max<int64_t>(1, pairs / active), active, N, A->cols, direct,
                                       small, tr_of(*A, *B), false);
    dg::BlockArgs a = block_args(*A, *B, C, ldc, out_dtype);
    a.mode = dg::BLOCK_EXPERTS;
    a.M = (int)P;
    a.E = (int)E;
    a.offsets = plan->offsets;
    a.counts = plan->counts;
    a.rows = gather ? plan->rows : nullptr;
    a.tiles_m = (int)std::max<int64_t>(1, P / p.bm + std::min(E, P));  // no plan has more; one clears rows without experts
    a.tiles_n = (int)ceil_div(N, p.bn);
    return launch(p, a, (int64_t)a.tiles_m * a.tiles_n, A->dtype, B->dtype, (hipStream_t)stream);
}

int gemm_experts_gradient(const gemm_block_matrix* A, const gemm_block_matrix* B, const gemm_expert_plan* plan,
                          void* C, int64_t ldc, int64_t stride_c, int out_dtype, void* stream) {
    dg::clear_error();
    DG_TRY(check_plan(plan));
    DG_TRY(check_block("A", A));
    DG_TRY(check_block("B", B));
    const int64_t M = A->rows, N = B->rows, E = plan->experts;
    if (A->cols != plan->capacity || B->cols != plan->capacity) {
        set_error("A has %lld columns and B %lld, the plan %lld rows", (long long)A->cols, (long long)B->cols,
                  (long long)plan->capacity);
        return GEMM_ERR_INVALID_VALUE;
    }
    if (M == 0 || N == 0 || E == 0) {
        DG_TRY(check_dtype("out_dtype", out_dtype));
        return check_ld("ldc", ldc, N);
    }
    DG_TRY(check_c(C, ldc, N, out_dtype));
    if (E > 1 && (stride_c < (M - 1) * ldc + N || stride_c >= ((int64_t)1 << 50))) {
        set_error("stride_c = %lld must be at least %lld", (long long)stride_c, (long long)((M - 1) * ldc + N));
        return GEMM_ERR_INVALID_VALUE;
    }
    DG_TRY(check_pointer("plan.offsets", plan->offsets));
    DG_TRY(check_overlap({range("C", C, span(M, N, ldc, elem_size(out_dtype), E, stride_c))},
                         {data_range("A.data", *A), scale_range("A.scale", *A), data_range("B.data", *B),
                          scale_range("B.scale", *B), range("plan.offsets", plan->offsets, (uint64_t)(E + 1) * 4)}));
    DG_TRY(check_device());
    const bool direct = direct_rows(*A, 1) && direct_rows(*B, 1), small = small_call(*A, *B);
    const dg::BlockPlan p = block_plan(dg::BLOCK_GRADIENT, M, E, N, ceil_div(plan->capacity, E), direct, small,
                                       tr_of(*A, *B), false);
    dg::BlockArgs a = block_args(*A, *B, C, ldc, out_dtype);
    a.mode = dg::BLOCK_GRADIENT;
    a.E = (int)E;
    a.offsets = plan->offsets;
    a.stride_c = stride_c;
    a.tiles_m = (int)ceil_div(M, p.bm);
    a.tiles_n = (int)ceil_div(N, p.bn);
    a.group_m = 1;
    return launch(p, a, ceil_div((int64_t)a.tiles_m * a.tiles_n, 8) * 8 * E, A->dtype, B->dtype, (hipStream_t)stream);
}

int gemm_experts_combine(const void* Y, int64_t cols, int64_t ldy, int dtype, const gemm_expert_plan* plan,
                         const float* weight, void* out, int64_t ldo, void* stream) {
    dg::clear_error();
    DG_TRY(check_dtype("dtype", dtype));
    DG_TRY(check_plan(plan));
    DG_TRY(check_size("cols", cols));
    DG_TRY(check_ld("ldy", ldy, cols));
    DG_TRY(check_ld("ldo", ldo, cols));
    const int64_t T = plan->tokens, n = T * plan->top_k, es = elem_size(dtype);
    if (T == 0 || cols == 0) return GEMM_OK;
    DG_TRY(check_pointer("out", out));
    if (n > 0) {
        DG_TRY(check_pointer("plan.position", plan->position));
        DG_TRY(check_pointer("weight", weight));
    }
    if (plan->capacity > 0) DG_TRY(check_pointer("Y", Y));
    DG_TRY(check_overlap({range("out", out, span(T, cols, ldo, es))},
                         {range("Y", Y, span(plan->capacity, cols, ldy, es)),
                          range("weight", weight, (uint64_t)n * 4), range("plan.position", plan->position, (uint64_t)n * 4)}));
    DG_TRY(check_device());
    dg::CombineArgs a;
    memset(&a, 0, sizeof a);
    a.Y = Y;
    a.ldy = ldy;
    a.cols = (int)cols;
    a.tokens = (int)T;
    a.top_k = (int)plan->top_k;
    a.capacity = (int)plan->capacity;
    a.position = plan->position;
    a.weight = weight;
    a.out = out;
    a.ldo = ldo;
    return launched(dg::launch_combine(a, dtype, (hipStream_t)stream), "experts combine");
}

int gemm_experts_combine_backward(const void* Y, int64_t cols, int64_t ldy, int dtype, const gemm_expert_plan* plan,
                                  const float* weight, const void* G, int64_t ldg, void* y_grad, int64_t ldyg,
                                  float* weight_grad, void* stream) {
    dg::clear_error();
    DG_TRY(check_dtype("dtype", dtype));
    DG_TRY(check_plan(plan));
    DG_TRY(check_size("cols", cols));
    DG_TRY(check_ld("ldy", ldy, cols));
    DG_TRY(check_ld("ldg", ldg, cols));
    DG_TRY(check_ld("ldyg", ldyg, cols));
    if (plan->top_k > dg::kMaxTopK) {
        set_error("plan.top_k = %lld must be at most %d", (long long)plan->top_k, dg::kMaxTopK);
        return GEMM_ERR_UNSUPPORTED;
    }
    const int64_t T = plan->tokens, n = T * plan->top_k, P = plan->capacity, es = elem_size(dtype);
    if (n == 0 && (P == 0 || cols == 0)) return GEMM_OK;
    if (n > 0) {
        DG_TRY(check_pointer("plan.position", plan->position));
        DG_TRY(check_pointer("weight", weight));
        DG_TRY(check_pointer("weight_grad", weight_grad));
        if (cols > 0) DG_TRY(check_pointer("G", G));
    }
    if (P > 0) DG_TRY(check_pointer("plan.rows", plan->rows));
    if (P > 0 && cols > 0) {
        DG_TRY(check_pointer("Y", Y));
        DG_TRY(check_pointer("y_grad", y_grad));
    }
    DG_TRY(check_overlap({range("y_grad", y_grad, span(P, cols, ldyg, es)), range("weight_grad", weight_grad, (uint64_t)n * 4)},
                         {range("Y", Y, span(P, cols, ldy, es)), range("G", G, span(T, cols, ldg, es)),
                          range("weight", weight, (uint64_t)n * 4), range("plan.position", plan->position, (uint64_t)n * 4),
                          range("plan.rows", plan->rows, (uint64_t)P * 4)}));
    DG_TRY(check_device());
    dg::CombineArgs a;
    memset(&a, 0, sizeof a);
    a.Y = Y;
    a.ldy = ldy;
    a.cols = (int)cols;
    a.tokens = (int)T;
    a.top_k = (int)plan->top_k;
    a.capacity = (int)P;
    a.position = plan->position;
    a.rows = plan->rows;
    a.weight = weight;
    a.G = G;
    a.ldg = ldg;
    a.y_grad = y_grad;
    a.ldyg = ldyg;
    a.weight_grad = weight_grad;
    return launched(dg::launch_combine_backward(a, dtype, (hipStream_t)stream), "experts combine's gradient");
}

}  // extern "C"
