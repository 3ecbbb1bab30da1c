// layers_api.cpp -- the C ABI declared in include/gemm_layers.h: validation, workspaces and
// the launches. Everything is validated before the first launch.
#include <hip/hip_runtime.h>
#include <string.h>

#include <algorithm>

#include "checks.h"
#include "launch.h"
#include "layers.h"
#include "plan.h"
#include "product.h"

namespace {

// Workspace that a plain product inside an operator may split K or pack its operands in.
constexpr int64_t kProductWorkspace = (int64_t)32 << 20;

int64_t align256(int64_t n) { return (n + 255) / 256 * 256; }

// Hands out the parts of a workspace; with a NULL base it only counts them.
struct Parts {
    char* base;
    int64_t at = 0;
    void* take(int64_t bytes) {
        char* p = base ? base + at : nullptr;
        at += align256(bytes);
        return p;
    }
};

int check_workspace(const void* workspace, int64_t bytes, int64_t need) {
    if (bytes < need) {
        set_error("workspace_bytes = %lld is less than the %lld that the call needs", (long long)bytes, (long long)need);
        return GEMM_ERR_INVALID_VALUE;
    }
    if (bytes == 0) return GEMM_OK;
    DG_TRY(check_pointer("workspace", workspace));
    if (((uintptr_t)workspace & 15) != 0) {
        set_error("the workspace must be 16-byte aligned (got %p)", workspace);
        return GEMM_ERR_INVALID_VALUE;
    }
    return GEMM_OK;
}

int check_threads(const char* what, int64_t a, int64_t b, int64_t each) {
    if ((unsigned __int128)a * (uint64_t)b * (uint64_t)each <= (unsigned __int128)kMaxThreads) return GEMM_OK;
    set_error("%s = %lld * %lld needs more threads than a launch holds", what, (long long)a, (long long)b);
    return GEMM_ERR_UNSUPPORTED;
}

// A product inside an operator: C of type out_dtype, plus beta C for fp32 C.
int product(int opB, int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, const void* B, int64_t ldb, void* C,
            int64_t ldc, int dtype, int out_dtype, float beta, void* ws, int64_t ws_bytes, void* stream) {
    dg::Epilogue ep = dg::plain_epilogue();
    if (out_dtype != GEMM_F32 || beta != 0.0f) {
        ep.kind = 1;
        ep.out_dt = out_dtype;
        ep.beta = beta;
        ep.R = beta != 0.0f ? C : nullptr;
        ep.ldr = ldc;
    }
    return dg::run_product(GEMM_OP_N, opB, M, N, K, A, std::max<int64_t>(1, lda), B, std::max<int64_t>(1, ldb), C, ldc,
                           dtype, ep, nullptr, ws, ws_bytes, stream);
}

// Sizes that the calls take (check_product, check_adapters); for others a workspace's size is 0.
bool sizes_ok(std::initializer_list<int64_t> sizes) {
    for (int64_t n : sizes)
        if (n < 0 || n >= (int64_t)1 << 30) return false;
    return true;
}
bool adapters_ok(int64_t adapters, int64_t rank) {
    return adapters >= 0 && adapters <= dg::kMaxAdapters && rank >= 0 && rank <= dg::kMaxRank;
}

struct Named {
    const char* what;
    int64_t value;
};
// What the products' kernels take: they count rows and columns in 32 bits with a tile to spare, and
// address 256 rows of an operand from one place with 32 bits.
int check_product(std::initializer_list<Named> sizes, std::initializer_list<Named> lds) {
    for (const Named& n : sizes)
        if (n.value >= (int64_t)1 << 30) {
            set_error("%s = %lld must be below 2^30", n.what, (long long)n.value);
            return GEMM_ERR_UNSUPPORTED;
        }
    for (const Named& n : lds)
        if (n.value >= (int64_t)1 << 23) {
            set_error("%s = %lld must be below 2^23", n.what, (long long)n.value);
            return GEMM_ERR_UNSUPPORTED;
        }
    return GEMM_OK;
}

// ---------------------------------------------------------------- adapters
int check_adapters(const gemm_adapter_set* s, int64_t N, int64_t K) {
    DG_TRY(check_pointer("set", s));
    DG_TRY(check_size("set.adapters", s->adapters));
    if (s->adapters > dg::kMaxAdapters) {
        set_error("set.adapters = %lld must be at most %d", (long long)s->adapters, dg::kMaxAdapters);
        return GEMM_ERR_UNSUPPORTED;
    }
    if (s->rank < (s->adapters > 0 ? 1 : 0) || s->rank > dg::kMaxRank) {
        set_error("set.rank = %lld must be 1 .. %d", (long long)s->rank, dg::kMaxRank);
        return s->rank > dg::kMaxRank ? GEMM_ERR_UNSUPPORTED : GEMM_ERR_INVALID_VALUE;
    }
    DG_TRY(check_ld("set.lda", s->lda, K));
    DG_TRY(check_ld("set.ldb", s->ldb, s->rank));
    if (s->stride_a < 0 || s->stride_b < 0 || s->stride_a >= ((int64_t)1 << 40) || s->stride_b >= ((int64_t)1 << 40)) {
        set_error("set: strides must be non-negative and below 2^40");
        return GEMM_ERR_INVALID_VALUE;
    }
    if (s->adapters > 0) {
        if (K > 0) DG_TRY(check_pointer("set.a", s->a));
        if (N > 0) DG_TRY(check_pointer("set.b", s->b));
    }
    return GEMM_OK;
}

// Threads of the first product's widest launch on 16-bit matrices (see shrink16); fp32 kernels walk their
// tokens, as does the form for few tokens and ranks.
bool shrink_by_rows(int64_t tokens, int64_t rank) { return tokens * rank <= 8192; }
int check_shrink_threads(int64_t tokens, int64_t rank, int dtype, bool direct) {
    if (dtype == GEMM_F32 || rank == 0 || shrink_by_rows(tokens, rank)) return GEMM_OK;
    DG_TRY(check_threads("tokens * rank", tokens, ceil_div(rank, 16) * 2, 2));  // an eighth of the padded rank, or more
    return check_threads("blocks of tokens", ceil_div(tokens, direct ? 64 : 16), 1, direct ? 256 : 512);
}
// And of the second's: in tiles, on its own, or with up to 64 tokens by strips of 16 columns (those of
// 64 of the stream are no more).
int check_expand_threads(int64_t tokens, int64_t cols, int dtype, bool tiles, bool few) {
    if (dtype == GEMM_F32) return GEMM_OK;
    if (few) return check_threads("blocks of columns", ceil_div(cols, 16), 1, 512);
    if (tiles) return check_threads("tiles of tokens * columns", ceil_div(tokens, 256), ceil_div(cols, 256), 512);
    return check_threads("blocks of tokens * columns", ceil_div(tokens, 32), ceil_div(cols, 64), 256);
}

Range a_range(const gemm_adapter_set& s, int64_t K, int64_t es) {
    return range("set.a", s.a, span(s.rank, K, s.lda, es, s.adapters, s.stride_a));
}
Range b_range(const gemm_adapter_set& s, int64_t N, int64_t es) {
    return range("set.b", s.b, span(N, s.rank, s.ldb, es, s.adapters, s.stride_b));
}
Range scale_of(const gemm_adapter_set& s) { return range("set.scale", s.scale, (uint64_t)s.adapters * 4); }

int64_t rank_padded(int64_t rank) { return rank <= 16 ? 16 : rank <= 32 ? 32 : rank <= 64 ? 64 : 128; }

#define DG_BY_TYPE(name, dtype, ...) \
    ((dtype) == GEMM_F16 ? dg::name##_f16(__VA_ARGS__) : dg::name##_bf16(__VA_ARGS__))

dg::AdapterArgs adapter_args(const gemm_adapter_set& s, int64_t tokens, const int32_t* index) {
    dg::AdapterArgs a;
    memset(&a, 0, sizeof a);
    a.tokens = (int)tokens;
    a.rank = (int)s.rank;
    a.rank_p = (int)rank_padded(s.rank);
    a.adapters = (int)s.adapters;
    a.index = index;
    return a;
}

void with_a(dg::AdapterArgs& a, const gemm_adapter_set& s, int64_t K) {
    a.m = s.a;
    a.ldm = s.lda;
    a.stride_m = s.stride_a;
    a.turned = 0;
    a.cols = (int)K;
}

void with_b(dg::AdapterArgs& a, const gemm_adapter_set& s, int64_t N) {
    a.m = s.b;
    a.ldm = s.ldb;
    a.stride_m = s.stride_b;
    a.turned = 1;
    a.rank_m = (int)s.rank;
    a.cols = (int)N;
}

// Tokens up to which one workgroup has all of them (kernel_skinny.h).
constexpr int64_t kSkinny = 64;

// Whether 256 x 256 tiles of the result give enough compute units work for the kernel that adds
// the adapters to the product in its tiles.
bool adapter_tiles(int64_t tokens, int64_t cols) { return ceil_div(tokens, 256) * ceil_div(cols, 256) >= 128; }

int tile_group(int64_t rows, int64_t cols, int64_t tile = 256) {
    const int64_t m = ceil_div(rows, tile);
    return (int)std::max<int64_t>(1, std::min<int64_t>(dg::default_group_m(m, ceil_div(cols, tile)), m));
}

// How the kernels on 16-bit matrices read x (rows x len) and w (op T: cols x len, op N: len x cols):
// 0 not at all, 1 through registers, 2 straight to LDS.
bool whole_pieces(const void* p, int64_t ld, int64_t cols) {
    return ((uintptr_t)p & 15) == 0 && ld % 8 == 0 && cols % 8 == 0;
}
int tiles_form(const void* x, int64_t ldx, const void* w, int64_t ldw, int64_t cols, int64_t len, int opb, int dtype) {
    if (dtype == GEMM_F32 || len < 8 || (opb == GEMM_OP_N && cols < 8)) return 0;
    return whole_pieces(x, ldx, len) && whole_pieces(w, ldw, opb == GEMM_OP_T ? len : cols) ? 2 : 1;
}

// k cut into slices of whole stages (128) so that `tiles` of them make two workgroups for each
// compute unit.
struct Slices {
    int64_t count, k;
};
Slices slices_of(int64_t tiles, int64_t K, int64_t others = 0, bool equal = false) {
    const int64_t stages = std::max<int64_t>(1, ceil_div(K, 128)), most = 2 * dg::kCus;
    tiles = std::max<int64_t>(1, tiles);  // none where the result is empty
    int64_t want = ceil_div(most, tiles);
    // room for `others` workgroups beside them, rather than after them, and with many rows of x, whose
    // copies take longer, slices of equally many stages or nearly so (17, 33 and 64 tokens of 4096 x 4096,
    // rank 16: 14.4, 17.0, 18.9 us without the room, 13.0, 16.5, 18.7 with it in 7 slices, 13.0, 16.0, 17.4 in 4;
    // rank 64: 17.5, 21.5, 25.8, then 16.3, 23.4, 24.3, then 16.4, 20.5, 24.9; 4096 x 14336: 28.3, 33.3, 35.1,
    // then 25.3, 33.7, 35.3; 32 tokens of 4096 x 4096 in 4 slices 13.9, in 7 13.3)
    if (others > 0 && want * tiles <= most && tiles <= most - others) {
        want = (most - others) / tiles;
        for (int64_t n = want; equal && n >= 2 && 2 * n >= want; --n)
            if (16 * (n * ceil_div(stages, n) - stages) <= stages) {
                want = n;
                break;
            }
    }
    want = std::min({want, stages, (int64_t)32});
    const int64_t k = ceil_div(stages, want) * 128;
    return {std::max<int64_t>(1, ceil_div(K, k)), k};
}

struct AdapterSpace {
    Slices mid = {1, 0};      // of the shared product in 128 x 128 tiles
    float* base = nullptr;    // the shared product (16-bit matrices without a kernel for both)
    void* product = nullptr;
    float* part = nullptr;    // sums of slices of k
    uint16_t* us = nullptr;   // scale u (or v) as two 16-bit numbers
    uint16_t* us_b = nullptr; // scale u in the backward pass
    float* unit = nullptr;    // fp16: their powers of two
    float* unit_b = nullptr;
    float* v = nullptr;       // backward
    void* a_turned = nullptr; // adapters x K x rank_m, adapters x rank x N (16-bit matrices)
    void* b_turned = nullptr;
    float* sums = nullptr;    // the gradients' slots
    Slices slices = {1, 0};
    int64_t rank_m = 0, chunk = 0, slots = 0, bytes = 0;
};

// What the first product over `len` of 16-bit matrices needs, and the second's u.
void shrink_space(AdapterSpace& s, Parts& p, int64_t tokens, int64_t len, int64_t rank, int dtype) {
    // half as many as elsewhere: a tile's second adapter has a workgroup of its own, which finds room
    s.slices = slices_of(2 * ceil_div(tokens, 64), len);
    s.part = static_cast<float*>(p.take(s.slices.count * tokens * rank_padded(rank) * 4));
    s.us = static_cast<uint16_t*>(p.take(tokens * rank_padded(rank) * 4));
    if (dtype == GEMM_F16) s.unit = static_cast<float*>(p.take(tokens * 4));
}

// The shared product of a call without one kernel for both (sliced: it may come in slices of k).
void product_space(AdapterSpace& s, Parts& p, int64_t tokens, int64_t cols, int64_t len, int dtype, bool one_kernel, bool sliced) {
    if (one_kernel) return;
    if (dtype != GEMM_F32) {
        if (sliced) s.mid = slices_of(ceil_div(tokens, 128) * ceil_div(cols, 128), len);
        s.base = static_cast<float*>(p.take(s.mid.count * tokens * ceil_div(cols, 4) * 16));
    }
    s.product = p.take(kProductWorkspace);
}

// A forward call of 16-bit matrices: few tokens
bool few_tokens(int64_t tokens, int64_t K, int dtype) { return dtype != GEMM_F32 && K > 0 && tokens <= kSkinny; }
// or one kernel for the product and the adapters in its tiles, in either direction
bool in_tiles(int64_t tokens, int64_t cols, int64_t len, int64_t rank, int dtype) {
    return dtype != GEMM_F32 && cols >= 8 && len >= 8 && rank <= 64 && adapter_tiles(tokens, cols);
}

AdapterSpace adapter_space(void* workspace, int64_t tokens, int64_t N, int64_t K, int64_t rank, int dtype) {
    AdapterSpace s;
    Parts p{static_cast<char*>(workspace)};
    if (few_tokens(tokens, K, dtype)) {
        s.slices = slices_of(ceil_div(N, 64), K, tokens > 16 ? tokens * rank_padded(rank) / 16 : 0, tokens > 32);
        s.part = static_cast<float*>(p.take(s.slices.count * tokens * ceil_div(N, 4) * 16));
    } else {
        product_space(s, p, tokens, N, K, dtype, in_tiles(tokens, N, K, rank, dtype), true);
        if (dtype != GEMM_F32) shrink_space(s, p, tokens, K, rank, dtype);
    }
    s.bytes = p.at;
    return s;
}

AdapterSpace adapter_backward_space(void* workspace, int64_t tokens, int64_t N, int64_t K, int64_t adapters,
                                    int64_t rank, int dtype) {
    AdapterSpace s;
    Parts p{static_cast<char*>(workspace)};
    product_space(s, p, tokens, K, N, dtype, in_tiles(tokens, K, N, rank, dtype), false);
    s.v = static_cast<float*>(p.take(tokens * rank * 4));
    if (dtype != GEMM_F32) {
        shrink_space(s, p, tokens, N, rank, dtype);
        s.rank_m = ceil_div(rank, 16) * 16;
        s.a_turned = p.take(adapters * K * s.rank_m * 2);
        s.b_turned = p.take(adapters * N * rank * 2);
        // chunks of 512 rows (what the kernel holds), fewer where that leaves compute units idle
        s.chunk = 512;
        while (s.chunk > 64 && ceil_div(tokens, s.chunk) * (ceil_div(N, 64) + ceil_div(K, 64)) < 1024) s.chunk /= 2;
        s.slots = adapters + ceil_div(tokens, s.chunk);
        s.sums = static_cast<float*>(p.take(s.slots * rank * (N + K) * 4));
        s.us_b = static_cast<uint16_t*>(p.take(tokens * rank_padded(rank) * 4));
        if (dtype == GEMM_F16) s.unit_b = static_cast<float*>(p.take(tokens * 4));
    }
    s.bytes = p.at;
    return s;
}

#define DG_BY_TYPE(name, dtype, ...) \
    ((dtype) == GEMM_F16 ? dg::name##_f16(__VA_ARGS__) : dg::name##_bf16(__VA_ARGS__))

// Whether the first product's rows come by direct copies (a.m of rank x cols).
bool shrink_direct(const dg::AdapterArgs& a) {
    return whole_pieces(a.x, a.ldx, a.cols) && whole_pieces(a.m, a.ldm, a.cols) && a.stride_m % 8 == 0;
}

// u and us of 16-bit matrices for a.m of rank x cols.
int shrink16(const dg::AdapterArgs& a, const AdapterSpace& sp, int dtype, hipStream_t s) {
    // each token by itself where all of them together read no more than 8192 rows of the adapters
    if (shrink_by_rows(a.tokens, a.rank)) return DG_BY_TYPE(launch_adapter_shrink_row, dtype, a, s);
    return DG_BY_TYPE(launch_adapter_shrink16, dtype, a, shrink_direct(a), (int)sp.slices.count, (int)sp.slices.k, sp.part, s);
}

// ---------------------------------------------------------------- loss
// What d may take as it is, and transposed again. Larger pieces mean fewer rounds of adding to x's
// gradient (4096 tokens, 65536 words of 4096, bf16: 7.90, 7.71 and 7.54 ms with 32, 64 and 128 MB),
// and these still fit the last level of cache.
constexpr int64_t kPieceBytes = (int64_t)128 << 20;
constexpr int64_t kPieceMost = (int64_t)1 << 22;  // it is a leading dimension of a product

// Columns of a piece: whole blocks of 256, as many as kPieceBytes hold, and of those as many as
// make whole rounds of 256 x 256 tiles, but one block at least.
int64_t piece_of(int64_t tokens, int64_t vocabulary, int64_t each) {
    const int64_t blocks = std::max<int64_t>(1, kPieceBytes / std::max<int64_t>(1, tokens * each) / 256);
    const int64_t tm = std::max<int64_t>(1, ceil_div(tokens, 256)), rounds = tm * blocks / dg::kCus;
    const int64_t whole = rounds > 0 ? std::max<int64_t>(1, rounds * dg::kCus / tm) : blocks;
    return std::max<int64_t>(1, std::min({whole * 256, vocabulary, kPieceMost}));
}

struct LossSpace {
    void* part = nullptr;   // fused: maxima and sums of strips
    float* logits = nullptr;
    float* top = nullptr;
    float* sum = nullptr;
    float* picked = nullptr;
    float* factor = nullptr;
    float* apart = nullptr;
    float* rest = nullptr;
    void* d = nullptr;
    void* dt = nullptr;
    void* xp = nullptr;     // x with rows of zeros up to lddt
    float* x_acc = nullptr;
    float* w_acc = nullptr;
    void* product = nullptr;
    int64_t piece = 0, ldd = 0, lddt = 0, ldxp = 0, product_bytes = 0, bytes = 0;
};

// 16-bit logits are never stored but for the shortest sums.
bool loss_fused(int64_t vocabulary, int64_t K, int dtype) { return dtype != GEMM_F32 && K >= 8 && vocabulary > 0; }
// How tokens x n logits are cut into tiles: the first `wide` columns in 256 x 256 ones, the rest in
// 128 x 128 ones; up to 64 tokens need none. A round of 256 wide tiles takes about as long as three
// of narrow ones (2048 long, 32768 columns: 62 us for 256 wide tiles, 31 for 256 narrow ones and 62
// for 768), so a last round of few wide tiles, and wide tiles that are mostly empty, are done better
// by narrow ones.
struct LossTiles {
    int64_t wide, strips;   // strips: wide ones and narrow ones
};
LossTiles loss_tiles(int64_t tokens, int64_t n, bool direct) {
    const int64_t tm = ceil_div(tokens, 256), tn = ceil_div(n, 256), rounds = tm * tn / dg::kCus;
    const int64_t part = std::min(tn, rounds * dg::kCus / tm);  // columns of tiles in whole rounds
    auto narrow = [&](int64_t cols) { return ceil_div(ceil_div(tokens, 128) * ceil_div(cols, 128), dg::kCus); };
    const int64_t all_wide = 3 * ceil_div(tm * tn, dg::kCus), all_narrow = narrow(n);
    const int64_t both = part > 0 && part < tn ? 3 * rounds + narrow(n - part * 256) : all_wide;
    if (!direct || (all_wide <= all_narrow && all_wide <= both)) return {n, tn};
    if (all_narrow <= both) return {0, ceil_div(n, 128)};
    return {part * 256, part + ceil_div(n - part * 256, 128)};
}
int64_t loss_strips(int64_t tokens, int64_t vocabulary) {
    if (tokens <= kSkinny) return ceil_div(vocabulary, 16);
    return std::max(loss_tiles(tokens, vocabulary, false).strips, loss_tiles(tokens, vocabulary, true).strips);
}

LossSpace loss_space(void* workspace, int64_t tokens, int64_t vocabulary, int64_t K, int dtype) {
    LossSpace s;
    Parts p{static_cast<char*>(workspace)};
    if (loss_fused(vocabulary, K, dtype)) {
        s.part = p.take(loss_strips(tokens, vocabulary) * tokens * dg::kLossPartBytes);
        s.picked = static_cast<float*>(p.take(tokens * 4));
        s.bytes = p.at;
        return s;
    }
    s.piece = piece_of(tokens, vocabulary, 4);
    s.logits = static_cast<float*>(p.take(tokens * s.piece * 4));
    s.top = static_cast<float*>(p.take(tokens * 4));
    s.sum = static_cast<float*>(p.take(tokens * 4));
    s.picked = static_cast<float*>(p.take(tokens * 4));
    s.product = p.take(kProductWorkspace);
    s.bytes = p.at;
    return s;
}

// Whether d comes from the stream of w, or from 128 x 128 tiles once these fill the card (backward
// pass in bf16, tiles against stream: 1 token, 8192 x 1024: 39.4 and 31.2 us; 16, 32768 x 1024: 74 and 69;
// 60, 8192 x 1024: 43.2 and 40.9; 60, 32768 x 2048: 116 and 120).
bool loss_few(int64_t tokens, int64_t n) { return tokens <= 32 || (tokens <= kSkinny && ceil_div(n, 128) < dg::kCus); }

// Whether w's gradient (n x K) takes 128 x 128 tiles, by the same rounds; these need x transposed, and
// the others a copy where tokens are no multiple of 32 (d and w's gradient, bf16, wide against
// narrow: 200 tokens, 4000 x 512: 28.2 and 22.4 us; 500, 8192 x 1024: 41.8 and 37.2; 512: 36.5 and 36.9;
// 4000, 2000 x 512: 134 and 86).
bool loss_w_narrow(int64_t n, int64_t K) {
    return ceil_div(ceil_div(n, 128) * ceil_div(K, 128), dg::kCus) <
           3 * ceil_div(ceil_div(n, 256) * ceil_div(K, 256), dg::kCus);
}

// Workspace of x_grad's product: its sum over a piece is cut into up to eight slices.
int64_t x_product_bytes(int64_t tokens, int64_t K) {
    const int64_t most = (int64_t)128 << 20;
    return std::max(kProductWorkspace, tokens * K < most / 32 ? 8 * tokens * K * 4 : most);
}

LossSpace loss_backward_space(void* workspace, int64_t tokens, int64_t vocabulary, int64_t K, int dtype, bool x_grad,
                              bool w_grad, int64_t piece) {
    LossSpace s;
    Parts p{static_cast<char*>(workspace)};
    const int64_t es = elem_size(dtype);
    s.piece = piece > 0 ? std::min({piece, std::max<int64_t>(1, vocabulary), kPieceMost}) : piece_of(tokens, vocabulary, es);
    s.lddt = (tokens + 31) / 32 * 32;
    s.factor = static_cast<float*>(p.take(8));
    s.apart = static_cast<float*>(p.take(tokens * 4));
    s.rest = static_cast<float*>(p.take(tokens * 4));
    if (!loss_fused(vocabulary, K, dtype)) s.logits = static_cast<float*>(p.take(tokens * s.piece * 4));
    s.ldd = dtype == GEMM_F32 ? s.piece : ceil_div(s.piece, 8) * 8;
    if (x_grad) s.d = s.logits && dtype == GEMM_F32 ? s.logits : p.take(tokens * s.ldd * es);  // in place in fp32
    if (w_grad) s.dt = p.take(s.piece * s.lddt * es);
    // 16-bit sums over tokens run in whole stages and pieces of 16 bytes, over a copy of x with zeros at
    // its ends where x has others
    s.ldxp = ceil_div(K, 8) * 8;
    if (w_grad && loss_fused(vocabulary, K, dtype)) s.xp = p.take(s.lddt * s.ldxp * es);
    if (x_grad && dtype != GEMM_F32) s.x_acc = static_cast<float*>(p.take(tokens * K * 4));
    if (w_grad && dtype == GEMM_F16 && !loss_fused(vocabulary, K, dtype)) s.w_acc = static_cast<float*>(p.take(s.piece * K * 4));
    s.product_bytes = x_grad ? x_product_bytes(tokens, K) : kProductWorkspace;
    s.product = p.take(s.product_bytes);
    s.bytes = p.at;
    return s;
}

dg::LossProduct loss_product(const void* x, int64_t ldx, const void* w, int64_t ldw, int64_t tokens, int64_t n,
                             int64_t K, int dtype, int64_t tile) {
    return {x, w, ldx, ldw, (int)tokens, (int)n, (int)K, tile_group(tokens, n, tile),
            tiles_form(x, ldx, w, ldw, n, K, GEMM_OP_T, dtype) == 2, (int)tile};
}

// ---------------------------------------------------------------- activations
int check_activation(int activation, int64_t cols, int gated) {
    if (activation != GEMM_ACT_RELU && activation != GEMM_ACT_GELU_TANH && activation != GEMM_ACT_SILU) {
        set_error("activation = %d is not GEMM_ACT_RELU, GEMM_ACT_GELU_TANH or GEMM_ACT_SILU", activation);
        return GEMM_ERR_INVALID_VALUE;
    }
    if (gated && cols > kMaxDim / 2) {
        set_error("2 cols = %lld must be below 2^31", (long long)(2 * cols));
        return GEMM_ERR_UNSUPPORTED;
    }
    return GEMM_OK;
}

int check_codes(const gemm_block_matrix& m, int64_t rows, int64_t zcols) {
    DG_TRY(check_op_n("codes", m));
    if (m.rows == rows && m.cols == zcols) return GEMM_OK;
    set_error("codes is %lld x %lld, not %lld x %lld", (long long)m.rows, (long long)m.cols, (long long)rows,
              (long long)zcols);
    return GEMM_ERR_INVALID_VALUE;
}

// Matrices of 128 MB and more, half the last level of cache, pass it (8192 x 8192 gated bf16, both
// ways: 254 to 233 us); smaller ones are found there (2001 x 5003 fp16: 35 us, past it 41).
bool past_caches(int64_t rows, int64_t cols, int64_t es) { return rows * cols >= ((int64_t)128 << 20) / es; }

dg::QuantOut codes_of(const gemm_block_matrix& m) {
    dg::QuantOut o;
    o.q = static_cast<uint8_t*>(m.data);
    o.s = m.scale;
    o.ld = m.ld;
    o.s_row = m.scale_row;
    o.s_blk = m.scale_block;
    o.type = m.dtype == GEMM_E4M3 ? 0 : 1;
    o.block_rows = m.block_rows;
    return o;
}

}  // namespace

extern "C" {

// ---------------------------------------------------------------- adapters
int64_t gemm_adapters_workspace(int64_t tokens, int64_t N, int64_t K, int64_t rank, int dtype) {
    if (!sizes_ok({tokens, N, K}) || !adapters_ok(0, rank) || !is_wide(dtype)) return 0;
    return adapter_space(nullptr, tokens, N, K, rank, dtype).bytes;
}

int gemm_adapters_product(const void* x, int64_t tokens, int64_t K, int64_t ldx, const void* w, int64_t N, int64_t ldw,
                          int dtype, const gemm_adapter_set* set, const int32_t* index, void* y, int64_t ldy, float* u,
                          void* workspace, int64_t workspace_bytes, void* stream) {
    dg::clear_error();
    DG_TRY(check_dtype("dtype", dtype));
    DG_TRY(check_size("tokens", tokens));
    DG_TRY(check_size("K", K));
    DG_TRY(check_size("N", N));
    DG_TRY(check_ld("ldx", ldx, K));
    DG_TRY(check_ld("ldw", ldw, K));
    DG_TRY(check_ld("ldy", ldy, N));
    DG_TRY(check_adapters(set, N, K));
    DG_TRY(check_product({{"tokens", tokens}, {"K", K}, {"N", N}},
                         {{"ldx", ldx}, {"ldw", ldw}, {"set.lda", set->lda}, {"set.ldb", set->ldb}}));
    if (tokens == 0) return GEMM_OK;
    const int64_t es = elem_size(dtype);
    const AdapterSpace sp = adapter_space(workspace, tokens, N, K, set->rank, dtype);
    if (K > 0) DG_TRY(check_pointer("x", x));
    if (K > 0 && N > 0) DG_TRY(check_pointer("w", w));
    if (N > 0) DG_TRY(check_pointer("y", y));
    if (set->rank > 0) DG_TRY(check_pointer("u", u));
    DG_TRY(check_pointer("index", index));
    DG_TRY(check_workspace(workspace, workspace_bytes, sp.bytes));
    DG_TRY(check_overlap({range("y", y, span(tokens, N, ldy, es)), range("u", u, (uint64_t)tokens * set->rank * 4),
                          range("workspace", workspace, (uint64_t)workspace_bytes)},
                         {range("x", x, span(tokens, K, ldx, es)), range("w", w, span(N, K, ldw, es)),
                          a_range(*set, K, es), b_range(*set, N, es), scale_of(*set),
                          range("index", index, (uint64_t)tokens * 4)}));
    dg::AdapterArgs a = adapter_args(*set, tokens, index);
    a.x = x;
    a.ldx = ldx;
    a.u = u;
    with_a(a, *set, K);
    const bool wide = dtype == GEMM_F32, few = few_tokens(tokens, K, dtype), tiles = in_tiles(tokens, N, K, set->rank, dtype);
    if (!few) DG_TRY(check_shrink_threads(tokens, set->rank, dtype, shrink_direct(a)));
    DG_TRY(check_expand_threads(tokens, N, dtype, tiles, few));
    DG_TRY(check_device());
    const hipStream_t s = (hipStream_t)stream;
    const int form = tiles_form(x, ldx, w, ldw, N, K, GEMM_OP_T, dtype);
    const dg::AdapterProduct p{x, w, ldx, ldw, (int)N, (int)K, GEMM_OP_T, form == 2};
    dg::AdapterArgs b = a;
    with_b(b, *set, N);
    b.scale = set->scale;
    b.out = y;
    b.ldo = ldy;
    // the stream of w, where there is enough of it; kernel_skinny.h's otherwise
    if (few && form == 2 && N >= 64)
        return launched(DG_BY_TYPE(launch_adapter_decode, dtype, p, a, b, (int)sp.slices.count, (int)sp.slices.k, sp.part, s),
                        "adapters' products");
    if (set->rank > 0) {
        a.us = b.us = sp.us;
        a.unit = b.unit = sp.unit;
        a.scale = wide ? nullptr : set->scale;
        DG_TRY(launched(wide  ? dg::launch_adapter_shrink(a, s)
                        : few ? DG_BY_TYPE(launch_adapter_shrink_row, dtype, a, s)
                              : shrink16(a, sp, dtype, s),
                        "adapters' first product"));
    }
    if (N == 0) return GEMM_OK;
    if (few) return launched(DG_BY_TYPE(launch_adapter_skinny, dtype, p, b, s), "adapters' products");
    if (tiles)
        return launched(DG_BY_TYPE(launch_adapter_tiles, dtype, p, b, tile_group(tokens, N), s), "adapters' products");
    b.slices = 1;
    if (form == 2) {
        DG_TRY(launched(DG_BY_TYPE(launch_mid_part, dtype, p, (int)tokens, tile_group(tokens, N, 128), (int)sp.mid.count,
                                   (int)sp.mid.k, sp.base, s), "adapters' shared product"));
        b.base = sp.base;
        b.ld_base = ceil_div(N, 4) * 4;
        b.slices = (int)sp.mid.count;
        return launched(DG_BY_TYPE(launch_adapter_expand16, dtype, b, s), "adapters' second product");
    }
    float* base = wide ? static_cast<float*>(y) : sp.base;
    const int64_t ldb = wide ? ldy : N;
    DG_TRY(product(GEMM_OP_T, tokens, N, K, x, ldx, w, ldw, base, ldb, dtype, GEMM_F32, 0.0f, sp.product,
                   kProductWorkspace, stream));
    b.base = base;
    b.ld_base = ldb;
    return launched(wide ? dg::launch_adapter_expand(b, s) : DG_BY_TYPE(launch_adapter_expand16, dtype, b, s),
                    "adapters' second product");
}

int64_t gemm_adapters_backward_workspace(int64_t tokens, int64_t N, int64_t K, int64_t adapters, int64_t rank,
                                         int dtype) {
    if (!sizes_ok({tokens, N, K}) || !adapters_ok(adapters, rank) || !is_wide(dtype)) return 0;
    return adapter_backward_space(nullptr, tokens, N, K, adapters, rank, dtype).bytes;
}

int gemm_adapters_backward(const void* grad, int64_t tokens, int64_t N, int64_t ldg, const void* x, int64_t K,
                           int64_t ldx, const float* u, const void* w, int64_t ldw, int dtype,
                           const gemm_adapter_set* set, const int32_t* index, const gemm_expert_plan* plan, void* x_grad,
                           int64_t ldxg, void* a_grad, void* b_grad, void* workspace, int64_t workspace_bytes,
                           void* stream) {
    dg::clear_error();
    DG_TRY(check_dtype("dtype", dtype));
    DG_TRY(check_size("tokens", tokens));
    DG_TRY(check_size("K", K));
    DG_TRY(check_size("N", N));
    DG_TRY(check_ld("ldg", ldg, N));
    DG_TRY(check_ld("ldx", ldx, K));
    DG_TRY(check_ld("ldw", ldw, K));
    if (x_grad) DG_TRY(check_ld("ldxg", ldxg, K));
    DG_TRY(check_adapters(set, N, K));
    DG_TRY(check_product({{"tokens", tokens}, {"K", K}, {"N", N}},
                         {{"ldg", ldg}, {"ldx", ldx}, {"ldw", ldw}, {"set.lda", set->lda}, {"set.ldb", set->ldb}}));
    const bool adapters = (a_grad || b_grad) && set->adapters > 0;
    if (adapters && ((a_grad == nullptr && K > 0) || (b_grad == nullptr && N > 0))) {
        set_error("a_grad and b_grad come together or are both NULL");
        return GEMM_ERR_NULL_POINTER;
    }
    const int64_t es = elem_size(dtype);
    if (adapters) {
        DG_TRY(check_plan(plan));
        if (plan->experts != set->adapters || plan->tokens != tokens || plan->top_k != 1) {
            set_error("plan of %lld experts, %lld tokens, top_k %lld, not of %lld adapters, %lld tokens, 1",
                      (long long)plan->experts, (long long)plan->tokens, (long long)plan->top_k,
                      (long long)set->adapters, (long long)tokens);
            return GEMM_ERR_INVALID_VALUE;
        }
        if (plan->capacity > tokens) {
            set_error("plan.capacity = %lld must be at most the %lld tokens (a plan with align 1)",
                      (long long)plan->capacity, (long long)tokens);
            return GEMM_ERR_INVALID_VALUE;
        }
        if (dtype != GEMM_F32 && ceil_div(tokens, 512) + set->adapters > 65535) {
            set_error("tokens = %lld with %lld adapters need more chunks than a launch holds", (long long)tokens,
                      (long long)set->adapters);
            return GEMM_ERR_UNSUPPORTED;
        }
        DG_TRY(check_pointer("plan.offsets", plan->offsets));
        DG_TRY(check_pointer("plan.counts", plan->counts));
        if (plan->capacity > 0) DG_TRY(check_pointer("plan.rows", plan->rows));
    }
    if (tokens == 0 && !adapters) return GEMM_OK;
    const AdapterSpace sp = adapter_backward_space(workspace, tokens, N, K, set->adapters, set->rank, dtype);
    if (tokens > 0) {
        if (N > 0) DG_TRY(check_pointer("grad", grad));
        if (K > 0) DG_TRY(check_pointer("x", x));
        if (x_grad && N > 0 && K > 0) DG_TRY(check_pointer("w", w));
        if (set->rank > 0) DG_TRY(check_pointer("u", u));
        DG_TRY(check_pointer("index", index));
    }
    DG_TRY(check_workspace(workspace, workspace_bytes, sp.bytes));
    const Range none = range("", nullptr, 0);
    const uint64_t each = (uint64_t)set->adapters * set->rank * es;
    DG_TRY(check_overlap(
        {range("x_grad", x_grad, span(tokens, K, ldxg, es)), range("a_grad", a_grad, each * K),
         range("b_grad", b_grad, each * N), range("workspace", workspace, (uint64_t)workspace_bytes)},
        {range("grad", grad, span(tokens, N, ldg, es)), range("x", x, span(tokens, K, ldx, es)),
         range("u", u, (uint64_t)tokens * set->rank * 4), range("w", w, span(N, K, ldw, es)), a_range(*set, K, es),
         b_range(*set, N, es), scale_of(*set), range("index", index, (uint64_t)tokens * 4),
         adapters ? range("plan.offsets", plan->offsets, (uint64_t)(plan->experts + 1) * 4) : none,
         adapters ? range("plan.counts", plan->counts, (uint64_t)plan->experts * 4) : none,
         adapters ? range("plan.rows", plan->rows, (uint64_t)plan->capacity * 4) : none}));
    const bool wide = dtype == GEMM_F32, any = set->adapters > 0 && set->rank > 0;
    const bool tiles = in_tiles(tokens, K, N, set->rank, dtype);
    // v = scale grad b
    dg::AdapterArgs a = adapter_args(*set, tokens, index);
    a.x = grad;
    a.ldx = ldg;
    a.u = sp.v;
    a.us = sp.us;
    a.unit = sp.unit;
    a.fold = 1;
    a.scale = set->scale;
    with_b(a, *set, N);
    if (!wide) {
        a.m = sp.b_turned;
        a.ldm = N;
        a.stride_m = set->rank * N;
        a.turned = 0;
    }
    DG_TRY(check_shrink_threads(tokens, set->rank, dtype, shrink_direct(a)));
    if (x_grad) DG_TRY(check_expand_threads(tokens, K, dtype, tiles, false));
    if (any) DG_TRY(check_threads("blocks of N + K", ceil_div(N, 64) + ceil_div(K, 64), 2, 256));  // layout, gradients
    DG_TRY(check_device());
    const hipStream_t s = (hipStream_t)stream;
    if (!wide && any && (N > 0 || K > 0)) {
        // the adapters' other layout: a as K x rank_m for x_grad, b as rank x N for v
        auto turn = [](const void* in, int64_t ld, int64_t stride, int64_t rows, int64_t cols, void* out, int64_t out_ld) {
            return dg::TurnArgs{in,          ld, stride, (int)rows, (int)cols, out, (int)out_ld, (int)ceil_div(out_ld, 64),
                                (int)ceil_div(cols, 64)};
        };
        const dg::TurnArgs p = turn(set->a, set->lda, set->stride_a, set->rank, x_grad ? K : 0, sp.a_turned, sp.rank_m);
        const dg::TurnArgs q = turn(set->b, set->ldb, set->stride_b, N, set->rank, sp.b_turned, N);
        // and u, for b's gradient, as hi and lo only
        dg::AdapterArgs of_u = adapter_args(*set, tokens, index);
        of_u.us = sp.us_b;
        of_u.unit = sp.unit_b;
        of_u.scale = set->scale;
        if (!adapters) of_u.tokens = 0;
        if (p.tiles_r * p.tiles_c + q.tiles_r * q.tiles_c > 0)
            DG_TRY(launched(DG_BY_TYPE(launch_adapter_prepare, dtype, p, q, (int)set->adapters, of_u, u, s), "adapters' layout"));
    }
    if (tokens > 0 && set->rank > 0)
        DG_TRY(launched(wide ? dg::launch_adapter_shrink(a, s) : shrink16(a, sp, dtype, s), "adapters' v"));
    if (x_grad && tokens > 0 && K > 0) {
        with_a(a, *set, K);
        if (!wide) {
            a.m = sp.a_turned;
            a.ldm = sp.rank_m;
            a.stride_m = K * sp.rank_m;
            a.rank_m = (int)sp.rank_m;
            a.turned = 1;
        }
        a.scale = nullptr;
        a.out = x_grad;
        a.ldo = ldxg;
        if (tiles) {
            dg::AdapterProduct p{grad, w, ldg, ldw, (int)K, (int)N, GEMM_OP_N,
                                 tiles_form(grad, ldg, w, ldw, K, N, GEMM_OP_N, dtype) == 2};
            DG_TRY(launched(DG_BY_TYPE(launch_adapter_tiles, dtype, p, a, tile_group(tokens, K), s), "adapters' x_grad"));
        } else {
            float* base = wide ? static_cast<float*>(x_grad) : sp.base;
            const int64_t ldb = wide ? ldxg : K;
            DG_TRY(product(GEMM_OP_N, tokens, K, N, grad, ldg, w, ldw, base, ldb, dtype, GEMM_F32, 0.0f, sp.product,
                           kProductWorkspace, stream));
            a.base = base;
            a.ld_base = ldb;
            a.slices = 1;
            DG_TRY(launched(wide ? dg::launch_adapter_expand(a, s) : DG_BY_TYPE(launch_adapter_expand16, dtype, a, s),
                            "adapters' x_grad"));
        }
    }
    if (!adapters) return GEMM_OK;
    a.offsets = plan->offsets;
    a.counts = plan->counts;
    a.rows = plan->rows;
    a.capacity = (int)plan->capacity;
    a.chunk = (int)sp.chunk;
    a.work = sp.sums;
    dg::AdapterArgs b = a;
    a.x = x;
    a.ldx = ldx;
    a.scale = nullptr;  // it is in v
    with_a(a, *set, K);
    a.out = a_grad;
    b.x = grad;
    b.ldx = ldg;
    b.u = const_cast<float*>(u);
    b.us = sp.us_b;
    b.unit = sp.unit_b;
    b.scale = wide ? set->scale : nullptr;  // us_b holds scale u
    with_b(b, *set, N);
    b.out = b_grad;
    b.work = sp.sums + sp.slots * set->rank * K;
    if (N == 0 && K == 0) return GEMM_OK;
    return launched(wide ? dg::launch_adapter_gradient(a, b, s)
                         : DG_BY_TYPE(launch_adapter_gradient16, dtype, a, b, (int)sp.slots, s),
                    "adapters' gradients");
}

// ---------------------------------------------------------------- loss
int64_t gemm_loss_workspace(int64_t tokens, int64_t vocabulary, int64_t K, int dtype) {
    if (!sizes_ok({tokens, vocabulary, K}) || !is_wide(dtype)) return 0;
    return loss_space(nullptr, tokens, vocabulary, K, dtype).bytes;
}

int gemm_loss(const void* x, int64_t tokens, int64_t K, int64_t ldx, const void* w, int64_t vocabulary, int64_t ldw,
              int dtype, const int64_t* target, float* loss, float* lse, void* workspace, int64_t workspace_bytes,
              void* stream) {
    dg::clear_error();
    DG_TRY(check_dtype("dtype", dtype));
    DG_TRY(check_size("tokens", tokens));
    DG_TRY(check_size("K", K));
    DG_TRY(check_size("vocabulary", vocabulary));
    DG_TRY(check_ld("ldx", ldx, K));
    DG_TRY(check_ld("ldw", ldw, K));
    DG_TRY(check_product({{"tokens", tokens}, {"K", K}, {"vocabulary", vocabulary}}, {{"ldx", ldx}, {"ldw", ldw}}));
    if (tokens == 0) return GEMM_OK;
    const int64_t es = elem_size(dtype);
    const LossSpace sp = loss_space(workspace, tokens, vocabulary, K, dtype);
    if (K > 0) DG_TRY(check_pointer("x", x));
    if (K > 0 && vocabulary > 0) DG_TRY(check_pointer("w", w));
    DG_TRY(check_pointer("target", target));
    DG_TRY(check_pointer("loss", loss));
    DG_TRY(check_pointer("lse", lse));
    DG_TRY(check_workspace(workspace, workspace_bytes, sp.bytes));
    const uint64_t n4 = (uint64_t)tokens * 4;
    DG_TRY(check_overlap({range("loss", loss, n4), range("lse", lse, n4),
                          range("workspace", workspace, (uint64_t)workspace_bytes)},
                         {range("x", x, span(tokens, K, ldx, es)), range("w", w, span(vocabulary, K, ldw, es)),
                          range("target", target, n4 * 2)}));
    DG_TRY(check_threads("tokens", tokens, 1, sp.part ? 16 : 256));
    DG_TRY(check_threads("tiles of tokens * vocabulary", ceil_div(tokens, 256),
                         ceil_div(vocabulary, tokens <= kSkinny ? 16 : 256), 512));
    DG_TRY(check_device());
    if (sp.part) {
        const hipStream_t s = (hipStream_t)stream;
        int64_t strips = loss_strips(tokens, vocabulary);
        if (tokens <= kSkinny) {
            const dg::LossProduct p = loss_product(x, ldx, w, ldw, tokens, vocabulary, K, dtype, 256);
            DG_TRY(launched(DG_BY_TYPE(launch_loss_skinny, dtype, p, target, sp.part, sp.picked, s), "loss"));
        } else {
            const LossTiles t = loss_tiles(tokens, vocabulary, whole_pieces(x, ldx, K) && whole_pieces(w, ldw, K));
            strips = t.strips;
            if (t.wide > 0) {
                const dg::LossProduct p = loss_product(x, ldx, w, ldw, tokens, t.wide, K, dtype, 256);
                DG_TRY(launched(DG_BY_TYPE(launch_loss_tiles, dtype, p, 0, target, sp.part, sp.picked, s), "loss"));
            }
            if (t.wide < vocabulary) {
                const dg::LossProduct p = loss_product(x, ldx, static_cast<const char*>(w) + (size_t)t.wide * ldw * es, ldw,
                                                       tokens, vocabulary - t.wide, K, dtype, 128);
                void* part = static_cast<char*>(sp.part) + t.wide / 256 * tokens * dg::kLossPartBytes;
                DG_TRY(launched(DG_BY_TYPE(launch_loss_tiles, dtype, p, (int)t.wide, target, part, sp.picked, s), "loss"));
            }
        }
        return launched(dg::launch_loss_finish(sp.part, (int)strips, (int)tokens, target, (int)vocabulary, sp.picked,
                                               loss, lse, s), "loss");
    }
    dg::LossArgs a;
    memset(&a, 0, sizeof a);
    a.logits = sp.logits;
    a.tokens = (int)tokens;
    a.vocabulary = (int)vocabulary;
    a.target = target;
    a.top = sp.top;
    a.sum = sp.sum;
    a.picked = sp.picked;
    a.loss = loss;
    a.lse = lse;
    int64_t v0 = 0;
    do {
        a.n = (int)std::min(sp.piece, vocabulary - v0);
        a.ld = std::max(1, a.n);
        a.v0 = (int)v0;
        a.first = v0 == 0;
        a.last = v0 + a.n >= vocabulary;
        DG_TRY(product(GEMM_OP_T, tokens, a.n, K, x, ldx, static_cast<const char*>(w) + (size_t)v0 * ldw * es, ldw,
                       sp.logits, a.ld, dtype, GEMM_F32, 0.0f, sp.product, kProductWorkspace, stream));
        DG_TRY(launched(dg::launch_loss_stats(a, (hipStream_t)stream), "loss"));
        v0 += a.n;
    } while (v0 < vocabulary);
    return GEMM_OK;
}

int64_t gemm_loss_backward_workspace(int64_t tokens, int64_t vocabulary, int64_t K, int dtype, int want_x_grad,
                                     int want_w_grad, int64_t piece) {
    if (!sizes_ok({tokens, vocabulary, K}) || piece < 0 || piece > kMaxDim || !is_wide(dtype)) return 0;
    return loss_backward_space(nullptr, tokens, vocabulary, K, dtype, want_x_grad != 0, want_w_grad != 0, piece).bytes;
}

int gemm_loss_backward(const float* grad, const void* x, int64_t tokens, int64_t K, int64_t ldx, const void* w,
                       int64_t vocabulary, int64_t ldw, int dtype, const int64_t* target, const float* lse, void* x_grad,
                       int64_t ldxg, void* w_grad, int64_t ldwg, int64_t piece, void* workspace,
                       int64_t workspace_bytes, void* stream) {
    dg::clear_error();
    DG_TRY(check_dtype("dtype", dtype));
    DG_TRY(check_size("tokens", tokens));
    DG_TRY(check_size("K", K));
    DG_TRY(check_size("vocabulary", vocabulary));
    DG_TRY(check_size("piece", piece));
    DG_TRY(check_ld("ldx", ldx, K));
    DG_TRY(check_ld("ldw", ldw, K));
    if (x_grad) DG_TRY(check_ld("ldxg", ldxg, K));
    if (w_grad) DG_TRY(check_ld("ldwg", ldwg, K));
    DG_TRY(check_product({{"tokens", tokens}, {"K", K}, {"vocabulary", vocabulary}},
                         {{"ldx", ldx}, {"ldw", ldw}, {"tokens of w_grad", w_grad ? tokens + 31 : 0}}));
    if (K == 0 || (x_grad == nullptr && w_grad == nullptr)) return GEMM_OK;
    if ((tokens == 0 || x_grad == nullptr) && (vocabulary == 0 || w_grad == nullptr)) return GEMM_OK;
    const int64_t es = elem_size(dtype);
    const LossSpace sp =
        loss_backward_space(workspace, tokens, vocabulary, K, dtype, x_grad != nullptr, w_grad != nullptr, piece);
    if (tokens > 0) {
        DG_TRY(check_pointer("grad", grad));
        DG_TRY(check_pointer("x", x));
        DG_TRY(check_pointer("target", target));
        DG_TRY(check_pointer("lse", lse));
    }
    if (vocabulary > 0) DG_TRY(check_pointer("w", w));
    DG_TRY(check_workspace(workspace, workspace_bytes, sp.bytes));
    const uint64_t n4 = (uint64_t)tokens * 4;
    DG_TRY(check_overlap({range("x_grad", x_grad, span(tokens, K, ldxg, es)),
                          range("w_grad", w_grad, span(vocabulary, K, ldwg, es)),
                          range("workspace", workspace, (uint64_t)workspace_bytes)},
                         {range("grad", grad, n4), range("x", x, span(tokens, K, ldx, es)),
                          range("w", w, span(vocabulary, K, ldw, es)), range("target", target, n4 * 2),
                          range("lse", lse, n4)}));
    DG_TRY(check_threads("blocks of tokens * piece", ceil_div(tokens, 64), ceil_div(sp.piece, 64), 256));
    if (sp.xp) DG_TRY(check_threads("blocks of tokens * K", ceil_div(sp.lddt, 64), ceil_div(K, 64), 256));
    DG_TRY(check_device());
    const hipStream_t s = (hipStream_t)stream;
    // fp16 holds d times a power of two that brings the largest |grad| near 2^14
    const bool wide = dtype == GEMM_F32, scaled = dtype == GEMM_F16;
    dg::LossArgs a;
    memset(&a, 0, sizeof a);
    a.logits = sp.logits;
    a.tokens = (int)tokens;
    a.vocabulary = (int)vocabulary;
    a.target = target;
    a.lse_in = lse;
    a.grad = grad;
    a.factor = scaled ? sp.factor : nullptr;
    a.d = sp.d;
    a.apart = sp.apart;
    a.rest = sp.rest;
    a.dt = sp.dt;
    a.lddt = sp.lddt;
    if (scaled) DG_TRY(launched(dg::launch_loss_factor(grad, (int)tokens, sp.factor, s), "loss gradient's factor"));
    const void* xw = x;  // x for w_grad's product
    int64_t ldxw = ldx;
    const bool narrow = loss_w_narrow(std::min(sp.piece, vocabulary), K);
    if (sp.xp && tokens > 0 && narrow) {
        DG_TRY(launched(dg::launch_loss_turn(x, ldx, (int)tokens, (int)K, sp.xp, sp.lddt, s), "loss gradient's copy of x"));
        xw = sp.xp;
        ldxw = sp.lddt;
    } else if (sp.xp && tokens > 0 && (tokens % 32 != 0 || !whole_pieces(x, ldx, K))) {
        const dg::PackJob job{x, sp.xp, ldx, (int)tokens, (int)K, (int)sp.lddt, (int)sp.ldxp}, none_left{x, sp.xp, ldx, 0, 0, 0, 8};
        DG_TRY(launched(dg::launch_pack((int)es, job, none_left, s), "loss gradient's copy of x"));
        xw = sp.xp;
        ldxw = sp.ldxp;
    }
    float* xa = wide ? static_cast<float*>(x_grad) : sp.x_acc;
    const int64_t ldxa = wide ? ldxg : K;
    int64_t v0 = 0;
    do {
        const int64_t n = std::min(sp.piece, vocabulary - v0);
        a.n = (int)n;
        a.ld = std::max<int64_t>(1, n);
        a.ldd = wide ? a.ld : sp.ldd;
        a.v0 = (int)v0;
        const char* wp = static_cast<const char*>(w) + (size_t)v0 * ldw * es;
        if (tokens > 0 && n > 0) {
            if (sp.logits) {
                DG_TRY(product(GEMM_OP_T, tokens, n, K, x, ldx, wp, ldw, sp.logits, a.ld, dtype, GEMM_F32, 0.0f,
                               sp.product, sp.product_bytes, stream));
                DG_TRY(launched(dg::launch_loss_grad(a, dtype, s), "loss gradient"));
            } else {
                // few rows all at once; else wide tiles and then narrow ones
                const bool few = loss_few(tokens, n);
                const LossTiles t = few ? LossTiles{n, 0} : loss_tiles(tokens, n, whole_pieces(x, ldx, K) && whole_pieces(wp, ldw, K));
                for (int64_t c = 0; c < n; c = t.wide > c ? t.wide : n) {
                    const bool is_wide = t.wide > c;
                    dg::LossArgs b = a;
                    b.n = (int)((is_wide ? t.wide : n) - c);
                    b.v0 = (int)(v0 + c);
                    if (b.d) b.d = static_cast<char*>(b.d) + c * es;
                    if (b.dt) b.dt = static_cast<char*>(b.dt) + c * b.lddt * es;
                    const dg::LossProduct p = loss_product(x, ldx, wp + (size_t)c * ldw * es, ldw, tokens, b.n, K, dtype,
                                                           few ? 16 : is_wide ? 256 : 128);
                    DG_TRY(launched(DG_BY_TYPE(launch_loss_grad_tiles, dtype, p, b, s), "loss gradient"));
                }
            }
        }
        if (x_grad) {
            // of a 16-bit piece, whole stages first: rows of w beyond the last piece are not read
            const int64_t main = !wide && n >= 32 ? n / 32 * 32 : n;
            DG_TRY(product(GEMM_OP_N, tokens, K, main, sp.d, a.ldd, wp, ldw, xa, ldxa, dtype, GEMM_F32,
                           v0 == 0 ? 0.0f : 1.0f, sp.product, sp.product_bytes, stream));
            if (n > main)
                DG_TRY(product(GEMM_OP_N, tokens, K, n - main, static_cast<const char*>(sp.d) + main * es, a.ldd,
                               wp + (size_t)main * ldw * es, ldw, xa, ldxa, dtype, GEMM_F32, 1.0f, sp.product,
                               sp.product_bytes, stream));
        }
        if (w_grad && n > 0) {
            char* wg = static_cast<char*>(w_grad) + (size_t)v0 * ldwg * es;
            if (sp.xp && tokens > 0) {
                DG_TRY(launched(DG_BY_TYPE(launch_loss_w, dtype, a, x, ldx, xw, ldxw, narrow, (int)K,
                                           tile_group(n, K, narrow ? 128 : 256), wg, ldwg, s), "loss gradient of w"));
            } else {
                DG_TRY(product(GEMM_OP_N, n, K, tokens, sp.dt, sp.lddt, x, ldx, sp.w_acc ? (void*)sp.w_acc : wg,
                               sp.w_acc ? K : ldwg, dtype, sp.w_acc ? GEMM_F32 : dtype, 0.0f, sp.product,
                               sp.product_bytes, stream));
                if (sp.w_acc)
                    DG_TRY(launched(dg::launch_scaled_cast(sp.w_acc, K, (int)n, (int)K, sp.factor, wg, ldwg, nullptr, 0,
                                                           nullptr, 0, nullptr, nullptr, dtype, s), "loss gradient's rounding"));
            }
        }
        v0 += n;
    } while (v0 < vocabulary);
    if (x_grad && !wide && tokens > 0)
        DG_TRY(launched(dg::launch_scaled_cast(sp.x_acc, K, (int)tokens, (int)K, a.factor, x_grad, ldxg,
                                               sp.logits ? nullptr : w, ldw, target, (int)vocabulary, grad, sp.apart,
                                               dtype, s),
                        "loss gradient's rounding"));
    return GEMM_OK;
}

// ---------------------------------------------------------------- activations
int gemm_activation_forward(const void* z, int64_t rows, int64_t cols, int64_t ldz, int dtype, int activation,
                            int gated, void* y, int64_t ldy, const gemm_block_matrix* codes, void* stream) {
    dg::clear_error();
    DG_TRY(check_dtype("dtype", dtype));
    DG_TRY(check_size("rows", rows));
    DG_TRY(check_size("cols", cols));
    DG_TRY(check_activation(activation, cols, gated));
    const int64_t zcols = gated ? 2 * cols : cols, es = elem_size(dtype);
    DG_TRY(check_ld("ldz", ldz, zcols));
    DG_TRY(check_ld("ldy", ldy, cols));
    if (codes) {
        DG_TRY(check_block("codes", codes));
        DG_TRY(check_codes(*codes, rows, zcols));
        if (codes->block_rows != 1) {
            set_error("codes.block_rows = %d must be 1", codes->block_rows);
            return GEMM_ERR_INVALID_VALUE;
        }
    }
    if (rows == 0 || cols == 0) return GEMM_OK;
    DG_TRY(check_pointer("z", z));
    DG_TRY(check_pointer("y", y));
    const Range none = range("", nullptr, 0);
    DG_TRY(check_overlap({range("y", y, span(rows, cols, ldy, es)), codes ? data_range("codes.data", *codes) : none,
                          codes ? scale_range("codes.scale", *codes) : none},
                         {range("z", z, span(rows, zcols, ldz, es))}));
    DG_TRY(check_device());
    dg::ActArgs a;
    memset(&a, 0, sizeof a);
    a.z = z;
    a.ldz = ldz;
    if (codes) a.codes = codes_of(*codes);
    a.rows = (int)rows;
    a.cols = (int)cols;
    a.act = activation;
    a.gated = gated != 0;
    a.y = y;
    a.ldy = ldy;
    a.passing = past_caches(rows, cols, es);
    return launched(dg::launch_activation(a, dtype, (hipStream_t)stream), "activation");
}

int gemm_activation_backward(const gemm_block_matrix* codes, const void* grad, int64_t rows, int64_t cols, int64_t ldg,
                             int dtype, int activation, int gated, void* z_grad, int64_t ldzg, void* y, int64_t ldy,
                             void* stream) {
    dg::clear_error();
    DG_TRY(check_dtype("dtype", dtype));
    DG_TRY(check_size("rows", rows));
    DG_TRY(check_size("cols", cols));
    DG_TRY(check_activation(activation, cols, gated));
    const int64_t zcols = gated ? 2 * cols : cols, es = elem_size(dtype);
    if (grad || z_grad) {
        DG_TRY(check_ld("ldg", ldg, cols));
        DG_TRY(check_ld("ldzg", ldzg, zcols));
    }
    if (y) DG_TRY(check_ld("ldy", ldy, cols));
    DG_TRY(check_block("codes", codes));
    DG_TRY(check_codes(*codes, rows, zcols));
    if (rows == 0 || cols == 0) return GEMM_OK;
    if (grad || z_grad || y == nullptr) {
        DG_TRY(check_pointer("grad", grad));
        DG_TRY(check_pointer("z_grad", z_grad));
    }
    DG_TRY(check_overlap({range("z_grad", z_grad, span(rows, zcols, ldzg, es)),
                          range("y", y, span(rows, cols, ldy, es))},
                         {range("grad", grad, span(rows, cols, ldg, es)), data_range("codes.data", *codes),
                          scale_range("codes.scale", *codes)}));
    DG_TRY(check_device());
    dg::ActArgs a;
    memset(&a, 0, sizeof a);
    a.codes = codes_of(*codes);
    a.rows = (int)rows;
    a.cols = (int)cols;
    a.act = activation;
    a.gated = gated != 0;
    a.y = y;
    a.ldy = ldy;
    a.grad = grad;
    a.ldg = ldg;
    a.z_grad = z_grad;
    a.ldzg = ldzg;
    a.passing = past_caches(rows, grad ? zcols : cols, es);
    return launched(dg::launch_activation_backward(a, dtype, (hipStream_t)stream), "activation's backward pass");
}

}  // extern "C"
