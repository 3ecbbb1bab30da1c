// checks.h -- the checks that the C entry points of gemm_experts.h and gemm_layers.h share:
// each returns a gemm_status and leaves the reason for gemm_last_error.
#pragma once
#include <hip/hip_runtime.h>
#include <stdio.h>
#include <string.h>

#include <algorithm>
#include <atomic>
#include <initializer_list>

#include "experts.h"
#include "plan.h"

namespace {

using dg::ceil_div;
using dg::set_error;

constexpr int64_t kMaxDim = ((int64_t)1 << 31) - 1;
constexpr int64_t kMaxThreads = ((int64_t)1 << 32) - 1;  // of one launch

int64_t elem_size(int dtype) { return dtype == GEMM_F32 ? 4 : dtype == GEMM_F16 || dtype == GEMM_BF16 ? 2 : 1; }
bool is_wide(int dtype) { return dtype == GEMM_F32 || dtype == GEMM_F16 || dtype == GEMM_BF16; }

int check_dtype(const char* what, int dtype) {
    if (is_wide(dtype)) return GEMM_OK;
    set_error("%s = %d is not GEMM_F32, GEMM_F16 or GEMM_BF16", what, dtype);
    return GEMM_ERR_INVALID_VALUE;
}

int check_size(const char* what, int64_t n) {
    if (n < 0) {
        set_error("%s = %lld must be non-negative", what, (long long)n);
        return GEMM_ERR_INVALID_VALUE;
    }
    if (n > kMaxDim) {
        set_error("%s = %lld must be below 2^31", what, (long long)n);
        return GEMM_ERR_UNSUPPORTED;
    }
    return GEMM_OK;
}

int check_ld(const char* what, int64_t ld, int64_t cols) {
    if (ld >= std::max<int64_t>(1, cols) && ld < ((int64_t)1 << 40)) return GEMM_OK;
    set_error("%s = %lld must be at least %lld and below 2^40", what, (long long)ld,
              (long long)std::max<int64_t>(1, cols));
    return GEMM_ERR_INVALID_VALUE;
}

int check_pointer(const char* what, const void* p) {
    if (p != nullptr) return GEMM_OK;
    set_error("%s is NULL", what);
    return GEMM_ERR_NULL_POINTER;
}

#define DG_TRY(x)                      \
    do {                               \
        const int st_ = (x);           \
        if (st_ != GEMM_OK) return st_; \
    } while (0)

struct Range {
    const char* name;
    uintptr_t at;
    uint64_t len;
};

// Bytes that `batch` matrices of rows x cols span, saturating.
uint64_t span(int64_t rows, int64_t cols, int64_t ld, int64_t es, int64_t batch = 1, int64_t stride = 0) {
    if (rows <= 0 || cols <= 0 || batch <= 0) return 0;
    const unsigned __int128 n = (unsigned __int128)(batch - 1) * (uint64_t)stride +
                                (unsigned __int128)(rows - 1) * (uint64_t)ld + (uint64_t)cols;
    const unsigned __int128 b = n * (uint64_t)es;
    return b >> 62 ? (uint64_t)1 << 62 : (uint64_t)b;
}

Range range(const char* name, const void* p, uint64_t len) { return {name, (uintptr_t)p, p ? len : 0}; }

// No output may overlap an input or another output.
int check_overlap(std::initializer_list<Range> outs, std::initializer_list<Range> ins) {
    for (const Range* o = outs.begin(); o != outs.end(); ++o) {
        auto meets = [&](const Range& r) { return o->len && r.len && o->at < r.at + r.len && r.at < o->at + o->len; };
        for (const Range& r : ins)
            if (meets(r)) {
                set_error("%s overlaps %s", o->name, r.name);
                return GEMM_ERR_INVALID_VALUE;
            }
        for (const Range* q = o + 1; q != outs.end(); ++q)
            if (meets(*q)) {
                set_error("%s overlaps %s", o->name, q->name);
                return GEMM_ERR_INVALID_VALUE;
            }
    }
    return GEMM_OK;
}

int check_block(const char* name, const gemm_block_matrix* m, int64_t batch = 1) {
    char what[64];
    auto field = [&](const char* f) {
        snprintf(what, sizeof what, "%s.%s", name, f);
        return what;
    };
    DG_TRY(check_pointer(name, m));
    DG_TRY(check_size(field("rows"), m->rows));
    DG_TRY(check_size(field("cols"), m->cols));
    if (m->op != GEMM_OP_N && m->op != GEMM_OP_T) {
        set_error("%s.op = %d is not GEMM_OP_N or GEMM_OP_T", name, m->op);
        return GEMM_ERR_INVALID_VALUE;
    }
    DG_TRY(check_ld(field("ld"), m->ld, m->op == GEMM_OP_T ? m->rows : m->cols));
    if (m->dtype != GEMM_E4M3 && m->dtype != GEMM_E5M2) {
        set_error("%s.dtype = %d is not GEMM_E4M3 or GEMM_E5M2", name, m->dtype);
        return GEMM_ERR_INVALID_VALUE;
    }
    if (m->block_rows != 1 && m->block_rows != dg::kBlock) {
        set_error("%s.block_rows = %d must be 1 or 128", name, m->block_rows);
        return GEMM_ERR_INVALID_VALUE;
    }
    if (m->scale_row < 0 || m->scale_block < 0 || m->stride < 0 || m->scale_stride < 0 ||
        m->scale_row >= ((int64_t)1 << 40) || m->scale_block >= ((int64_t)1 << 40)) {
        set_error("%s: strides must be non-negative (scale strides below 2^40)", name);
        return GEMM_ERR_INVALID_VALUE;
    }
    if (m->rows > 0 && m->cols > 0 && batch > 0) {
        DG_TRY(check_pointer(field("data"), m->data));
        DG_TRY(check_pointer(field("scale"), m->scale));
    }
    return GEMM_OK;
}

int check_op_n(const char* name, const gemm_block_matrix& m) {
    if (m.op == GEMM_OP_N) return GEMM_OK;
    set_error("%s.op = GEMM_OP_T: its rows have to be contiguous here", name);
    return GEMM_ERR_UNSUPPORTED;
}

Range data_range(const char* name, const gemm_block_matrix& m, int64_t batch = 1) {
    return range(name, m.data, m.op == GEMM_OP_T ? span(m.cols, m.rows, m.ld, 1, batch, m.stride)
                                                 : span(m.rows, m.cols, m.ld, 1, batch, m.stride));
}

Range scale_range(const char* name, const gemm_block_matrix& m, int64_t batch = 1) {
    const int64_t r = ceil_div(m.rows, m.block_rows), b = ceil_div(m.cols, dg::kBlock);
    if (r <= 0 || b <= 0 || batch <= 0) return range(name, m.scale, 0);
    // the span of a strided array: its last element
    return range(name, m.scale, span(1, (r - 1) * m.scale_row + 1, 0, 4) + span(1, (b - 1) * m.scale_block, 0, 4) +
                                    span(1, (batch - 1) * std::min<int64_t>(m.scale_stride, (int64_t)1 << 30), 0, 4));
}

// The current device, which has to be a gfx950 (asked once for each of the first 64).
std::atomic<uint64_t> g_checked{0};

int check_device() {
    int dev = 0, cus = 0;
    char arch[64];
    const hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) {
        set_error("hipGetDevice failed: %s", hipGetErrorString(e));
        return GEMM_ERR_DEVICE;
    }
    const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
    if (g_checked.load(std::memory_order_relaxed) & bit) return GEMM_OK;
    DG_TRY(gemm_device_info(dev, &cus, arch, (int)sizeof arch));
    if (strncmp(arch, "gfx950", 6) != 0) {
        set_error("device architecture '%s' is not gfx950; the kernels are built for gfx950 only", arch);
        return GEMM_ERR_DEVICE;
    }
    g_checked.fetch_or(bit, std::memory_order_relaxed);
    return GEMM_OK;
}

int launched(int rc, const char* what) {
    if (rc == 0) return GEMM_OK;
    set_error("%s: launch failed: %s", what, hipGetErrorString((hipError_t)rc));
    return GEMM_ERR_LAUNCH;
}

int check_plan(const gemm_expert_plan* p) {
    DG_TRY(check_pointer("plan", p));
    DG_TRY(check_size("plan.experts", p->experts));
    DG_TRY(check_size("plan.tokens", p->tokens));
    DG_TRY(check_size("plan.top_k", p->top_k));
    DG_TRY(check_size("plan.capacity", p->capacity));
    if (p->tokens > 0 && p->top_k > kMaxDim / p->tokens) {
        set_error("plan: tokens * top_k = %lld * %lld must be below 2^31", (long long)p->tokens, (long long)p->top_k);
        return GEMM_ERR_UNSUPPORTED;
    }
    return GEMM_OK;
}

}  // namespace
