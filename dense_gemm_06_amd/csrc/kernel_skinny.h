// kernel_skinny.h -- x w^T of up to 64 rows x, fp16 or bf16, for any alignment and for the fewest
// rows of w: fragments straight from memory, the sum in one launch (kernel_stream.h has the others).
//
// A workgroup has 16 rows of w; its eight waves cut k in pieces of 64, so that what the
// workgroup reads (128 KB at k = 4096) is in flight almost at once, and their sums are joined in
// LDS in the waves' order. What becomes of a finished 16 x 16 piece is up to EPI: lane l of a wave
// has row x t = 16 tt + l % 16 and rows w n .. n + 3, n = n0 + 4 (l / 16).
#pragma once
#include "device_common.h"
#include "kernel_adapters.h"

namespace dg {

struct SkinnyArgs {
    const void* x;
    const void* w;
    int64_t ldx, ldw;
    int T, N, K;
};

template <int DT, int TT, class EPI>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 4))) void skinny_product(SkinnyArgs a,
                                                                                                EPI epi) {
    __shared__ __attribute__((aligned(16))) float part[8][TT][64][4];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int l16 = lane & 15, lg = lane >> 4;
    const int n0 = (int)blockIdx.x * 16;
    const uint16_t* w = static_cast<const uint16_t*>(a.w) + (size_t)min(n0 + l16, a.N - 1) * (size_t)a.ldw + 8 * lg;
    const uint16_t* x[TT];
    f32x4 acc[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) {
        x[t] = static_cast<const uint16_t*>(a.x) + (size_t)min(16 * t + l16, a.T - 1) * (size_t)a.ldx + 8 * lg;
        acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    // pieces of 64 of k: wave, wave + 8, ..
    const int whole = a.K & ~63, all = whole >> 6;
    const int mine = wave < all ? (all - wave + 7) >> 3 : 0;
    auto k_of = [&](int p) { return 64 * (wave + 8 * p); };
    // U pieces at a time, all of their loads before the first product
    int at = 0;
    auto pieces_of = [&](auto u_tag) {
        constexpr int U = decltype(u_tag)::value;
        u32x4 wv[U][2], xv[U][2][TT];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int s = 0; s < 2; ++s) __builtin_memcpy(&wv[u][s], w + k_of(at + u) + 32 * s, 16);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int t = 0; t < TT; ++t) __builtin_memcpy(&xv[u][s][t], x[t] + k_of(at + u) + 32 * s, 16);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int t = 0; t < TT; ++t) acc[t] = mfma_16<DT>(wv[u][s], xv[u][s][t], acc[t]);
        at += U;
    };
    constexpr int U = TT == 1 ? 8 : TT == 2 ? 4 : 3;
    while (at + U <= mine) pieces_of(std::integral_constant<int, U>{});
    while (at < mine) pieces_of(std::integral_constant<int, 1>{});
    const int k = whole;
    if (whole < a.K && wave == (all & 7))
        for (int s = 0; s < 2; ++s) {
            const int valid = max(0, min(8, (int)(a.K - (k + 32 * s + 8 * lg))));
            const u32x4 wv = load_frag8(w + k + 32 * s, valid);
#pragma unroll
            for (int t = 0; t < TT; ++t) acc[t] = mfma_16<DT>(wv, load_frag8(x[t] + k + 32 * s, valid), acc[t]);
        }
#pragma unroll
    for (int t = 0; t < TT; ++t) *reinterpret_cast<f32x4*>(part[wave][t][lane]) = acc[t];
    __syncthreads();
    if (wave >= TT) return;
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int p = 0; p < 8; ++p) v += *reinterpret_cast<const f32x4*>(part[p][wave][lane]);
    epi(16 * wave + l16, n0 + 4 * lg, v);
}

// y = sum + scale b_i u[t] for up to four columns n .. n + 3
template <int DT>
struct AdapterRowEpi {
    AdapterArgs a;  // m: cols x rank
    __device__ __forceinline__ void operator()(int t, int n, f32x4 v) const {
        if (t < a.tokens && n < a.cols) adapter_row_store<DT>(a, t, n, v + adapter_row<DT>(a, a.index[t], t, n));
    }
};

}  // namespace dg
