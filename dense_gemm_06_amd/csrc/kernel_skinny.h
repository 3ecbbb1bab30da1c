// kernel_skinny.h -- x w^T of up to 64 rows x, fp16 or bf16: w is read once, past everything else.
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
    const int whole = a.K & ~63;
    int64_t k = wave * 64;
    // U pieces of 64 at a time, all of their loads before the first product
    auto pieces_of = [&](auto u_tag) {
        constexpr int U = decltype(u_tag)::value;
        u32x4 wv[U][2], xv[U][2][TT];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int s = 0; s < 2; ++s) __builtin_memcpy(&wv[u][s], w + k + 512 * u + 32 * s, 16);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int t = 0; t < TT; ++t) __builtin_memcpy(&xv[u][s][t], x[t] + k + 512 * u + 32 * s, 16);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int t = 0; t < TT; ++t) acc[t] = mfma_16<DT>(wv[u][s], xv[u][s][t], acc[t]);
        k += 512 * U;
    };
    constexpr int U = TT == 1 ? 8 : TT == 2 ? 4 : 3;
    while (k + 512 * (U - 1) < whole) pieces_of(std::integral_constant<int, U>{});
    while (k < whole) pieces_of(std::integral_constant<int, 1>{});
    if (k == whole && whole < a.K)
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
        if (t >= a.tokens || n >= a.cols) return;
        const int i = a.index[t], left = a.cols - n;
        if (i >= 0 && i < a.adapters) {
            const uint16_t* m = static_cast<const uint16_t*>(a.m) + (size_t)i * (size_t)a.stride_m;
            f32x4 d = {0.f, 0.f, 0.f, 0.f};
            for (int j = 0; j < a.rank; j += 8) {
                float u[8];
                load_f8(u, a.u + (size_t)t * (size_t)a.rank + j, a.rank - j);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const u32x4 p = load_frag8(m + (size_t)(n + min(e, left - 1)) * (size_t)a.ldm + j, a.rank - j);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        d[e] = fmaf(u[2 * q], decode<DT>((uint16_t)p[q]), d[e]);
                        d[e] = fmaf(u[2 * q + 1], decode<DT>((uint16_t)(p[q] >> 16)), d[e]);
                    }
                }
            }
            const float scale = a.scale ? a.scale[i] : 1.0f;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = fmaf(scale, d[e], v[e]);
        }
        const size_t at = (size_t)t * (size_t)a.ldo + n;
        if (left >= 4) store_out4(a.out, DT, at, v);
        else
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (e < left) store_out(a.out, DT, at + e, v[e]);
    }
};

}  // namespace dg
