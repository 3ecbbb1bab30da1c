// kernel_loss.h -- the loss over a vocabulary for fp16 and bf16: products whose epilogue turns a
// tile of logits into what is kept of it, so that no logits are stored.
//
// Forward: of each row and tile the maximum m and s = sum exp(l - m). A lane holds 32 logits of
// one row, so they take two passes over registers and one exchange; the four waves along a row
// are joined in LDS. Backward: d = (exp(l - lse) - [target]) grad, rounded to the matrices' type
// (fp16 after a power of two that keeps it in range), stored by rows for the product with w and
// turned for the product with x. Where the target's p is below 1/2 the rows hold p and not p - 1, and
// x's gradient gets the rest, most of such a row's d, unrounded when it is rounded itself.
#pragma once
#include "device_common.h"
#include "kernel_mid.h"
#include "kernel_skinny.h"
#include "kernel_stream.h"
#include "kernel_sp.h"
#include "layers.h"
#include "tile16.h"

namespace dg {

constexpr float kLog2e = 1.44269504f;

// (m, s) joined with (m2, s2); a part without anything is (-inf, 0). Equal infinities count 1.
__device__ __forceinline__ void loss_join(float& m, float& s, float m2, float s2) {
    const float M = fmaxf(m, m2);
    const float a = m == M ? 1.0f : __builtin_amdgcn_exp2f((m - M) * kLog2e);
    const float b = m2 == M ? 1.0f : __builtin_amdgcn_exp2f((m2 - M) * kLog2e);
    s = s * a + s2 * b;
    m = M;
}

struct LossPart {
    float m, s;
};

struct LossStatsHook {
    static constexpr bool kReplace = true;
    const int64_t* target;
    LossPart* part;   // strips x tokens
    float* picked;
    int tokens, n, v0;   // columns, and the first one's word

    template <int SI, int SJ, int WM, int WN>
    __device__ __forceinline__ void finish(f32x16 (&acc)[SI][SJ], int m0, int n0, int wm, int wn, char* lds, char*) const {
        constexpr int ROWS = WM * 32 * SI, COLS = WN * 32 * SJ;
        const int lane = threadIdx.x & 63, l32 = lane & 31, lh = lane >> 5;
        LossPart* joined = reinterpret_cast<LossPart*>(lds);  // waves along n x rows
        const bool cut = n0 + 32 * SJ > n;
#pragma unroll
        for (int i = 0; i < SI; ++i) {
            const int row = m0 + 32 * i + l32;
            float m = -INFINITY, s = 0.0f;
            if (cut) {
#pragma unroll
                for (int j = 0; j < SJ; ++j)
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        if (n0 + 32 * j + 8 * (r / 4) + 4 * lh + r % 4 >= n) acc[i][j][r] = -INFINITY;
            }
#pragma unroll
            for (int j = 0; j < SJ; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r) m = fmaxf(m, acc[i][j][r]);
            if (__any(!(fabsf(m) < INFINITY))) {
#pragma unroll
                for (int j = 0; j < SJ; ++j)
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        s += acc[i][j][r] == m ? 1.0f : __builtin_amdgcn_exp2f((acc[i][j][r] - m) * kLog2e);
            } else {
                const float c = -m * kLog2e;
#pragma unroll
                for (int j = 0; j < SJ; ++j)
#pragma unroll
                    for (int r = 0; r < 16; ++r) s += __builtin_amdgcn_exp2f(fmaf(acc[i][j][r], kLog2e, c));
            }
            const int64_t at = row < tokens ? target[row] - v0 - n0 : -1;
            const bool has = at >= 0 && at < 32 * SJ;
            if (__any(has)) {
                const int t = has ? (int)at - 4 * lh : -1;
                float v = 0.0f;
                bool mine = false;
#pragma unroll
                for (int j = 0; j < SJ; ++j)
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        const bool hit = t == 32 * j + 8 * (r / 4) + r % 4;
                        v = hit ? acc[i][j][r] : v;
                        mine = mine || hit;
                    }
                if (mine && n0 + at < n) picked[row] = v;
            }
            loss_join(m, s, __shfl_xor(m, 32), __shfl_xor(s, 32));
            if (lh == 0) joined[wn * ROWS + wm * (32 * SI) + 32 * i + l32] = {m, s};
        }
        __syncthreads();
        const int r = threadIdx.x, row = m0 - wm * (32 * SI) + r;
        if (r < ROWS && row < tokens) {
            float m = joined[r].m, s = joined[r].s;
#pragma unroll
            for (int w = 1; w < WN; ++w) loss_join(m, s, joined[w * ROWS + r].m, joined[w * ROWS + r].s);
            part[(size_t)((n0 - wn * 32 * SJ) / COLS) * (size_t)tokens + row] = {m, s};
        }
    }
};

// The same of up to 64 rows: a strip is 16 columns.
struct LossSkinnyEpi {
    const int64_t* target;
    LossPart* part;
    float* picked;
    int tokens, n;
    __device__ __forceinline__ void operator()(int t, int c, f32x4 v) const {
        const int left = n - c;
        float m = -INFINITY, s = 0.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[e] = e < left ? v[e] : -INFINITY;
            m = fmaxf(m, v[e]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) s += v[e] == m ? 1.0f : __builtin_amdgcn_exp2f((v[e] - m) * kLog2e);
        const int64_t at = t < tokens ? target[t] - c : -1;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (at == e && e < left) picked[t] = v[e];
#pragma unroll
        for (int d = 16; d < 64; d <<= 1) loss_join(m, s, __shfl_xor(m, d), __shfl_xor(s, d));
        if (t < tokens && (threadIdx.x & 63) < 16) part[(size_t)(c >> 4) * (size_t)tokens + t] = {m, s};
    }
};

// Few rows x against a stream of w, 64 words to a workgroup.
template <int DT, int TT, class EPI>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2, 4))) void loss_stream(StreamArgs a, EPI epi) {
    __shared__ __attribute__((aligned(1024))) StreamLds<TT, true> lds;
    f32x4 acc[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int r0 = (int)blockIdx.x * kStreamRows, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    stream_sum<DT, TT, true>(acc, a, lds, r0, 0, a.K);
    if (r0 + 16 * wave >= a.rows) return;
#pragma unroll
    for (int t = 0; t < TT; ++t) epi(16 * t + (lane & 15), r0 + 16 * wave + 4 * (lane >> 4), acc[t]);
}

// Joins the strips of each row. A workgroup has `width` tokens (a power of two up to 64) and as
// many threads to each as are left.
static __global__ __launch_bounds__(1024) void loss_finish(const LossPart* part, int strips, int tokens, int width,
                                                           const int64_t* target, int vocabulary, const float* picked,
                                                           float* loss, float* lse) {
    __shared__ LossPart buf[1024];
    const int tid = threadIdx.x, t = (int)blockIdx.x * width + (tid & (width - 1)), groups = 1024 / width;
    float m = -INFINITY, s = 0.0f;
    if (t < tokens)
#pragma unroll 4
        for (int k = tid / width; k < strips; k += groups) {
            const LossPart p = part[(size_t)k * (size_t)tokens + t];
            loss_join(m, s, p.m, p.s);
        }
    buf[tid] = {m, s};
    for (int half = 512; half >= width; half >>= 1) {
        __syncthreads();
        if (tid < half) {
            loss_join(m, s, buf[tid + half].m, buf[tid + half].s);
            buf[tid] = {m, s};
        }
    }
    if (tid >= width || t >= tokens) return;
    const float l = m + logf(s);
    const int64_t k = target[t];
    lse[t] = l;
    loss[t] = k >= 0 && k < vocabulary ? l - picked[t] : 0.0f;
}

// d of a tile leaves as 16-bit rows (tile16.h).
template <int DT>
struct LossGradHook {
    static constexpr bool kReplace = true;
    const int64_t* target;
    const float* lse;
    const float* grad;
    const float* factor;   // or NULL
    uint16_t* d;           // tokens x n, or NULL: where p < 1/2 without the target's -1
    float* apart;          // tokens, with d: 1 where it was left out, else 0
    uint16_t* dt;          // n x lddt, or NULL
    float* rest;           // tokens, with dt: what rounding took from the target's d
    int64_t ldd, lddt;
    int tokens, n, v0, vocabulary;

    template <int SI, int SJ, int WM, int WN>
    __device__ __forceinline__ void finish(f32x16 (&acc)[SI][SJ], int m0, int n0, int wm, int wn, char* lds,
                                           char* lds2) const {
        typedef Tile16<SI, SJ, WM, WN> Tile;
        const Tile tile{lds, lds2};
        const int lane = threadIdx.x & 63, l32 = lane & 31, lh = lane >> 5;
        const float f = factor ? factor[0] : 1.0f;
        uint32_t hit[SI];      // the target's (p - 1) grad, where this lane has it and d does not hold it,
        int hit_at[SI];        // and its column in the wave's tile, or -1
#pragma unroll
        for (int i = 0; i < SI; ++i) {
            const int r = wm * Tile::HALF + 32 * i + l32, row = m0 + 32 * i + l32;
            int64_t at = -1;
            float g = 0.0f, c = 0.0f;
            if (row < tokens) {
                at = target[row];
                if (at >= 0 && at < vocabulary) {
                    g = grad[row] * f;
                    c = -lse[row] * kLog2e;
                    at -= (int64_t)v0 + n0;
                } else {
                    at = -1;
                }
            }
            const bool live = g != 0.0f;  // a NaN is live
            const int t = at >= 0 && at < 32 * SJ ? (int)at - 4 * lh : -1;
            float mine = 0.0f;
            bool has = false, low = false;
#pragma unroll
            for (int j = 0; j < SJ; ++j) {
                if constexpr (SI == 4) asm volatile("" : "+a"(acc[i][j]));  // see full_epilogue
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float v[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float p = __builtin_amdgcn_exp2f(fmaf(acc[i][j][4 * q + e], kLog2e, c));
                        const bool here = t == 32 * j + 8 * q + e;
                        const float all = (p - 1.0f) * g;
                        v[e] = live ? (here && !(p < 0.5f) ? all : p * g) : 0.0f;
                        mine = here ? all : mine;
                        low = here ? p < 0.5f : low;
                        has = has || here;
                    }
                    tile.template put<DT>(r, wn, j, q, lh, v);
                }
            }
            hit[i] = DT == DT_F16 ? (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)mine) : (uint32_t)f32_to_bf16_rne(mine);
            hit_at[i] = has && low && live ? (int)at : -1;
            if (d && has) apart[row] = low && live ? 1.0f : 0.0f;
            const float left = mine - decode<DT>((uint16_t)hit[i]);
            if (dt && has) rest[row] = live && left == left ? left : 0.0f;  // an infinite d leaves nothing
        }
        __syncthreads();
        const int wave = threadIdx.x >> 6, tile_m = m0 - wm * Tile::HALF, tile_n = n0 - wn * 32 * SJ;
        if (d) tile.store(d, ldd, tile_m, tile_n, tokens, n);
        if (dt) {
            if (d) __syncthreads();
#pragma unroll
            for (int i = 0; i < SI; ++i)
                if (hit_at[i] >= 0) {
                    const int col = wn * 32 * SJ + hit_at[i];
                    *reinterpret_cast<uint16_t*>(tile.at(wm * Tile::HALF + 32 * i + l32, col >> 3) + (col & 7) * 2) = (uint16_t)hit[i];
                }
            __syncthreads();
            // a wave: 32 columns, 32 rows at a time: 16 lanes get eight rows of 16 columns
            static_assert(Tile::COLS / Tile::WAVES == 32, "columns of a wave");
            const int l16 = lane & 15, lg = lane >> 4;
#pragma unroll 2
            for (int it = 0; it < 2 * (2 * Tile::HALF / 32); ++it) {
                const int cb = wave * 32 + 16 * (it & 1), rb = 32 * (it >> 1) + 8 * lg;
                u32x4 v;
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    const int col = cb + 4 * (l16 & 3);
                    char* p = tile.at(rb + 4 * hh + (l16 >> 2), col >> 3) + (col & 7) * 2;
                    const u32x2 x = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4f16(DG_LDS_PTR(fp16x4_t, p)));
                    v[2 * hh] = x[0];
                    v[2 * hh + 1] = x[1];
                }
                const int c = tile_n + cb + l16, row = tile_m + rb;
                if (c < n && row < lddt) __builtin_memcpy(dt + (size_t)c * (size_t)lddt + row, &v, 16);
            }
        }
    }
};

// The same of up to 64 rows, 16 of them and four words to a lane's call.
template <int DT>
struct LossGradSkinnyEpi {
    LossGradHook<DT> h;
    __device__ __forceinline__ void operator()(int t, int c, f32x4 v) const {
        const int left = h.n - c;
        if (left <= 0) return;
        int64_t at = -1;
        float g = 0.0f, k = 0.0f;
        if (t < h.tokens) {
            at = h.target[t];
            if (at >= 0 && at < h.vocabulary) {
                g = h.factor ? h.grad[t] * h.factor[0] : h.grad[t];
                k = -h.lse[t] * kLog2e;
                at -= (int64_t)h.v0 + c;
            } else {
                at = -1;
            }
        }
        const bool live = g != 0.0f;  // a NaN is live
        uint32_t in_row[4], in_turn[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float p = __builtin_amdgcn_exp2f(fmaf(v[e], kLog2e, k));
            const bool here = at == e && e < left, low = here && p < 0.5f;
            const float all = live ? (here ? p - 1.0f : p) * g : 0.0f, some = low && live ? p * g : all;
            const uint16_t r = DT == DT_F16 ? __builtin_bit_cast(uint16_t, (_Float16)all) : f32_to_bf16_rne(all);
            in_turn[e] = r;
            in_row[e] = DT == DT_F16 ? __builtin_bit_cast(uint16_t, (_Float16)some) : f32_to_bf16_rne(some);
            if (here) {
                const float rest = all - decode<DT>(r);
                if (h.d) h.apart[t] = low && live ? 1.0f : 0.0f;
                if (h.dt) h.rest[t] = rest == rest ? rest : 0.0f;  // an infinite d leaves nothing
            }
        }
        if (h.d && t < h.tokens) {
            uint16_t* d = h.d + (size_t)t * (size_t)h.ldd + c;
            const u32x2 two = {in_row[0] | (in_row[1] << 16), in_row[2] | (in_row[3] << 16)};
            if (left >= 4) __builtin_memcpy(d, &two, 8);
            else
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (e < left) d[e] = (uint16_t)in_row[e];
        }
        if (h.dt && t < h.lddt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (e < left) {
                    uint16_t* turned = h.dt + (size_t)(c + e) * (size_t)h.lddt + t;
                    *turned = (uint16_t)in_turn[e];
                    if (h.tokens <= 16) turned[16] = 0;  // rows of dt are 32 long
                }
    }
};

// w's gradient of a tile (256 words from v0 on): the product, plus for each token whose target is
// among the words what rounding took from its d, times its row of x. A word's gradient is mostly its
// own tokens' d, so the result comes as near as its own rounding allows (relative error 0.0024 to
// 0.0017 in bf16; the whole of 4096 tokens, 65536 words, 4096 long, both ways: 7.25 to 7.37 ms). The
// rests are few to a tile: one more sum, over the tokens that the tile finds among all, 16 at a time
// on the matrix instructions.
template <int DT>
struct LossWHook {
    static constexpr bool kReplace = true;
    uint16_t* out;
    int64_t ld;
    int rows, cols;
    const float* factor;   // or NULL
    const int64_t* target;
    const float* rest;
    const uint16_t* x;
    int64_t ldx;
    int tokens, v0;

    template <int SI, int SJ, int WM, int WN>
    __device__ __forceinline__ void finish(f32x16 (&acc)[SI][SJ], int m0, int n0, int wm, int wn, char* lds,
                                           char* lds2) const {
        typedef Tile16<SI, SJ, WM, WN> Tile;
        constexpr int WAVES = WM * WN, BLOCK = WAVES * 512;  // tokens looked at together
        const Tile tile{lds, lds2};
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l32 = lane & 31, lh = lane >> 5;
        const int tile_m = m0 - wm * Tile::HALF;
        int* token = reinterpret_cast<int*>(lds);                            // the tile's tokens in order
        int* word = reinterpret_cast<int*>(lds + BLOCK * 4 + 64);            // and their rows
        int* counts = reinterpret_cast<int*>(lds2);
        const int64_t first = (int64_t)v0 + tile_m;
        for (int64_t t0 = 0; t0 < tokens; t0 += BLOCK) {
            uint64_t hit[8];
            int row[8], mine = 0;
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const int64_t t = t0 + wave * 512 + 64 * q + lane;
                const int64_t at = target[min(t, (int64_t)tokens - 1)] - first;  // all loads before the first wait
                row[q] = t < tokens && at >= 0 && at < 2 * Tile::HALF && tile_m + at < rows ? (int)at : -1;
            }
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                hit[q] = __ballot(row[q] >= 0);
                mine += (int)__popcll(hit[q]);
            }
            if (lane == 0) counts[wave] = mine;
            __syncthreads();
            int before = 0, all = 0;
#pragma unroll
            for (int w = 0; w < WAVES; ++w) {
                before += w < wave ? counts[w] : 0;
                all += counts[w];
            }
            all = __builtin_amdgcn_readfirstlane(all);
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                if (row[q] >= 0) {
                    const int at = before + (int)__popcll(hit[q] & (((uint64_t)1 << lane) - 1));
                    token[at] = (int)(t0 + wave * 512 + 64 * q + lane);
                    word[at] = row[q];
                }
                before += (int)__popcll(hit[q]);
            }
            if (threadIdx.x < 16) {  // the last 16 are filled up with none
                token[all + threadIdx.x] = 0;
                word[all + threadIdx.x] = -1;
            }
            __syncthreads();
            for (int k0 = 0; k0 < all; k0 += 16) {
                int w[8];
                float left[8];
                u32x4 p[SJ];
                uint16_t xs[SJ][8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int t = token[k0 + 8 * lh + k];
                    w[k] = word[k0 + 8 * lh + k];
                    left[k] = rest[t];
                    const uint16_t* xr = x + (size_t)t * (size_t)ldx;
#pragma unroll
                    for (int j = 0; j < SJ; ++j) xs[j][k] = xr[min(n0 + 32 * j + l32, cols - 1)];
                }
                __builtin_amdgcn_sched_barrier(0);  // every load before the first wait
                uint32_t r16[8];
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    r16[k] = DT == DT_F16 ? (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)left[k])
                                          : (uint32_t)f32_to_bf16_rne(left[k]);
#pragma unroll
                for (int j = 0; j < SJ; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) p[j][e] = (uint32_t)xs[j][2 * e] | ((uint32_t)xs[j][2 * e + 1] << 16);
#pragma unroll
                for (int i = 0; i < SI; ++i) {
                    const int r = wm * Tile::HALF + 32 * i + l32;
                    u32x4 q;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        q[e] = (w[2 * e] == r ? r16[2 * e] : 0u) | (w[2 * e + 1] == r ? r16[2 * e + 1] << 16 : 0u);
#pragma unroll
                    for (int j = 0; j < SJ; ++j) acc[i][j] = mfma_32<DT>(p[j], q, acc[i][j]);
                }
            }
            __syncthreads();
        }
        const float f = factor ? factor[1] : 1.0f;
#pragma unroll
        for (int i = 0; i < SI; ++i)
#pragma unroll
            for (int j = 0; j < SJ; ++j) {
                if constexpr (SI == 4) asm volatile("" : "+a"(acc[i][j]));  // see full_epilogue
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float v[4] = {acc[i][j][4 * q] * f, acc[i][j][4 * q + 1] * f, acc[i][j][4 * q + 2] * f,
                                        acc[i][j][4 * q + 3] * f};
                    tile.template put<DT>(wm * Tile::HALF + 32 * i + l32, wn, j, q, lh, v);
                }
            }
        __syncthreads();
        tile.template store<true>(out, ld, tile_m, n0 - wn * 32 * SJ, rows, cols);
    }
};

template <int DT, bool REG>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2))) void loss_tiles(GemmArgs g, LossStatsHook h) {
    mfma32_sp_body<DT, 1, 8, REG, false, false>(g, nullptr, h);
}

template <int DT, bool REG>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2))) void loss_grad_tiles(GemmArgs g,
                                                                                                 LossGradHook<DT> h) {
    mfma32_sp_body<DT, 1, 8, REG, false, false>(g, nullptr, h);
}

// w's gradient: d^T (rows of whole stages) x
template <int DT>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2))) void loss_w_tiles(GemmArgs g, LossWHook<DT> h) {
    mfma32_sp_body<DT, 0, 8, false, false, false>(g, nullptr, h);
}

// The same in 128 x 128 tiles, of a transposed x.
template <int DT>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2, 2))) void loss_w_mid(MidArgs g, LossWHook<DT> h) {
    __shared__ __attribute__((aligned(1024))) MidLds lds;
    mid_body<DT>(g, lds, h);
}

static __global__ __launch_bounds__(256) void loss_turn(TurnArgs t) {
    __shared__ __attribute__((aligned(16))) uint16_t buf[64][72];
    turn_tile(t, (int)blockIdx.x, 0, buf);
}

template <int DT>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2, 2))) void loss_mid(MidArgs g, LossStatsHook h) {
    __shared__ __attribute__((aligned(1024))) MidLds lds;
    mid_body<DT>(g, lds, h);
}

template <int DT>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2, 2))) void loss_grad_mid(MidArgs g,
                                                                                               LossGradHook<DT> h) {
    __shared__ __attribute__((aligned(1024))) MidLds lds;
    mid_body<DT>(g, lds, h);
}

}  // namespace dg
