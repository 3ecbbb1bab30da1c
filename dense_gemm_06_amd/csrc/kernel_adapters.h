// kernel_adapters.h -- low-rank adapters of fp16 and bf16 on the matrix instructions.
//
// The rows of a tile may belong to any adapters. Where u m^T is added to a product, 32 rows
// are taken at a time and each adapter among them in turn, and what the instruction gives in the
// other adapters' rows is dropped, so that nothing of one adapter (a NaN least of all) reaches
// another's rows. u enters as the sum of two numbers of the matrices' type, its rounding and what
// that leaves: off by 2^-16 (bf16) or 2^-22 of u, against the single rounding of y that follows,
// for twice 2 T N rank operations. fp16 would hold a small u, or v of the backward pass, by its
// subnormal numbers, and a large one not at all, so there each token's numbers come after a power of
// two that brings the largest near 2^14 (what lies below it is off by 2^-39 of it at most; backward passes of
// up to 700 tokens take 1 to 2 us longer for it, of 4096 tokens 0.7%).
#pragma once
#include "device_common.h"
#include "extents.h"
#include "kernel_sp.h"
#include "layers.h"
#include "tile16.h"

namespace dg {

// Eight 16-bit elements from p, of which `valid` lie inside (the rest zero).
__device__ __forceinline__ u32x4 load_frag8(const uint16_t* p, int valid) {
    u32x4 r = {0, 0, 0, 0};
    if (valid >= 8) {
        __builtin_memcpy(&r, p, 16);
    } else if (valid > 0) {
#pragma unroll
        for (int e = 0; e < 7; ++e)
            if (e < valid) r[e >> 1] |= (uint32_t)p[e] << (16 * (e & 1));
    }
    return r;
}

// Eight fp32 numbers from p, of which `valid` lie inside (the rest zero).
__device__ __forceinline__ void load_f8(float (&v)[8], const float* p, int valid) {
    if (valid >= 8) {
        __builtin_memcpy(v, p, 32);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = e < valid ? p[e] : 0.0f;
    }
}

// x as hi + lo; an infinite or NaN x is all in hi.
template <int DT>
__device__ __forceinline__ void split_one(float x, uint16_t& hi, uint16_t& lo) {
    hi = DT == DT_F16 ? __builtin_bit_cast(uint16_t, (_Float16)x) : f32_to_bf16_rne(x);
    float rest = x - decode<DT>(hi);
    rest = fabsf(rest) < INFINITY ? rest : 0.0f;
    lo = DT == DT_F16 ? __builtin_bit_cast(uint16_t, (_Float16)rest) : f32_to_bf16_rne(rest);
}
// The power of two by which a token's numbers are divided before fp16 holds them: the largest finite
// magnitude, of bits `top`, comes to 2^14 .. 2^15.
__device__ __forceinline__ float split_unit(uint32_t top) {
    const int e = top == 0 ? 0 : max((int)(top >> 23) - 127 - 14, -100);
    return __uint_as_float((uint32_t)(e + 127) << 23);
}
// The bits of a finite |x|, else 0.
__device__ __forceinline__ uint32_t finite_bits(float x) {
    const uint32_t b = __float_as_uint(x) & 0x7fffffffu;
    return b < 0x7f800000u ? b : 0u;
}
// 1 / unit, a power of two
__device__ __forceinline__ float over(float unit) { return __uint_as_float((254u << 23) - __float_as_uint(unit)); }
template <int DT>
__device__ __forceinline__ void split_hi_lo(const float (&v)[8], u32x4& hi, u32x4& lo) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        uint16_t h[2], l[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) split_one<DT>(v[2 * e + k], h[k], l[k]);
        hi[e] = (uint32_t)h[0] | ((uint32_t)h[1] << 16);
        lo[e] = (uint32_t)l[0] | ((uint32_t)l[1] << 16);
    }
}

// The other operand's infinities meet hi alone, since lo is 0 or may have the other sign: lo's product
// takes them as zeros.
// Not 0 where one of the eight is infinite or NaN.
template <int DT>
__device__ __forceinline__ uint32_t has_special(u32x4 p) {
    const uint32_t up = DT == DT_F16 ? 0x04000400u : 0x00800080u;  // a full exponent carries into the sign's place
    uint32_t r = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) r |= (p[e] & 0x7fff7fffu) + up;
    return r & 0x80008000u;
}
template <int DT>
__device__ __forceinline__ u32x4 without_special(u32x4 p) {
    const uint32_t up = DT == DT_F16 ? 0x04000400u : 0x00800080u;
#pragma unroll
    for (int e = 0; e < 4; ++e) p[e] &= ~(((((p[e] & 0x7fff7fffu) + up) >> 15) & 0x00010001u) * 0xffffu);
    return p;
}

template <int DT>
__device__ __forceinline__ f32x16 mfma_32(u32x4 p, u32x4 q, f32x16 c) {
    if (DT == DT_F16)
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, p), __builtin_bit_cast(f16x8, q), c, 0,
                                                      0, 0);
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, p), __builtin_bit_cast(bf16x8, q), c, 0,
                                                   0, 0);
}
template <int DT>
__device__ __forceinline__ f32x4 mfma_16(u32x4 p, u32x4 q, f32x4 c) {
    if (DT == DT_F16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, p), __builtin_bit_cast(f16x8, q), c, 0,
                                                      0, 0);
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, p), __builtin_bit_cast(bf16x8, q), c, 0,
                                                   0, 0);
}

// sum + d unit, d being a product with us
template <int DT>
__device__ __forceinline__ float adapter_sum(float sum, float d, float unit) {
    return DT == DT_F16 ? fmaf(d, unit, sum) : sum + d;
}

// acc[j] += scale u m^T for rows m0 .. m0 + 31 and columns n0 + 32 j .. + 31 (m: columns x rank).
// Lane l holds row m0 + l % 32; register r column 8 (r / 4) + 4 (l / 32) + r % 4 of a subtile. Of
// the adapters among the rows, every parts-th one from the part-th on.
template <int DT, int SJ>
__device__ __forceinline__ void adapter_add(f32x16 (&acc)[SJ], int m0, int n0, const AdapterArgs& a, int part = 0,
                                            int parts = 1) {
    const int lane = threadIdx.x & 63, l32 = lane & 31, lh = lane >> 5;
    const int row = m0 + l32;
    int mine = row < a.tokens ? a.index[row] : -1;
    if (mine >= a.adapters) mine = -1;
    const uint16_t* us = a.us + (size_t)min(row, a.tokens - 1) * (size_t)(2 * a.rank_p) + 8 * lh;
    const float unit = DT == DT_F16 && mine >= 0 ? a.unit[row] : 1.0f;
    const uint16_t* cols[SJ];
#pragma unroll
    for (int j = 0; j < SJ; ++j)
        cols[j] = static_cast<const uint16_t*>(a.m) + (size_t)min(n0 + 32 * j + l32, a.cols - 1) * (size_t)a.ldm + 8 * lh;
    uint64_t todo = __ballot(mine >= 0);
    for (int turn = 0; todo; ++turn) {
        const int i = __builtin_amdgcn_readlane(mine, (int)__builtin_ctzll(todo));
        const bool here = mine == i;
        todo &= ~__ballot(here);
        if (turn % parts != part) continue;
        const size_t at = (size_t)i * (size_t)a.stride_m;
        f32x16 d[SJ];
#pragma unroll
        for (int j = 0; j < SJ; ++j) d[j] = f32x16{};
        int r = 0;
        // whole pieces of 32: the loads of both halves before the first product
        for (; r + 32 <= a.rank_m; r += 32) {
            u32x4 hi[2], lo[2], p[2][SJ];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                __builtin_memcpy(&hi[h], us + r + 16 * h, 16);
                __builtin_memcpy(&lo[h], us + a.rank_p + r + 16 * h, 16);
#pragma unroll
                for (int j = 0; j < SJ; ++j) __builtin_memcpy(&p[h][j], cols[j] + at + r + 16 * h, 16);
            }
            uint32_t special = 0;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int j = 0; j < SJ; ++j) {
                    d[j] = mfma_32<DT>(p[h][j], hi[h], d[j]);
                    special |= has_special<DT>(p[h][j]);
                }
            if (__any(special != 0))
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int j = 0; j < SJ; ++j) p[h][j] = without_special<DT>(p[h][j]);
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int j = 0; j < SJ; ++j) d[j] = mfma_32<DT>(p[h][j], lo[h], d[j]);
        }
        for (; r < a.rank; r += 16) {
            u32x4 hi, lo;
            __builtin_memcpy(&hi, us + r, 16);
            __builtin_memcpy(&lo, us + a.rank_p + r, 16);
#pragma unroll
            for (int j = 0; j < SJ; ++j) {
                const u32x4 p = load_frag8(cols[j] + at + r, a.rank_m - r - 8 * lh);
                d[j] = mfma_32<DT>(p, hi, d[j]);
                d[j] = mfma_32<DT>(without_special<DT>(p), lo, d[j]);
            }
        }
#pragma unroll
        for (int j = 0; j < SJ; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[j][e] = adapter_sum<DT>(acc[j][e], here ? d[j][e] : 0.0f, unit);
    }
}

// ---------------------------------------------------------------- shared product and adapters in one
// A tile's u (256 rows, hi and lo) and an adapter's rows of m (256 columns), of rank up to 64, are
// brought to LDS by all waves together, whole lines at a time: fragments loaded by each wave
// straight from memory touch a line for every two lanes, and each is loaded by several waves. The
// adapters among 32 rows of each half of the tile take turns.
// 16-byte piece c of row r of `pieces` pieces lies at piece c ^ swz: reads of 32 rows meet in no bank.
__device__ __forceinline__ int rank_swz(int r, int pieces) {
    return pieces == 16 ? r & 15 : pieces == 8 ? (r >> 1) & 7 : pieces == 4 ? (r >> 2) & 3 : (r >> 3) & 1;
}

template <int DT>
struct AdapterHook {
    static constexpr bool kReplace = true;
    AdapterArgs a;
    template <int SI, int SJ, int WM, int WN>
    __device__ __forceinline__ void finish(f32x16 (&acc)[SI][SJ], int m, int n, int wm, int wn, char* lds,
                                           char* lds2) const {
        typedef Tile16<SI, SJ, WM, WN> Tile;
        const int m0 = m - wm * Tile::HALF, n0 = n - wn * 32 * SJ;
        if (a.adapters > 0) {  // else there may be no u, and a rank of 0
            add<SI, SJ, WM, WN>(acc, m0, n0, wm, wn, lds, lds2);
            __syncthreads();
        }
        const Tile tile{lds, lds2};
        const int lane = threadIdx.x & 63, l32 = lane & 31, lh = lane >> 5;
#pragma unroll
        for (int i = 0; i < SI; ++i)
#pragma unroll
            for (int j = 0; j < SJ; ++j) {
                asm volatile("" : "+a"(acc[i][j]));  // see full_epilogue
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float v[4] = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
                    tile.template put<DT>(wm * Tile::HALF + 32 * i + l32, wn, j, q, lh, v);
                }
            }
        __syncthreads();
        tile.store(static_cast<uint16_t*>(a.out), a.ldo, m0, n0, a.tokens, a.cols);
    }
    template <int SI, int SJ, int WM, int WN>
    __device__ __forceinline__ void add(f32x16 (&acc)[SI][SJ], int m0, int n0, int wm, int wn, char* us_lds,
                                        char* m_lds) const {
        constexpr int ROWS = WM * 32 * SI, COLS = WN * 32 * SJ, THREADS = WM * WN * 64;
        static_assert(WM == 2, "halves of the tile");
        const int tid = threadIdx.x, lane = tid & 63, l32 = lane & 31, lh = lane >> 5;
        const int mp = a.rank_p / 8, up = 2 * mp;  // pieces of a row of m, of u
        const int lmp = 31 - __builtin_clz(mp);
        // lanes 0-31: rows 32 b .. of the tile's first half, 32-63: of its second; the same in all waves
        int of[SI];
        float unit[SI];  // of this wave's rows
#pragma unroll
        for (int b = 0; b < SI; ++b) {
            const int row = m0 + lh * (32 * SI) + 32 * b + l32;
            of[b] = row < a.tokens ? a.index[row] : -1;
            unit[b] = DT == DT_F16 ? a.unit[min(m0 + wm * (32 * SI) + 32 * b + l32, a.tokens - 1)] : 1.0f;
        }
#pragma unroll
        for (int b = 0; b < SI; ++b) of[b] = of[b] >= a.adapters ? -1 : of[b];
        // n pieces, four loads of a thread in flight; whether this thread's hold infinities
        auto bring = [&](int n, auto load, char* to, int lp) {
            const int pieces = 1 << lp;
            uint32_t special = 0;
            for (int e = tid; e < n; e += 4 * THREADS) {
                u32x4 v[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int at = min(e + k * THREADS, n - 1);
                    v[k] = load(at >> lp, at & (pieces - 1));
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int at = e + k * THREADS, r = at >> lp, c = at & (pieces - 1);
                    if (at < n) *reinterpret_cast<u32x4*>(to + (size_t)(r * pieces + (c ^ rank_swz(r, pieces))) * 16) = v[k];
                    special |= has_special<DT>(v[k]);
                }
            }
            return special;
        };
        bring(
            ROWS * up,
            [&](int r, int c) {
                u32x4 v;
                __builtin_memcpy(&v, a.us + (size_t)min(m0 + r, a.tokens - 1) * (size_t)(2 * a.rank_p) + 8 * c, 16);
                return v;
            },
            us_lds, lmp + 1);
        // two adapters stay in LDS (2 x 32 KB at rank 64): a tile in which one request ends and the
        // next begins brings each once
        int staged[2] = {-1, -1}, next = 0;
        uint32_t infinite[2] = {0, 0};               // of each place
        __shared__ uint32_t special[2][WM * WN];     // and wave
#pragma unroll
        for (int b = 0; b < SI; ++b) {
            uint64_t todo = __ballot(of[b] >= 0);
            while (todo) {
                const int i = __builtin_amdgcn_readlane(of[b], (int)__builtin_ctzll(todo));
                const uint64_t rows = __ballot(of[b] == i);
                todo &= ~rows;
                int at = staged[0] == i ? 0 : 1;
                if (staged[0] != i && staged[1] != i) {
                    at = next;
                    next ^= 1;
                    __syncthreads();  // the last reads of that place are done
                    const uint16_t* m = static_cast<const uint16_t*>(a.m) + (size_t)i * (size_t)a.stride_m;
                    const bool any = __any(bring(
                        COLS * mp,
                        [&](int r, int c) {
                            return load_frag8(m + (size_t)min(n0 + r, a.cols - 1) * (size_t)a.ldm + 8 * c,
                                              a.rank_m - 8 * c);
                        },
                        m_lds + at * 32768, lmp) != 0);
                    if (lane == 0) special[at][wm * WN + wn] = any;
                    __syncthreads();
                    uint32_t all = 0;
#pragma unroll
                    for (int w = 0; w < WM * WN; ++w) all |= special[at][w];
                    all = __builtin_amdgcn_readfirstlane(all);
                    if (at == 0) staged[0] = i, infinite[0] = all;
                    else staged[1] = i, infinite[1] = all;
                }
                const char* m_at = m_lds + at * 32768;
                const bool clear = (at == 0 ? infinite[0] : infinite[1]) != 0;
                const uint32_t own = (uint32_t)(wm == 0 ? rows : rows >> 32);
                const bool here = (own >> l32) & 1;
                const int ur = wm * 32 * SI + 32 * b + l32, us = rank_swz(ur, up);
                const char* u_row = us_lds + (size_t)(ur * up) * 16;
                f32x16 d[SJ];
#pragma unroll
                for (int j = 0; j < SJ; ++j) d[j] = f32x16{};
                auto products = [&](auto special_tag) {
                    for (int c = own != 0 ? lh : mp; c < mp; c += 2) {
                        const u32x4 hi = *reinterpret_cast<const u32x4*>(u_row + ((c ^ us) << 4));
                        const u32x4 lo = *reinterpret_cast<const u32x4*>(u_row + (((mp + c) ^ us) << 4));
    #pragma unroll
                        for (int j = 0; j < SJ; ++j) {
                            const int mr = wn * 32 * SJ + 32 * j + l32;
                            const u32x4 p =
                                *reinterpret_cast<const u32x4*>(m_at + (size_t)(mr * mp + (c ^ rank_swz(mr, mp))) * 16);
                            d[j] = mfma_32<DT>(p, hi, d[j]);
                            d[j] = mfma_32<DT>(decltype(special_tag)::value ? without_special<DT>(p) : p, lo, d[j]);
                        }
                    }
                };
                if (clear) products(std::true_type{});
                else products(std::false_type{});
#pragma unroll
                for (int j = 0; j < SJ; ++j)
#pragma unroll
                    for (int e = 0; e < 16; ++e) acc[b][j][e] = adapter_sum<DT>(acc[b][j][e], here ? d[j][e] : 0.0f, unit[b]);
            }
        }
    }
};

template <int DT, int OPB, bool REG>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2))) void adapter_product(
    GemmArgs g, AdapterHook<DT> h) {
    mfma32_sp_body<DT, OPB, 8, REG, false, false>(g, nullptr, h);
}

// ---------------------------------------------------------------- second product on its own
// out = the slices' sum of base + scale u m^T, 32 rows x 64 columns to a workgroup, whose four waves
// share the adapters among the rows and are joined in LDS in their order.
template <int DT>
__global__ __launch_bounds__(256) void adapter_expand16(AdapterArgs a, int tiles_n) {
    __shared__ __attribute__((aligned(16))) float sums[4][32][68];
    const int tm = (int)blockIdx.x / tiles_n, tn = (int)blockIdx.x - tm * tiles_n;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l32 = lane & 31, lh = lane >> 5;
    const int m0 = tm * 32, n0 = tn * 64;
    f32x16 acc[2] = {f32x16{}, f32x16{}};
    adapter_add<DT, 2>(acc, m0, n0, a, wave, 4);
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q)
            *reinterpret_cast<f32x4*>(&sums[wave][l32][32 * j + 8 * q + 4 * lh]) =
                f32x4{acc[j][4 * q], acc[j][4 * q + 1], acc[j][4 * q + 2], acc[j][4 * q + 3]};
    __syncthreads();
    const int c = n0 + (threadIdx.x & 15) * 4, left = a.cols - c;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int r = (threadIdx.x >> 4) + 16 * h, row = m0 + r;
        if (row >= a.tokens || left <= 0) continue;
        f32x4 v = {0.f, 0.f, 0.f, 0.f};
        const float* base = a.base + (size_t)row * (size_t)a.ld_base + c;
        const size_t step = (size_t)a.tokens * (size_t)a.ld_base;
        auto add = [&](auto n, int k) {  // n slices, loaded together
            constexpr int U = decltype(n)::value;
            f32x4 b[U];
#pragma unroll
            for (int e = 0; e < U; ++e) {
                b[e] = f32x4{0.f, 0.f, 0.f, 0.f};
                if (left >= 4) __builtin_memcpy(&b[e], base + (size_t)(k + e) * step, 16);
                else
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        if (q < left) b[e][q] = base[(size_t)(k + e) * step + q];
            }
#pragma unroll
            for (int e = 0; e < U; ++e) v += b[e];
        };
        int k = 0;
        for (; k + 8 <= a.slices; k += 8) add(std::integral_constant<int, 8>{}, k);
        for (; k + 2 <= a.slices; k += 2) add(std::integral_constant<int, 2>{}, k);
        if (k < a.slices) add(std::integral_constant<int, 1>{}, k);
#pragma unroll
        for (int w = 0; w < 4; ++w) v += *reinterpret_cast<const f32x4*>(&sums[w][r][(threadIdx.x & 15) * 4]);
        const size_t at = (size_t)row * (size_t)a.ldo + c;
        if (left >= 4) store_out4(a.out, DT, at, v);
        else
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (e < left) store_out(a.out, DT, at + e, v[e]);
    }
}

// ---------------------------------------------------------------- first product
// A wave: rank numbers j .. j + 3 of token t, whose adapter is i, 8 elements to a lane and step: lane l
// up to 3 returns that of j + l, unscaled (zero without an adapter and past the rank).
template <int DT>
__device__ __forceinline__ float adapter_shrink_four(const AdapterArgs& a, int t, int i, int j) {
    const int lane = threadIdx.x & 63;
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    if (i >= 0 && i < a.adapters && j < a.rank) {
        const uint16_t* x = static_cast<const uint16_t*>(a.x) + (size_t)t * (size_t)a.ldx;
        const uint16_t* m[4];
#pragma unroll
        for (int r = 0; r < 4; ++r)
            m[r] = static_cast<const uint16_t*>(a.m) + (size_t)i * (size_t)a.stride_m +
                   (size_t)min(j + r, a.rank - 1) * (size_t)a.ldm;
        auto add = [&](u32x4 p, u32x4 q, float& s) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                s = fmaf(decode<DT>((uint16_t)p[e]), decode<DT>((uint16_t)q[e]), s);
                s = fmaf(decode<DT>((uint16_t)(p[e] >> 16)), decode<DT>((uint16_t)(q[e] >> 16)), s);
            }
        };
        int64_t k = lane * 8;
        for (; k + 3 * 512 + 8 <= a.cols; k += 4 * 512) {
            u32x4 p[4], q[4][4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                __builtin_memcpy(&p[e], x + k + 512 * e, 16);
#pragma unroll
                for (int r = 0; r < 4; ++r) __builtin_memcpy(&q[r][e], m[r] + k + 512 * e, 16);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int r = 0; r < 4; ++r) add(p[e], q[r][e], sum[r]);
        }
        for (; k < a.cols; k += 512) {
            const int valid = (int)min((int64_t)8, a.cols - k);
            const u32x4 p = load_frag8(x + k, valid);
#pragma unroll
            for (int r = 0; r < 4; ++r) add(p, load_frag8(m[r] + k, valid), sum[r]);
        }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) sum[r] += __shfl_xor(sum[r], d);
    return j + lane >= a.rank ? 0.0f : lane == 0 ? sum[0] : lane == 1 ? sum[1] : lane == 2 ? sum[2] : sum[3];
}

// For tokens few enough that each can read its adapter by itself: u and, in bf16 where wanted, us (see
// adapter_shrink_finish). A wave has four rank numbers of one token.
template <int DT>
__device__ __forceinline__ void adapter_shrink_wave(const AdapterArgs& a, int64_t unit) {
    const int lane = threadIdx.x & 63, each = a.rank_p >> 2;
    if (unit >= (int64_t)a.tokens * each) return;
    const int t = (int)(unit / each), j = (int)(unit - (int64_t)t * each) * 4;
    if (j >= a.rank && a.us == nullptr) return;
    const int i = a.index[t];
    const float scale = a.scale && i >= 0 && i < a.adapters ? a.scale[i] : 1.0f;
    const float v = adapter_shrink_four<DT>(a, t, i, j);
    if (lane >= 4) return;
    if (j + lane < a.rank) a.u[(size_t)t * (size_t)a.rank + j + lane] = a.fold ? v * scale : v;
    if (a.us) {
        uint16_t hi, lo;
        split_one<DT>(v * scale, hi, lo);
        uint16_t* us = a.us + (size_t)t * (size_t)(2 * a.rank_p) + j + lane;
        us[0] = hi;
        us[a.rank_p] = lo;
    }
}

template <int DT>
__global__ __launch_bounds__(256) void adapter_shrink_row(AdapterArgs a) {
    adapter_shrink_wave<DT>(a, (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6));
}

// The same with us in fp16, whose power of two is the whole token's: a workgroup to a token.
template <int DT>
__global__ __launch_bounds__(1024) void adapter_shrink_token(AdapterArgs a) {
    __shared__ float sums[kMaxRank];
    const int t = (int)blockIdx.x, tid = threadIdx.x, lane = tid & 63;
    const int i = a.index[t];
    const float scale = a.scale && i >= 0 && i < a.adapters ? a.scale[i] : 1.0f;
    for (int j = (tid >> 6) * 4; j < a.rank_p; j += (int)blockDim.x >> 4) {
        const float v = adapter_shrink_four<DT>(a, t, i, j);
        if (lane < 4) sums[j + lane] = v;
    }
    __syncthreads();
    if (tid >= a.rank_p && tid >= 64) return;  // every wave left has whole rows of the exchange
    uint32_t top = 0;
    for (int j = lane; j < a.rank_p; j += 64) top = max(top, finite_bits(sums[j] * scale));
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, d));
    const float unit = split_unit(top);
    if (tid == 0) a.unit[t] = unit;
    if (tid >= a.rank_p) return;
    const float v = sums[tid], w = v * scale;
    if (tid < a.rank) a.u[(size_t)t * (size_t)a.rank + tid] = a.fold ? w : v;
    uint16_t hi, lo;
    split_one<DT>(w * over(unit), hi, lo);
    uint16_t* us = a.us + (size_t)t * (size_t)(2 * a.rank_p) + tid;
    us[0] = hi;
    us[a.rank_p] = lo;
}

// The same sums as kernel_stream.h's for any alignment, fragments loaded straight from memory: 16
// tokens against each adapter among them (shared out over grid y), k cut over the workgroup's
// eight waves in pieces of 64 and joined in LDS in their order. To part, tokens x 16 NT.
template <int DT, int NT>
__global__ __launch_bounds__(512) void adapter_shrink_any(AdapterArgs a, float* part_out) {
    __shared__ __attribute__((aligned(16))) float part[8][NT][64][4];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int l16 = lane & 15, lg = lane >> 4;
    const int row = (int)blockIdx.x * 16 + l16;
    int mine = row < a.tokens ? a.index[row] : -1;
    if (mine >= a.adapters) mine = -1;
    const uint16_t* x = static_cast<const uint16_t*>(a.x) + (size_t)min(row, a.tokens - 1) * (size_t)a.ldx;
    uint32_t todo = (uint32_t)(__ballot(mine >= 0) & 0xffffu);
    for (uint32_t turn = 0; todo; ++turn) {
        const int i = __builtin_amdgcn_readlane(mine, (int)__builtin_ctz(todo));
        const bool here = mine == i;
        todo &= ~(uint32_t)__ballot(here);
        if (turn % gridDim.y != blockIdx.y) continue;
        const uint16_t* m = static_cast<const uint16_t*>(a.m) + (size_t)i * (size_t)a.stride_m;
        f32x4 acc[NT];
        const uint16_t* mr[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            acc[n] = f32x4{0.f, 0.f, 0.f, 0.f};
            mr[n] = m + (size_t)min(16 * n + l16, a.rank - 1) * (size_t)a.ldm;  // past the rank: not stored
        }
        // pieces of 64 of k: wave, wave + 8, ..
        const int whole = a.cols & ~63, all = whole >> 6;
        const int cnt = wave < all ? (all - wave + 7) >> 3 : 0;
        auto k_of = [&](int p) { return 64 * (wave + 8 * p) + 8 * lg; };
        u32x4 xv[2][2], mv[2][2][NT];  // two pieces in turn
        auto load = [&](int b, int p) {
            const int k = k_of(p);
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                __builtin_memcpy(&xv[b][s], x + k + 32 * s, 16);
#pragma unroll
                for (int n = 0; n < NT; ++n) __builtin_memcpy(&mv[b][s][n], mr[n] + k + 32 * s, 16);
            }
        };
        auto use = [&](int b) {
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int n = 0; n < NT; ++n) acc[n] = mfma_16<DT>(mv[b][s][n], xv[b][s], acc[n]);
        };
        if (cnt > 0) load(0, 0);
        int p = 0;
        for (; p + 2 < cnt; p += 2) {
            load(1, p + 1);
            __builtin_amdgcn_sched_barrier(0);
            use(0);
            load(0, p + 2);
            __builtin_amdgcn_sched_barrier(0);
            use(1);
        }
        if (p + 1 < cnt) {
            load(1, p + 1);
            use(0);
            use(1);
        } else if (p < cnt) {
            use(0);
        }
        if (whole < a.cols && wave == (all & 7))
            for (int s = 0; s < 2; ++s) {
                const int k = whole + 32 * s + 8 * lg, valid = max(0, min(8, a.cols - k));
                const u32x4 xt = load_frag8(x + k, valid);
#pragma unroll
                for (int n = 0; n < NT; ++n) acc[n] = mfma_16<DT>(load_frag8(mr[n] + k, valid), xt, acc[n]);
            }
#pragma unroll
        for (int n = 0; n < NT; ++n) *reinterpret_cast<f32x4*>(part[wave][n][lane]) = acc[n];
        __syncthreads();
        if (wave < NT && here) {  // lane: token l16, rank numbers 16 wave + 4 lg .. + 3
            f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int p = 0; p < 8; ++p) v += *reinterpret_cast<const f32x4*>(part[p][wave][lane]);
            *reinterpret_cast<f32x4*>(part_out + (size_t)row * (16 * NT) + 16 * wave + 4 * lg) = v;
        }
        __syncthreads();
    }
}

// u = the sum of the slices (rows of ld numbers), zeros in rows without an adapter, as fp32 (a.u,
// NULL: not wanted) and, times the scale, as hi and lo of the matrices' type (a.us: tokens x 2 x
// rank_p, zeros past the rank; fp16 after a.unit). a.fold: the scale is in the fp32 numbers too. A
// thread: eight rank numbers of one token, whose threads are neighbours.
template <int DT>
__device__ __forceinline__ void adapter_split(const AdapterArgs& a, int slices, const float* part, int ld, int64_t at) {
    const int rank_p = a.rank_p;
    const int each = rank_p >> 3;
    if (at >= (int64_t)a.tokens * each) return;
    const int t = (int)(at / each), j = (int)(at - (int64_t)t * each) * 8;
    const int i = a.index[t];
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    float scale = 1.0f;
    if (i >= 0 && i < a.adapters) {
        const float* p = part + (size_t)t * (size_t)ld + j;
        const size_t step = (size_t)a.tokens * (size_t)ld;
        int s = 0;
        for (; s + 4 <= slices; s += 4) {
            float q[4][8];
#pragma unroll
            for (int k = 0; k < 4; ++k) load_f8(q[k], p + (s + k) * step, ld - j);
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] += q[k][e];
        }
        for (; s < slices; ++s) {
            float q[8];
            load_f8(q, p + s * step, ld - j);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += q[e];
        }
        if (a.scale) scale = a.scale[i];
    }
    float w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        v[e] = j + e < a.rank ? v[e] : 0.0f;
        w[e] = v[e] * scale;
        if (a.u && j + e < a.rank) a.u[(size_t)t * (size_t)a.rank + j + e] = a.fold ? w[e] : v[e];
    }
    if constexpr (DT == DT_F16) {
        uint32_t top = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) top = max(top, finite_bits(w[e]));
        for (int d = 1; d < each; d <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, d));
        const float unit = split_unit(top), down = over(unit);
        if (j == 0) a.unit[t] = unit;
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] *= down;
    }
    u32x4 hi, lo;
    split_hi_lo<DT>(w, hi, lo);
    uint16_t* us = a.us + (size_t)t * (size_t)(2 * rank_p) + j;
    *reinterpret_cast<u32x4*>(us) = hi;
    *reinterpret_cast<u32x4*>(us + rank_p) = lo;
}

template <int DT>
__global__ __launch_bounds__(64) void adapter_shrink_finish(AdapterArgs a, int slices, const float* part, int ld) {
    adapter_split<DT>(a, slices, part, ld, (int64_t)blockIdx.x * 64 + threadIdx.x);
}

// scale b_i u[t] for columns n .. n + 3 (a.m: cols x rank), i = index[t]. Sixteen rank numbers at a time, their
// loads before the first product.
template <int DT>
__device__ __forceinline__ f32x4 adapter_row(const AdapterArgs& a, int i, int t, int n) {
    f32x4 d = {0.f, 0.f, 0.f, 0.f};
    if (i < 0 || i >= a.adapters) return d;
    const int left = a.cols - n;
    const uint16_t* m = static_cast<const uint16_t*>(a.m) + (size_t)i * (size_t)a.stride_m;
    const float* ut = a.u + (size_t)t * (size_t)a.rank;
    const float scale = a.scale ? a.scale[i] : 1.0f;
    for (int j = 0; j < a.rank; j += 16) {
        float u[2][8];
        u32x4 p[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            load_f8(u[h], ut + j + 8 * h, a.rank - j - 8 * h);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                p[h][e] = load_frag8(m + (size_t)(n + min(e, left - 1)) * (size_t)a.ldm + j + 8 * h, a.rank - j - 8 * h);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    d[e] = fmaf(u[h][2 * q], decode<DT>((uint16_t)p[h][e][q]), d[e]);
                    d[e] = fmaf(u[h][2 * q + 1], decode<DT>((uint16_t)(p[h][e][q] >> 16)), d[e]);
                }
    }
    return d * scale;
}

// Columns n .. n + 3 of row t of the result.
template <int DT>
__device__ __forceinline__ void adapter_row_store(const AdapterArgs& a, int t, int n, f32x4 v) {
    const int left = a.cols - n;
    const size_t at = (size_t)t * (size_t)a.ldo + n;
    if (left >= 4) store_out4(a.out, DT, at, v);
    else
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (e < left) store_out(a.out, DT, at + e, v[e]);
}

// ---------------------------------------------------------------- adapters' transposes
// Each in_i (rows x cols) as its transpose of cols x out_ld, zeros past column `rows`. A
// workgroup turns 64 x 64 through LDS.
__device__ __forceinline__ void turn_tile(const TurnArgs& t, int tile, int i, uint16_t (*buf)[72]) {
    const int tr = tile / t.tiles_c, tc = tile - tr * t.tiles_c;
    const int c8 = (threadIdx.x & 7) * 8, r0 = threadIdx.x >> 3;
    const uint16_t* in = static_cast<const uint16_t*>(t.in) + (size_t)i * (size_t)t.stride;
    uint16_t* out = static_cast<uint16_t*>(t.out) + (size_t)i * (size_t)t.cols * (size_t)t.out_ld;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int r = tr * 64 + r0 + 32 * h, c = tc * 64 + c8;
        *reinterpret_cast<u32x4*>(&buf[r0 + 32 * h][c8]) =
            load_frag8(in + (size_t)min(r, t.rows - 1) * (size_t)t.ld + c, r < t.rows ? t.cols - c : 0);
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int cc = tc * 64 + r0 + 32 * h, r = tr * 64 + c8, left = t.out_ld - r;
        if (cc >= t.cols || left <= 0) continue;
        u32x4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            v[e] = (uint32_t)buf[c8 + 2 * e][r0 + 32 * h] | ((uint32_t)buf[c8 + 2 * e + 1][r0 + 32 * h] << 16);
        uint16_t* dst = out + (size_t)cc * (size_t)t.out_ld + r;
        if (left >= 8) __builtin_memcpy(dst, &v, 16);
        else
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < left) dst[e] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
    }
}

// What the backward pass has to lay out before it starts, in one launch: both of an adapter's
// matrices (grid y, grid x the tiles of one and then of the other) and, from grid y `adapters` on, the
// forward pass's u as hi and lo.
template <int DT>
__global__ __launch_bounds__(256) void adapter_prepare(TurnArgs p, TurnArgs q, int adapters, AdapterArgs a,
                                                       const float* u) {
    __shared__ __attribute__((aligned(16))) uint16_t buf[64][72];
    const int first = p.tiles_r * p.tiles_c, x = (int)blockIdx.x, y = (int)blockIdx.y;
    if (y < adapters) {
        if (x < first) turn_tile(p, x, y, buf);
        else turn_tile(q, x - first, y, buf);
        return;
    }
    const int64_t all = (int64_t)a.tokens * (a.rank_p >> 3), step = (int64_t)(gridDim.y - adapters) * gridDim.x * 256;
    for (int64_t at = ((int64_t)(y - adapters) * gridDim.x + x) * 256 + threadIdx.x; at < all; at += step)
        adapter_split<DT>(a, 1, u, a.rank, at);
}

// ---------------------------------------------------------------- gradients
// The plan's rows are cut into chunks; slot i + c of the grid (y) is what adapter i has in chunk
// c, so that slots are distinct for distinct pairs. An adapter within one chunk is finished by
// its slot; the others' slots leave fp32 sums, which adapter_join adds in their order.
struct AdapterSpan {
    int from, to;  // rows of the plan
};
__device__ __forceinline__ AdapterSpan adapter_span(const AdapterArgs& a, int i) {
    const int from = max(0, min(a.offsets[i], a.capacity));
    return {from, capped_sum(from, max(0, a.counts[i]), a.capacity)};
}

// A workgroup: 128 columns of z (x or grad) and the whole rank, over an adapter's rows of a chunk
// (at most kChunkMax) in steps of 32, loaded two steps ahead. z and h (v or u as hi and lo) lie in
// LDS by rows and are read transposed, so that a lane gets eight consecutive rows of one column.
constexpr int kChunkMax = 512, kGradientCols = 128;

template <int NT>
struct GradientLds {
    uint16_t z[2][32 * kGradientCols];
    uint16_t h[2][2][32 * NT * 16];
    int rows[kChunkMax + 64];
    int odd[4];            // of each wave
};

// fp16: the powers of two that the rows of h leave out, as one for the whole chunk (the largest, in
// `unit`) and the rest of each row, of which h is multiplied with two factors of fp16's range.
struct GradientUnits {
    float row[kChunkMax + 64];
    float top[4];
};
__device__ __forceinline__ u32x4 scaled_f16(u32x4 h, float f) {
    const float first = fmaxf(f, 6.103515625e-05f);  // 2^-14
    const _Float16 p = (_Float16)first, q = (_Float16)(f * over(first));
    f16x8 v = __builtin_bit_cast(f16x8, h);
    v = v * p;
    v = v * q;
    return __builtin_bit_cast(u32x4, v);
}

template <int DT, int NT, bool TURNED>
__device__ __forceinline__ void adapter_gradient_body(const AdapterArgs& a, GradientLds<NT>& lds, GradientUnits* units) {
    constexpr int HC = NT * 2;               // 16-byte pieces of a row of h
    constexpr int HN = 32 * 2 * HC;          // pieces of a step: hi and lo
    constexpr int HP = (HN + 255) / 256;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int l16 = lane & 15, lg = lane >> 4;
    const int slot = (int)blockIdx.y, c0 = (int)blockIdx.x * kGradientCols;
    // the adapter of this slot: the last one whose first slot is not past it
    int lo = 0, hi = a.adapters - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (adapter_span(a, mid).from / a.chunk + mid <= slot) lo = mid;
        else hi = mid - 1;
    }
    const int i = lo;
    const AdapterSpan sp = adapter_span(a, i);
    const int first = sp.from / a.chunk, ch = slot - i;
    if (ch < first || (int64_t)ch * a.chunk >= sp.to) return;
    const int from = max(sp.from, ch * a.chunk), to = (int)min((int64_t)sp.to, ((int64_t)ch + 1) * a.chunk);
    if (from >= to) return;
    const bool alone = (sp.to - 1) / a.chunk == first;
    // the chunk's rows, -1 for padding and past its end
    float unit = 0.0f;
    for (int e = tid; e < kChunkMax + 64; e += 256) {
        int t = from + e < to ? a.rows[from + e] : -1;
        t = t >= 0 && t < a.tokens ? t : -1;
        lds.rows[e] = t;
        if constexpr (DT == DT_F16) {
            const float u = t >= 0 ? a.unit[t] : 0.0f;
            units->row[e] = u;
            unit = fmaxf(unit, u);
        }
    }
    if constexpr (DT == DT_F16) {
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) unit = fmaxf(unit, __shfl_xor(unit, d));
        if (lane == 0) units->top[wave] = unit;
    }
    __syncthreads();
    if constexpr (DT == DT_F16) {
        unit = fmaxf(fmaxf(units->top[0], units->top[1]), fmaxf(units->top[2], units->top[3]));
        if (unit == 0.0f) unit = 1.0f;  // a chunk of padding
    }
    const float down = DT == DT_F16 ? over(unit) : 1.0f;

    const uint16_t* z = static_cast<const uint16_t*>(a.x);
    // the two 16-byte pieces of z that this thread moves: rows zr and zr + 16
    const int zr = tid >> 4, zc = tid & 15, zleft = a.cols - (c0 + zc * 8);
    struct Step {
        u32x4 z[2], h[HP];
    };
    auto load = [&](Step& s, int p0) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int t = lds.rows[p0 + zr + 16 * q];
            s.z[q] = load_frag8(z + (size_t)max(t, 0) * (size_t)a.ldx + c0 + zc * 8, t < 0 ? 0 : zleft);
        }
#pragma unroll
        for (int q = 0; q < HP; ++q) {
            const int piece = q * 256 + tid, r = (piece / (2 * HC)) & 31, c = piece % (2 * HC);
            const int th = lds.rows[p0 + r];
            s.h[q] = load_frag8(a.us + (size_t)max(th, 0) * (size_t)(2 * NT * 16) + c * 8, th < 0 ? 0 : 8);
        }
    };
    auto put = [&](const Step& s, int b, int p0) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int r = zr + 16 * q;
            *reinterpret_cast<u32x4*>(&lds.z[b][r * kGradientCols + ((zc ^ nmaj_swz<16>(r)) << 3)]) = s.z[q];
        }
#pragma unroll
        for (int q = 0; q < HP; ++q) {
            const int piece = q * 256 + tid, r = piece / (2 * HC), c = piece % (2 * HC);
            if (HN < 256 && piece >= HN) break;
            u32x4 h = s.h[q];
            if constexpr (DT == DT_F16) h = scaled_f16(h, units->row[p0 + r] * down);
            *reinterpret_cast<u32x4*>(&lds.h[b][c / HC][r * (HC * 8) + (((c % HC) ^ nmaj_swz<HC>(r)) << 3)]) = h;
        }
    };
    // rows 8 lg .. + 7 of column c0 + l16 of a tile of CH chunks a row
    auto turned = [&](const uint16_t* base, int c, auto chunks) {
        constexpr int CH = decltype(chunks)::value;
        u32x4 r;
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
            const int k = 8 * lg + 4 * hh + (l16 >> 2), col = c + 4 * (l16 & 3);
            const uint16_t* p = base + k * (CH * 8) + (((col >> 3) ^ nmaj_swz<CH>(k)) << 3) + (col & 7);
            const u32x2 v = __builtin_bit_cast(
                u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4f16(DG_LDS_PTR(fp16x4_t, const_cast<uint16_t*>(p))));
            r[2 * hh] = v[0];
            r[2 * hh + 1] = v[1];
        }
        return r;
    };
    f32x4 acc[2][NT];  // of columns 32 wave .. + 15 and the 16 after them
    auto use = [&](int b, auto clear) {
        u32x4 zf[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) zf[q] = turned(lds.z[b], wave * 32 + 16 * q, std::integral_constant<int, 16>{});
        u32x4 zl[2] = {zf[0], zf[1]};  // with lo
        if constexpr (decltype(clear)::value)
#pragma unroll
            for (int q = 0; q < 2; ++q) zl[q] = without_special<DT>(zf[q]);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const u32x4 hf = turned(lds.h[b][0], n * 16, std::integral_constant<int, HC>{});
            const u32x4 lf = turned(lds.h[b][1], n * 16, std::integral_constant<int, HC>{});
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                acc[q][n] = TURNED ? mfma_16<DT>(hf, zf[q], acc[q][n]) : mfma_16<DT>(zf[q], hf, acc[q][n]);
                acc[q][n] = TURNED ? mfma_16<DT>(lf, zl[q], acc[q][n]) : mfma_16<DT>(zl[q], lf, acc[q][n]);
            }
        }
    };
    // steps two at a time; rows past the chunk's end load nothing and count as zeros
    const int n = to - from;
    Step s0, s1;
    auto run = [&](auto clear) {
#pragma unroll
        for (int k = 0; k < NT; ++k) acc[0][k] = acc[1][k] = f32x4{0.f, 0.f, 0.f, 0.f};
        load(s0, 0);
        load(s1, 32);
        put(s0, 0, 0);
        for (int p = 0; p < n; p += 64) {
            __syncthreads();
            if (p + 64 < n) load(s0, p + 64);
            use(0, clear);
            put(s1, 1, p + 32);
            __syncthreads();
            if (p + 64 < n) load(s1, p + 96);
            use(1, clear);
            if (p + 64 < n) put(s0, 0, p + 64);
        }
    };
    run(std::false_type{});
    // where a sum is infinite or NaN a second time, z's infinities with hi alone
    f32x4 nan = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < NT; ++k) nan += (acc[0][k] - acc[0][k]) + (acc[1][k] - acc[1][k]);
    const bool odd = __any((nan[0] + nan[1]) + (nan[2] + nan[3]) != 0.0f);
    if (lane == 0) lds.odd[wave] = odd;
    __syncthreads();
    if (lds.odd[0] | lds.odd[1] | lds.odd[2] | lds.odd[3]) run(std::true_type{});
    // TURNED: lane has column c + l16 and rank numbers 16 n + 4 lg .. + 3; else rank number
    // 16 n + l16 and columns c + 4 lg .. + 3
    const size_t each = (size_t)a.rank * (size_t)a.cols;
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const f32x4 v = DT == DT_F16 ? acc[q][n] * unit : acc[q][n];
            const int c = c0 + wave * 32 + 16 * q + (TURNED ? l16 : 4 * lg), j = 16 * n + (TURNED ? 4 * lg : l16);
            if (c >= a.cols || j >= a.rank) continue;
            const int left = TURNED ? a.rank - j : a.cols - c;
            const size_t at = TURNED ? (size_t)c * (size_t)a.rank + j : (size_t)j * (size_t)a.cols + c;
            float* w = a.work + (size_t)slot * each + at;
            if (left >= 4) {
                if (alone) store_out4(a.out, DT, (size_t)i * each + at, v);
                else __builtin_memcpy(w, &v, 16);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (e < left) {
                        if (alone) store_out(a.out, DT, (size_t)i * each + at + e, v[e]);
                        else w[e] = v[e];
                    }
            }
        }
}

// Both gradients in one launch: grid z 0 is a's, 1 b's.
template <int DT, int NT>
__global__ __launch_bounds__(256) void adapter_gradient16(AdapterArgs a, AdapterArgs b) {
    __shared__ __attribute__((aligned(16))) GradientLds<NT> lds;
    GradientUnits* units = nullptr;
    if constexpr (DT == DT_F16) {
        __shared__ GradientUnits space;
        units = &space;
    }
    if (blockIdx.z == 0) {
        if ((int64_t)blockIdx.x * kGradientCols < a.cols) adapter_gradient_body<DT, NT, false>(a, lds, units);
    } else {
        if ((int64_t)blockIdx.x * kGradientCols < b.cols) adapter_gradient_body<DT, NT, true>(b, lds, units);
    }
}

// An adapter (grid y) of several chunks: the sum of its slots; one without rows: zeros.
template <int DT>
__global__ __launch_bounds__(256) void adapter_join(AdapterArgs p, AdapterArgs q, int slots) {
    const AdapterArgs& a = blockIdx.z == 0 ? p : q;
    const int i = (int)blockIdx.y;
    const AdapterSpan sp = adapter_span(a, i);
    const bool none = sp.to <= sp.from;
    const int first = sp.from / a.chunk + i, last = none ? first : min((sp.to - 1) / a.chunk + i, slots - 1);
    if (!none && first == last) return;
    const size_t each = (size_t)a.rank * (size_t)a.cols;
    for (size_t at = ((size_t)blockIdx.x * 256 + threadIdx.x) * 4; at < each; at += (size_t)gridDim.x * 1024) {
        const int left = (int)min((size_t)4, each - at);
        f32x4 v = {0.f, 0.f, 0.f, 0.f};
        if (!none)
            for (int s = first; s <= last; ++s) {
                const float* w = a.work + (size_t)s * each + at;
                if (left == 4) {
                    f32x4 p;
                    __builtin_memcpy(&p, w, 16);
                    v += p;
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (e < left) v[e] += w[e];
                }
            }
        if (left == 4) store_out4(a.out, DT, (size_t)i * each + at, v);
        else
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (e < left) store_out(a.out, DT, (size_t)i * each + at + e, v[e]);
    }
}

}  // namespace dg
