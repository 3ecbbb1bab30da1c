// kernel_block.h -- products of block-scaled 8-bit matrices, for gfx950.
//
//   C[m][n] = sum_b SA(m,b) SB(n,b) sum_{k in block b} a(m,k) b(n,k)
//
// with blocks of 128 k. The inner sums run on the matrix cores from a zero accumulator;
// each block's sum is then multiplied by both scales and added in fp32, since the scales
// are arbitrary fp32 numbers and the 8-bit instruction's own scales are powers of two.
//
// The codes become fp16 (exactly: e5m2 is fp16's upper byte, e4m3 a subset) in registers, and
// v_mfma_f32_*_f16 has exact products and fp32 sums. The 8-bit instructions, twice as fast,
// do not hold such sums: measured on gfx950 (v_mfma_f32_32x32x16_fp8_fp8 and both f8f6f4
// shapes, bit for bit alike), the products of 8 neighbouring k are cut, towards zero, to whole
// multiples of 2^-13 of the power of two under the largest before they are added, so
// 448 * 448 - 448 * 448 + 1 is 0. 8192 x 4096 x 4096 to bf16 took 128 us on them.
//
// The rows of B are the instruction's first operand, so a lane holds one row m of C and four
// consecutive n per accumulator quad: SA is one value per lane and subtile, and with 128 x 128
// blocks of B both scales are one factor per subtile and block.
//
// The order of k inside a fragment is free as long as both operands share it: the lanes
// with the same row take 16-byte chunks in whichever order is cheapest to read.
#pragma once
#include <type_traits>

#include "device_common.h"
#include "experts.h"
#include "extents.h"
#include "lds_layout.h"

#define DG_LDS_ADDR(a) ((__attribute__((address_space(3))) void*)(uintptr_t)(uint32_t)(a))

namespace dg {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x2 __attribute__((ext_vector_type(2)));

// Source of the chunks that lie past the end of a row.
__device__ const uint32_t block_zeros[4] = {0, 0, 0, 0};

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

// Eight codes as eight fp16 numbers.
template <int T>
__device__ __forceinline__ f16x8 widen8(int lo, int hi) {
    uint32_t w[4];
    if constexpr (T == 0) {
        w[0] = __builtin_bit_cast(uint32_t, (f16x2)__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false));
        w[1] = __builtin_bit_cast(uint32_t, (f16x2)__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true));
        w[2] = __builtin_bit_cast(uint32_t, (f16x2)__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false));
        w[3] = __builtin_bit_cast(uint32_t, (f16x2)__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true));
    } else {  // each code becomes the upper byte of a half (selector 12: zero)
        w[0] = __builtin_amdgcn_perm(0u, (uint32_t)lo, 0x010c000cu);
        w[1] = __builtin_amdgcn_perm(0u, (uint32_t)lo, 0x030c020cu);
        w[2] = __builtin_amdgcn_perm(0u, (uint32_t)hi, 0x010c000cu);
        w[3] = __builtin_amdgcn_perm(0u, (uint32_t)hi, 0x030c020cu);
    }
    return __builtin_bit_cast(f16x8, u32x4{w[0], w[1], w[2], w[3]});
}

// Two codes (of the low or the high half of a dword) as two fp16 numbers.
template <int T>
__device__ __forceinline__ uint32_t widen2(int v, bool high) {
    if constexpr (T == 0)
        return high ? __builtin_bit_cast(uint32_t, (f16x2)__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(v, 1.0f, true))
                    : __builtin_bit_cast(uint32_t, (f16x2)__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(v, 1.0f, false));
    else return __builtin_amdgcn_perm(0u, (uint32_t)v, high ? 0x030c020cu : 0x010c000cu);
}

// One workgroup's piece of a product: rows m0 .. m_end-1 of C (in whole tiles of BM),
// columns from n0, blocks kb0 .. kb0+nkb-1 of k, the last one holding krem elements.
struct BlockTile {
    int m0, m_end, n0;
    int m_live;          // experts: rows from here on are padding
    int expert;
    int kb0, nkb, krem;
    bool bad;            // gradient: rows that start inside a block or end inside 16
};

// Offsets of expert e, kept inside 0 .. P whatever the array holds.
__device__ __forceinline__ void expert_range(const int* offsets, int e, int P, int& lo, int& hi) {
    lo = min(max(offsets[e], 0), P);
    hi = min(max(offsets[e + 1], lo), P);
}

// Linear tile of this workgroup among `total`, each XCD (hardware id mod 8) taking a
// contiguous run; -1 if none is left for it. The grid holds at least `total` workgroups.
__device__ __forceinline__ int xcd_tile(int total) {
    const int bid = (int)blockIdx.x, x = bid & 7, i = bid >> 3;
    const int q = total >> 3, rem = total & 7;
    return i < q + (x < rem ? 1 : 0) ? x * q + min(x, rem) + i : -1;
}

// The expert that owns a tile of BM rows: every wave adds up the experts' tile counts, 64
// experts at a time. Returns false when the grid has no tile for this workgroup.
template <int BM>
__device__ __forceinline__ bool expert_tile(const BlockArgs& g, BlockTile& t) {
    const int lane = threadIdx.x & 63;
    int total = 0;
    for (int64_t e0 = 0; e0 < g.E; e0 += 64) {
        int lo = 0, hi = 0;
        if (e0 + lane < g.E) expert_range(g.offsets, (int)(e0 + lane), g.M, lo, hi);
        int n = pieces<BM>(hi - lo);
#pragma unroll
        for (int d = 32; d; d >>= 1) n += __shfl_xor(n, d);
        total = capped_sum(total, n, g.tiles_m);  // a plan's never pass tiles_m, overlapping offsets may
    }
    total = __builtin_amdgcn_readfirstlane(total);
    const int id = xcd_tile(total * g.tiles_n);
    if (id < 0) return false;
    const int q = id / g.tiles_n;  // lies in the tiles of the wanted expert, as all of its row tiles have tiles_n columns
    int before = 0;
    for (int64_t e0 = 0; e0 < g.E; e0 += 64) {
        int lo = 0, hi = 0;
        if (e0 + lane < g.E) expert_range(g.offsets, (int)(e0 + lane), g.M, lo, hi);
        const int n = pieces<BM>(hi - lo);
        int sum = n;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int v = __shfl_up(sum, d);
            if (lane >= d) sum += v;
        }
        const unsigned long long hit = __ballot(q < before + sum);
        if (hit) {
            const int l = __builtin_ctzll(hit);
            const int first = __builtin_amdgcn_readlane(before + sum - n, l);
            const int tiles = __builtin_amdgcn_readlane(n, l);
            int tm, tn;
            raster(id - first * g.tiles_n, tiles, g.tiles_n, min(g.group_m, tiles), tm, tn);
            t.expert = (int)(e0 + l);
            const int base = __builtin_amdgcn_readlane(lo, l);
            t.m0 = base + tm * BM;
            t.m_end = __builtin_amdgcn_readlane(hi, l);
            t.m_live = min(t.m_end, base + max(__builtin_amdgcn_readfirstlane(g.counts[t.expert]), 0));
            t.n0 = tn;  // in tiles; the caller scales it
            return true;
        }
        before += __builtin_amdgcn_readlane(sum, 63);
    }
    return false;
}

// Narrows a tile to this workgroup's slice of K (grid y), whose sums go to its plane of the
// workspace in fp32.
__device__ __forceinline__ void split_k(BlockArgs& g, BlockTile& t) {
    if (g.k_split <= 1) return;
    t.kb0 = (int)blockIdx.y * g.kb_chunk;
    const int left = t.nkb - t.kb0;
    if (left > g.kb_chunk) {
        t.nkb = g.kb_chunk;
        t.krem = kBlock;
    } else {
        t.nkb = left;
    }
    g.C = g.work + (size_t)blockIdx.y * (size_t)g.work_slice;
    g.ldc = g.work_ld;
    g.out_dt = DT_F32;
}

// The tile of this workgroup; false when there is none (the caller still takes part in
// clearing the rows past the last expert).
template <int BM, int BN>
__device__ __forceinline__ bool block_tile_of(BlockArgs& g, BlockTile& t) {
    t.bad = false;
    t.expert = 0;
    t.kb0 = 0;
    t.nkb = pieces<kBlock>(g.K);
    t.krem = g.K - (t.nkb - 1) * kBlock;
    t.m_end = g.M;
    t.m_live = g.M;
    if (g.mode == BLOCK_EXPERTS) {
        if (!expert_tile<BM>(g, t)) return false;
        t.n0 *= BN;
        if (t.m0 >= t.m_live || g.a_rows == 0) t.nkb = 0;  // nothing but padding: zeros, and nothing is read
        g.B += (size_t)t.expert * (size_t)g.stride_b;
        g.SB += (size_t)t.expert * (size_t)g.stride_sb;
        return true;
    }
    const int per = g.tiles_m * g.tiles_n;
    int tm, tn;
    if (g.mode == BLOCK_PLAIN && g.M % BM != 0 && g.tiles_m > 1) {
        // tiles of the cut last row, which are less work, start last on each XCD: in front of
        // whole ones they would leave those to a round of their own
        const int x = (int)blockIdx.x & 7, i = (int)blockIdx.x >> 3;
        const int whole = per - g.tiles_n, hq = whole >> 3, hr = whole & 7, q = per >> 3, r = per & 7;
        const int mine = hq + (x < hr ? 1 : 0);
        if (i < mine) {
            raster(x * hq + min(x, hr) + i, g.tiles_m - 1, g.tiles_n, min(g.group_m, g.tiles_m - 1), tm, tn);
        } else {
            tm = g.tiles_m - 1;
            tn = (x * q + min(x, r)) - (x * hq + min(x, hr)) + i - mine;
        }
        split_k(g, t);
        t.m0 = tm * BM;
        t.n0 = tn * BN;
        return true;
    }
    int id;
    if (g.mode == BLOCK_GRADIENT) {
        // each XCD takes a run of every expert's tiles, row by row, so that experts of many and
        // of few rows are shared out evenly; a run reads its own rows of A and all of B (the
        // experts in turn to the XCDs: 350 us against 298 at 64 experts of 20 to 2310 rows)
        const int x = (int)blockIdx.x & 7, i = (int)blockIdx.x >> 3, q = per >> 3, r = per & 7, most = (per + 7) >> 3;
        t.expert = i / most;
        const int k = i - t.expert * most;
        if (k >= q + (x < r ? 1 : 0)) return false;
        id = x * q + min(x, r) + k;
        int lo, hi;
        expert_range(g.offsets, t.expert, g.K, lo, hi);
        lo = __builtin_amdgcn_readfirstlane(lo);
        hi = __builtin_amdgcn_readfirstlane(hi);
        t.bad = ((lo & (kBlock - 1)) != 0 || (hi & 15) != 0) && hi > lo;  // chunks are 16 bytes
        t.kb0 = lo / kBlock;
        t.nkb = t.bad ? 0 : pieces<kBlock>(hi - lo);
        t.krem = hi - lo - (t.nkb - 1) * kBlock;
        g.C = static_cast<char*>(g.C) + (size_t)t.expert * (size_t)g.stride_c * (g.out_dt == DT_F32 ? 4 : 2);
    } else {
        id = xcd_tile((int)gridDim.x);
        split_k(g, t);
    }
    raster(id, g.tiles_m, g.tiles_n, g.group_m, tm, tn);
    t.m0 = tm * BM;
    t.n0 = tn * BN;
    return true;
}

// Row of A for row m of C, or -1 for a row of zeros.
__device__ __forceinline__ int block_a_row(const BlockArgs& g, const BlockTile& t, int m) {
    if (g.mode != BLOCK_EXPERTS) return m < t.m_end ? m : -1;
    if (m >= t.m_live) return -1;
    const int r = g.rows ? g.rows[m] : m;
    return r >= 0 && r < g.a_rows ? r : -1;
}

// Columns n .. n+3 of row m of C (columns at or past N skipped).
__device__ __forceinline__ void block_store4(const BlockArgs& g, int m, int n, f32x4 v) {
    const size_t at = (size_t)m * (size_t)g.ldc + n;
    if (n + 4 <= g.N) {
        store_out4(g.C, g.out_dt, at, v);
        return;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (n + e < g.N) store_out(g.C, g.out_dt, at + e, v[e]);
}

// Two fp32 values as two 16-bit ones of type DT, the first in the low half.
template <int DT>
__device__ __forceinline__ uint32_t pack16(float x, float y) {
    if constexpr (DT == DT_F16)
        return (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)x) | ((uint32_t)__builtin_bit_cast(uint16_t, (_Float16)y) << 16);
    else return (uint32_t)f32_to_bf16_rne(x) | ((uint32_t)f32_to_bf16_rne(y) << 16);
}

// Whether row m of C (below m_end) is computed: the others, padding, become zeros. One bit a lane.
__device__ __forceinline__ uint64_t live_rows(const BlockArgs& g, const BlockTile& t, int first) {
    if (g.mode != BLOCK_EXPERTS) return ~0ull;
    const int m = first + ((int)threadIdx.x & 63);
    return __ballot(m < t.m_end && block_a_row(g, t, m) >= 0);
}

// Zeros in the rows past the last expert's, spread over the whole grid.
__device__ __forceinline__ void clear_tail(const BlockArgs& g) {
    const int first = min(max(g.offsets[g.E], 0), g.M);
    stride_walk((int64_t)first + blockIdx.x, g.M, gridDim.x, [&](int m) {
        stride_walk(threadIdx.x * 4, g.N, blockDim.x * 4, [&](int n) { block_store4(g, m, n, f32x4{0, 0, 0, 0}); });
    });
}

// 16 bytes of a row from p, of which the first `valid` lie inside it.
__device__ __forceinline__ u32x4 load_codes(const uint8_t* p, int valid) {
    u32x4 v = {0, 0, 0, 0};
    if (valid >= 16) {
        __builtin_memcpy(&v, p, 16);
    } else if (valid > 0) {
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            uint32_t x = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (w * 4 + e < valid) x |= (uint32_t)p[w * 4 + e] << (8 * e);
            v[w] = x;
        }
    }
    return v;
}

// Whether, in the tile's blocks, some row's scale (lane: row r of A) and B's, one for the whole
// tile, multiply to no normal fp32 number though neither is zero. Their product serves as one
// factor otherwise; here the scaled sums may be normal numbers all the same.
__device__ __forceinline__ bool odd_scales(const BlockArgs& g, const BlockTile& t, int r) {
    const float* a = g.SA + (size_t)(r >> g.a_shift) * (size_t)g.sa_row + (size_t)t.kb0 * (size_t)g.sa_blk;
    const float* b = g.SB + (size_t)(t.n0 >> g.b_shift) * (size_t)g.sb_row + (size_t)t.kb0 * (size_t)g.sb_blk;
    bool odd = false;
    for (int kb = 0; kb < t.nkb; ++kb) {
        const float x = a[(size_t)kb * (size_t)g.sa_blk], y = b[(size_t)kb * (size_t)g.sb_blk];
        odd |= !__builtin_amdgcn_classf(x * y, 0x108) & (x != 0.0f) & (y != 0.0f);
    }
    return __ballot(odd) != 0;
}

// A wave's 64 x 64 tile of C, at (m, n) of its workgroup's, from the codes in global memory, for
// 16-byte aligned rows and one scale of B for the tile: each block's sum by A's scale and then by
// B's. For scales out of the ordinary only, so nothing is done for speed.
template <int TA, int TB>
__device__ __forceinline__ void block_again(const BlockArgs& g, const BlockTile& t, int m, int n, int l16, int lg,
                                            f32x4 (&acc)[4][4]) {
    auto codes = [&](const uint8_t* p, int rem) {  // chunks lg and lg + 4 of a row
        u32x4 x = {0, 0, 0, 0}, y = {0, 0, 0, 0};
        if (16 * lg < rem) __builtin_memcpy(&x, p + 16 * lg, 16);
        if (64 + 16 * lg < rem) __builtin_memcpy(&y, p + 64 + 16 * lg, 16);
        return i32x8{(int)x[0], (int)x[1], (int)x[2], (int)x[3], (int)y[0], (int)y[1], (int)y[2], (int)y[3]};
    };
    const float* const sb = g.SB + (size_t)(t.n0 >> g.b_shift) * (size_t)g.sb_row;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
#pragma unroll 1
    for (int kb = t.kb0; kb < t.kb0 + t.nkb; ++kb) {
        const int rem = kb - t.kb0 == t.nkb - 1 ? t.krem : kBlock;
        const float b_scale = sb[(size_t)kb * (size_t)g.sb_blk];
        i32x8 b[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int row = min(t.n0 + n + j * 16 + l16, g.N - 1);
            b[j] = codes(g.B + (size_t)row * (size_t)g.ldb + (size_t)kb * kBlock, rem);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = max(block_a_row(g, t, min(t.m0 + m + i * 16 + l16, t.m_end - 1)), 0);
            const i32x8 a = codes(g.A + (size_t)row * (size_t)g.lda + (size_t)kb * kBlock, rem);
            const float s = g.SA[(size_t)(row >> g.a_shift) * (size_t)g.sa_row + (size_t)kb * (size_t)g.sa_blk];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                f32x4 part = {0, 0, 0, 0};
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    part = __builtin_amdgcn_mfma_f32_16x16x32_f16(widen8<TB>(b[j][2 * u], b[j][2 * u + 1]),
                                                                  widen8<TA>(a[2 * u], a[2 * u + 1]), part, 0, 0, 0);
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][j][e] = fmaf(part[e] * s, b_scale, acc[i][j][e]);
            }
        }
    }
}

// ---------------------------------------------------------------------------- aligned rows
// (64 WM) x 128 tiles for 16-byte aligned rows on 2 WM waves of 64 x 64 (WM = 2, S = 2: two
// workgroups to a compute unit; with B turned WM = 4, S = 3: one), each 4 x 4 tiles of
// v_mfma_f32_16x16x32_f16, four instructions to a block of k. Codes are copied
// straight to LDS (S stages of rows of 128 bytes, 16-byte chunk c of row r at c ^ ((r >> 1) & 7),
// so that the phases of a read cover all banks) S - 1 blocks ahead and widened in
// the fragments: a wave holds the block's four fragments of B as halves (64 registers),
// widens those of A one ahead and, behind the last use of each of B's, the next block's.
// Vector and matrix instructions are even (with a scale for each row of B: 256 of 4 cycles
// and 64 of 16 for each wave and block); widening on the way into LDS instead, as the next
// kernel does, halves the conversions, but its writes and conflicts keep LDS busy longer than
// the matrix cores. 8192 x 4096 x 4096 to bf16: 252 us, 1090 TFLOP/s (a library's product in
// bf16 reaches 1290 at 8192 x 8192 x 8192), 49% of the SIMDs' cycles in matrix instructions and
// 63% in vector ones; 2056 x 4000 x 8176 to fp32, scales for each row of B: 149 us.
// TRB: B is stored with its rows adjacent; its stage then holds 128 rows of k, 16-byte chunk c
// of row k at c ^ (((k >> 1) & 3) | ((k >> 2) & 4)), and 8 k of a row of B come from
// ds_read_b64_tr_b8: in each 16 lanes, lane i addresses 8 bytes of row k0 + i/2 at half i%2 of a
// chunk and receives column i of the 8 rows. The 32 lanes of a phase see 16 rows of k, two groups
// of 8 that lie 16 apart, at one chunk, in 16 different places.
template <int TA, int TB, bool BROW, int WM, int S, bool TRB = false>
__global__ __launch_bounds__(WM * 128, 2) void block_direct(BlockArgs g) {
    constexpr int NW = 2 * WM, BM = 64 * WM, BN = 128, FM = 4, FN = 4;
    constexpr int CB = BN / 8 / NW;  // copies of 1 KB (8 rows) of B for each wave; 4 of A
    constexpr int AHEAD = WM == 2 || TRB ? 1 : 2;  // fragments of codes read ahead (as registers allow)
    constexpr int STAGE_A = BM * kBlock, STAGE_B = BN * kBlock, STAGE_S = (BM + BN) * 4;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[S * (STAGE_A + STAGE_B + STAGE_S)];
    uint8_t* const sA = lds;
    uint8_t* const sB = lds + S * STAGE_A;
    float* const fS = reinterpret_cast<float*>(lds + S * (STAGE_A + STAGE_B));
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 1, wn = wave & 1;
    const int l16 = lane & 15, lg = lane >> 4;

    BlockTile t;
    const bool any = block_tile_of<BM, BN>(g, t);
    if (g.mode == BLOCK_EXPERTS) clear_tail(g);
    if (!any) return;

    const uint8_t* ba = g.A + (size_t)t.kb0 * kBlock;
    const size_t step_b = TRB ? (size_t)kBlock * (size_t)g.ldb : kBlock;
    const uint8_t* bb = g.B + (size_t)t.kb0 * step_b;
    uint32_t oa[4], ob[CB];
    int ka[2], kb2[2];  // the k of a chunk: the same for every other copy
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const int row = (wave * 4 + c) * 8 + (lane >> 3);
        ka[c & 1] = ((lane & 7) ^ ((row >> 1) & 7)) * 16;
        const int r = max(block_a_row(g, t, min(t.m0 + row, t.m_end - 1)), 0);
        oa[c] = (uint32_t)r * (uint32_t)g.lda + (uint32_t)ka[c & 1];
    }
#pragma unroll
    for (int c = 0; c < CB; ++c) {
        const int row = (wave * CB + c) * 8 + (lane >> 3);
        if constexpr (TRB) {  // rows of k at chunk n; past N (a multiple of 16) the last, which is not stored
            const int n = t.n0 + ((lane & 7) ^ (((row >> 1) & 3) | ((row >> 2) & 4))) * 16;
            // n is the same for the copies of 16 rows: rows 8 c are added at the copy (registers)
            ob[c >> 1] = (uint32_t)(row - 8 * c) * (uint32_t)g.ldb + (uint32_t)min(n, g.N - 16);
        } else {
            kb2[c & 1] = ((lane & 7) ^ ((row >> 1) & 7)) * 16;
            ob[c] = (uint32_t)min(t.n0 + row, g.N - 1) * (uint32_t)g.ldb + (uint32_t)kb2[c & 1];
        }
    }
    // scales: the first WM waves copy those of A's rows, two those of B's, the others none
    const bool scales = wave < WM + 2;
    const float* ps;
    int64_t ps_step;
    if (wave < WM) {
        const int r = max(block_a_row(g, t, min(t.m0 + tid, t.m_end - 1)), 0);
        ps = g.SA + (size_t)(r >> g.a_shift) * (size_t)g.sa_row + (size_t)t.kb0 * (size_t)g.sa_blk;
        ps_step = g.sa_blk;
    } else {
        const int n = min(t.n0 + (tid - BM) % BN, g.N - 1);
        ps = g.SB + (size_t)(n >> g.b_shift) * (size_t)g.sb_row + (size_t)t.kb0 * (size_t)g.sb_blk;
        ps_step = g.sb_blk;
    }
    const uint32_t dA = (uint32_t)reinterpret_cast<uintptr_t>(DG_LDSV(sA)) + (uint32_t)wave * 4096u;
    const uint32_t dB = (uint32_t)reinterpret_cast<uintptr_t>(DG_LDSV(sB)) + (uint32_t)wave * (CB * 1024u);
    const uint32_t dS = (uint32_t)reinterpret_cast<uintptr_t>(DG_LDSV(fS)) + (uint32_t)wave * 256u;
    auto issue = [&](int kb, int st) {  // block kb into stage st: 4 + CB (+ 1) copies
        const size_t k = (size_t)kb * kBlock;
        const int rem = kb < t.nkb - 1 ? kBlock : t.krem;
        if (scales) __builtin_amdgcn_global_load_lds(DG_GLB(ps), DG_LDS_ADDR(dS + st * STAGE_S), 4, 0, 0);
        ps += ps_step;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const void* a = ka[c & 1] < rem ? static_cast<const void*>(ba + k + oa[c]) : block_zeros;
            __builtin_amdgcn_global_load_lds(DG_GLB(a), DG_LDS_ADDR(dA + st * STAGE_A + c * 1024u), 16, 0, 0);
        }
#pragma unroll
        for (int c = 0; c < CB; ++c) {
            const bool in = (TRB ? (wave * CB + c) * 8 + (lane >> 3) : kb2[c & 1]) < rem;
            const void* b = in ? static_cast<const void*>(bb + (size_t)kb * step_b +
                                                            (TRB ? ob[c >> 1] + (uint32_t)(8 * c) * (uint32_t)g.ldb : ob[c]))
                              : block_zeros;
            __builtin_amdgcn_global_load_lds(DG_GLB(b), DG_LDS_ADDR(dB + st * STAGE_B + c * 1024u), 16, 0, 0);
        }
    };
    // this wave's copies but those of the `behind` newest blocks have landed (0 or S - 2), and
    // after the barrier everybody's
    auto published = [&](bool behind) {
        if (S > 2 && behind) {
            if (scales) asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((S - 2) * (5 + CB)) : "memory");
            else asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((S - 2) * (4 + CB)) : "memory");
        } else {
            asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
        }
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    };

    // a lane's 32 codes of a fragment row: chunks lg and lg + 4, 16 codes each; halves u = 0 .. 3
    const int off = l16 * kBlock + ((lg ^ ((l16 >> 1) & 7)) << 4);
    auto codes_of = [&](const uint8_t* base) {
        const u32x4 x = *reinterpret_cast<const u32x4*>(base + off);
        const u32x4 y = *reinterpret_cast<const u32x4*>(base + (off ^ 64));
        return i32x8{(int)x[0], (int)x[1], (int)x[2], (int)x[3], (int)y[0], (int)y[1], (int)y[2], (int)y[3]};
    };
    const uint8_t* const aw = sA + wm * 64 * kBlock;
    // fragment j of B from a stage
    const int tr_row = (l16 >> 1) + 16 * lg, tr_swz = ((l16 >> 2) & 3) | ((lg & 1) << 2);
    auto b_codes = [&](int stage, int j) {
        const uint8_t* b = sB + stage * STAGE_B;
        if constexpr (TRB) {
            // 8 rows of k from 64 (u / 2) + 16 lg + 8 (u % 2); the rows' (k >> 1) & 3 and bit 4 are the lane's
            const uint8_t* p = b + tr_row * kBlock + (((wn * 4 + j) ^ tr_swz) << 4) + (l16 & 1) * 8;
            i32x8 r;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const i32x2 v = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
                    DG_LDS_PTR(i32x2, p + (64 * (u >> 1) + 8 * (u & 1)) * kBlock));
                r[2 * u] = v[0];
                r[2 * u + 1] = v[1];
            }
            return r;
        } else {
            return codes_of(b + (wn * 64 + j * 16) * kBlock);
        }
    };
    const float* const fa = fS + wm * 64 + l16;
    const float* const fb = fS + BM + wn * 64;

    f32x4 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = t.bad ? f32x4{1, 1, 1, 1} * __builtin_nanf("") : f32x4{0, 0, 0, 0};
    const bool active = t.m0 + wm * 64 < t.m_end;  // this wave has rows of C

    // lanes (rows of the wave's tile) that met a product of scales that is no normal number
    uint64_t odd = 0;
    float row_scale = 0;
    u32x4 af[4], bf[FN][4];    // halves: step u (32 k) of a fragment
    i32x8 raw[2], rawb[2];     // codes
    f32x4 part[2][FN], sb[BROW ? FN : 1];
    float sa[2];
    auto read_sb = [&](int st) {
        const float* f = fb + st * (BM + BN);
        if constexpr (BROW) {
#pragma unroll
            for (int j = 0; j < FN; ++j) sb[j] = *reinterpret_cast<const f32x4*>(f + j * 16 + lg * 4);
        } else {
            sb[0][0] = f[0];
        }
    };
    // one number of a part, scaled and added: by A's scale and then by B's, or, where B has one for
    // the whole tile, by their product, a fifth fewer vector instructions (8192 x 4096 x 4096: 244
    // against 264 us)
    auto add1 = [&](int i, int q, float s) {
        const int j = q >> 2, e = q & 3;
        if constexpr (BROW) acc[i][j][e] = fmaf(part[i & 1][j][e] * s, sb[j][e], acc[i][j][e]);
        else acc[i][j][e] = fmaf(part[i & 1][j][e], s, acc[i][j][e]);
    };
    // dword d (two codes) of step u of a fragment
    auto widen_a = [&](const i32x8& r, int u, int d) { af[u][d] = widen2<TA>(r[2 * u + (d >> 1)], d & 1); };
    auto widen_b = [&](const i32x8& r, int j, int u, int d) { bf[j][u][d] = widen2<TB>(r[2 * u + (d >> 1)], d & 1); };
    auto mfma = [&](int i, int j, int u) {
        part[i & 1][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, bf[j][u]),
                                                                __builtin_bit_cast(f16x8, af[u]),
                                                                u ? part[i & 1][j] : f32x4{0, 0, 0, 0}, 0, 0, 0);
    };

    if (t.nkb > 0) {
        issue(0, 0);
        if (t.nkb > 1) issue(1, 1);
        if (S > 2 && t.nkb > 2) {
            issue(2, 2);
            asm volatile("s_waitcnt vmcnt(%0)" ::"n"(2 * (4 + CB)) : "memory");  // at least block 0's
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
        } else {
            published(false);
        }
        if (active) {
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                const i32x8 r = b_codes(0, j);
#pragma unroll
                for (int q = 0; q < 16; ++q) widen_b(r, j, q >> 2, q & 3);
            }
            raw[0] = codes_of(aw);
            if (AHEAD > 1) raw[1] = codes_of(aw + 16 * kBlock);
            sa[0] = fa[0];
#pragma unroll
            for (int q = 0; q < 16; ++q) widen_a(raw[0], q >> 2, q & 3);
            read_sb(0);
        }
    }
    // A step is 16 instructions of the matrix core, and behind each a few of the vector unit
    // that run in its shadow, pinned there: a number of the step before's part (first of the
    // block: of the last block's) scaled and added, two codes of the next fragment widened
    // over those just used. (In one piece each, with the other wave of the SIMD left to fill
    // the gaps, the two units hardly overlapped: 5300 cycles a block for 2048 of matrix and
    // 2400 of vector instructions.)
    float s_last = 0;  // factor of the last step's part
    int st = 0;
    for (int kb = 0; kb < t.nkb; ++kb) {
        const int next = st + 1 == S ? 0 : st + 1;
        if (active) {
#pragma unroll
            for (int i = 0; i < FM - 1; ++i) {
                // codes AHEAD fragments ahead; the scale of the next
                if (i + AHEAD < FM) raw[(i + AHEAD) & 1] = codes_of(aw + st * STAGE_A + (i + AHEAD) * 16 * kBlock);
                const float s = sa[i & 1];
                sa[(i + 1) & 1] = fa[st * (BM + BN) + (i + 1) * 16];
#pragma unroll
                for (int q = 0; q < 16; ++q) {
                    mfma(i, q & 3, q >> 2);
                    if (i > 0) add1(i - 1, q, s_last);
                    else if (kb > 0) add1(FM - 1, q, s_last);
                    if (q >= 4) widen_a(raw[(i + 1) & 1], (q >> 2) - 1, q & 3);
                    __builtin_amdgcn_sched_barrier(0);
                }
#pragma unroll
                for (int q = 0; q < 4; ++q) widen_a(raw[(i + 1) & 1], 3, q);
                if (i == 0) {
                    read_sb(st);
                    if constexpr (!BROW) row_scale = fS[st * (BM + BN) + wm * 64 + lane];
                }
                s_last = BROW ? s : s * sb[0][0];
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        // in the shadow of the wait for the next block
        if constexpr (!BROW) odd |= __ballot(!__builtin_amdgcn_classf(row_scale * sb[0][0], 0x108));
        if (kb + 1 < t.nkb) {
            // block kb + 1 is there, and everybody has read the last of block kb from its stage
            published(kb + S - 1 < t.nkb);
            if (kb + S < t.nkb) issue(kb + S, st);
        }
        if (active) {
            // past the end of k the reads find old data, which nothing uses
            rawb[0] = b_codes(next, 0);
            rawb[1] = b_codes(next, 1);
            const float s = sa[(FM - 1) & 1];
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int j = 0; j < FN; ++j) {
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    mfma(FM - 1, j, u);
                    add1(FM - 2, 4 * j + u, s_last);
                    if (j > 0) {
#pragma unroll
                        for (int d = 0; d < 4; ++d) widen_b(rawb[(j - 1) & 1], j - 1, u, d);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
                if (j == 1) rawb[0] = b_codes(next, 2);
                if (j == 2) {
                    rawb[1] = b_codes(next, 3);
                    raw[0] = codes_of(aw + next * STAGE_A);
                    if (AHEAD > 1) raw[1] = codes_of(aw + next * STAGE_A + 16 * kBlock);
                    sa[0] = fa[next * (BM + BN)];
                }
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int q = 0; q < 16; ++q) widen_b(rawb[1], 3, q >> 2, q & 3);
#pragma unroll
            for (int q = 0; q < 16; ++q) widen_a(raw[0], q >> 2, q & 3);
            s_last = BROW ? s : s * sb[0][0];
            __builtin_amdgcn_sched_barrier(0);
        }
        st = next;
    }
    if (active && t.nkb > 0) {
#pragma unroll
        for (int q = 0; q < 16; ++q) add1(FM - 1, q, s_last);
    }

    // lanes counted anew, so that nothing of this waits in registers through the loop
    int at = (int)__builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u));
    asm("" : "+v"(at));
    const int r16 = at & 15, rg = at >> 4;
    if constexpr (!BROW) {
        if (active && odd != 0 && odd_scales(g, t, max(block_a_row(g, t, min(t.m0 + wm * 64 + at, t.m_end - 1)), 0)))
            block_again<TA, TB>(g, t, wm * 64, wn * 64, r16, rg, acc);
    }
    const uint64_t live = live_rows(g, t, t.m0 + wm * 64);
    if (g.out_dt != DT_F32) {
        // ---- C of 16 bits through LDS, so that each store instruction writes whole 128-byte
        // rows: the wave's 64 rows, 16-byte chunks permuted by (row >> 1) & 7
        __builtin_amdgcn_s_barrier();  // every wave has read its last fragments
        asm volatile("" ::: "memory");
        if (!active) return;
        uint8_t* const stage = lds + wave * (64 * 128);
        auto to_lds = [&](auto dt) {
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FN; ++j) {
                    const f32x4 v = acc[i][j];
                    const u32x2 h = {pack16<decltype(dt)::value>(v[0], v[1]), pack16<decltype(dt)::value>(v[2], v[3])};
                    *reinterpret_cast<u32x2*>(stage + (i * 16 + r16) * 128 + (((2 * j + (rg >> 1)) ^ ((r16 >> 1) & 7)) << 4) +
                                              (rg & 1) * 8) = h;
                }
        };
        if (g.out_dt == DT_F16) to_lds(std::integral_constant<int, DT_F16>{});
        else to_lds(std::integral_constant<int, DT_BF16>{});
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        uint16_t* const C = static_cast<uint16_t*>(g.C);
        const int n = t.n0 + wn * 64 + (at & 7) * 8;
#pragma unroll 4
        for (int p = 0; p < 8; ++p) {
            const int row = p * 8 + (at >> 3), m = t.m0 + wm * 64 + row;
            u32x4 v = *reinterpret_cast<const u32x4*>(stage + row * 128 + (((at & 7) ^ ((row >> 1) & 7)) << 4));
            if (!((live >> row) & 1)) v = u32x4{0, 0, 0, 0};
            if (m >= t.m_end || n >= g.N) continue;
            uint16_t* const c = C + (size_t)m * (size_t)g.ldc + n;
            if (n + 8 <= g.N) {
                __builtin_memcpy(c, &v, 16);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (n + e < g.N) c[e] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
            }
        }
        return;
    }
    // ---- fp32 C from the registers: a lane's four columns are 16 bytes, four lanes' 64 of a row
    if (!active) return;
    float* const C = static_cast<float*>(g.C);
    const bool whole = t.n0 + BN <= g.N;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        const int m = t.m0 + wm * 64 + i * 16 + r16;
        const bool zero = !((live >> (i * 16 + r16)) & 1);
        float* const c = C + (size_t)m * (size_t)g.ldc + t.n0 + wn * 64 + rg * 4;
        if (m >= t.m_end) continue;
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            const f32x4 v = zero ? f32x4{0, 0, 0, 0} : acc[i][j];
            if (whole) {
                __builtin_memcpy(c + j * 16, &v, 16);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (t.n0 + wn * 64 + j * 16 + rg * 4 + e < g.N) c[j * 16 + e] = v[e];
            }
        }
    }
}

// ---------------------------------------------------------------------------- any layout
// 128 x 128 tiles for rows at any byte address and for operands with adjacent rows, on 2 x 2
// tiles of v_mfma_f32_32x32x16_f16 for each wave: the codes go through registers and are
// widened on their way into LDS, once for the whole workgroup. LDS holds one
// block of k (64 KB of halves, so that two workgroups share a compute unit and each fills
// the other's waits), the next block's codes wait in registers.
//
// Rows of 256 bytes, 16-byte chunk c of row r at c ^ (r & 15): the 16 lanes of a read phase
// see one chunk of 16 rows that differ in the low bits, so all places. TR: bit 0, B is
// stored with its rows adjacent (element (n, k) at k*ldb + n), bit 1 the same for A; such an
// operand is held as 128 rows of k, its 32-byte units of 16 rows permuted by 2 (k & 3), and
// read through ds_read_b64_tr_b16. 8192 x 4096 x 4090 to bf16: 354 us, LDS busy with conflicts
// in a third of its active cycles.
template <int TA, int TB, bool BROW, int TR>
__global__ __launch_bounds__(256, 2) void block_staged(BlockArgs g) {
    constexpr int BM = 128, BN = 128, FM = 2, FN = 2, ROW = 68;
    constexpr bool TRB = (TR & 1) != 0, TRA = (TR & 2) != 0;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * 128 * 256 + (BM + BN) * 4];
    uint8_t* const sA = lds;
    uint8_t* const sB = lds + 128 * 256;
    float* const fS = reinterpret_cast<float*>(lds + 2 * 128 * 256);
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 1, wn = wave & 1;
    const int l32 = lane & 31, lh = lane >> 5, l16 = lane & 15, lg = lane >> 4;

    BlockTile t;
    const bool any = block_tile_of<BM, BN>(g, t);
    if (g.mode == BLOCK_EXPERTS) clear_tail(g);
    if (!any) return;

    // ---- this thread's codes: chunk tid & 7 of rows (tid >> 3) + 32 c, c = 0 .. 3; rows of C
    // and columns of k, or the other way round for an operand with adjacent rows
    const int chunk = (tid & 7) * 16;
    const uint8_t* pa[4];
    const uint8_t* pb[4];
    const size_t step_a = TRA ? (size_t)kBlock * (size_t)g.lda : kBlock;
    const size_t step_b = TRB ? (size_t)kBlock * (size_t)g.ldb : kBlock;
    const int va = g.M - t.m0 - chunk, vb = g.N - t.n0 - chunk;  // bytes of a transposed chunk inside the matrix
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const int row = (tid >> 3) + 32 * c;
        if constexpr (TRA) {
            pa[c] = g.A + ((size_t)t.kb0 * kBlock + row) * (size_t)g.lda + (t.m0 + chunk);
        } else {
            const int r = max(block_a_row(g, t, min(t.m0 + row, t.m_end - 1)), 0);
            pa[c] = g.A + (size_t)r * (size_t)g.lda + (size_t)t.kb0 * kBlock + chunk;
        }
        if constexpr (TRB) pb[c] = g.B + ((size_t)t.kb0 * kBlock + row) * (size_t)g.ldb + (t.n0 + chunk);
        else pb[c] = g.B + (size_t)min(t.n0 + row, g.N - 1) * (size_t)g.ldb + (size_t)t.kb0 * kBlock + chunk;
    }
    const float* ps;
    int64_t ps_step;
    if (wave < 2) {
        const int r = max(block_a_row(g, t, min(t.m0 + tid, t.m_end - 1)), 0);
        ps = g.SA + (size_t)(r >> g.a_shift) * (size_t)g.sa_row + (size_t)t.kb0 * (size_t)g.sa_blk;
        ps_step = g.sa_blk;
    } else {
        const int n = min(t.n0 + tid - 128, g.N - 1);
        ps = g.SB + (size_t)(n >> g.b_shift) * (size_t)g.sb_row + (size_t)t.kb0 * (size_t)g.sb_blk;
        ps_step = g.sb_blk;
    }

    u32x4 ra[4], rb[4];
    float rs;
    auto load = [&](int kb) {
        const int rem = kb == t.nkb - 1 ? t.krem : kBlock;
        rs = *ps;
        ps += ps_step;
        const bool plain = rem == kBlock && (!TRA || t.m0 + BM <= g.M) && (!TRB || t.n0 + BN <= g.N);
        if (plain) {  // whole chunks, without a branch for each
#pragma unroll
            for (int c = 0; c < 4; ++c) __builtin_memcpy(&ra[c], pa[c], 16);
#pragma unroll
            for (int c = 0; c < 4; ++c) __builtin_memcpy(&rb[c], pb[c], 16);
        } else {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int row = (tid >> 3) + 32 * c;
                ra[c] = load_codes(pa[c], TRA ? (row < rem ? va : 0) : rem - chunk);
                rb[c] = load_codes(pb[c], TRB ? (row < rem ? vb : 0) : rem - chunk);
            }
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            pa[c] += step_a;
            pb[c] += step_b;
        }
    };
    auto widen_to = [&](uint8_t* s, u32x4 v, int row, auto type, bool tr) {
        constexpr int T = decltype(type)::value;
        const f16x8 x = widen8<T>((int)v[0], (int)v[1]), y = widen8<T>((int)v[2], (int)v[3]);
        if (tr) {
            uint8_t* p = s + row * 256 + (((tid & 7) ^ (2 * (row & 3))) << 5);
            *reinterpret_cast<f16x8*>(p) = x;
            *reinterpret_cast<f16x8*>(p + 16) = y;
        } else {
            const int at = ((2 * (tid & 7)) ^ (row & 15)) << 4;
            *reinterpret_cast<f16x8*>(s + row * 256 + at) = x;
            *reinterpret_cast<f16x8*>(s + row * 256 + (at ^ 16)) = y;
        }
    };
    auto settle = [&]() {
        fS[tid] = rs;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int row = (tid >> 3) + 32 * c;
            widen_to(sA, ra[c], row, std::integral_constant<int, TA>{}, TRA);
            widen_to(sB, rb[c], row, std::integral_constant<int, TB>{}, TRB);
        }
    };

    // ---- fragments: step u, lane (l32, lh): k 16u + 8lh .. +7 of row l32 of a subtile
    auto frag = [&](const uint8_t* s, int sub, int u) {
        return *reinterpret_cast<const f16x8*>(s + (sub * 32 + l32) * 256 + (((2 * u + lh) ^ l16) << 4));
    };
    auto frag_tr = [&](const uint8_t* s, int sub, int u) {
        const int k = 8 * lh + (l16 >> 2);  // of rows 16u + k and + 4
        const uint8_t* p = s + (16 * u + k) * 256 + (((2 * sub + (lg & 1)) ^ (2 * (k & 3))) << 5) + (l16 & 3) * 8;
        const fp16x4_t x = __builtin_amdgcn_ds_read_tr16_b64_v4f16(DG_LDS_PTR(fp16x4_t, p));
        const fp16x4_t y = __builtin_amdgcn_ds_read_tr16_b64_v4f16(DG_LDS_PTR(fp16x4_t, p + 4 * 256));
        const u32x2 a = __builtin_bit_cast(u32x2, x), b = __builtin_bit_cast(u32x2, y);
        return __builtin_bit_cast(f16x8, u32x4{a[0], a[1], b[0], b[1]});
    };
    auto a_frag = [&](int i, int u) {
        if constexpr (TRA) return frag_tr(sA, wm * FM + i, u);
        else return frag(sA, wm * FM + i, u);
    };
    auto b_frag = [&](int j, int u) {
        if constexpr (TRB) return frag_tr(sB, wn * FN + j, u);
        else return frag(sB, wn * FN + j, u);
    };

    f32x16 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = f32x16{0};
    // subtiles of 32 rows of this wave that hold rows of C
    const int subs = min(max((t.m_end - t.m0 + 31) / 32 - wm * FM, 0), FM);

    if (t.nkb > 0) {
        load(0);
        settle();
    }
    for (int kb = 0; kb < t.nkb; ++kb) {
        __syncthreads();
        if (kb + 1 < t.nkb) load(kb + 1);
        auto block = [&](auto whole_tag) {
            constexpr bool WHOLE = decltype(whole_tag)::value;
            f32x16 part[FM][FN];
            f16x8 af[2][FM], bf[2][FN];
#pragma unroll
            for (int j = 0; j < FN; ++j) bf[0][j] = b_frag(j, 0);
#pragma unroll
            for (int i = 0; i < FM; ++i) af[0][i] = a_frag(i, 0);
#pragma unroll
            for (int u = 0; u < 8; ++u) {
#pragma unroll
                for (int i = 0; i < FM; ++i)
#pragma unroll
                    for (int j = 0; j < FN; ++j) {
                        if (WHOLE || i < subs)
                            part[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(bf[u & 1][j], af[u & 1][i],
                                                                                u ? part[i][j] : f32x16{0}, 0, 0, 0);
                        if (i == 0 && j == 0 && u < 7) {
                            // the next step's fragments, behind the wait for this one's
                            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                            for (int q = 0; q < FN; ++q) bf[(u + 1) & 1][q] = b_frag(q, u + 1);
#pragma unroll
                            for (int q = 0; q < FM; ++q) af[(u + 1) & 1][q] = a_frag(q, u + 1);
                            __builtin_amdgcn_sched_barrier(0);
                        }
                    }
            }
            // A's scale and B's of each row of B; or, where B has one for the tile, both as one factor,
            // unless that is no normal number in some lane: then one after the other too
            float f[FM];
            uint64_t odd = 0;
#pragma unroll
            for (int i = 0; i < FM; ++i) {
                f[i] = fS[wm * 64 + i * 32 + l32];
                if constexpr (!BROW) {
                    f[i] *= fS[BM + wn * 64];
                    odd |= __ballot(!__builtin_amdgcn_classf(f[i], 0x108));
                }
            }
            if (odd != 0) {
#pragma unroll
                for (int i = 0; i < FM; ++i) {
                    const float sa = fS[wm * 64 + i * 32 + l32];
#pragma unroll
                    for (int j = 0; j < FN; ++j) part[i][j] *= sa;
                    f[i] = fS[BM + wn * 64];
                }
            }
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FN; ++j) {
                    if (!(WHOLE || i < subs)) continue;
                    const float* sb = fS + BM + wn * 64 + j * 32 + lh * 4;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        f32x4 t = {1, 1, 1, 1};
                        if constexpr (BROW) t = *reinterpret_cast<const f32x4*>(sb + q * 8);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int r = 4 * q + e;
                            if constexpr (BROW) acc[i][j][r] = fmaf(part[i][j][r] * f[i], t[e], acc[i][j][r]);
                            else acc[i][j][r] = fmaf(part[i][j][r], f[i], acc[i][j][r]);
                        }
                    }
                }
        };
        if (subs == FM) block(std::true_type{});
        else if (subs > 0) block(std::false_type{});
        __syncthreads();
        if (kb + 1 < t.nkb) settle();
    }

    // ---- C through LDS, 32 rows of the wave's 64 columns at a time (no wave reads or writes
    // the operands' stage any more)
    // lanes counted anew, so that nothing of this waits in registers through the loop
    int at = (int)__builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u));
    asm("" : "+v"(at));
    const int r32 = at & 31, rh = at >> 5, r16 = at & 15, rg = at >> 4;
    float* const stage = reinterpret_cast<float*>(lds) + wave * (32 * ROW);
    const int n = t.n0 + wn * 64 + r16 * 4;
    const bool whole = t.n0 + BN <= g.N;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        if (i >= subs) continue;
        const int first = t.m0 + wm * 64 + i * 32;
        const uint64_t live = live_rows(g, t, first);
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                f32x4 v = {acc[i][j][q * 4], acc[i][j][q * 4 + 1], acc[i][j][q * 4 + 2], acc[i][j][q * 4 + 3]};
                if (t.bad) v = f32x4{1, 1, 1, 1} * __builtin_nanf("");
                *reinterpret_cast<f32x4*>(stage + r32 * ROW + j * 32 + q * 8 + rh * 4) = v;
            }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        auto rows_out = [&](auto put) {
#pragma unroll
            for (int p = 0; p < 8; ++p) {
                const int row = p * 4 + rg, m = first + row;
                f32x4 v = *reinterpret_cast<const f32x4*>(stage + row * ROW + r16 * 4);
                if (!((live >> row) & 1)) v = f32x4{0, 0, 0, 0};
                if (m < t.m_end && n < g.N) put((size_t)m * (size_t)g.ldc + n, m, v);
            }
        };
        if (!whole) rows_out([&](size_t, int m, f32x4 v) { block_store4(g, m, n, v); });
        else if (g.out_dt == DT_F32)
            // a weight's gradient is far larger than the codes, which other tiles read again:
            // past the caches (64 experts, 512 rows each, 2048 x 1024: 273 against 279 us)
            rows_out([&](size_t c, int, f32x4 v) { store_passing(static_cast<float*>(g.C) + c, v); });
        else rows_out([&](size_t c, int, f32x4 v) { store_out4(g.C, g.out_dt, c, v); });
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
}

// ---------------------------------------------------------------------------- few rows
// At most 16 * SM rows of A: the time is that of reading B once. A workgroup takes 16 * NT
// rows of B, its NW waves every NW-th block of k, fragments straight from global memory
// (a row's 128 bytes from four lanes); the waves' sums meet in LDS and are added in the
// waves' order. NT = 4 where that leaves enough workgroups: a wave then has four times the
// bytes in flight behind one search for its expert and one reading of A (16 tokens x 4 of 64
// experts of 2048 x 2048: 50 -> 45 us, 3.9 TB/s of their matrices; one token x 4096 x 4096,
// NT = 1: 6 us).
template <int TA, int TB, int SM, int NT, bool DIRECT>
__global__ __launch_bounds__(512) void block_skinny(BlockArgs g) {
    constexpr int NW = 8, BM = 16 * SM, BN = 16 * NT;
    __shared__ f32x4 sums[NW][SM * NT][64];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int l16 = lane & 15, lg = lane >> 4;
    BlockTile t;
    const bool any = block_tile_of<BM, BN>(g, t);
    if (g.mode == BLOCK_EXPERTS) clear_tail(g);
    if (!any) return;

    const uint8_t* pa[SM];
    const float* fa[SM];
    const size_t k0 = (size_t)t.kb0 * kBlock;
#pragma unroll
    for (int i = 0; i < SM; ++i) {
        const int r = max(block_a_row(g, t, min(t.m0 + i * 16 + l16, t.m_end - 1)), 0);
        pa[i] = g.A + (size_t)r * (size_t)g.lda + k0 + lg * 32;
        fa[i] = g.SA + (size_t)(r >> g.a_shift) * (size_t)g.sa_row + (size_t)t.kb0 * (size_t)g.sa_blk;
    }
    const uint8_t* pb[NT];
    const float* fb[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        pb[j] = g.B + (size_t)min(t.n0 + j * 16 + l16, g.N - 1) * (size_t)g.ldb + k0 + lg * 32;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int n = min(t.n0 + j * 16 + lg * 4 + e, g.N - 1);
            fb[j][e] = g.SB + (size_t)(n >> g.b_shift) * (size_t)g.sb_row + (size_t)t.kb0 * (size_t)g.sb_blk;
        }
    }
    auto frag = [&](const uint8_t* p, int rem) {
        u32x4 x, y;
        if constexpr (DIRECT) {
            const uint8_t* z = reinterpret_cast<const uint8_t*>(block_zeros);
            x = *reinterpret_cast<const u32x4*>(rem > 0 ? p : z);
            y = *reinterpret_cast<const u32x4*>(rem > 16 ? p + 16 : z);
        } else {
            x = load_codes(p, rem);
            y = load_codes(p + 16, rem - 16);
        }
        return i32x8{(int)x[0], (int)x[1], (int)x[2], (int)x[3], (int)y[0], (int)y[1], (int)y[2], (int)y[3]};
    };
    f32x4 acc[SM][NT];
#pragma unroll
    for (int i = 0; i < SM; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
#pragma unroll(DIRECT ? (NT == 1 ? 4 : 2) : 1)
    for (int kb = wave; kb < t.nkb; kb += NW) {
        const int rem = (kb == t.nkb - 1 ? t.krem : kBlock) - lg * 32;
        i32x8 bf[NT];
        f32x4 sb[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) bf[j] = frag(pb[j] + (size_t)kb * kBlock, rem);
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) sb[j][e] = fb[j][e][(size_t)kb * (size_t)g.sb_blk];
#pragma unroll
        for (int i = 0; i < SM; ++i) {
            const i32x8 af = frag(pa[i] + (size_t)kb * kBlock, rem);
            const float sa = fa[i][(size_t)kb * (size_t)g.sa_blk];
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                f32x4 part = {0, 0, 0, 0};
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    part = __builtin_amdgcn_mfma_f32_16x16x32_f16(widen8<TB>(bf[j][2 * u], bf[j][2 * u + 1]),
                                                                  widen8<TA>(af[2 * u], af[2 * u + 1]), part, 0, 0, 0);
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][j][e] = fmaf(part[e] * sa, sb[j][e], acc[i][j][e]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < SM; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) sums[wave][i * NT + j][lane] = acc[i][j];
    __syncthreads();
    if (wave >= SM * NT) return;
    f32x4 v = sums[0][wave][lane];
#pragma unroll
    for (int w = 1; w < NW; ++w) v += sums[w][wave][lane];
    const int m = t.m0 + (wave / NT) * 16 + l16, n = t.n0 + (wave % NT) * 16 + lg * 4;
    if (m >= t.m_end || n >= g.N) return;
    if (t.bad) v = f32x4{1, 1, 1, 1} * __builtin_nanf("");
    else if (block_a_row(g, t, m) < 0) v = f32x4{0, 0, 0, 0};
    block_store4(g, m, n, v);
}

template <int TA, int TB>
int launch_block(const BlockPlan& p, const BlockArgs& a, dim3 grid, hipStream_t s) {
    const bool brow = a.b_shift == 0;
    if (p.kernel == BLOCK_DIRECT)
        return brow ? launch_status(block_direct<TA, TB, true, 2, 2>, grid, dim3(256), s, a)
                    : launch_status(block_direct<TA, TB, false, 2, 2>, grid, dim3(256), s, a);
    // operands with adjacent rows: one kernel for either kind of scales, each row's its own
    if (p.kernel == BLOCK_TURNED) return launch_status(block_direct<TA, TB, true, 4, 3, true>, grid, dim3(512), s, a);
    if (p.kernel == BLOCK_STAGED) {
        if (p.tr == 1) return launch_status(block_staged<TA, TB, true, 1>, grid, dim3(256), s, a);
        if (p.tr == 2) return launch_status(block_staged<TA, TB, true, 2>, grid, dim3(256), s, a);
        if (p.tr == 3) return launch_status(block_staged<TA, TB, true, 3>, grid, dim3(256), s, a);
        return brow ? launch_status(block_staged<TA, TB, true, 0>, grid, dim3(256), s, a)
                    : launch_status(block_staged<TA, TB, false, 0>, grid, dim3(256), s, a);
    }
    if (p.direct) {
        if (p.bn == 64) return launch_status(block_skinny<TA, TB, 1, 4, true>, grid, dim3(512), s, a);
        return p.bm == 16   ? launch_status(block_skinny<TA, TB, 1, 1, true>, grid, dim3(512), s, a)
               : p.bm == 32 ? launch_status(block_skinny<TA, TB, 2, 1, true>, grid, dim3(512), s, a)
                            : launch_status(block_skinny<TA, TB, 4, 1, true>, grid, dim3(512), s, a);
    }
    return p.bm == 16   ? launch_status(block_skinny<TA, TB, 1, 1, false>, grid, dim3(512), s, a)
           : p.bm == 32 ? launch_status(block_skinny<TA, TB, 2, 1, false>, grid, dim3(512), s, a)
                        : launch_status(block_skinny<TA, TB, 4, 1, false>, grid, dim3(512), s, a);
}

}  // namespace dg
