// kernel_adapters.h -- low-rank adapters of fp16 and bf16 on the matrix instructions.
//
// The rows of a tile may belong to any adapters. Where u m^T is added to a product, 32 rows
// are taken at a time and each adapter among them in turn: u's rows of other adapters count
// as zeros, and what the instruction gives in their rows is dropped, so that nothing of one
// adapter (a NaN least of all) reaches another's rows. u enters as the sum of two numbers of
// the matrices' type, its rounding and what that leaves: off by 2^-16 (bf16) or 2^-22 of u,
// against the single rounding of y that follows, for twice 2 T N rank operations.
#pragma once
#include "device_common.h"
#include "extents.h"
#include "kernel_sp.h"
#include "layers.h"

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

// v as hi + lo; an infinite or NaN v is all in hi.
template <int DT>
__device__ __forceinline__ void split_hi_lo(const float (&v)[8], u32x4& hi, u32x4& lo) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        uint32_t h[2], l[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float x = v[2 * e + k];
            const uint16_t b = DT == DT_F16 ? __builtin_bit_cast(uint16_t, (_Float16)x) : f32_to_bf16_rne(x);
            float rest = x - decode<DT>(b);
            rest = fabsf(rest) < INFINITY ? rest : 0.0f;
            h[k] = b;
            l[k] = DT == DT_F16 ? __builtin_bit_cast(uint16_t, (_Float16)rest) : f32_to_bf16_rne(rest);
        }
        hi[e] = h[0] | (h[1] << 16);
        lo[e] = l[0] | (l[1] << 16);
    }
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

// acc[j] += scale u m^T for rows m0 .. m0 + 31 and columns n0 + 32 j .. + 31 (m: columns x rank).
// Lane l holds row m0 + l % 32; register r column 8 (r / 4) + 4 (l / 32) + r % 4 of a subtile.
template <int DT, int SJ>
__device__ __forceinline__ void adapter_add(f32x16 (&acc)[SJ], int m0, int n0, const AdapterArgs& a) {
    const int lane = threadIdx.x & 63, l32 = lane & 31, lh = lane >> 5;
    const int row = m0 + l32;
    int mine = row < a.tokens ? a.index[row] : -1;
    if (mine >= a.adapters) mine = -1;
    uint64_t todo = __ballot(mine >= 0);
    while (todo) {
        const int i = __builtin_amdgcn_readlane(mine, (int)__builtin_ctzll(todo));
        const bool here = mine == i;
        const float scale = a.scale ? a.scale[i] : 1.0f;
        const uint16_t* m = static_cast<const uint16_t*>(a.m) + (size_t)i * (size_t)a.stride_m;
        f32x16 d[SJ];
#pragma unroll
        for (int j = 0; j < SJ; ++j) d[j] = f32x16{};
        for (int r0 = 0; r0 < a.rank; r0 += 16) {
            const int r = r0 + 8 * lh;
            float v[8];
            load_f8(v, a.u + (size_t)row * (size_t)a.rank + r, here ? a.rank - r : 0);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] *= scale;
            u32x4 hi, lo;
            split_hi_lo<DT>(v, hi, lo);
#pragma unroll
            for (int j = 0; j < SJ; ++j) {
                const int col = n0 + 32 * j + l32;
                const u32x4 p = load_frag8(m + (size_t)col * (size_t)a.ldm + r, col < a.cols ? a.rank_m - r : 0);
                d[j] = mfma_32<DT>(p, hi, d[j]);
                d[j] = mfma_32<DT>(p, lo, d[j]);
            }
        }
#pragma unroll
        for (int j = 0; j < SJ; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[j][e] += here ? d[j][e] : 0.0f;
        todo &= ~__ballot(here);
    }
}

// ---------------------------------------------------------------- shared product and adapters in one
template <int DT>
struct AdapterHook {
    static constexpr bool kReplace = false, kAdd = true;
    AdapterArgs a;
    template <int SJ>
    __device__ __forceinline__ void add(f32x16 (&acc)[4][SJ], int m, int n) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) adapter_add<DT, SJ>(acc[i], m + 32 * i, n, a);
    }
};

template <int DT, int OPB, bool REG>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2))) void adapter_product(
    GemmArgs g, AdapterHook<DT> h) {
    mfma32_sp_body<DT, OPB, 8, REG, false, false>(g, nullptr, h);
}

// ---------------------------------------------------------------- second product on its own
// out = base + scale u m^T; a wave has 32 rows x 64 columns.
template <int DT>
__global__ __launch_bounds__(256) void adapter_expand16(AdapterArgs a, int tiles_n) {
    const int tm = (int)blockIdx.x / tiles_n, tn = (int)blockIdx.x - tm * tiles_n;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int m0 = tm * 32, n0 = tn * 256 + wave * 64;
    const int row = m0 + (lane & 31), lh = lane >> 5;
    f32x16 acc[2];
    const float* base = a.base + (size_t)min(row, a.tokens - 1) * (size_t)a.ld_base;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int c = n0 + 32 * j + 8 * q + 4 * lh;
            float v[4] = {0.f, 0.f, 0.f, 0.f};
            if (c + 3 < a.cols) __builtin_memcpy(v, base + c, 16);
            else
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (c + e < a.cols) v[e] = base[c + e];
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[j][4 * q + e] = v[e];
        }
    adapter_add<DT, 2>(acc, m0, n0, a);
    if (row >= a.tokens) return;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int c = n0 + 32 * j + 8 * q + 4 * lh;
            const size_t at = (size_t)row * (size_t)a.ldo + c;
            const f32x4 v = {acc[j][4 * q], acc[j][4 * q + 1], acc[j][4 * q + 2], acc[j][4 * q + 3]};
            if (c + 3 < a.cols) store_out4(a.out, DT, at, v);
            else
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (c + e < a.cols) store_out(a.out, DT, at + e, v[e]);
        }
}

// ---------------------------------------------------------------- first product
// A wave: one token and one of its rank numbers, 8 elements to a lane and step. For few tokens,
// whose adapters mostly differ.
template <int DT>
__global__ __launch_bounds__(256) void adapter_shrink_row(AdapterArgs a) {
    const int64_t unit = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    if (unit >= (int64_t)a.tokens * a.rank) return;
    const int t = (int)(unit / a.rank), j = (int)(unit - (int64_t)t * a.rank);
    const int i = a.index[t];
    float sum = 0.0f;
    if (i >= 0 && i < a.adapters) {
        const uint16_t* x = static_cast<const uint16_t*>(a.x) + (size_t)t * (size_t)a.ldx;
        const uint16_t* m = static_cast<const uint16_t*>(a.m) + (size_t)i * (size_t)a.stride_m + (size_t)j * (size_t)a.ldm;
#pragma unroll 4
        for (int64_t k = lane * 8; k < a.cols; k += 512) {
            const int valid = (int)min((int64_t)8, a.cols - k);
            const u32x4 p = load_frag8(x + k, valid), q = load_frag8(m + k, valid);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                sum = fmaf(decode<DT>((uint16_t)p[e]), decode<DT>((uint16_t)q[e]), sum);
                sum = fmaf(decode<DT>((uint16_t)(p[e] >> 16)), decode<DT>((uint16_t)(q[e] >> 16)), sum);
            }
        }
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d);
        if (a.scale) sum *= a.scale[i];
    }
    if (lane == 0) a.u[unit] = sum;
}

// A workgroup: 16 tokens against each adapter among them (the adapters shared out over grid y),
// the sum over k cut over its eight waves in pieces of 64 and joined in LDS in their order.
template <int DT, int NT>
__global__ __launch_bounds__(512) void adapter_shrink16(AdapterArgs a) {
    __shared__ __attribute__((aligned(16))) float part[8][NT][64][4];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int l16 = lane & 15, lg = lane >> 4;
    const int row = (int)blockIdx.x * 16 + l16;
    int mine = row < a.tokens ? a.index[row] : -1;
    if (mine >= a.adapters) mine = -1;
    const uint16_t* x = static_cast<const uint16_t*>(a.x) + (size_t)min(row, a.tokens - 1) * (size_t)a.ldx;
    if (blockIdx.y == 0 && mine < 0 && row < a.tokens)
        for (int j = wave * 4 + lg; j < a.rank; j += 32) a.u[(size_t)row * (size_t)a.rank + j] = 0.0f;
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
        int64_t k0 = wave * 64;
        const int whole = a.cols & ~63;
#pragma unroll 2
        for (; k0 < whole; k0 += 512) {
            u32x4 xv[2], mv[2][NT];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                __builtin_memcpy(&xv[s], x + k0 + 32 * s + 8 * lg, 16);
#pragma unroll
                for (int n = 0; n < NT; ++n) __builtin_memcpy(&mv[s][n], mr[n] + k0 + 32 * s + 8 * lg, 16);
            }
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int n = 0; n < NT; ++n) acc[n] = mfma_16<DT>(mv[s][n], xv[s], acc[n]);
        }
        if (k0 == whole && whole < a.cols)
            for (int s = 0; s < 2; ++s) {
                const int64_t k = k0 + 32 * s + 8 * lg;
                const int valid = (int)max((int64_t)0, min((int64_t)8, a.cols - k));
                const u32x4 xv = load_frag8(x + k, valid);
#pragma unroll
                for (int n = 0; n < NT; ++n) acc[n] = mfma_16<DT>(load_frag8(mr[n] + k, valid), xv, acc[n]);
            }
#pragma unroll
        for (int n = 0; n < NT; ++n) *reinterpret_cast<f32x4*>(part[wave][n][lane]) = acc[n];
        __syncthreads();
        if (wave < NT && here) {  // lane: token l16, rank numbers 16 wave + 4 lg .. + 3
            f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int p = 0; p < 8; ++p) v += *reinterpret_cast<const f32x4*>(part[p][wave][lane]);
            const float scale = a.scale ? a.scale[i] : 1.0f;
            const int j = 16 * wave + 4 * lg;
            float* u = a.u + (size_t)row * (size_t)a.rank + j;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (j + e < a.rank) u[e] = v[e] * scale;
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------- adapters' transposes
// Each in_i (rows x cols) as its transpose of cols x out_ld, zeros past column `rows`. A
// workgroup turns 64 x 64 through LDS.
__device__ __forceinline__ void turn_tile(const TurnArgs& t, int tile, int i, uint16_t (*buf)[66]) {
    const int tr = tile / t.tiles_c, tc = tile - tr * t.tiles_c;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint16_t* in = static_cast<const uint16_t*>(t.in) + (size_t)i * (size_t)t.stride;
    uint16_t* out = static_cast<uint16_t*>(t.out) + (size_t)i * (size_t)t.cols * (size_t)t.out_ld;
    const int c = tc * 64 + lane;
    for (int e = wave; e < 64; e += 4) {
        const int r = tr * 64 + e;
        buf[e][lane] = r < t.rows && c < t.cols ? in[(size_t)r * (size_t)t.ld + c] : (uint16_t)0;
    }
    __syncthreads();
    const int r = tr * 64 + lane;
    for (int e = wave; e < 64; e += 4) {
        const int cc = tc * 64 + e;
        if (cc < t.cols && r < t.out_ld) out[(size_t)cc * (size_t)t.out_ld + r] = buf[lane][e];
    }
}

// Both of an adapter's matrices in one launch: grid x the tiles of one and then of the other,
// grid y the adapters.
static __global__ __launch_bounds__(256) void adapter_turn(TurnArgs p, TurnArgs q) {
    __shared__ uint16_t buf[64][66];
    const int first = p.tiles_r * p.tiles_c;
    if ((int)blockIdx.x < first) turn_tile(p, (int)blockIdx.x, (int)blockIdx.y, buf);
    else turn_tile(q, (int)blockIdx.x - first, (int)blockIdx.y, buf);
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

// A workgroup: 64 columns of z (x or grad) and the whole rank, over an adapter's rows of a chunk
// in steps of 32. z and h (v or u, split in two) lie in LDS by rows and are read transposed, so
// that a lane gets eight consecutive rows of one column.
template <int DT, int NT, bool TURNED>
__global__ __launch_bounds__(256) void adapter_gradient16(AdapterArgs a) {
    constexpr int HC = NT * 2;  // 16-byte chunks of a row of h
    __shared__ __attribute__((aligned(16))) uint16_t sz[2][32 * 64];
    __shared__ __attribute__((aligned(16))) uint16_t sh[2][2][32 * NT * 16];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int l16 = lane & 15, lg = lane >> 4;
    const int slot = (int)blockIdx.y, c0 = (int)blockIdx.x * 64;
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

    const uint16_t* z = static_cast<const uint16_t*>(a.x);
    const int zr = tid >> 3, zc = tid & 7;   // the 16 bytes of z this thread moves
    constexpr int HN = NT * 32 * 16 / 8;     // pieces of eight numbers of h
    constexpr int HP = HN < 256 ? 1 : HN / 256;
    u32x4 zreg;
    float hreg[HP][8];
    auto load = [&](int p0) {
        int t = p0 + zr < to ? a.rows[p0 + zr] : -1;
        if (t >= a.tokens) t = -1;
        const int c = c0 + zc * 8;
        zreg = load_frag8(z + (size_t)max(t, 0) * (size_t)a.ldx + c, t < 0 ? 0 : a.cols - c);
#pragma unroll
        for (int q = 0; q < HP; ++q) {
            const int piece = q * 256 + tid, r = piece / HC, j = (piece % HC) * 8;
            int th = r < 32 && p0 + r < to ? a.rows[p0 + r] : -1;
            if (th >= a.tokens) th = -1;
            load_f8(hreg[q], a.u + (size_t)max(th, 0) * (size_t)a.rank + j, th < 0 ? 0 : a.rank - j);
        }
    };
    auto put = [&](int b) {
        *reinterpret_cast<u32x4*>(&sz[b][zr * 64 + ((zc ^ nmaj_swz<8>(zr)) << 3)]) = zreg;
#pragma unroll
        for (int q = 0; q < HP; ++q) {
            const int piece = q * 256 + tid, r = piece / HC, c = piece % HC;
            if (HN < 256 && piece >= HN) break;
            u32x4 hv, lv;
            split_hi_lo<DT>(hreg[q], hv, lv);
            const int at = r * (HC * 8) + ((c ^ nmaj_swz<HC>(r)) << 3);
            *reinterpret_cast<u32x4*>(&sh[b][0][at]) = hv;
            *reinterpret_cast<u32x4*>(&sh[b][1][at]) = lv;
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
    f32x4 acc[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[n] = f32x4{0.f, 0.f, 0.f, 0.f};
    load(from);
    put(0);
    int b = 0;
    for (int p0 = from; p0 < to; p0 += 32, b ^= 1) {
        __syncthreads();
        const bool more = p0 + 32 < to;
        if (more) load(p0 + 32);
        const u32x4 zf = turned(sz[b], wave * 16, std::integral_constant<int, 8>{});
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const u32x4 hf = turned(sh[b][0], n * 16, std::integral_constant<int, HC>{});
            const u32x4 lf = turned(sh[b][1], n * 16, std::integral_constant<int, HC>{});
            if (TURNED) {
                acc[n] = mfma_16<DT>(hf, zf, acc[n]);
                acc[n] = mfma_16<DT>(lf, zf, acc[n]);
            } else {
                acc[n] = mfma_16<DT>(zf, hf, acc[n]);
                acc[n] = mfma_16<DT>(zf, lf, acc[n]);
            }
        }
        if (more) put(b ^ 1);
    }
    // TURNED: lane has column c0 + l16 and rank numbers 16 n + 4 lg .. + 3; else rank number
    // 16 n + l16 and columns c0 + 4 lg .. + 3
    const float scale = a.scale ? a.scale[i] : 1.0f;
    const size_t each = (size_t)a.rank * (size_t)a.cols;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const f32x4 v = acc[n] * scale;
        const int c = c0 + wave * 16 + (TURNED ? l16 : 4 * lg), j = 16 * n + (TURNED ? 4 * lg : l16);
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

// An adapter (grid y) of several chunks: the sum of its slots; one without rows: zeros.
template <int DT>
__global__ __launch_bounds__(256) void adapter_join(AdapterArgs a, int slots) {
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
