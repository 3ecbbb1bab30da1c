// block_quantize.hip -- fp32, fp16 or bf16 values into 8-bit codes with a scale for each
// block of 1 x 128 or 128 x 128, as they are, transposed, or both from one read.
//
//   amax = max(max |x|, 2^-100)   scale = amax / qmax   code = round(x * (qmax / amax))
//
// The maximum is taken on the values' bits without their sign, as whole numbers: the same
// order, and a NaN is larger than everything, so its block becomes NaN.
#include "device_common.h"
#include "experts.h"
#include "launch.h"

namespace dg {

constexpr uint32_t kAmaxFloor = (127u - 100u) << 23;  // the bits of 2^-100

__device__ __forceinline__ float qmax_of(int type) { return type == 0 ? 448.0f : 57344.0f; }

// four values as four codes, the first in the low byte; rounds to nearest even
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d, int type) {
    int r = 0;
    if (type == 0) {
        r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, r, false);
        r = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true);
    } else {
        r = __builtin_amdgcn_cvt_pk_bf8_f32(a, b, r, false);
        r = __builtin_amdgcn_cvt_pk_bf8_f32(c, d, r, true);
    }
    return (uint32_t)r;
}

// Eight elements of a row from p, of which `valid` (> 0) lie inside it (the rest zero).
template <typename T>
__device__ __forceinline__ void load8(T (&raw)[8], const T* p, int valid) {
    if (valid >= 8) {
        __builtin_memcpy(raw, p, sizeof raw);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) raw[e] = e < valid ? p[e] : T(0);
    }
}

// One workgroup: a 128 x 128 block of X in registers, thread (rg, cg) holding rows
// 8 rg .. 8 rg + 7 at columns 8 cg .. 8 cg + 7. The transposed codes go through LDS (rows
// of 128 bytes, 16-byte pieces permuted by the column's bits 3 to 5 against bank conflicts).
// Bound by memory: 8192 x 4096 bf16 into codes both ways moves 136 MB in 30 us, 4.5 TB/s of
// the 5.1 that a copy reaches; the fewest rows take 5 us, of which a launch is 2.5.
template <int DT>
__global__ __launch_bounds__(256) void block_quantize(QuantArgs a) {
    typedef typename Elem<DT>::type T;
    __shared__ uint32_t wave_max[4][128];
    __shared__ __attribute__((aligned(16))) uint8_t turned[128 * 128];
    const int tid = threadIdx.x, wave = tid >> 6;
    const int cg = tid & 15, rg = tid >> 4;
    const int across = (a.cols + 127) >> 7;
    const int by = (int)blockIdx.x / across, bx = (int)blockIdx.x - by * across;
    const int r0 = by * 128 + rg * 8, c0 = bx * 128 + cg * 8;
    const int left = a.cols - c0;
    const T* X = static_cast<const T*>(a.X);

    // every load is issued before the first is used: rows outside the matrix read row 0 and
    // become zeros
    T raw[8][8];
    bool in[8];
    size_t at[8];
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        int r = r0 + p;
        in[p] = r < a.rows;
        if (a.gather) r = a.gather[min(r, a.rows - 1)];
        in[p] = in[p] && r >= 0 && r < a.x_rows && left > 0;
        at[p] = (size_t)(in[p] ? r : 0) * (size_t)a.ldx;
    }
    if (a.x_rows > 0) {  // there is a row 0
        if (bx * 128 + 128 <= a.cols) {  // whole columns, without a branch at each load
#pragma unroll
            for (int p = 0; p < 8; ++p) __builtin_memcpy(raw[p], X + at[p] + c0, sizeof raw[p]);
        } else {
#pragma unroll
            for (int p = 0; p < 8; ++p) load8<T>(raw[p], X + at[p] + (left > 0 ? c0 : 0), left > 0 ? left : a.cols);
        }
    }
    float v[8][8];
#pragma unroll
    for (int p = 0; p < 8; ++p)
#pragma unroll
        for (int e = 0; e < 8; ++e) v[p][e] = in[p] ? decode<DT>(raw[p][e]) : 0.0f;
    uint32_t rmax[8], cmax[8];
#pragma unroll
    for (int p = 0; p < 8; ++p) rmax[p] = cmax[p] = kAmaxFloor;
#pragma unroll
    for (int p = 0; p < 8; ++p)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t u = __float_as_uint(v[p][e]) & 0x7fffffffu;
            rmax[p] = max(rmax[p], u);
            cmax[e] = max(cmax[e], u);
        }
    const bool need_rows = a.nat.q && a.nat.block_rows == 1;
    const bool need_cols = a.tr.q && a.tr.block_rows == 1;
    const bool need_block = (a.nat.q && a.nat.block_rows != 1) || (a.tr.q && a.tr.block_rows != 1);
    if (need_rows || need_block) {
#pragma unroll
        for (int p = 0; p < 8; ++p)
#pragma unroll
            for (int d = 1; d < 16; d <<= 1) rmax[p] = max(rmax[p], (uint32_t)__shfl_xor((int)rmax[p], d));
    }
    uint32_t bmax = kAmaxFloor;
    if (need_block) {
#pragma unroll
        for (int p = 0; p < 8; ++p) bmax = max(bmax, rmax[p]);
        bmax = max(bmax, (uint32_t)__shfl_xor((int)bmax, 16));
        bmax = max(bmax, (uint32_t)__shfl_xor((int)bmax, 32));
        if ((tid & 63) == 0) wave_max[wave][0] = bmax;
        __syncthreads();
        bmax = max(max(wave_max[0][0], wave_max[1][0]), max(wave_max[2][0], wave_max[3][0]));
        __syncthreads();
    }
    if (a.nat.q) {
        const float top = qmax_of(a.nat.type);
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            const int r = r0 + p;
            const float amax = __uint_as_float(need_rows ? rmax[p] : bmax);
            const float inv = top / amax;
            u32x2 q;
            q[0] = encode4(v[p][0] * inv, v[p][1] * inv, v[p][2] * inv, v[p][3] * inv, a.nat.type);
            q[1] = encode4(v[p][4] * inv, v[p][5] * inv, v[p][6] * inv, v[p][7] * inv, a.nat.type);
            if (r >= a.rows) continue;
            uint8_t* dst = a.nat.q + (size_t)r * (size_t)a.nat.ld + c0;
            if (left >= 8) {
                __builtin_memcpy(dst, &q, 8);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (e < left) dst[e] = (uint8_t)(q[e >> 2] >> (8 * (e & 3)));
            }
            if (cg == 0 && (need_rows || (rg == 0 && p == 0))) {
                const int sr = need_rows ? r : by;
                a.nat.s[(size_t)sr * (size_t)a.nat.s_row + (size_t)bx * (size_t)a.nat.s_blk] = amax / top;
            }
        }
    }
    if (!a.tr.q) return;
    if (need_cols) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            cmax[e] = max(cmax[e], (uint32_t)__shfl_xor((int)cmax[e], 16));
            cmax[e] = max(cmax[e], (uint32_t)__shfl_xor((int)cmax[e], 32));
        }
        if ((tid & 48) == 0)
#pragma unroll
            for (int e = 0; e < 8; ++e) wave_max[wave][cg * 8 + e] = cmax[e];
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 8; ++e)
            cmax[e] = max(max(wave_max[0][cg * 8 + e], wave_max[1][cg * 8 + e]),
                          max(wave_max[2][cg * 8 + e], wave_max[3][cg * 8 + e]));
    }
    const float top = qmax_of(a.tr.type);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float amax = __uint_as_float(need_cols ? cmax[e] : bmax);
        const float inv = top / amax;
        u32x2 q;
        q[0] = encode4(v[0][e] * inv, v[1][e] * inv, v[2][e] * inv, v[3][e] * inv, a.tr.type);
        q[1] = encode4(v[4][e] * inv, v[5][e] * inv, v[6][e] * inv, v[7][e] * inv, a.tr.type);
        const int c = cg * 8 + e;
        // the reader takes 16-byte pieces: pieces 2i, 2i + 1 stay neighbours
        *reinterpret_cast<u32x2*>(&turned[c * 128 + (((rg >> 1) ^ ((c >> 3) & 7)) << 4) + ((rg & 1) << 3)]) = q;
        if (rg == 0 && e < left && (need_cols || c == 0)) {
            const int sr = need_cols ? c0 + e : bx;
            a.tr.s[(size_t)sr * (size_t)a.tr.s_row + (size_t)by * (size_t)a.tr.s_blk] = amax / top;
        }
    }
    __syncthreads();
    const int piece = tid & 7;  // 16 rows of X
    const int row = by * 128 + piece * 16, valid = a.rows - row;
    if (valid <= 0) return;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const int c = p * 32 + (tid >> 3), col = bx * 128 + c;
        if (col >= a.cols) continue;
        const u32x4 q = *reinterpret_cast<const u32x4*>(&turned[c * 128 + ((piece ^ ((c >> 3) & 7)) << 4)]);
        uint8_t* dst = a.tr.q + (size_t)col * (size_t)a.tr.ld + row;
        if (valid >= 16) {
            // read by a later pass, if at all: past the caches (both ways 8192 x 4096: 30.4 against
            // 32.1 us). The others' reader comes next: with them and the products' C past the caches
            // too this takes 26.7 us, but two products with their quantizing 305 instead of 300.
            store_passing(dst, q);
        } else {
#pragma unroll
            for (int e = 0; e < 16; ++e)
                if (e < valid) dst[e] = (uint8_t)(q[e >> 2] >> (8 * (e & 3)));
        }
    }
}

int launch_block_quantize(const QuantArgs& a, int dtype, hipStream_t s) {
    const dim3 grid((unsigned)((a.cols + 127) / 128) * (unsigned)((a.rows + 127) / 128));
    if (dtype == DT_F32) return launch_status(block_quantize<DT_F32>, grid, dim3(256), s, a);
    if (dtype == DT_F16) return launch_status(block_quantize<DT_F16>, grid, dim3(256), s, a);
    return launch_status(block_quantize<DT_BF16>, grid, dim3(256), s, a);
}

}  // namespace dg
