// tile16.h -- a tile's results as 16-bit rows, through LDS, for the kernels built on the 128 x 128
// and 256 x 256 tiles.
#pragma once
#include "device_common.h"

namespace dg {

// A tile as 16-bit rows in LDS (a half of its rows to each half of LDS), their 16-byte pieces
// permuted by the row, so that neither the writes (32 rows of one piece) nor the whole-row reads
// meet in a bank. From there whole rows leave, 512 bytes of a 256 x 256 tile's at a time.
template <int SI, int SJ, int WM, int WN>
struct Tile16 {
    static_assert(WM == 2, "a half of LDS for each");
    static constexpr int HALF = 32 * SI, COLS = WN * 32 * SJ, PITCH = COLS * 2, PIECES = COLS / 8, WAVES = WM * WN;
    char* lds;
    char* lds2;
    __device__ __forceinline__ char* at(int r, int piece) const {
        return (r < HALF ? lds : lds2) + (r % HALF) * PITCH + ((piece ^ (r & (PIECES - 1))) << 4);
    }
    // columns 32 SJ wn + 32 j + 8 q + 4 lh .. + 3 of row r
    template <int DT>
    __device__ __forceinline__ void put(int r, int wn, int j, int q, int lh, const float (&v)[4]) const {
        uint32_t h[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            h[e] = DT == DT_F16 ? (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)v[e]) : (uint32_t)f32_to_bf16_rne(v[e]);
        *reinterpret_cast<u32x2*>(at(r, wn * (4 * SJ) + 4 * j + q) + 8 * lh) = u32x2{h[0] | (h[1] << 16), h[2] | (h[3] << 16)};
    }
    // rows x cols of the tile at (m, n) to out, past the caches with PASSING
    template <bool PASSING = false>
    __device__ __forceinline__ void store(uint16_t* out, int64_t ld, int m, int n, int rows, int cols) const {
        constexpr int RI = 64 / PIECES, IT = 2 * HALF / WAVES / RI;  // rows of a load, loads of a wave
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
        const int piece = lane % PIECES, c = n + 8 * piece, left = cols - c;
#pragma unroll 4
        for (int it = 0; it < IT; ++it) {
            const int r = wave * (2 * HALF / WAVES) + RI * it + lane / PIECES, row = m + r;
            const u32x4 v = *reinterpret_cast<const u32x4*>(at(r, piece));
            if (row >= rows || left <= 0) continue;
            uint16_t* dst = out + (size_t)row * (size_t)ld + c;
            if (left >= 8) {
                if constexpr (PASSING) store_passing(dst, v);
                else __builtin_memcpy(dst, &v, 16);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (e < left) dst[e] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
            }
        }
    }
};

}  // namespace dg
