// kernel_mid.h -- x w^T of fp16 or bf16 in 128 x 128 tiles, for sizes whose 256 x 256 tiles would be
// few or mostly empty.
//
// Four waves of 64 x 64 (2 x 2 accumulators of v_mfma_f32_32x32x16) over stages of 64 k that come
// by direct copies, whole 128-byte lines of a row; two stages (64 KB), so that two workgroups share
// a compute unit and one computes while the other waits for its stage or stores its tile. A row's
// 16-byte pieces lie permuted by (row / 2) % 8, which keeps the reads of 32 rows free of bank
// conflicts. Rows are 16-byte aligned and k a multiple of 8. Grid y: slices of k.
#pragma once
#include "kernel_adapters.h"

namespace dg {

struct MidArgs {
    const void* A;
    const void* B;
    int64_t lda, ldb;
    int M, N, K;
    int tiles_m, tiles_n, group_m, xcd_remap;
    int slice_k;   // a multiple of 64
};

constexpr int kMid = 128, kMidK = 64;

struct MidLds {
    uint16_t a[2][kMid * kMidK];
    uint16_t b[2][kMid * kMidK];
};

template <int DT, class HOOK>
__device__ __forceinline__ void mid_body(const MidArgs& g, MidLds& lds, const HOOK& h) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int l32 = lane & 31, lh = lane >> 5;
    const int wm = wave >> 1, wn = wave & 1;
    int tm, tn;
    raster(round_tile(0, g.tiles_m * g.tiles_n, g.xcd_remap), g.tiles_m, g.tiles_n, g.group_m, tm, tn);
    const int m0 = tm * kMid, n0 = tn * kMid;
    const int k0 = (int)blockIdx.y * g.slice_k, k1 = min(g.K, k0 + g.slice_k);
    const uint32_t wave_u = (uint32_t)__builtin_amdgcn_readfirstlane(wave);
    // a wave copies 32 rows of each operand, 8 rows at a time
    const uint16_t* src_a[4];
    const uint16_t* src_b[4];
    int kc[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 32 * wave + 8 * i + (lane >> 3);
        kc[i] = ((lane & 7) ^ ((r >> 1) & 7)) << 3;
        src_a[i] = static_cast<const uint16_t*>(g.A) + (size_t)min(m0 + r, g.M - 1) * (size_t)g.lda;
        src_b[i] = static_cast<const uint16_t*>(g.B) + (size_t)min(n0 + r, g.N - 1) * (size_t)g.ldb;
    }
    const uint32_t dst_a = (uint32_t)reinterpret_cast<uintptr_t>(DG_LDSV(&lds.a[0][0])) + wave_u * 4096u;
    const uint32_t dst_b = (uint32_t)reinterpret_cast<uintptr_t>(DG_LDSV(&lds.b[0][0])) + wave_u * 4096u;
    // pieces at or past K are taken from the row's start; the products leave them out
    auto copy = [&](int k, uint32_t st) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int kk = k + kc[i] < g.K ? k + kc[i] : 0;
            __builtin_amdgcn_global_load_lds(DG_GLB(src_a[i] + kk), DG_LDS_AT(dst_a + st * 16384u + i * 1024u), 16, 0, 0);
            __builtin_amdgcn_global_load_lds(DG_GLB(src_b[i] + kk), DG_LDS_AT(dst_b + st * 16384u + i * 1024u), 16, 0, 0);
        }
    };
    f32x16 acc[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = f32x16{};
    auto step = [&](int st, int left) {
#pragma unroll
        for (int ks = 0; ks < kMidK / 16; ++ks) {
            const int c = 2 * ks + lh, sw = (c ^ ((l32 >> 1) & 7)) << 3;
            u32x4 q[2], p[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                q[i] = *reinterpret_cast<const u32x4*>(&lds.a[st][(wm * 64 + 32 * i + l32) * kMidK + sw]);
                p[i] = *reinterpret_cast<const u32x4*>(&lds.b[st][(wn * 64 + 32 * i + l32) * kMidK + sw]);
            }
            if (left < kMidK && 8 * c >= left) q[0] = q[1] = p[0] = p[1] = u32x4{0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) acc[i][j] = mfma_32<DT>(p[j], q[i], acc[i][j]);
        }
    };
    copy(k0, 0);
    int st = 0;
    for (int k = k0; k < k1; k += kMidK, st ^= 1) {
        vm_wait_n<0>();
        asm volatile("s_barrier" ::: "memory");
        // every wave is past the reads of the other stage
        if (k + kMidK < k1) copy(k + kMidK, (uint32_t)(st ^ 1));
        step(st, k1 - k);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
    __syncthreads();
    h.template finish<2, 2, 2, 2>(acc, m0 + wm * 64, n0 + wn * 64, wm, wn, reinterpret_cast<char*>(&lds.a[0][0]),
                                  reinterpret_cast<char*>(&lds.b[0][0]));
}

// Sums of a slice of k as fp32 rows: part (slices x M x ld), ld a multiple of 4.
struct MidPartHook {
    float* part;
    int64_t ld;
    int M, N;
    template <int SI, int SJ, int WM, int WN>
    __device__ __forceinline__ void finish(f32x16 (&acc)[SI][SJ], int m0, int n0, int wm, int wn, char* lds,
                                           char* lds2) const {
        // a wave's 64 x 64 tile through its own 16 KB: rows of 256 bytes, 16-byte pieces permuted by
        // the row
        const int lane = threadIdx.x & 63, l32 = lane & 31, lh = lane >> 5;
        char* slot = (wm == 0 ? lds : lds2) + wn * 16384;
#pragma unroll
        for (int i = 0; i < SI; ++i)
#pragma unroll
            for (int j = 0; j < SJ; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int r = 32 * i + l32, c = 8 * j + 2 * q + lh;
                    *reinterpret_cast<f32x4*>(slot + r * 256 + ((c ^ (r & 15)) << 4)) =
                        f32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
                }
        __builtin_amdgcn_wave_barrier();
        const int c = lane & 15, n = n0 + 4 * c;
        float* out = part + (size_t)blockIdx.y * (size_t)M * (size_t)ld;
#pragma unroll 4
        for (int it = 0; it < 16; ++it) {
            const int r = 4 * it + (lane >> 4);
            const f32x4 v = *reinterpret_cast<const f32x4*>(slot + r * 256 + ((c ^ (r & 15)) << 4));
            if (m0 + r < M && n < ld) *reinterpret_cast<f32x4*>(out + (size_t)(m0 + r) * (size_t)ld + n) = v;
        }
    }
};

template <int DT>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2, 2))) void mid_part(MidArgs g, MidPartHook h) {
    __shared__ __attribute__((aligned(1024))) MidLds lds;
    mid_body<DT>(g, lds, h);
}

}  // namespace dg
