// kernel_stream.h -- products of a tall matrix with a few rows, fp16 or bf16: the tall one is read
// once and bounds the time.
//
// A workgroup of four waves has 64 rows of the tall matrix and up to 16 TT rows of the other, over
// a range of k. Both come by direct copies, whole lines of a row at a time, into a ring of two to
// five stages; two to four workgroups share a compute unit, which keeps about 100 KB in flight there.
// Loading fragments straight into registers instead touches 16 lines with every 16 lanes and
// reached a third of this on operands out of L2.
//
// A row's pieces of 16 bytes lie permuted by the row's number, so that neither the copies nor
// the fragment reads meet in a bank. Rows are 16-byte aligned and k a multiple of 8.
#pragma once
#include "kernel_adapters.h"

namespace dg {

struct StreamArgs {
    const void* tall;
    const void* few;
    int64_t ld_tall, ld_few;
    int rows, few_rows, K;   // of tall and of few, length of the sum
};

constexpr int kStreamRows = 64;

// S stages of KS k: of 128, or 64 where the few rows are many. A large matrix out of HBM wants deep rings
// (loss of 16 tokens, 32768 words of 2048: four stages, two workgroups to a compute unit, 62.5 us, two
// stages, four workgroups, 66; adapters of 60 tokens, 14336 x 4096: five of 64 63.5, two of 128 66), one
// token and the adapters' first product more workgroups or longer stages (1 token, 4096 x 4096: 23.5
// against 25.1; training step of 4096 tokens, rank 64: 360 against 370, caches cold in each case).
template <int TT, bool DEEP>
struct StreamLds {
    static constexpr int KS = TT <= 2 || (TT == 4 && !DEEP) ? 128 : 64;
    static constexpr int S = TT == 1 ? (DEEP ? 4 : 2) : TT == 4 ? (DEEP ? 5 : 2) : 3;
    uint16_t tall[S][kStreamRows * KS];
    uint16_t few[S][TT * 16 * KS];
};

// Wait until the copies of at most `later` stages of CP copies are in flight.
template <int CP, int MAX>
__device__ __forceinline__ void stream_wait(int later) {
    if constexpr (MAX == 0) {
        vm_wait_n<0>();
    } else {
        if (later >= MAX) vm_wait_n<CP * MAX>();
        else stream_wait<CP, MAX - 1>(later);
    }
}

// acc[t] += the sums over k0 <= k < k1 (k0 a multiple of 128) for tall rows r0 + 16 wave + .. and
// few rows 16 t + ..; TALL_FIRST: lane l has few row 16 t + l % 16 and tall rows 4 (l / 16) .. + 3
// of the wave's 16, else tall row l % 16 and few rows 16 t + 4 (l / 16) .. + 3. Ends with every
// wave past its reads.
template <int DT, int TT, bool TALL_FIRST, class L>
__device__ __forceinline__ void stream_sum(f32x4 (&acc)[TT], const StreamArgs& a, L& lds, int r0, int k0, int k1) {
    constexpr int KS = L::KS, S = L::S, D = S - 1;
    constexpr int CH = KS / 8;               // 16-byte pieces of a stage's row
    constexpr int RC = 64 / CH;              // rows of one copy
    constexpr int CT = 16 / RC;              // copies of a wave's 16 tall rows
    constexpr int CF = TT * 16 / RC / 4;     // and of its share of the few rows
    constexpr int CP = CT + CF;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int l16 = lane & 15, lg = lane >> 4;
    const int piece = lane % CH, crow = lane / CH;
    const uint32_t wave_u = (uint32_t)__builtin_amdgcn_readfirstlane(wave);
    const uint16_t* src_t[CT];
    const uint16_t* src_f[CF];
    int kc_t[CT], kc_f[CF];
#pragma unroll
    for (int i = 0; i < CT; ++i) {
        const int r = 16 * wave + RC * i + crow;
        kc_t[i] = (piece ^ (r & (CH - 1))) << 3;
        src_t[i] = static_cast<const uint16_t*>(a.tall) + (size_t)min(r0 + r, a.rows - 1) * (size_t)a.ld_tall;
    }
#pragma unroll
    for (int i = 0; i < CF; ++i) {
        const int r = RC * (4 * i + wave) + crow;
        kc_f[i] = (piece ^ (r & (CH - 1))) << 3;
        src_f[i] = static_cast<const uint16_t*>(a.few) + (size_t)min(r, a.few_rows - 1) * (size_t)a.ld_few;
    }
    const uint32_t dst_t = (uint32_t)reinterpret_cast<uintptr_t>(DG_LDSV(&lds.tall[0][0])) + wave_u * (16u * KS * 2);
    const uint32_t dst_f = (uint32_t)reinterpret_cast<uintptr_t>(DG_LDSV(&lds.few[0][0])) + wave_u * 1024u;
    // pieces at or past K are taken from the row's start; the products below leave them out
    auto copy = [&](int k, uint32_t st) {
#pragma unroll
        for (int i = 0; i < CT; ++i) {
            const int kk = k + kc_t[i];
            __builtin_amdgcn_global_load_lds(DG_GLB(src_t[i] + (kk < a.K ? kk : 0)),
                                             DG_LDS_AT(dst_t + st * (kStreamRows * KS * 2) + i * 1024u), 16, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < CF; ++i) {
            const int kk = k + kc_f[i];
            __builtin_amdgcn_global_load_lds(DG_GLB(src_f[i] + (kk < a.K ? kk : 0)),
                                             DG_LDS_AT(dst_f + st * (TT * 16 * KS * 2) + i * 4096u), 16, 0, 0);
        }
    };
    const int steps = (k1 - k0 + KS - 1) / KS;
    for (int s = 0; s < D && s < steps; ++s) copy(k0 + s * KS, (uint32_t)s);
    int st = 0, next = D;  // stages of this step and of the one copied during it
    for (int s = 0; s < steps; ++s) {
        stream_wait<CP, D - 1>(steps - 1 - s);
        asm volatile("s_barrier" ::: "memory");
        const int left = k1 - (k0 + s * KS);
        // the barrier also shows that every wave is past step s - 1, whose stage this refills
        if (s + D < steps) copy(k0 + (s + D) * KS, (uint32_t)next);
#pragma unroll
        for (int q = 0; q < KS / 32; ++q) {
            const int c = 4 * q + lg, sw = (c ^ (l16 & (CH - 1))) << 3;
            u32x4 tf = *reinterpret_cast<const u32x4*>(&lds.tall[st][(16 * wave + l16) * KS + sw]);
            u32x4 ff[TT];
#pragma unroll
            for (int t = 0; t < TT; ++t) ff[t] = *reinterpret_cast<const u32x4*>(&lds.few[st][(16 * t + l16) * KS + sw]);
            if (left < KS && 8 * c >= left) {
                tf = u32x4{0, 0, 0, 0};
#pragma unroll
                for (int t = 0; t < TT; ++t) ff[t] = u32x4{0, 0, 0, 0};
            }
#pragma unroll
            for (int t = 0; t < TT; ++t)
                acc[t] = TALL_FIRST ? mfma_16<DT>(tf, ff[t], acc[t]) : mfma_16<DT>(ff[t], tf, acc[t]);
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        st = st + 1 == S ? 0 : st + 1;
        next = next + 1 == S ? 0 : next + 1;
    }
    asm volatile("s_barrier" ::: "memory");
}

// ---------------------------------------------------------------- few tokens
// The first `groups` workgroups: the shared product, 64 rows of w and a slice of k each, as sums to
// part (slices x tokens x N); those after them: u (adapter_shrink_wave).
template <int DT, int TT>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2, 4))) void adapter_decode(
    StreamArgs a, AdapterArgs u, int groups, int slices, int slice_k, float* part) {
    __shared__ __attribute__((aligned(1024))) StreamLds<TT, (TT > 1)> lds;
    const int bid = (int)blockIdx.x;
    if (bid >= groups) {
        adapter_shrink_wave<DT>(u, (int64_t)(bid - groups) * 4 + (threadIdx.x >> 6));
        return;
    }
    const int strip = bid / slices, slice = bid - strip * slices;
    f32x4 acc[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int k0 = slice * slice_k;
    stream_sum<DT, TT, true>(acc, a, lds, strip * kStreamRows, k0, min(a.K, k0 + slice_k));
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int n = strip * kStreamRows + 16 * wave + 4 * (lane >> 4), ld = (a.rows + 3) & ~3;
    if (n >= a.rows) return;
#pragma unroll
    for (int t = 0; t < TT; ++t) {
        const int row = 16 * t + (lane & 15);
        if (row < a.few_rows)
            *reinterpret_cast<f32x4*>(part + ((size_t)slice * a.few_rows + row) * (size_t)ld + n) = acc[t];
    }
}

// y = the slices' sum + scale b u. A thread: four columns of one token.
template <int DT>
__global__ __launch_bounds__(64) void adapter_decode_finish(AdapterArgs a, int slices, const float* part) {
    const int t = (int)blockIdx.y, n = ((int)blockIdx.x * 64 + (int)threadIdx.x) * 4;
    if (n >= a.cols) return;
    const int ld = (a.cols + 3) & ~3;
    const int i = a.index[t];
    const float* p = part + (size_t)t * (size_t)ld + n;
    const size_t step = (size_t)a.tokens * (size_t)ld;
    f32x4 b[8], v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < 8; ++s) b[s] = *reinterpret_cast<const f32x4*>(p + (size_t)min(s, slices - 1) * step);
    const f32x4 d = adapter_row<DT>(a, i, t, n);  // its loads join those in flight
#pragma unroll
    for (int s = 0; s < 8; ++s)
        if (s < slices) v += b[s];
#pragma unroll 8
    for (int s = 8; s < slices; ++s) v += *reinterpret_cast<const f32x4*>(p + (size_t)s * step);
    adapter_row_store<DT>(a, t, n, v + d);
}

// ---------------------------------------------------------------- many tokens: u
// 64 tokens against each adapter among them, over a slice of k: sums to part (slices x tokens x
// rank_p). The adapters of a tile are shared out over grid z.
template <int DT, int TT>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2, 4))) void adapter_shrink_part(
    StreamArgs a, AdapterArgs u, int slice_k, float* part) {
    __shared__ __attribute__((aligned(1024))) StreamLds<TT, false> lds;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int r0 = (int)blockIdx.x * kStreamRows;
    int mine = r0 + lane < a.rows ? u.index[r0 + lane] : -1;  // of row r0 + lane
    if (mine >= u.adapters) mine = -1;
    const int at = __shfl(mine, 16 * wave + (lane & 15));     // of the row whose sums this lane gets
    uint64_t todo = __ballot(mine >= 0);
    const int k0 = (int)blockIdx.y * slice_k, k1 = min(a.K, k0 + slice_k);
    for (uint32_t turn = 0; todo; ++turn) {
        const int i = __builtin_amdgcn_readlane(mine, (int)__builtin_ctzll(todo));
        todo &= ~__ballot(mine == i);
        if (turn % gridDim.z != blockIdx.z) continue;
        f32x4 acc[TT];
#pragma unroll
        for (int t = 0; t < TT; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
        StreamArgs b = a;
        b.few = static_cast<const uint16_t*>(u.m) + (size_t)i * (size_t)u.stride_m;
        stream_sum<DT, TT, false>(acc, b, lds, r0, k0, k1);
        if (at != i) continue;
        float* p = part + ((size_t)blockIdx.y * a.rows + r0 + 16 * wave + (lane & 15)) * (size_t)(TT * 16) + 4 * (lane >> 4);
#pragma unroll
        for (int t = 0; t < TT; ++t) *reinterpret_cast<f32x4*>(p + 16 * t) = acc[t];
    }
}

}  // namespace dg
