// block_plan.h -- which kernel a block-scaled product takes: plain C++, no device needed.
#pragma once
#include <stdint.h>

#include <algorithm>

namespace dg {

constexpr int kBlock = 128;     // elements of k (or of a row) that share a scale
constexpr int64_t kCus = 256;   // compute units

enum BlockMode { BLOCK_PLAIN = 0, BLOCK_EXPERTS = 1, BLOCK_GRADIENT = 2 };

enum BlockKernel {
    BLOCK_SKINNY = 0,  // few rows: block_skinny
    BLOCK_DIRECT = 1,  // 128 x 128 tiles copied straight to LDS: block_direct
    BLOCK_TURNED = 2,  // 256 x 128 tiles, B stored with its rows adjacent: block_direct
    BLOCK_STAGED = 3   // 128 x 128 tiles through registers, any layout: block_staged
};

// What a call launches.
struct BlockPlan {
    int kernel;       // BlockKernel
    int bm, bn;
    int direct;       // rows of whole 16-byte chunks (the kernel for few rows loads them whole)
    int split;        // K slices
    int tr;           // bit 0: B stored with its rows adjacent, bit 1: A
};

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// rows: rows of C that share a B (for experts the average); n_products: B's in the call;
// direct: 16-byte aligned rows of whole chunks; small: byte offsets within an operand fit 32
// bits; may_split: whether K may be split (plain products with a workspace).
//
// Both sides of each rule, in us (e4m3, B in 128 x 128 blocks, C bf16 where not said):
//  - rows <= 64, few rows against tiles: 64 x 4096 x 4096 12.9 : 16.4, 64 x 1024 x 2048 10.3 : 12.8,
//    17 x 4096 x 512 9.5 : 9.7; 96 rows would take two passes over B.
//  - 64 columns to a workgroup against 16: 64 experts of 2048 x 2048 over 16 x 4 rows 38.4 : 45.2,
//    of 2048 x 512 16.9 : 31.9, 32 of 2048 x 1024 15.8 : 21.5; behind, where they leave fewer
//    than 2048 workgroups with more than 1024 k: 32 of 2048 x 4096 46.8 : 36.2, 16 of 2048 x 2048
//    15.9 : 15.0.
//  - 256 x 128 tiles against 128 x 128, two to a compute unit, of which one computes while the
//    other loads or stores: behind with straight rows (8192 x 4096 x 4096 254 : 236, x 512 47 : 42,
//    experts of 4096 x 8 rows 368 : 319), so there are none; with B turned, where the smaller ones
//    go through registers, ahead in single products (8192 x 4096 x 4096 316 : 335, x 1024 93 : 96),
//    behind for experts (453 : 421, gradients of 2048 x 1024 over 512 rows 340 : 268).
inline BlockPlan block_plan(BlockMode mode, int64_t rows, int64_t n_products, int64_t N, int64_t K, bool direct, bool small,
                            int tr, bool may_split) {
    BlockPlan p;
    p.tr = tr;
    p.direct = direct;
    p.split = 1;
    const int64_t nkb = ceil_div(K, kBlock);
    if (rows <= 64 && tr == 0) {
        p.kernel = BLOCK_SKINNY;
        p.bm = rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
        const int64_t wide = n_products * ceil_div(N, 64);
        p.bn = direct && p.bm == 16 && wide >= (K <= 1024 ? 4 : 8) * kCus ? 64 : 16;
        const int64_t wgs = n_products * ceil_div(N, p.bn);
        if (may_split && wgs < kCus) p.split = (int)std::max<int64_t>(1, std::min<int64_t>(kCus / wgs, nkb / 16));
    } else {
        const bool turned = mode == BLOCK_PLAIN && tr == 1 && direct && small &&
                            ceil_div(rows, 256) * ceil_div(N, 128) >= kCus * 3 / 4;
        p.kernel = turned ? BLOCK_TURNED : tr == 0 && direct && small ? BLOCK_DIRECT : BLOCK_STAGED;
        p.bm = turned ? 256 : 128;
        p.bn = 128;
        const int64_t wgs = n_products * ceil_div(rows, p.bm) * ceil_div(N, p.bn);
        if (may_split && wgs < kCus) p.split = (int)std::max<int64_t>(1, std::min<int64_t>(2 * kCus / wgs, nkb / 4));
    }
    // whole slices
    const int64_t chunk = ceil_div(std::max<int64_t>(nkb, 1), p.split);
    p.split = (int)std::max<int64_t>(1, ceil_div(nkb, chunk));
    return p;
}

// Rows past whole tiles that run as a launch of their own, on the kernel for few rows: a cut
// tile takes a third of a whole one's time or more, and where it makes some compute unit's
// share a tile longer, behind all the others (2056 x 4096 x 4096 71 against 91 us, with 64 rows
// past 2048 76 : 89, 1064 rows 53 : 58, 8200 x 1024 x 2048 40 : 49, 2056 x 4096 x 1024 26 : 29; through
// registers 2056 x 4096 x 4090 110 : 145). Where shares stay as they are, K is split over the units
// that are left or the tiles are short, the launch only adds its own time (576 x 1024 x 2048
// 24 : 17, 264 x 4096 x 4096 32 : 27, 1088 x 1024 x 2048 29 : 26, 8256 x 4096 x 512 50 : 46).
inline int64_t rest_rows(const BlockPlan& p, int64_t M, int64_t N, int64_t K) {
    if ((p.kernel != BLOCK_DIRECT && p.kernel != BLOCK_STAGED) || p.tr != 0 || p.split > 1 || M <= p.bm || K <= 512) return 0;
    const int64_t rest = M % p.bm, across = ceil_div(N, p.bn), wgs = ceil_div(M, p.bm) * across;
    return rest <= 64 && ceil_div(wgs, kCus) > ceil_div(wgs - across, kCus) ? rest : 0;
}

}  // namespace dg
