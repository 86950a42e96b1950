// fp4_plan.h -- which variant of the 4-bit kernels a call takes, by its sizes.
// Arithmetic on sizes alone and no CUDA, so that a host compiler can ask for the
// plan of any size too.
#pragma once

#include <stdint.h>

#include "bitnet_b200.h"

#ifdef __CUDACC__
#include "common.cuh"
#endif

namespace bitnet {

#ifndef __CUDACC__  // (else those of common.cuh)
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t k_pad(int64_t K) { return ceil_div(K, 128) * 128; }
#endif

constexpr int kFp4TileRows = 128;  // rows of a scale tile
constexpr int kFp4PatchK = 256;    // k of a patch that a CTA quantises or reads back
constexpr int kFp4Rows = 128;      // weight rows per tile of the small kernel (UMMA M)
constexpr int kFp4StageK = 256;    // k per stage of a product: a 128-byte swizzled row of codes
constexpr int kFp4MaxSplit = 8;    // largest portable cluster

// Patches of `r` rows x 256 k in the 128-row bands of a matrix, and the rows
// that a launch takes: 32 where patches of 64 are fewer than four to each of the
// B200's 148 SMs.
inline int64_t fp4_patches(int64_t rows, int64_t K, int r) {
    return ceil_div(rows, kFp4TileRows) * (kFp4TileRows / r) * ceil_div(k_pad(K), kFp4PatchK);
}
inline int fp4_patch_rows(int64_t rows, int64_t K) { return fp4_patches(rows, K, 64) < 4 * 148 ? 32 : 64; }

// Tokens that the small kernel takes; more go to the pair kernel.
// (64 x 2560 x 6912 takes 6.8 us in the small kernel, 9.0 in the other, 64 x
// 27648 x 5120 15.2 and 18.3; 128 x 13824 x 2560 10.6 and 8.0).
constexpr int kFp4SmallTokens = 64;

// CTAs per weight tile of the small kernel: as many as leave 240 CTAs or fewer,
// 150 from 17 tokens up (a CTA lives some 3 us beside its loads, so more of
// them than the SMs hold at once cost more than the shorter ranges of k save)
// and two stages to each.
// Measured, in us, for 1, 2, 4 and 8: 1 x 2560 x 6912 10.9, 7.4, 5.5, 5.1;
// 1 x 6912 x 2560 5.3, 5.2, 4.6, 8.1; 1 x 13824 x 5120 10.1, 9.5, 11.8, 14.9;
// 1 x 55296 x 5120 23.2, 26.7, 34.4, 48.4; 33 x 3200 x 4800 8.1, 6.5, 5.6, 6.1;
// 64 x 13824 x 2560 7.7, 8.5, 13.4, 25.8.  From the sizes alone, so that the
// sums' grouping depends on nothing else.
inline int fp4_split(int64_t M, int64_t N, int64_t K) {
    const int64_t tiles = ceil_div(N, kFp4Rows), nk = ceil_div(k_pad(K), kFp4StageK), most = M <= 16 ? 240 : 150;
    int s = 1;
    while (2 * s <= kFp4MaxSplit && tiles * 2 * s <= most && nk >= 4 * s) s *= 2;
    return s;
}

// Weight rows per tile of the pair kernel: the width whose rounds over the
// B200's 74 pairs take the least time.  Measured on 2048 x 9472 x K: a 256-k
// stage of a tile takes kStage ns and the tile kEnd more (its accumulators are
// emptied while the next tile's first MMAs wait, or run beside).  NV stages
// bring more scales.  A tile's stores run beside the next tile and take kLeast
// ns, which a short k does not cover, and more where rows of y are off 16-byte
// boundaries (1791 x 6643 x 1113: 22.5, 17.5, 20.0, 15.9 and 22.3 us with 384
// to 64 rows).  2048 x 13824 x 2560 MX takes 62, 38, 33, 30.0 and 29.7 us
// with 64, 128, 192, 256 and 384 rows, 512 x 6912 x 2560 11.4, 9.9, 7.7, 8.8
// and 10.8.
//   Where tiles of 64 or 128 rows leave pairs idle and k is long, 2 or 4 pairs
// share a tile (clusters of 4 or 8 CTAs, which fill some 64 pairs' SMs at once)
// for an exchange of some kExchange ns: 100 x 500 x 20000 MX takes 21.6 us with
// one pair to a tile, 12.3 with two, 8.3 with four; 448 x 1664 x 18022 19.4
// with one, 14.7 with two and 128 rows.  (77 x 3211 x 4801 NV, two pairs and 10
// stages each, takes 8.6, with half that k 7.6, with 512 k and one pair to a
// tile 3.3: a shared tile costs some 3 us beside its stages, which kExchange
// does not count.)
//   The numbers of pairs are the B200's and not the device's, so that the split,
// and with it the sums, are the same wherever the library runs.
struct Fp4PairPlan {
    int width, split;
};
inline Fp4PairPlan fp4_pair_plan(int64_t M, int64_t N, int64_t K, int format, bool vec) {
    constexpr int kWidths[5] = {384, 256, 192, 128, 64};
    constexpr int kStage[2][5] = {{490, 358, 288, 240, 207}, {520, 385, 345, 241, 207}};
    constexpr int kEnd[5] = {1400, 760, 590, 410, 370}, kExchange = 200;
    constexpr int kLeast[2][5] = {{2900, 1410, 1300, 760, 710}, {9000, 4500, 3900, 2300, 1800}};
    const int64_t nk = ceil_div(k_pad(K), kFp4StageK), tm = ceil_div(M, 256);
    auto plan = [&](int most, int off) {
        Fp4PairPlan best{256, 1};
        int64_t cost = INT64_MAX;
        for (int i = 0; i < 5; ++i) {
            const int64_t tiles = tm * ceil_div(N, kWidths[i]);
            for (int s = 1; s <= (kWidths[i] <= 128 ? most : 1); s *= 2) {
                if (s > 1 && (tiles * s > 64 || nk < 4 * s)) break;
                const int64_t t = ceil_div(nk, s) * kStage[format == BITNET_FP4_MX ? 0 : 1][i] + kEnd[i];
                const int64_t c = ceil_div(tiles * s, 74) * (t > kLeast[off][i] ? t : kLeast[off][i]) + (s > 1 ? kExchange : 0);
                if (c < cost) cost = c, best = {kWidths[i], s};
            }
        }
        return best;
    };
    // the split, which groups the sums, follows from the sizes alone; the width
    // leaves each sum's order as it is and may follow y's alignment too
    const Fp4PairPlan best = plan(4, 0);
    return vec || best.split > 1 ? best : plan(1, 1);
}

}  // namespace bitnet
