// Which tile an MXFP4 matrix product takes (mxfp4.hip): a rule on its sizes and the number of CUs, on the host and without HIP,
// so that it can be checked without a device.
#pragma once

#include <cstdint>

namespace ep {

// A tile of bm rows and bn columns whose waves form ks groups along K, and what it costs: step_us for 256 ks columns of K,
// tile_us for its start and end, and `share` of a round for each further round of tiles over the CUs (below 1 where a CU
// holds several blocks).
struct MxTile {
    int bm, bn, ks;
    float step_us, tile_us, share;
};

// A product with one weight takes the tile of the least (1 + share (rounds - 1)) (steps step_us + tile_us). The figures are fitted
// to 120 products (M 1 ... 4096; N x K 1024 x 2048 ... 8192 x 8192 and 4096 x 16384, weights that come from HBM), each tile for
// itself, but for 16 x 32 with four K groups: its own fit (0.436, 1.42) lost to two groups at 1 x 4096 x 16384 by a rounding. Over the 120 the
// picked tile takes 1.3% longer than the fastest of 20 tiles on average and 15% at most (800 x 2048 x 8192: 128 x 64 18.3 us, 64 x
// 64 15.9). They pick, e.g., 256 x 256 for 4096 x 8192 x 8192 (117-122 us; 256 x 192: 145, 256 x 128: 154, 128 x 128: 165), 256 x 192
// for 1024 x 11520 x 3840 (28; 256 x 256: 29, 256 x 128: 39), 128 x 128 for 512 x 8192 x 8192 (25; 128 x 64: 30), 128 x 64 for 333 x
// 5003 x 3968 (11.7; 64 x 64: 11.8, 128 x 128: 12.3), 64 x 64 for 256 x 4096 x 4096 (7.7; 128 x 64: 10.8), 32 x 32 for 64 x 4096 x
// 4096 (5.6; 64 x 64: 7.0), 16 x 32 with two K groups for 1 x 11520 x 3840 (7.1; with four: 10.3) and with four for 1 x 4096
// x 16384 (10.4; two: 13.1). They know nothing of the weight's bytes: 64 x 8192 x 8192 takes 64 x 64 (13.7 us) where 32 x 32 takes 13.1, and
// where 64 x 64 is faster by as much (27 x 12148 x 10112: 15.6 and 16.5). Nor are they a model of the times themselves: of 4096 x 8192 x 8192
// they make 90 us.
constexpr MxTile kMxTiles[] = {
    {256, 256, 1, 1.309f, 3.06f, 1.0f}, {256, 192, 1, 1.088f, 2.90f, 1.0f}, {256, 128, 1, 0.848f, 2.22f, 1.0f},
    {128, 128, 1, 0.553f, 0.76f, 1.0f}, {128, 64, 1, 0.431f, 0.91f, 0.86f}, {64, 64, 1, 0.257f, 0.25f, 0.91f},
    {32, 32, 2, 0.246f, 0.53f, 0.95f},  {16, 32, 2, 0.259f, 0.10f, 0.65f},  {16, 32, 4, 0.400f, 1.10f, 1.0f},
};
constexpr int kMxTileCount = sizeof kMxTiles / sizeof *kMxTiles;

inline int64_t mx_over(int64_t n, int64_t by) { return (n + by - 1) / by; }

inline float mx_cost(const MxTile& t, int64_t row_tiles, int64_t N, int64_t K, int64_t cus) {
    const int64_t rounds = mx_over(row_tiles * mx_over(N, t.bn), cus);
    return (1.0f + t.share * (float)(rounds - 1)) * ((float)mx_over(K, 256 * t.ks) * t.step_us + t.tile_us);
}

// The tile of a product with one weight, of kMxTiles.
inline int mx_tile(int64_t M, int64_t N, int64_t K, int64_t cus) {
    int best = 0;
    float least = 0.0f;
    for (int i = 0; i < kMxTileCount; ++i) {
        const float us = mx_cost(kMxTiles[i], mx_over(M, kMxTiles[i].bm), N, K, cus);
        if (i == 0 || us < least) best = i, least = us;
    }
    return best;
}

}  // namespace ep
