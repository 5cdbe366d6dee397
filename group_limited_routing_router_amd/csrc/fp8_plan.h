// fp8_plan.h -- which tiles the FP8 products run on: host side, from the shape
// alone.
#pragma once

#include "fp8_kernels.h"
#include "tile_plan.h"

namespace moe {

// Parts of a long reduction on 32 rows keep at most 32 stages: 40 tiles of 160
// stages (one row, 5120 x 20480, weights from HBM) 65, 40, 39, 29, 34 us in 1, 2,
// 4, 8, 16 parts; as an input gradient 93, 55, 49, 36 in 1, 2, 4, 8.
inline TilePlan long_parts(TilePlan p, int red) {
    while (p.rows == 32 && p.splits > 1 && p.splits < 16 && blocks_of(red) >= 32 * p.splits) p.splits *= 2;
    return p;
}

inline TilePlan product_plan(int64_t P, int E, int N, int K) {
    return long_parts(plan_tiles(P, E, N, K, K, 1), K);
}

// red: length of the sums (twice N, in whole blocks, for two matrices at once)
inline TilePlan input_grad_plan(int64_t P, int E, int red, int K) {
    return long_parts(plan_tiles(P, E, K, red, K, 1), red);
}

inline int pair_red(int N) { return 2 * blocks_of(N) * kBlock; }

// The gated products, by the mean expert's rows (256, 128 or 32 a tile, never
// split).  256 experts of 2 x 2560 x 5120, microseconds on 32, 128 and 256
// rows: 4 rows an expert 1051, 1201, -; 16 rows 1088, 1243, -; 32 rows 1375,
// 1223, 1388; 64 rows 2125, 1283, 1408; 128 rows -, 1750, 1556.
// The large tile from one for every compute unit on (8 experts of 225 rows, 2 x
// 704 x 1152, 64 tiles: 30 us, on 128 rows 18).  Weights that do not fit the
// caches stream past them where their rows are whole lines and few rows reuse
// them (4 rows 1141 us through the caches, 32 rows 1265; 64 rows the same).  On
// 32 rows the operands are multiplied as bf16 (gemm_fp8.h).
inline TilePlan gated_plan(int64_t P, int E, int N, int K) {
    const int64_t met = E < P ? E : P;
    const float rows = static_cast<float>(P) / static_cast<float>(met);
    const bool stream = 2 * met * N * K > kStreamBytes && K % 128 == 0 && rows <= 32.0f;
    if (rows <= 24.0f) return TilePlan{32, stream, 1};
    const float each = rows / 256 + 0.45f;  // row tiles of an expert, with half a tile for the ragged end
    const float tiles = static_cast<float>(met) * (each > 1.0f ? each : 1.0f) * static_cast<float>(blocks_of(N));
    if (rows > 96.0f && tiles >= kNumCu) return TilePlan{256, false, 1};
    return TilePlan{128, stream, 1};
}

}  // namespace moe
