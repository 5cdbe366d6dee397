// tile_plan.h -- which tile a grouped product runs on and into how many parts
// its reduction is split: host side, from the shape alone.
#pragma once

#include <math.h>

#include "common.h"
#include "kernels.h"

namespace moe {

constexpr int kNumCu = 256;

// Workgroups of a tiled launch (an upper bound: the host does not read the
// experts' counts).
inline int64_t tile_grid(int64_t P, int E, int cols, int bx, int by) {
    const int64_t row_tiles = (P + by - 1) / by + (E < P ? E : P);
    const int64_t tiles = row_tiles * ((cols + bx - 1) / bx);
    return (tiles + kNumXcd - 1) / kNumXcd * kNumXcd;
}

// How the product and the input gradient of a shape run.
struct TilePlan {
    int rows;    // tile: 32 x 128, 128 x 128 or 256 x 256
    bool nt;     // weights stream past the caches
    int splits;  // parts of the reduction
};

// Microseconds of `tiles` workgroups over `stages` stages each.  A round holds
// one 256-row tile on each compute unit or two of the smaller ones.  Measured:
// a stage (128 bytes of reduction) takes 1.85 us on 256 rows with the whole
// chip busy, 1.05 with little of it; 0.6 on 128 and 0.22 on 32 rows with a
// compute unit to itself, 1.1 and 0.5 with two on it; a round costs 11, 5.5
// and 4 us beside its stages (first loads, writing out).
inline float tile_time(int rows, float tiles, float stages) {
    const float slots = rows == 256 ? kNumCu : 2.0f * kNumCu;
    float rounds = tiles / slots;
    // the last round of a few is not full, but then runs faster
    if (rounds <= 2.0f)
        rounds = ceilf(rounds);
    else if (rounds < 4.0f)
        rounds = 0.5f * (rounds + ceilf(rounds));
    if (rows == 256)
        return rounds * ((1.05f + 0.8f * (tiles < kNumCu ? tiles / kNumCu : 1.0f)) * stages + 11.0f);
    const bool alone = tiles <= kNumCu;
    if (rows == 128) return rounds * ((alone ? 0.6f : 1.1f) * stages + 5.5f);
    return rounds * ((alone ? 0.22f : 0.5f) * stages + 4.0f);
}

// The host does not read the experts' counts: a mean expert is taken, with
// half a tile more for the ragged end.
//   cols, red  columns of the output and length of its sums (a weight matrix
//              has cols x red elements of eb bytes)
//   row_bytes  bytes of a row of the weights in memory
inline TilePlan plan_tiles(int64_t P, int E, int cols, int red, int64_t row_bytes, int eb) {
    const int64_t met = E < P ? E : P;  // experts that can have rows
    const float experts = static_cast<float>(met);
    const float mean_rows = static_cast<float>(P) / experts;
    const bool large = met * cols * red * eb > kStreamBytes;
    const bool whole_lines = row_bytes % 128 == 0;
    const float stages = static_cast<float>((red + 128 / eb - 1) / (128 / eb));
    auto tiles_of = [&](int rows) {
        const float each = met == 1 ? static_cast<float>((P + rows - 1) / rows) : mean_rows / rows + 0.45f;
        const int width = rows == 256 ? 256 : 128;
        return experts * (each > 1.0f ? each : 1.0f) * static_cast<float>((cols + width - 1) / width);
    };
    TilePlan p{256, false, 1};
    const bool stream = large && mean_rows <= 32;
    if (stream) {
        // the weight stream is the time: the tile that takes an expert's rows
        // at once and keeps the most loads in flight (256 experts of 2560 x
        // 5120: 4 rows each 0.97 ms on 32, 1.07 on 128 rows; 24 rows each 1.10
        // and 1.09 ms)
        p.rows = mean_rows <= 24 ? 32 : 128;
        // past the caches where rows are whole lines (0.97 against 1.07 ms;
        // rows of 1776 bytes: 452 against 381 us)
        p.nt = whole_lines;
    }
    float best = -1.0f;
    // a large weight stream with more rows and tiles for every compute unit:
    // the tile that reads the weights least often (4096 tokens over 256 busy
    // and idle experts: 1.46 against 1.68 ms on 128 rows)
    if (large && !stream && tiles_of(256) >= kNumCu) return p;
    for (int rows : {32, 128, 256}) {
        if (stream && rows != p.rows) continue;
        // more tiles than a launch takes (2^31 - 1 rows of width 8 on 128
        // rows); outputs of up to kMaxOutputs always fit on 256
        if (rows < 256 && tile_grid(P, E, cols, 128, rows) > kMaxWorkgroups) continue;
        for (int splits = 1; splits <= 16; splits *= 2) {
            if (splits > 1 && stages < 4 * splits) break;
            // rows that are not whole lines take more lines a stage, which
            // shows most where the tile's part of a row is short (185 x 4
            // rows, K 2232: 112 us on 128 rows, 76 on 256)
            const float lines = whole_lines ? 1.0f : (rows == 256 ? 1.1f : 1.3f);
            float t = tile_time(rows, tiles_of(rows) * splits, lines * stages / splits);
            // the sums written and read, one more launch, and 5% for the parts'
            // own first loads.  Of 1, 2, 4, 8, 16 parts: 32 rows, 512 x 16384:
            // 58, 36, 24, 19, 19 us, 16 taken; 256 rows, 2048 x 4096: 21, 22,
            // 20, 22, 26, 1 taken; 8192 rows, 5120 x 20480: 1367, 1350, 1446,
            // 1708, 2249, 1 taken; worst of twelve shapes: 8 x 128 rows, 1024 x
            // 4096: 22, 30, 28, 31, 43, 2 taken
            if (splits > 1) t = 1.05f * t + 4.0f + 2.0f * splits * static_cast<float>(P) * cols * 4.0f / 5e6f;
            if (best < 0.0f || t < best) {
                best = t;
                p.rows = rows;
                p.splits = splits;
            }
        }
    }
    return p;
}

}  // namespace moe
