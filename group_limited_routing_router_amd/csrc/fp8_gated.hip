// fp8_gated.hip -- launches of the gated feed-forward products in FP8: gate and
// up, their activation and product and its quantisation in one kernel, and the
// same with the gradients (gemm_fp8.h).
#include "gemm_fp8.h"

namespace moe {
namespace {

// By the mean expert's rows.  256 experts of 2 x 2560 x 5120, microseconds on
// 32, 128 and 256 rows: 4 rows an expert 1051, 1201, -; 16 rows 1088, 1243, -;
// 32 rows 1375, 1223, 1388; 64 rows 2125, 1283, 1408; 128 rows -, 1750, 1556.
// The large tile from one for every compute unit on (8 experts of 225 rows, 2 x
// 704 x 1152, 64 tiles: 30 us, on 128 rows 18).  Weights that do not fit the
// caches stream past them where their rows are whole lines and few rows reuse
// them (4 rows 1141 us through the caches, 32 rows 1265; 64 rows the same).  On
// 32 rows the operands are multiplied as bf16 (gemm_fp8.h).
template <int MODE>
hipError_t launch_gated(const Fp8Args& g, hipStream_t s) {
    const int64_t met = g.E < g.P ? g.E : g.P;
    const float rows = static_cast<float>(g.P) / static_cast<float>(met);
    const bool stream = 2 * met * g.N * g.K > kStreamBytes && g.K % 128 == 0 && rows <= 32.0f;
    if (rows <= 24.0f) return stream ? launch_tiles<MODE, 256, 32, true, true>(g, s) : launch_tiles<MODE, 256, 32, false, true>(g, s);
    const float each = rows / 256 + 0.45f;  // row tiles of an expert, with half a tile for the ragged end
    const float tiles = static_cast<float>(met) * (each > 1.0f ? each : 1.0f) * static_cast<float>(blocks_of(g.N));
    if (rows > 96.0f && tiles >= kNumCu) return launch_tiles<MODE, 256, 256>(g, s);
    return stream ? launch_tiles<MODE, 256, 128, true>(g, s) : launch_tiles<MODE, 256, 128>(g, s);
}

}  // namespace

hipError_t launch_fp8_gate_up(const Fp8Args& g, hipStream_t s) {
    return g.dh ? launch_gated<kF8GateUpGrad>(g, s) : launch_gated<kF8GateUp>(g, s);
}

}  // namespace moe
