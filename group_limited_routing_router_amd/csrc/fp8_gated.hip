// fp8_gated.hip -- launches of the gated feed-forward products in FP8: gate and
// up, their activation and product and its quantisation in one kernel, and the
// same with the gradients (gemm_fp8.h).
#include "gemm_fp8.h"

namespace moe {
namespace {

template <int MODE>
hipError_t launch_gated(const Fp8Args& g, hipStream_t s) {
    const int64_t met = g.E < g.P ? g.E : g.P;
    const float mean_rows = static_cast<float>(g.P) / static_cast<float>(met);
    if (mean_rows <= 24.0f) return launch_tiles<MODE, 256, 32>(g, s);
    if (mean_rows <= 96.0f) return launch_tiles<MODE, 256, 128>(g, s);
    return launch_tiles<MODE, 256, 256>(g, s);
}

}  // namespace

hipError_t launch_fp8_gate_up(const Fp8Args& g, hipStream_t s) {
    return g.dh ? launch_gated<kF8GateUpGrad>(g, s) : launch_gated<kF8GateUp>(g, s);
}

}  // namespace moe
