// fp8_gated.hip -- launches of the gated feed-forward products in FP8: gate and
// up, their activation and product and its quantisation in one kernel, and the
// same with the gradients (gemm_fp8.h).
#include "fp8_plan.h"
#include "gemm_fp8.h"

namespace moe {
namespace {

template <int MODE>
hipError_t launch_gated(const Fp8Args& g, hipStream_t s) {
    const TilePlan p = gated_plan(g.P, g.E, g.N, g.K);
    if (p.rows == 256) return launch_tiles<MODE, 256, 256>(g, s);
    if (p.rows == 32) return p.nt ? launch_tiles<MODE, 256, 32, true, true>(g, s) : launch_tiles<MODE, 256, 32, false, true>(g, s);
    return p.nt ? launch_tiles<MODE, 256, 128, true>(g, s) : launch_tiles<MODE, 256, 128>(g, s);
}

}  // namespace

hipError_t launch_fp8_gate_up(const Fp8Args& g, hipStream_t s) {
    return g.dh ? launch_gated<kF8GateUpGrad>(g, s) : launch_gated<kF8GateUp>(g, s);
}

}  // namespace moe
