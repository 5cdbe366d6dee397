// norm_api.hip -- the C ABI of include/moe_norm.h: argument checks and
// launches.  Host side only.
#include "moe_norm.h"

#include "api.h"
#include "norm_kernels.h"

using namespace moe::api;

namespace {

moe_status check_norm(int64_t rows, int32_t H) {
    if (rows < 0 || rows > 0x7fffffffLL)
        return fail(MOE_ERR_INVALID_ARG, "rows=%lld must be in [0, 2^31)", (long long)rows);
    if (H <= 0 || H % 8 != 0) return fail(MOE_ERR_INVALID_ARG, "H=%d must be a positive multiple of 8", H);
    if (H > moe::kNormMaxH) return fail(MOE_ERR_UNSUPPORTED, "H=%d > %d", H, moe::kNormMaxH);
    return MOE_OK;
}

moe_status check_dtype(moe_dtype d, const char* name) {
    if (d != MOE_DTYPE_F32 && d != MOE_DTYPE_BF16)
        return fail(MOE_ERR_INVALID_ARG, "%s=%d is not MOE_DTYPE_F32/BF16", name, (int)d);
    return MOE_OK;
}

}  // namespace

MOE_EXPORT moe_status moe_norm(int64_t rows, int32_t H, const void* x, moe_dtype x_dtype, const float* weight,
                               const float* bias, float eps, int center, void* out, moe_dtype out_dtype,
                               float* stats, hipStream_t stream) {
    MOE_TRY(check_norm(rows, H));
    MOE_TRY(check_dtype(x_dtype, "x_dtype"));
    MOE_TRY(check_dtype(out_dtype, "out_dtype"));
    if (!(eps > 0.0f) || !isfinite(eps)) return fail(MOE_ERR_INVALID_ARG, "eps must be positive and finite");
    if (rows == 0) return ok();
    MOE_TRY(check_ptr(x, "x"));
    MOE_TRY(check_ptr(weight, "weight"));
    MOE_TRY(check_ptr(bias, "bias", true));
    MOE_TRY(check_ptr(out, "out"));
    MOE_TRY(check_ptr(stats, "stats", true));
    if (out == x && out_dtype != x_dtype)
        return fail(MOE_ERR_INVALID_ARG, "out is x, in another type");
    moe::NormArgs a{};
    a.rows = rows;
    a.H = H;
    a.x = x;
    a.x_f32 = x_dtype == MOE_DTYPE_F32;
    a.weight = weight;
    a.bias = bias;
    a.eps = eps;
    a.center = center != 0;
    a.out = out;
    a.out_f32 = out_dtype == MOE_DTYPE_F32;
    a.stats = stats;
    return hip_status(moe::launch_norm(a, stream), "norm launch");
}

MOE_EXPORT size_t moe_norm_workspace_bytes(int64_t rows, int32_t H) {
    if (check_norm(rows, H) != MOE_OK) return 0;
    ok();
    return moe::norm_ws_bytes(rows, H);
}

MOE_EXPORT moe_status moe_norm_backward(int64_t rows, int32_t H, const void* dy, moe_dtype dy_dtype, const void* x,
                                        moe_dtype x_dtype, const float* weight, const float* stats, int center,
                                        void* dx, moe_dtype dx_dtype, float* dweight, float* dbias, int accumulate,
                                        void* ws, size_t ws_bytes, hipStream_t stream) {
    MOE_TRY(check_norm(rows, H));
    MOE_TRY(check_dtype(dy_dtype, "dy_dtype"));
    MOE_TRY(check_dtype(x_dtype, "x_dtype"));
    MOE_TRY(check_dtype(dx_dtype, "dx_dtype"));
    const bool empty = rows == 0;
    MOE_TRY(check_ptr(dy, "dy", empty));
    MOE_TRY(check_ptr(x, "x", empty));
    MOE_TRY(check_ptr(weight, "weight"));
    MOE_TRY(check_ptr(stats, "stats", empty));
    MOE_TRY(check_ptr(dx, "dx", empty));
    MOE_TRY(check_ptr(dweight, "dweight"));
    MOE_TRY(check_ptr(dbias, "dbias", true));
    if (!empty && dx == dy && dx_dtype != dy_dtype) return fail(MOE_ERR_INVALID_ARG, "dx is dy, in another type");
    if (!empty && dx == x && dx_dtype != x_dtype) return fail(MOE_ERR_INVALID_ARG, "dx is x, in another type");
    MOE_TRY(check_ws_bytes(moe::norm_ws_bytes(rows, H), ws, ws_bytes));
    moe::NormArgs a{};
    a.rows = rows;
    a.H = H;
    a.dy = dy;
    a.dy_f32 = dy_dtype == MOE_DTYPE_F32;
    a.x = x;
    a.x_f32 = x_dtype == MOE_DTYPE_F32;
    a.weight = weight;
    a.stats = const_cast<float*>(stats);
    a.center = center != 0;
    a.out = dx;
    a.out_f32 = dx_dtype == MOE_DTYPE_F32;
    a.dweight = dweight;
    a.dbias = dbias;
    a.accumulate = accumulate != 0;
    a.ws = static_cast<float*>(ws);
    return hip_status(moe::launch_norm_backward(a, stream), "norm backward launch");
}
