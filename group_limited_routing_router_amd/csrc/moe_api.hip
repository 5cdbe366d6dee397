// moe_api.hip -- the C ABI of libmoe.so (declared in include/moe.h).
//
// Host side only: argument checks, workspace layout and kernel launches.  All
// checks run before the first HIP call, so a rejected call enqueues nothing
// and touches no output.  No allocation, no synchronisation.
#include <mutex>

#include "api.h"

using namespace moe::api;

namespace {

// The workspace of moe_forward_noalloc: a fixed array in device memory, one
// copy per GPU that holds it until the process ends.  Host code never uses
// its name as an address: the device address of each GPU's copy comes from
// hipGetSymbolAddress (looked up on the first call on that GPU).
static __device__ __align__(256) unsigned char scratch[MOE_NOALLOC_SCRATCH_BYTES];

constexpr int kMaxDevices = 64;
std::mutex g_scratch_mutex;
void* g_scratch_ptr[kMaxDevices] = {};

// Device address of the current GPU's scratch array (looked up once per GPU).
moe_status device_scratch(void** out) {
    int dev = -1;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return hip_status(e, "hipGetDevice");
    if (dev < 0 || dev >= kMaxDevices)
        return fail(MOE_ERR_UNSUPPORTED, "device %d beyond the %d the library tracks", dev,
                    kMaxDevices);
    std::lock_guard<std::mutex> lock(g_scratch_mutex);
    if (!g_scratch_ptr[dev]) {
        void* ptr = nullptr;
        e = hipGetSymbolAddress(&ptr, HIP_SYMBOL(scratch));
        if (e != hipSuccess) return hip_status(e, "hipGetSymbolAddress(scratch)");
        if (!ptr) return fail(MOE_ERR_HIP, "hipGetSymbolAddress(scratch) gave NULL");
        g_scratch_ptr[dev] = ptr;
    }
    *out = g_scratch_ptr[dev];
    return MOE_OK;
}

}  // namespace

MOE_EXPORT size_t moe_workspace_bytes(const moe_problem* p) {
    if (check_problem(p) != MOE_OK) return 0;
    return layout_of(*p).total;
}

MOE_EXPORT moe_status moe_route(const moe_problem* p, const moe_bf16* x, const moe_bf16* w_router,
                                const float* bias, int32_t* topk_ids, float* topk_weights,
                                hipStream_t stream) {
    MOE_TRY(check_problem(p));
    if (p->T == 0) return ok();
    MOE_TRY(check_ptr(x, "x"));
    MOE_TRY(check_ptr(w_router, "w_router"));
    MOE_TRY(check_ptr(bias, "bias", true));
    MOE_TRY(check_ptr(topk_ids, "topk_ids"));
    MOE_TRY(check_ptr(topk_weights, "topk_weights"));
    return hip_status(moe::launch_route(to_internal(*p), x, w_router, bias, topk_ids, topk_weights,
                                        stream),
                      "route launch");
}

MOE_EXPORT moe_status moe_permute(const moe_problem* p, const int32_t* topk_ids,
                                  int32_t* expert_offsets, int32_t* sorted_pairs,
                                  int32_t* pair_rows, void* ws, size_t ws_bytes,
                                  hipStream_t stream) {
    MOE_TRY(check_problem(p));
    if (p->T == 0) return ok();
    MOE_TRY(check_ptr(topk_ids, "topk_ids"));
    MOE_TRY(check_ptr(expert_offsets, "expert_offsets"));
    MOE_TRY(check_ptr(sorted_pairs, "sorted_pairs"));
    MOE_TRY(check_ptr(pair_rows, "pair_rows"));
    MOE_TRY(check_ws(*p, ws, ws_bytes));
    const Layout L = layout_of(*p);
    return hip_status(moe::launch_permute(to_internal(*p), topk_ids, expert_offsets, sorted_pairs,
                                          pair_rows, at<int32_t>(ws, L.counts), stream),
                      "permute launch");
}

MOE_EXPORT moe_status moe_expert_ffn(const moe_problem* p, const moe_bf16* x,
                                     const int32_t* sorted_pairs, const int32_t* expert_offsets,
                                     const moe_bf16* w_gate, const moe_bf16* w_up,
                                     const moe_bf16* w_down, float* y, void* ws, size_t ws_bytes,
                                     hipStream_t stream) {
    MOE_TRY(check_problem(p));
    if (p->T == 0) return ok();
    MOE_TRY(check_ptr(x, "x"));
    MOE_TRY(check_ptr(sorted_pairs, "sorted_pairs"));
    MOE_TRY(check_ptr(expert_offsets, "expert_offsets"));
    MOE_TRY(check_ptr(w_gate, "w_gate"));
    MOE_TRY(check_ptr(w_up, "w_up"));
    MOE_TRY(check_ptr(w_down, "w_down"));
    MOE_TRY(check_ptr(y, "y"));
    MOE_TRY(check_ws(*p, ws, ws_bytes));
    const Layout L = layout_of(*p);
    return hip_status(moe::launch_expert_ffn(to_internal(*p), x, sorted_pairs, expert_offsets,
                                             w_gate, w_up, w_down, at<uint16_t>(ws, L.h), y,
                                             stream),
                      "expert ffn launch");
}

MOE_EXPORT moe_status moe_expert_gate_up(const moe_problem* p, const moe_bf16* x,
                                         const int32_t* sorted_pairs,
                                         const int32_t* expert_offsets, const moe_bf16* w_gate,
                                         const moe_bf16* w_up, moe_bf16* h, hipStream_t stream) {
    MOE_TRY(check_problem(p));
    if (p->T == 0) return ok();
    MOE_TRY(check_ptr(x, "x"));
    MOE_TRY(check_ptr(sorted_pairs, "sorted_pairs"));
    MOE_TRY(check_ptr(expert_offsets, "expert_offsets"));
    MOE_TRY(check_ptr(w_gate, "w_gate"));
    MOE_TRY(check_ptr(w_up, "w_up"));
    MOE_TRY(check_ptr(h, "h"));
    return hip_status(moe::launch_gate_up(to_internal(*p), x, sorted_pairs, expert_offsets, w_gate,
                                          w_up, h, stream),
                      "gate/up launch");
}

MOE_EXPORT moe_status moe_expert_down(const moe_problem* p, const moe_bf16* h,
                                      const int32_t* expert_offsets, const moe_bf16* w_down,
                                      float* y, hipStream_t stream) {
    MOE_TRY(check_problem(p));
    if (p->T == 0) return ok();
    MOE_TRY(check_ptr(h, "h"));
    MOE_TRY(check_ptr(expert_offsets, "expert_offsets"));
    MOE_TRY(check_ptr(w_down, "w_down"));
    MOE_TRY(check_ptr(y, "y"));
    return hip_status(moe::launch_down(to_internal(*p), h, expert_offsets, w_down, y, stream),
                      "down launch");
}

MOE_EXPORT moe_status moe_combine(const moe_problem* p, const float* y, const int32_t* pair_rows,
                                  const float* topk_weights, void* out, moe_dtype out_dtype,
                                  hipStream_t stream) {
    MOE_TRY(check_problem(p));
    if (out_dtype != MOE_DTYPE_F32 && out_dtype != MOE_DTYPE_BF16)
        return fail(MOE_ERR_INVALID_ARG, "out_dtype=%d is not MOE_DTYPE_F32/BF16", (int)out_dtype);
    if (p->T == 0) return ok();
    MOE_TRY(check_ptr(y, "y"));
    MOE_TRY(check_ptr(pair_rows, "pair_rows"));
    MOE_TRY(check_ptr(topk_weights, "topk_weights"));
    MOE_TRY(check_ptr(out, "out"));
    return hip_status(moe::launch_combine(to_internal(*p), y, pair_rows, topk_weights, out,
                                          out_dtype == MOE_DTYPE_BF16, stream),
                      "combine launch");
}

MOE_EXPORT moe_status moe_combine_residual(const moe_problem* p, const float* y,
                                           const int32_t* pair_rows, const float* topk_weights,
                                           const float* norm_weight, float eps, int32_t step,
                                           float* residual, hipStream_t stream) {
    MOE_TRY(check_problem(p));
    if (!(eps > 0.0f) || !isfinite(eps))
        return fail(MOE_ERR_INVALID_ARG, "eps=%g must be finite and > 0", (double)eps);
    if (step < 1) return fail(MOE_ERR_INVALID_ARG, "step=%d must be >= 1", step);
    if (p->H > moe::kResidualMaxH)
        return fail(MOE_ERR_UNSUPPORTED, "H=%d > %d for the fused epilogue", p->H, moe::kResidualMaxH);
    if (p->T == 0) return ok();
    MOE_TRY(check_ptr(y, "y"));
    MOE_TRY(check_ptr(pair_rows, "pair_rows"));
    MOE_TRY(check_ptr(topk_weights, "topk_weights"));
    MOE_TRY(check_ptr(norm_weight, "norm_weight"));
    MOE_TRY(check_ptr(residual, "residual"));
    // the stream weights in fp32, as the oracle takes them
    const float wa = sqrtf(static_cast<float>(step - 1) / static_cast<float>(step));
    const float wb = 1.0f / sqrtf(static_cast<float>(step));
    return hip_status(moe::launch_combine_residual(to_internal(*p), y, pair_rows, topk_weights,
                                                   norm_weight, eps, wa, wb, residual, stream),
                      "combine/residual launch");
}

MOE_EXPORT moe_status moe_dense_mlp(const moe_problem* p, const moe_bf16* x,
                                    const moe_bf16* w_gate, const moe_bf16* w_up,
                                    const moe_bf16* w_down, float* out, void* ws, size_t ws_bytes,
                                    hipStream_t stream) {
    MOE_TRY(check_problem(p));
    if (p->E != 1 || p->G != 1 || p->TG != 1 || p->k != 1)
        return fail(MOE_ERR_INVALID_ARG, "a dense MLP needs E=G=TG=k=1 (got E=%d G=%d TG=%d k=%d)",
                    p->E, p->G, p->TG, p->k);
    if (p->T == 0) return ok();
    MOE_TRY(check_ptr(x, "x"));
    MOE_TRY(check_ptr(w_gate, "w_gate"));
    MOE_TRY(check_ptr(w_up, "w_up"));
    MOE_TRY(check_ptr(w_down, "w_down"));
    MOE_TRY(check_ptr(out, "out"));
    MOE_TRY(check_ws(*p, ws, ws_bytes));
    const Layout L = layout_of(*p);
    const moe::Problem q = to_internal(*p);
    int32_t* off = at<int32_t>(ws, L.offsets);
    int32_t* sorted = at<int32_t>(ws, L.sorted);
    hipError_t e = moe::launch_identity_dispatch(p->T, off, sorted, stream);
    if (e != hipSuccess) return hip_status(e, "dispatch launch");
    e = moe::launch_expert_ffn(q, x, sorted, off, w_gate, w_up, w_down, at<uint16_t>(ws, L.h), out,
                               stream);
    return hip_status(e, "dense mlp launch");
}

MOE_EXPORT moe_status moe_expert_ffn_fp8(const moe_problem* p, const moe_bf16* x,
                                         const int32_t* sorted_pairs,
                                         const int32_t* expert_offsets, const uint8_t* w_gate,
                                         const float* s_gate, const uint8_t* w_up,
                                         const float* s_up, const uint8_t* w_down,
                                         const float* s_down, float* y, void* ws,
                                         size_t ws_bytes, hipStream_t stream) {
    MOE_TRY(check_problem(p));
    if (p->T == 0) return ok();
    MOE_TRY(check_ptr(x, "x"));
    MOE_TRY(check_ptr(sorted_pairs, "sorted_pairs"));
    MOE_TRY(check_ptr(expert_offsets, "expert_offsets"));
    MOE_TRY(check_ptr(w_gate, "w_gate"));
    MOE_TRY(check_ptr(s_gate, "s_gate"));
    MOE_TRY(check_ptr(w_up, "w_up"));
    MOE_TRY(check_ptr(s_up, "s_up"));
    MOE_TRY(check_ptr(w_down, "w_down"));
    MOE_TRY(check_ptr(s_down, "s_down"));
    MOE_TRY(check_ptr(y, "y"));
    MOE_TRY(check_ws(*p, ws, ws_bytes));
    const Layout L = layout_of(*p);
    return hip_status(moe::launch_expert_ffn_fp8(to_internal(*p), x, sorted_pairs, expert_offsets,
                                                 w_gate, s_gate, w_up, s_up, w_down, s_down,
                                                 at<uint16_t>(ws, L.h), y, stream),
                      "fp8 expert ffn launch");
}

MOE_EXPORT moe_status moe_forward_fp8(const moe_problem* p, const moe_bf16* x,
                                      const moe_bf16* w_router, const float* bias,
                                      const uint8_t* w_gate, const float* s_gate,
                                      const uint8_t* w_up, const float* s_up,
                                      const uint8_t* w_down, const float* s_down, void* out,
                                      moe_dtype out_dtype, int32_t* topk_ids,
                                      float* topk_weights, float* y, void* ws, size_t ws_bytes,
                                      hipStream_t stream) {
    MOE_TRY(check_problem(p));
    if (out_dtype != MOE_DTYPE_F32 && out_dtype != MOE_DTYPE_BF16)
        return fail(MOE_ERR_INVALID_ARG, "out_dtype=%d is not MOE_DTYPE_F32/BF16", (int)out_dtype);
    if (p->T == 0) return ok();
    MOE_TRY(check_ptr(x, "x"));
    MOE_TRY(check_ptr(w_router, "w_router"));
    MOE_TRY(check_ptr(bias, "bias", true));
    MOE_TRY(check_ptr(w_gate, "w_gate"));
    MOE_TRY(check_ptr(s_gate, "s_gate"));
    MOE_TRY(check_ptr(w_up, "w_up"));
    MOE_TRY(check_ptr(s_up, "s_up"));
    MOE_TRY(check_ptr(w_down, "w_down"));
    MOE_TRY(check_ptr(s_down, "s_down"));
    MOE_TRY(check_ptr(out, "out"));
    MOE_TRY(check_ptr(topk_ids, "topk_ids", true));
    MOE_TRY(check_ptr(topk_weights, "topk_weights", true));
    MOE_TRY(check_ptr(y, "y"));
    MOE_TRY(check_ws(*p, ws, ws_bytes));
    const Layout L = layout_of(*p);
    const moe::Problem q = to_internal(*p);
    int32_t* ids = topk_ids ? topk_ids : at<int32_t>(ws, L.ids);
    float* wts = topk_weights ? topk_weights : at<float>(ws, L.weights);
    int32_t* off = at<int32_t>(ws, L.offsets);
    int32_t* sorted = at<int32_t>(ws, L.sorted);
    int32_t* rows = at<int32_t>(ws, L.rows);
    // the h region is written only by the expert step, after routing: it
    // doubles as the router's score scratch
    const size_t h_bytes = static_cast<size_t>(p->T) * static_cast<size_t>(p->k) *
                           static_cast<size_t>(p->I) * 2;
    hipError_t e = moe::launch_route_scratch(q, x, w_router, bias, ids, wts, at<uint16_t>(ws, L.h),
                                             h_bytes, stream);
    if (e != hipSuccess) return hip_status(e, "route launch");
    e = moe::launch_permute(q, ids, off, sorted, rows, at<int32_t>(ws, L.counts), stream);
    if (e != hipSuccess) return hip_status(e, "permute launch");
    e = moe::launch_expert_ffn_fp8(q, x, sorted, off, w_gate, s_gate, w_up, s_up, w_down, s_down,
                                   at<uint16_t>(ws, L.h), y, stream);
    if (e != hipSuccess) return hip_status(e, "fp8 expert ffn launch");
    e = moe::launch_combine(q, y, rows, wts, out, out_dtype == MOE_DTYPE_BF16, stream);
    return hip_status(e, "combine launch");
}

MOE_EXPORT moe_status moe_forward(const moe_problem* p, const moe_bf16* x,
                                  const moe_bf16* w_router, const float* bias,
                                  const moe_bf16* w_gate, const moe_bf16* w_up,
                                  const moe_bf16* w_down, void* out, moe_dtype out_dtype,
                                  int32_t* topk_ids, float* topk_weights, float* y, void* ws,
                                  size_t ws_bytes, hipStream_t stream) {
    MOE_TRY(check_problem(p));
    if (out_dtype != MOE_DTYPE_F32 && out_dtype != MOE_DTYPE_BF16)
        return fail(MOE_ERR_INVALID_ARG, "out_dtype=%d is not MOE_DTYPE_F32/BF16", (int)out_dtype);
    if (p->T == 0) return ok();
    MOE_TRY(check_ptr(x, "x"));
    MOE_TRY(check_ptr(w_router, "w_router"));
    MOE_TRY(check_ptr(bias, "bias", true));
    MOE_TRY(check_ptr(w_gate, "w_gate"));
    MOE_TRY(check_ptr(w_up, "w_up"));
    MOE_TRY(check_ptr(w_down, "w_down"));
    MOE_TRY(check_ptr(out, "out"));
    MOE_TRY(check_ptr(topk_ids, "topk_ids", true));
    MOE_TRY(check_ptr(topk_weights, "topk_weights", true));
    MOE_TRY(check_ptr(y, "y"));
    MOE_TRY(check_ws(*p, ws, ws_bytes));
    const Layout L = layout_of(*p);
    const moe::Problem q = to_internal(*p);
    int32_t* ids = topk_ids ? topk_ids : at<int32_t>(ws, L.ids);
    float* wts = topk_weights ? topk_weights : at<float>(ws, L.weights);
    int32_t* off = at<int32_t>(ws, L.offsets);
    int32_t* sorted = at<int32_t>(ws, L.sorted);
    int32_t* rows = at<int32_t>(ws, L.rows);
    // the h region is written only by the expert step, after routing: it
    // doubles as the router's score scratch
    const size_t h_bytes = static_cast<size_t>(p->T) * static_cast<size_t>(p->k) *
                           static_cast<size_t>(p->I) * 2;
    hipError_t e = moe::launch_route_scratch(q, x, w_router, bias, ids, wts, at<uint16_t>(ws, L.h),
                                             h_bytes, stream);
    if (e != hipSuccess) return hip_status(e, "route launch");
    e = moe::launch_permute(q, ids, off, sorted, rows, at<int32_t>(ws, L.counts), stream);
    if (e != hipSuccess) return hip_status(e, "permute launch");
    e = moe::launch_expert_ffn(q, x, sorted, off, w_gate, w_up, w_down, at<uint16_t>(ws, L.h), y,
                               stream);
    if (e != hipSuccess) return hip_status(e, "expert ffn launch");
    e = moe::launch_combine(q, y, rows, wts, out, out_dtype == MOE_DTYPE_BF16, stream);
    return hip_status(e, "combine launch");
}

MOE_EXPORT moe_status moe_forward_noalloc(const moe_problem* p, const moe_bf16* x,
                                          const moe_bf16* w_router, const float* bias,
                                          const moe_bf16* w_gate, const moe_bf16* w_up,
                                          const moe_bf16* w_down, void* out, moe_dtype out_dtype,
                                          int32_t* topk_ids, float* topk_weights, float* y,
                                          hipStream_t stream) {
    MOE_TRY(check_problem(p));
    if (out_dtype != MOE_DTYPE_F32 && out_dtype != MOE_DTYPE_BF16)
        return fail(MOE_ERR_INVALID_ARG, "out_dtype=%d is not MOE_DTYPE_F32/BF16", (int)out_dtype);
    if (p->T == 0) return ok();
    MOE_TRY(check_ptr(x, "x"));
    MOE_TRY(check_ptr(w_router, "w_router"));
    MOE_TRY(check_ptr(bias, "bias", true));
    MOE_TRY(check_ptr(w_gate, "w_gate"));
    MOE_TRY(check_ptr(w_up, "w_up"));
    MOE_TRY(check_ptr(w_down, "w_down"));
    MOE_TRY(check_ptr(out, "out"));
    MOE_TRY(check_ptr(topk_ids, "topk_ids", true));
    MOE_TRY(check_ptr(topk_weights, "topk_weights", true));
    MOE_TRY(check_ptr(y, "y"));
    const size_t need = layout_of(*p).total;
    if (need > static_cast<size_t>(MOE_NOALLOC_SCRATCH_BYTES))
        return fail(MOE_ERR_UNSUPPORTED,
                    "the problem needs %zu bytes of scratch; the static scratch holds %zu "
                    "(call moe_forward with a workspace)",
                    need, static_cast<size_t>(MOE_NOALLOC_SCRATCH_BYTES));
    void* ws = nullptr;
    MOE_TRY(device_scratch(&ws));
    // the same kernels and workspace layout as moe_forward; nothing in the
    // workspace has to start at zero (every scratch value is written before
    // it is read), so the previous call's contents need no clearing
    return moe_forward(p, x, w_router, bias, w_gate, w_up, w_down, out, out_dtype, topk_ids,
                       topk_weights, y, ws, need, stream);
}

// ---- grouped products (moe_gemm.h) ----

MOE_EXPORT size_t moe_gemm_workspace_bytes(const moe_gemm_problem* g) {
    if (check_gemm(g, 8) != MOE_OK) return 0;
    ok();
    return all_gemm_ws_bytes(*g);
}

MOE_EXPORT moe_status moe_grouped_gemm(const moe_gemm_problem* g, const moe_bf16* a,
                                       const int32_t* sorted_pairs, const int32_t* expert_offsets,
                                       const moe_bf16* w, void* out, moe_dtype out_dtype, void* ws,
                                       size_t ws_bytes, hipStream_t stream) {
    MOE_TRY(check_gemm(g, 8));
    MOE_TRY(check_outputs(g->P, g->N));
    MOE_TRY(check_gemm_out(out_dtype, 0));
    MOE_TRY(check_rows(*g, sorted_pairs));
    if (g->P == 0) return ok();
    MOE_TRY(check_offsets(*g, expert_offsets));
    MOE_TRY(check_ptr(a, "a"));
    MOE_TRY(check_ptr(w, "w"));
    MOE_TRY(check_ptr(out, "out"));
    MOE_TRY(check_gemm_ws(*g, ws, ws_bytes));
    moe::GemmArgs x = gemm_args(*g);
    x.a = a;
    x.w = w;
    x.pairs = sorted_pairs;
    x.offsets = expert_offsets;
    x.out = out;
    x.out_bf16 = out_dtype == MOE_DTYPE_BF16;
    x.ws = ws;
    return hip_status(moe::launch_grouped_gemm(x, stream), "grouped gemm launch");
}

MOE_EXPORT moe_status moe_grouped_gemm_dgrad(const moe_gemm_problem* g, const moe_bf16* dout,
                                             const int32_t* expert_offsets, const moe_bf16* w,
                                             void* da, moe_dtype da_dtype, int accumulate, void* ws,
                                             size_t ws_bytes, hipStream_t stream) {
    MOE_TRY(check_gemm(g, 8));
    MOE_TRY(check_outputs(g->P, g->K));
    MOE_TRY(check_gemm_out(da_dtype, accumulate));
    if (g->P == 0) return ok();
    MOE_TRY(check_offsets(*g, expert_offsets));
    MOE_TRY(check_ptr(dout, "dout"));
    MOE_TRY(check_ptr(w, "w"));
    MOE_TRY(check_ptr(da, "da"));
    MOE_TRY(check_gemm_ws(*g, ws, ws_bytes));
    moe::GemmArgs x = gemm_args(*g);
    x.dout = dout;
    x.w = w;
    x.offsets = expert_offsets;
    x.out = da;
    x.out_bf16 = da_dtype == MOE_DTYPE_BF16;
    x.accumulate = accumulate != 0;
    x.ws = ws;
    return hip_status(moe::launch_grouped_dgrad(x, stream), "grouped gemm input gradient launch");
}

MOE_EXPORT moe_status moe_grouped_gemm_wgrad(const moe_gemm_problem* g, const moe_bf16* dout,
                                             const moe_bf16* a, const int32_t* sorted_pairs,
                                             const int32_t* expert_offsets, void* dw,
                                             moe_dtype dw_dtype, int accumulate, void* ws,
                                             size_t ws_bytes, hipStream_t stream) {
    MOE_TRY(check_gemm(g, 8));
    MOE_TRY(check_gemm_out(dw_dtype, accumulate));
    MOE_TRY(check_rows(*g, sorted_pairs));
    MOE_TRY(check_offsets(*g, expert_offsets));
    MOE_TRY(check_ptr(dout, "dout", g->P == 0));
    MOE_TRY(check_ptr(a, "a", g->P == 0));
    MOE_TRY(check_ptr(dw, "dw"));
    MOE_TRY(check_gemm_ws(*g, ws, ws_bytes));
    moe::GemmArgs x = gemm_args(*g);
    x.dout = dout;
    x.a = a;
    x.pairs = sorted_pairs;
    x.offsets = expert_offsets;
    x.out = dw;
    x.out_bf16 = dw_dtype == MOE_DTYPE_BF16;
    x.accumulate = accumulate != 0;
    x.ws = ws;
    return hip_status(moe::launch_grouped_wgrad(x, stream), "grouped gemm weight gradient launch");
}

MOE_EXPORT moe_status moe_quantize_rows_int8(int64_t rows, int32_t K, const moe_bf16* x,
                                             int8_t* codes, float* scales, hipStream_t stream) {
    if (rows < 0 || rows > 0x7fffffffLL)
        return fail(MOE_ERR_INVALID_ARG, "rows=%lld must be in [0, 2^31)", (long long)rows);
    if (K <= 0 || K % 16 != 0)
        return fail(MOE_ERR_INVALID_ARG, "K=%d must be a positive multiple of 16", K);
    if (K > kMaxDim) return fail(MOE_ERR_UNSUPPORTED, "K=%d > %d", K, kMaxDim);
    if (rows == 0) return ok();
    MOE_TRY(check_ptr(x, "x"));
    MOE_TRY(check_ptr(codes, "codes"));
    MOE_TRY(check_ptr(scales, "scales"));
    return hip_status(moe::launch_quantize_rows(rows, K, x, codes, scales, stream), "quantize launch");
}

MOE_EXPORT moe_status moe_grouped_gemm_int8(const moe_gemm_problem* g, const int8_t* a,
                                            const float* a_scale, const int32_t* sorted_pairs,
                                            const int32_t* expert_offsets, const int8_t* w,
                                            const float* w_scale, void* out, moe_dtype out_dtype,
                                            void* ws, size_t ws_bytes, hipStream_t stream) {
    MOE_TRY(check_gemm(g, 16));
    MOE_TRY(check_outputs(g->P, g->N));
    MOE_TRY(check_gemm_out(out_dtype, 0));
    MOE_TRY(check_rows(*g, sorted_pairs));
    if (g->P == 0) return ok();
    MOE_TRY(check_offsets(*g, expert_offsets));
    MOE_TRY(check_ptr(a, "a"));
    MOE_TRY(check_ptr(a_scale, "a_scale"));
    MOE_TRY(check_ptr(w, "w"));
    MOE_TRY(check_ptr(w_scale, "w_scale"));
    MOE_TRY(check_ptr(out, "out"));
    MOE_TRY(check_gemm_ws(*g, ws, ws_bytes));
    moe::GemmArgs x = gemm_args(*g);
    x.a = a;
    x.a_scale = a_scale;
    x.w = w;
    x.w_scale = w_scale;
    x.pairs = sorted_pairs;
    x.offsets = expert_offsets;
    x.out = out;
    x.out_bf16 = out_dtype == MOE_DTYPE_BF16;
    x.ws = ws;
    return hip_status(moe::launch_grouped_int8(x, stream), "grouped int8 gemm launch");
}

// ---- the experts on these products ----

namespace {

// What follows the forward pass's own workspace: the products' sums, their
// operands, the scratch of split reductions.
struct Int8Layout {
    size_t x, x_scale, g, u, h, h_scale, sums, total;
};

Int8Layout int8_layout(const moe_problem& p) {
    const size_t P = static_cast<size_t>(p.T) * static_cast<size_t>(p.k), T = static_cast<size_t>(p.T);
    const size_t H = static_cast<size_t>(p.H), I = static_cast<size_t>(p.I);
    const size_t a = gemm_ws_bytes(gate_shape(p)), b = gemm_ws_bytes(down_shape(p));
    Int8Layout L{};
    size_t o = layout_of(p).total;
    L.x = o;       o += align_up(T * H);
    L.x_scale = o; o += align_up(T * 4);
    L.g = o;       o += align_up(P * I * 4);
    L.u = o;       o += align_up(P * I * 4);
    L.h = o;       o += align_up(P * I);
    L.h_scale = o; o += align_up(P * 4);
    L.sums = o;    o += align_up(a > b ? a : b);
    L.total = o;
    return L;
}

struct BackwardLayout {
    size_t g, u, dh, h, dg, du, sums, total;
};

BackwardLayout backward_layout(const moe_problem& p) {
    const size_t PI = static_cast<size_t>(p.T) * static_cast<size_t>(p.k) * static_cast<size_t>(p.I);
    const size_t a = gemm_ws_bytes(gate_shape(p)), b = gemm_ws_bytes(down_shape(p));
    BackwardLayout L{};
    size_t o = 0;
    L.g = o;    o += align_up(PI * 4);
    L.u = o;    o += align_up(PI * 4);
    L.dh = o;   o += align_up(PI * 4);
    L.h = o;    o += align_up(PI * 2);
    L.dg = o;   o += align_up(PI * 2);
    L.du = o;   o += align_up(PI * 2);
    L.sums = o; o += align_up(a > b ? a : b);
    L.total = o;
    return L;
}

struct Int8Weights {
    const int8_t *gate, *up, *down;
    const float *s_gate, *s_up, *s_down;
};

hipError_t run_ffn_int8(const moe_problem& p, const moe_bf16* x, const int32_t* sorted, const int32_t* off,
                        const Int8Weights& w, float* y, void* ws, hipStream_t stream) {
    const Int8Layout L = int8_layout(p);
    int8_t* xc = at<int8_t>(ws, L.x);
    float* xs = at<float>(ws, L.x_scale);
    hipError_t e = moe::launch_quantize_rows(p.T, p.H, x, xc, xs, stream);
    if (e != hipSuccess) return e;
    moe::GemmArgs a = gemm_args(gate_shape(p));
    a.a = xc;
    a.a_scale = xs;
    a.pairs = sorted;
    a.offsets = off;
    a.ws = at<char>(ws, L.sums);
    a.w = w.gate;
    a.w_scale = w.s_gate;
    a.out = at<float>(ws, L.g);
    e = moe::launch_grouped_int8(a, stream);
    if (e != hipSuccess) return e;
    a.w = w.up;
    a.w_scale = w.s_up;
    a.out = at<float>(ws, L.u);
    e = moe::launch_grouped_int8(a, stream);
    if (e != hipSuccess) return e;
    e = moe::launch_swiglu_quantize(at<float>(ws, L.g), at<float>(ws, L.u), a.P, p.I, off, p.E,
                                    at<int8_t>(ws, L.h), at<float>(ws, L.h_scale), stream);
    if (e != hipSuccess) return e;
    moe::GemmArgs d = gemm_args(down_shape(p));
    d.a = at<int8_t>(ws, L.h);
    d.a_scale = at<float>(ws, L.h_scale);
    d.offsets = off;
    d.ws = at<char>(ws, L.sums);
    d.w = w.down;
    d.w_scale = w.s_down;
    d.out = y;
    return moe::launch_grouped_int8(d, stream);
}

moe_status check_int8_weights(const Int8Weights& w) {
    MOE_TRY(check_ptr(w.gate, "w_gate"));
    MOE_TRY(check_ptr(w.s_gate, "s_gate"));
    MOE_TRY(check_ptr(w.up, "w_up"));
    MOE_TRY(check_ptr(w.s_up, "s_up"));
    MOE_TRY(check_ptr(w.down, "w_down"));
    return check_ptr(w.s_down, "s_down");
}

}  // namespace

MOE_EXPORT size_t moe_int8_workspace_bytes(const moe_problem* p) {
    if (check_problem(p) != MOE_OK || check_expert_outputs(*p) != MOE_OK) return 0;
    return int8_layout(*p).total;
}

MOE_EXPORT moe_status moe_expert_ffn_int8(const moe_problem* p, const moe_bf16* x,
                                          const int32_t* sorted_pairs,
                                          const int32_t* expert_offsets, const int8_t* w_gate,
                                          const float* s_gate, const int8_t* w_up,
                                          const float* s_up, const int8_t* w_down,
                                          const float* s_down, float* y, void* ws, size_t ws_bytes,
                                          hipStream_t stream) {
    MOE_TRY(check_problem(p));
    MOE_TRY(check_expert_outputs(*p));
    if (p->T == 0) return ok();
    const Int8Weights w{w_gate, w_up, w_down, s_gate, s_up, s_down};
    MOE_TRY(check_ptr(x, "x"));
    MOE_TRY(check_ptr(sorted_pairs, "sorted_pairs"));
    MOE_TRY(check_ptr(expert_offsets, "expert_offsets"));
    MOE_TRY(check_int8_weights(w));
    MOE_TRY(check_ptr(y, "y"));
    MOE_TRY(check_ws_bytes(int8_layout(*p).total, ws, ws_bytes));
    return hip_status(run_ffn_int8(*p, x, sorted_pairs, expert_offsets, w, y, ws, stream),
                      "int8 expert ffn launch");
}

MOE_EXPORT moe_status moe_forward_int8(const moe_problem* p, const moe_bf16* x,
                                       const moe_bf16* w_router, const float* bias,
                                       const int8_t* w_gate, const float* s_gate,
                                       const int8_t* w_up, const float* s_up,
                                       const int8_t* w_down, const float* s_down, void* out,
                                       moe_dtype out_dtype, int32_t* topk_ids,
                                       float* topk_weights, float* y, void* ws, size_t ws_bytes,
                                       hipStream_t stream) {
    MOE_TRY(check_problem(p));
    MOE_TRY(check_expert_outputs(*p));
    if (out_dtype != MOE_DTYPE_F32 && out_dtype != MOE_DTYPE_BF16)
        return fail(MOE_ERR_INVALID_ARG, "out_dtype=%d is not MOE_DTYPE_F32/BF16", (int)out_dtype);
    if (p->T == 0) return ok();
    const Int8Weights w{w_gate, w_up, w_down, s_gate, s_up, s_down};
    MOE_TRY(check_ptr(x, "x"));
    MOE_TRY(check_ptr(w_router, "w_router"));
    MOE_TRY(check_ptr(bias, "bias", true));
    MOE_TRY(check_int8_weights(w));
    MOE_TRY(check_ptr(out, "out"));
    MOE_TRY(check_ptr(topk_ids, "topk_ids", true));
    MOE_TRY(check_ptr(topk_weights, "topk_weights", true));
    MOE_TRY(check_ptr(y, "y"));
    MOE_TRY(check_ws_bytes(int8_layout(*p).total, ws, ws_bytes));
    const Layout L = layout_of(*p);
    const moe::Problem q = to_internal(*p);
    int32_t* ids = topk_ids ? topk_ids : at<int32_t>(ws, L.ids);
    float* wts = topk_weights ? topk_weights : at<float>(ws, L.weights);
    int32_t* off = at<int32_t>(ws, L.offsets);
    int32_t* sorted = at<int32_t>(ws, L.sorted);
    int32_t* rows = at<int32_t>(ws, L.rows);
    const size_t h_bytes = static_cast<size_t>(p->T) * static_cast<size_t>(p->k) *
                           static_cast<size_t>(p->I) * 2;
    hipError_t e = moe::launch_route_scratch(q, x, w_router, bias, ids, wts, at<uint16_t>(ws, L.h),
                                             h_bytes, stream);
    if (e != hipSuccess) return hip_status(e, "route launch");
    e = moe::launch_permute(q, ids, off, sorted, rows, at<int32_t>(ws, L.counts), stream);
    if (e != hipSuccess) return hip_status(e, "permute launch");
    e = run_ffn_int8(*p, x, sorted, off, w, y, ws, stream);
    if (e != hipSuccess) return hip_status(e, "int8 expert ffn launch");
    e = moe::launch_combine(q, y, rows, wts, out, out_dtype == MOE_DTYPE_BF16, stream);
    return hip_status(e, "combine launch");
}

MOE_EXPORT size_t moe_backward_workspace_bytes(const moe_problem* p) {
    if (check_problem(p) != MOE_OK || check_expert_outputs(*p) != MOE_OK) return 0;
    return backward_layout(*p).total;
}

MOE_EXPORT moe_status moe_expert_ffn_backward(const moe_problem* p, const moe_bf16* x,
                                              const int32_t* sorted_pairs,
                                              const int32_t* expert_offsets,
                                              const moe_bf16* w_gate, const moe_bf16* w_up,
                                              const moe_bf16* w_down, const moe_bf16* dy, float* dx,
                                              void* dw_gate, void* dw_up, void* dw_down,
                                              moe_dtype dw_dtype, int accumulate, void* ws,
                                              size_t ws_bytes, hipStream_t stream) {
    MOE_TRY(check_problem(p));
    MOE_TRY(check_expert_outputs(*p));
    MOE_TRY(check_gemm_out(dw_dtype, accumulate));
    const bool empty = p->T == 0;
    MOE_TRY(check_ptr(x, "x", empty));
    MOE_TRY(check_ptr(sorted_pairs, "sorted_pairs", empty));
    MOE_TRY(check_ptr(expert_offsets, "expert_offsets", empty && p->E == 1));
    MOE_TRY(check_ptr(w_gate, "w_gate"));
    MOE_TRY(check_ptr(w_up, "w_up"));
    MOE_TRY(check_ptr(w_down, "w_down"));
    MOE_TRY(check_ptr(dy, "dy", empty));
    MOE_TRY(check_ptr(dx, "dx", empty));
    MOE_TRY(check_ptr(dw_gate, "dw_gate"));
    MOE_TRY(check_ptr(dw_up, "dw_up"));
    MOE_TRY(check_ptr(dw_down, "dw_down"));
    const BackwardLayout L = backward_layout(*p);
    MOE_TRY(check_ws_bytes(L.total, ws, ws_bytes));
    const char* what = "expert ffn backward launch";
    void* sums = at<char>(ws, L.sums);
    // the products again: g, u = x . w^T and dh = dy . w_down, in fp32
    moe::GemmArgs a = gemm_args(gate_shape(*p));
    a.a = x;
    a.pairs = sorted_pairs;
    a.offsets = expert_offsets;
    a.ws = sums;
    moe::GemmArgs d = gemm_args(down_shape(*p));
    d.offsets = expert_offsets;
    d.ws = sums;
    hipError_t e = hipSuccess;
    if (!empty) {
        a.w = w_gate;
        a.out = at<float>(ws, L.g);
        e = moe::launch_grouped_gemm(a, stream);
        if (e != hipSuccess) return hip_status(e, what);
        a.w = w_up;
        a.out = at<float>(ws, L.u);
        e = moe::launch_grouped_gemm(a, stream);
        if (e != hipSuccess) return hip_status(e, what);
        d.dout = dy;
        d.w = w_down;
        d.out = at<float>(ws, L.dh);
        e = moe::launch_grouped_dgrad(d, stream);
        if (e != hipSuccess) return hip_status(e, what);
        e = moe::launch_swiglu_backward(at<float>(ws, L.g), at<float>(ws, L.u), at<float>(ws, L.dh), a.P * p->I,
                                        at<uint16_t>(ws, L.h), at<uint16_t>(ws, L.dg), at<uint16_t>(ws, L.du),
                                        stream);
        if (e != hipSuccess) return hip_status(e, what);
        // dx = dg . w_gate + du . w_up
        a.dout = at<uint16_t>(ws, L.dg);
        a.w = w_gate;
        a.out = dx;
        e = moe::launch_grouped_dgrad(a, stream);
        if (e != hipSuccess) return hip_status(e, what);
        a.dout = at<uint16_t>(ws, L.du);
        a.w = w_up;
        a.accumulate = true;
        e = moe::launch_grouped_dgrad(a, stream);
        if (e != hipSuccess) return hip_status(e, what);
    }
    a.out_bf16 = dw_dtype == MOE_DTYPE_BF16;
    a.accumulate = accumulate != 0;
    a.dout = at<uint16_t>(ws, L.dg);
    a.out = dw_gate;
    e = moe::launch_grouped_wgrad(a, stream);
    if (e != hipSuccess) return hip_status(e, what);
    a.dout = at<uint16_t>(ws, L.du);
    a.out = dw_up;
    e = moe::launch_grouped_wgrad(a, stream);
    if (e != hipSuccess) return hip_status(e, what);
    d.out_bf16 = a.out_bf16;
    d.accumulate = a.accumulate;
    d.dout = dy;
    d.a = at<uint16_t>(ws, L.h);
    d.out = dw_down;
    return hip_status(moe::launch_grouped_wgrad(d, stream), what);
}

MOE_EXPORT const char* moe_status_string(moe_status s) {
    switch (s) {
        case MOE_OK: return "MOE_OK";
        case MOE_ERR_INVALID_ARG: return "MOE_ERR_INVALID_ARG";
        case MOE_ERR_UNSUPPORTED: return "MOE_ERR_UNSUPPORTED";
        case MOE_ERR_WORKSPACE: return "MOE_ERR_WORKSPACE";
        case MOE_ERR_HIP: return "MOE_ERR_HIP";
    }
    return "MOE_ERR_UNKNOWN";
}

MOE_EXPORT const char* moe_last_error(void) { return g_last_error.c_str(); }
