// fp8_api.hip -- the C ABI of include/moe_fp8.h: argument checks, workspace
// layout and kernel launches.  Host side only.
#include "moe_fp8.h"

#include "api.h"
#include "fp8_kernels.h"

using namespace moe::api;

namespace {

moe_status check_fp8_gemm(const moe_gemm_problem* g) {
    MOE_TRY(check_gemm(g, 16));
    if (g->N % 16 != 0) return fail(MOE_ERR_INVALID_ARG, "N=%d must be a positive multiple of 16", g->N);
    return MOE_OK;
}

// Gathered rows are addressed with 32-bit offsets.
moe_status check_gathered(int64_t rows, int64_t cols, const int32_t* sorted_pairs) {
    if (sorted_pairs && rows * cols > moe::kMaxGatherBytes)
        return fail(MOE_ERR_UNSUPPORTED, "%lld x %lld gathered codes > 4 GiB less 1 MiB", (long long)rows,
                    (long long)cols);
    return MOE_OK;
}

moe::Fp8Args fp8_args(const moe_gemm_problem& g, const int32_t* sorted_pairs, const int32_t* expert_offsets) {
    moe::Fp8Args a{};
    a.P = g.P;
    a.S = g.S;
    a.E = g.E;
    a.N = g.N;
    a.K = g.K;
    a.k = g.k;
    a.pairs = sorted_pairs;
    a.offsets = expert_offsets;
    return a;
}

void set_rows(moe::Fp8Args& a, const uint8_t* y, const uint8_t* scale, int cols) {
    a.y = y;
    a.y_cols = cols;
    a.y_scale = scale;
    a.y_pitch = moe::scale_pitch(cols);
}

struct Fp8Weights {
    const uint8_t *gate, *s_gate, *up, *s_up, *down, *s_down;
};

moe_status check_weights(const Fp8Weights& w) {
    MOE_TRY(check_ptr(w.gate, "w_gate"));
    MOE_TRY(check_ptr(w.s_gate, "s_gate"));
    MOE_TRY(check_ptr(w.up, "w_up"));
    MOE_TRY(check_ptr(w.s_up, "s_up"));
    MOE_TRY(check_ptr(w.down, "w_down"));
    return check_ptr(w.s_down, "s_down");
}

// The dispatch of the experts' calls: a dense layer may leave it out.
moe_status check_dispatch(const moe_problem& p, const int32_t* sorted_pairs, const int32_t* expert_offsets) {
    const bool dense = p.E == 1 && p.k == 1;
    MOE_TRY(check_ptr(sorted_pairs, "sorted_pairs", dense));
    MOE_TRY(check_ptr(expert_offsets, "expert_offsets", dense));
    return check_gathered(p.T, p.H, sorted_pairs);
}

// The workspace: the dispatch of the forward pass, x and h as codes and
// scales, the parts of split sums.
struct FfnLayout {
    size_t x, x_scale, h, h_scale, sums, total;
};

FfnLayout ffn_layout(const moe_problem& p) {
    const size_t T = static_cast<size_t>(p.T), P = T * static_cast<size_t>(p.k);
    FfnLayout L{};
    size_t o = layout_of(p).h;
    L.x = o;       o += align_up(T * static_cast<size_t>(p.H));
    L.x_scale = o; o += align_up(T * static_cast<size_t>(moe::scale_pitch(p.H)));
    L.h = o;       o += align_up(P * static_cast<size_t>(p.I));
    L.h_scale = o; o += align_up(P * static_cast<size_t>(moe::scale_pitch(p.I)));
    L.sums = o;    o += align_up(moe::fp8_ws_bytes(p.T * p.k, p.E, p.H, p.I));
    L.total = o;
    return L;
}

// Columns of [dg | du]: each part of whole blocks.
int pair_cols(int I) { return 2 * moe::blocks_of(I) * moe::kBlock; }

struct BackwardLayout {
    size_t x, x_scale, dy, dy_scale, dh, h, dg, du, d, d_scale, sums, total;
};

BackwardLayout backward_layout(const moe_problem& p) {
    const size_t T = static_cast<size_t>(p.T), P = T * static_cast<size_t>(p.k);
    const size_t H = static_cast<size_t>(p.H), PI = P * static_cast<size_t>(p.I);
    const size_t D = static_cast<size_t>(pair_cols(p.I));
    const size_t row_scales = static_cast<size_t>(moe::scale_pitch(p.H));
    size_t sums = gemm_ws_bytes(gate_shape(p));
    auto at_least = [&](size_t n) { sums = sums > n ? sums : n; };
    at_least(gemm_ws_bytes(down_shape(p)));
    at_least(moe::fp8_ws_bytes(p.T * p.k, p.E, p.H, p.I));
    at_least(moe::fp8_pair_ws_bytes(p.T * p.k, p.E, p.I, p.H));
    BackwardLayout L{};
    size_t o = 0;
    L.x = o;        o += align_up(T * H);
    L.x_scale = o;  o += align_up(T * row_scales);
    L.dy = o;       o += align_up(P * H);
    L.dy_scale = o; o += align_up(P * row_scales);
    L.dh = o;       o += align_up(PI * 4);
    L.h = o;        o += align_up(PI * 2);
    L.dg = o;       o += align_up(PI * 2);
    L.du = o;       o += align_up(PI * 2);
    L.d = o;        o += align_up(P * D);
    L.d_scale = o;  o += align_up(P * static_cast<size_t>(moe::scale_pitch(pair_cols(p.I))));
    L.sums = o;     o += align_up(sums);
    L.total = o;
    return L;
}

moe::Fp8Args gate_up_args(const moe_problem& p, const uint8_t* x, const uint8_t* x_scale, const int32_t* sorted,
                          const int32_t* off, const Fp8Weights& w) {
    moe::Fp8Args a = fp8_args(gate_shape(p), sorted, off);
    set_rows(a, x, x_scale, p.H);
    a.w[0] = w.gate;
    a.w[1] = w.up;
    a.w_scale[0] = w.s_gate;
    a.w_scale[1] = w.s_up;
    return a;
}

hipError_t run_gate_up(const moe_problem& p, const uint8_t* x, const uint8_t* x_scale, const int32_t* sorted,
                       const int32_t* off, const Fp8Weights& w, uint8_t* h, uint8_t* h_scale, hipStream_t s) {
    moe::Fp8Args a = gate_up_args(p, x, x_scale, sorted, off, w);
    a.q = h;
    a.q_cols = p.I;
    a.q_scale = h_scale;
    a.q_pitch = moe::scale_pitch(p.I);
    return moe::launch_fp8_gate_up(a, s);
}

hipError_t run_ffn(const moe_problem& p, const moe_bf16* x, const int32_t* sorted, const int32_t* off,
                   const Fp8Weights& w, void* y, bool y_bf16, void* ws, hipStream_t s) {
    const FfnLayout L = ffn_layout(p);
    uint8_t* xq = at<uint8_t>(ws, L.x);
    uint8_t* xs = at<uint8_t>(ws, L.x_scale);
    uint8_t* hq = at<uint8_t>(ws, L.h);
    uint8_t* hs = at<uint8_t>(ws, L.h_scale);
    hipError_t e = moe::launch_fp8_rows(p.T, p.H, x, xq, xs, s);
    if (e != hipSuccess) return e;
    e = run_gate_up(p, xq, xs, sorted, off, w, hq, hs, s);
    if (e != hipSuccess) return e;
    moe::Fp8Args d = fp8_args(down_shape(p), nullptr, off);
    set_rows(d, hq, hs, p.I);
    d.w[0] = w.down;
    d.w_scale[0] = w.s_down;
    d.out = y;
    d.out_bf16 = y_bf16;
    d.ws = at<char>(ws, L.sums);
    return moe::launch_fp8_product(d, s);
}

}  // namespace

MOE_EXPORT int32_t moe_fp8_block_scales(int32_t C) { return C <= 0 ? 0 : moe::scale_pitch(C); }

MOE_EXPORT moe_status moe_quantize_rows_fp8_block(int64_t rows, int32_t K, const moe_bf16* x, uint8_t* codes,
                                                  uint8_t* scales, hipStream_t stream) {
    if (rows < 0 || rows > 0x7fffffffLL)
        return fail(MOE_ERR_INVALID_ARG, "rows=%lld must be in [0, 2^31)", (long long)rows);
    if (K <= 0 || K % 16 != 0) return fail(MOE_ERR_INVALID_ARG, "K=%d must be a positive multiple of 16", K);
    if (K > kMaxDim) return fail(MOE_ERR_UNSUPPORTED, "K=%d > %d", K, kMaxDim);
    if (rows == 0) return ok();
    MOE_TRY(check_ptr(x, "x"));
    MOE_TRY(check_ptr(codes, "codes"));
    MOE_TRY(check_ptr(scales, "scales"));
    return hip_status(moe::launch_fp8_rows(rows, K, x, codes, scales, stream), "fp8 quantize launch");
}

MOE_EXPORT moe_status moe_quantize_weights_fp8_block(int32_t E, int32_t N, int32_t K, const moe_bf16* w,
                                                     uint8_t* codes, uint8_t* scales, hipStream_t stream) {
    const moe_gemm_problem g{0, 0, E, N, K, 1};
    MOE_TRY(check_fp8_gemm(&g));
    MOE_TRY(check_ptr(w, "w"));
    MOE_TRY(check_ptr(codes, "codes"));
    MOE_TRY(check_ptr(scales, "scales"));
    return hip_status(moe::launch_fp8_weights(E, N, K, w, codes, scales, stream), "fp8 weight quantize launch");
}

MOE_EXPORT moe_status moe_grouped_gemm_fp8_block(const moe_gemm_problem* g, const uint8_t* a,
                                                 const uint8_t* a_scale, const int32_t* sorted_pairs,
                                                 const int32_t* expert_offsets, const uint8_t* w,
                                                 const uint8_t* w_scale, void* out, moe_dtype out_dtype, void* ws,
                                                 size_t ws_bytes, hipStream_t stream) {
    MOE_TRY(check_fp8_gemm(g));
    MOE_TRY(check_outputs(g->P, g->N));
    MOE_TRY(check_gemm_out(out_dtype, 0));
    MOE_TRY(check_rows(*g, sorted_pairs));
    if (g->P == 0) return ok();
    MOE_TRY(check_gathered(g->S, g->K, sorted_pairs));
    MOE_TRY(check_offsets(*g, expert_offsets));
    MOE_TRY(check_ptr(a, "a"));
    MOE_TRY(check_ptr(a_scale, "a_scale"));
    MOE_TRY(check_ptr(w, "w"));
    MOE_TRY(check_ptr(w_scale, "w_scale"));
    MOE_TRY(check_ptr(out, "out"));
    MOE_TRY(check_ws_bytes(all_gemm_ws_bytes(*g), ws, ws_bytes));
    moe::Fp8Args x = fp8_args(*g, sorted_pairs, expert_offsets);
    set_rows(x, a, a_scale, g->K);
    x.w[0] = w;
    x.w_scale[0] = w_scale;
    x.out = out;
    x.out_bf16 = out_dtype == MOE_DTYPE_BF16;
    x.ws = ws;
    return hip_status(moe::launch_fp8_product(x, stream), "fp8 grouped gemm launch");
}

MOE_EXPORT moe_status moe_grouped_gemm_fp8_block_dgrad(const moe_gemm_problem* g, const uint8_t* dout,
                                                       const uint8_t* dout_scale, const int32_t* expert_offsets,
                                                       const uint8_t* w, const uint8_t* w_scale, void* da,
                                                       moe_dtype da_dtype, int accumulate, void* ws,
                                                       size_t ws_bytes, hipStream_t stream) {
    MOE_TRY(check_fp8_gemm(g));
    MOE_TRY(check_outputs(g->P, g->K));
    MOE_TRY(check_gemm_out(da_dtype, accumulate));
    if (g->P == 0) return ok();
    MOE_TRY(check_offsets(*g, expert_offsets));
    MOE_TRY(check_ptr(dout, "dout"));
    MOE_TRY(check_ptr(dout_scale, "dout_scale"));
    MOE_TRY(check_ptr(w, "w"));
    MOE_TRY(check_ptr(w_scale, "w_scale"));
    MOE_TRY(check_ptr(da, "da"));
    MOE_TRY(check_ws_bytes(all_gemm_ws_bytes(*g), ws, ws_bytes));
    moe::Fp8Args x = fp8_args(*g, nullptr, expert_offsets);
    set_rows(x, dout, dout_scale, g->N);
    x.w[0] = w;
    x.w_scale[0] = w_scale;
    x.out = da;
    x.out_bf16 = da_dtype == MOE_DTYPE_BF16;
    x.accumulate = accumulate != 0;
    x.ws = ws;
    return hip_status(moe::launch_fp8_input_grad(x, stream), "fp8 grouped gemm input gradient launch");
}

MOE_EXPORT moe_status moe_expert_gate_up_fp8_block(const moe_problem* p, const uint8_t* x, const uint8_t* x_scale,
                                                   const int32_t* sorted_pairs, const int32_t* expert_offsets,
                                                   const uint8_t* w_gate, const uint8_t* s_gate,
                                                   const uint8_t* w_up, const uint8_t* s_up, uint8_t* h,
                                                   uint8_t* h_scale, hipStream_t stream) {
    MOE_TRY(check_problem(p));
    MOE_TRY(check_expert_outputs(*p));
    if (p->T == 0) return ok();
    MOE_TRY(check_dispatch(*p, sorted_pairs, expert_offsets));
    MOE_TRY(check_ptr(x, "x"));
    MOE_TRY(check_ptr(x_scale, "x_scale"));
    MOE_TRY(check_ptr(w_gate, "w_gate"));
    MOE_TRY(check_ptr(s_gate, "s_gate"));
    MOE_TRY(check_ptr(w_up, "w_up"));
    MOE_TRY(check_ptr(s_up, "s_up"));
    MOE_TRY(check_ptr(h, "h"));
    MOE_TRY(check_ptr(h_scale, "h_scale"));
    const Fp8Weights w{w_gate, s_gate, w_up, s_up, nullptr, nullptr};
    return hip_status(run_gate_up(*p, x, x_scale, sorted_pairs, expert_offsets, w, h, h_scale, stream),
                      "fp8 gate up launch");
}

MOE_EXPORT size_t moe_fp8_block_workspace_bytes(const moe_problem* p) {
    if (check_problem(p) != MOE_OK || check_expert_outputs(*p) != MOE_OK) return 0;
    return ffn_layout(*p).total;
}

MOE_EXPORT moe_status moe_expert_ffn_fp8_block(const moe_problem* p, const moe_bf16* x, const int32_t* sorted_pairs,
                                               const int32_t* expert_offsets, const uint8_t* w_gate,
                                               const uint8_t* s_gate, const uint8_t* w_up, const uint8_t* s_up,
                                               const uint8_t* w_down, const uint8_t* s_down, void* y,
                                               moe_dtype y_dtype, void* ws, size_t ws_bytes, hipStream_t stream) {
    MOE_TRY(check_problem(p));
    MOE_TRY(check_expert_outputs(*p));
    MOE_TRY(check_gemm_out(y_dtype, 0));
    if (p->T == 0) return ok();
    const Fp8Weights w{w_gate, s_gate, w_up, s_up, w_down, s_down};
    MOE_TRY(check_ptr(x, "x"));
    MOE_TRY(check_dispatch(*p, sorted_pairs, expert_offsets));
    MOE_TRY(check_weights(w));
    MOE_TRY(check_ptr(y, "y"));
    MOE_TRY(check_ws_bytes(ffn_layout(*p).total, ws, ws_bytes));
    return hip_status(run_ffn(*p, x, sorted_pairs, expert_offsets, w, y, y_dtype == MOE_DTYPE_BF16, ws, stream),
                      "fp8 expert ffn launch");
}

MOE_EXPORT moe_status moe_forward_fp8_block(const moe_problem* p, const moe_bf16* x, const moe_bf16* w_router,
                                            const float* bias, const uint8_t* w_gate, const uint8_t* s_gate,
                                            const uint8_t* w_up, const uint8_t* s_up, const uint8_t* w_down,
                                            const uint8_t* s_down, void* out, moe_dtype out_dtype,
                                            int32_t* topk_ids, float* topk_weights, float* y, void* ws,
                                            size_t ws_bytes, hipStream_t stream) {
    MOE_TRY(check_problem(p));
    MOE_TRY(check_expert_outputs(*p));
    MOE_TRY(check_gemm_out(out_dtype, 0));
    if (p->T == 0) return ok();
    const Fp8Weights w{w_gate, s_gate, w_up, s_up, w_down, s_down};
    MOE_TRY(check_ptr(x, "x"));
    MOE_TRY(check_ptr(w_router, "w_router"));
    MOE_TRY(check_ptr(bias, "bias", true));
    MOE_TRY(check_weights(w));
    MOE_TRY(check_ptr(out, "out"));
    MOE_TRY(check_ptr(topk_ids, "topk_ids", true));
    MOE_TRY(check_ptr(topk_weights, "topk_weights", true));
    MOE_TRY(check_ptr(y, "y"));
    const FfnLayout F = ffn_layout(*p);
    MOE_TRY(check_ws_bytes(F.total, ws, ws_bytes));
    const Layout L = layout_of(*p);
    int32_t* sorted = at<int32_t>(ws, L.sorted);
    MOE_TRY(check_gathered(p->T, p->H, sorted));
    const moe::Problem q = to_internal(*p);
    int32_t* ids = topk_ids ? topk_ids : at<int32_t>(ws, L.ids);
    float* wts = topk_weights ? topk_weights : at<float>(ws, L.weights);
    int32_t* off = at<int32_t>(ws, L.offsets);
    int32_t* rows = at<int32_t>(ws, L.rows);
    // the scores pass through what later holds x and h
    hipError_t e = moe::launch_route_scratch(q, x, w_router, bias, ids, wts, at<char>(ws, F.x), F.total - F.x, stream);
    if (e != hipSuccess) return hip_status(e, "route launch");
    e = moe::launch_permute(q, ids, off, sorted, rows, at<int32_t>(ws, L.counts), stream);
    if (e != hipSuccess) return hip_status(e, "permute launch");
    e = run_ffn(*p, x, sorted, off, w, y, false, ws, stream);
    if (e != hipSuccess) return hip_status(e, "fp8 expert ffn launch");
    e = moe::launch_combine(q, y, rows, wts, out, out_dtype == MOE_DTYPE_BF16, stream);
    return hip_status(e, "combine launch");
}

MOE_EXPORT size_t moe_fp8_block_backward_workspace_bytes(const moe_problem* p) {
    if (check_problem(p) != MOE_OK || check_expert_outputs(*p) != MOE_OK) return 0;
    return backward_layout(*p).total;
}

MOE_EXPORT moe_status moe_expert_ffn_fp8_block_backward(
    const moe_problem* p, const moe_bf16* x, const int32_t* sorted_pairs, const int32_t* expert_offsets,
    const uint8_t* w_gate, const uint8_t* s_gate, const uint8_t* w_up, const uint8_t* s_up, const uint8_t* w_down,
    const uint8_t* s_down, const moe_bf16* dy, void* dx, moe_dtype dx_dtype, void* dw_gate, void* dw_up,
    void* dw_down, moe_dtype dw_dtype, int accumulate, void* ws, size_t ws_bytes, hipStream_t stream) {
    MOE_TRY(check_problem(p));
    MOE_TRY(check_expert_outputs(*p));
    MOE_TRY(check_gemm_out(dx_dtype, 0));
    MOE_TRY(check_gemm_out(dw_dtype, accumulate));
    const bool empty = p->T == 0;
    const Fp8Weights w{w_gate, s_gate, w_up, s_up, w_down, s_down};
    MOE_TRY(check_ptr(x, "x", empty));
    if (empty)
        MOE_TRY(check_ptr(expert_offsets, "expert_offsets", p->E == 1));
    else
        MOE_TRY(check_dispatch(*p, sorted_pairs, expert_offsets));
    MOE_TRY(check_weights(w));
    MOE_TRY(check_ptr(dy, "dy", empty));
    MOE_TRY(check_ptr(dx, "dx", empty));
    MOE_TRY(check_ptr(dw_gate, "dw_gate"));
    MOE_TRY(check_ptr(dw_up, "dw_up"));
    MOE_TRY(check_ptr(dw_down, "dw_down"));
    const BackwardLayout L = backward_layout(*p);
    MOE_TRY(check_ws_bytes(L.total, ws, ws_bytes));
    const char* what = "fp8 expert ffn backward launch";
    void* sums = at<char>(ws, L.sums);
    hipError_t e = hipSuccess;
    if (!empty) {
        const int64_t P = p->T * p->k;
        uint8_t *xq = at<uint8_t>(ws, L.x), *xs = at<uint8_t>(ws, L.x_scale);
        uint8_t *dyq = at<uint8_t>(ws, L.dy), *dys = at<uint8_t>(ws, L.dy_scale);
        uint8_t *dq = at<uint8_t>(ws, L.d), *ds = at<uint8_t>(ws, L.d_scale);
        e = moe::launch_fp8_rows(p->T, p->H, x, xq, xs, stream);
        if (e != hipSuccess) return hip_status(e, what);
        e = moe::launch_fp8_rows(P, p->H, dy, dyq, dys, stream);
        if (e != hipSuccess) return hip_status(e, what);
        // dh = dy . w_down
        moe::Fp8Args d = fp8_args(down_shape(*p), nullptr, expert_offsets);
        set_rows(d, dyq, dys, p->H);
        d.w[0] = w_down;
        d.w_scale[0] = s_down;
        d.out = at<float>(ws, L.dh);
        d.ws = sums;
        e = moe::launch_fp8_input_grad(d, stream);
        if (e != hipSuccess) return hip_status(e, what);
        // g and u again, then h, dg and du
        moe::Fp8Args a = gate_up_args(*p, xq, xs, sorted_pairs, expert_offsets, w);
        a.dh = at<float>(ws, L.dh);
        a.h = at<uint16_t>(ws, L.h);
        a.dg = at<uint16_t>(ws, L.dg);
        a.du = at<uint16_t>(ws, L.du);
        a.q = dq;
        a.q_cols = pair_cols(p->I);
        a.q_scale = ds;
        a.q_pitch = moe::scale_pitch(pair_cols(p->I));
        e = moe::launch_fp8_gate_up(a, stream);
        if (e != hipSuccess) return hip_status(e, what);
        // dx = dg . w_gate + du . w_up
        moe::Fp8Args b = gate_up_args(*p, nullptr, nullptr, nullptr, expert_offsets, w);
        set_rows(b, dq, ds, pair_cols(p->I));
        b.out = dx;
        b.out_bf16 = dx_dtype == MOE_DTYPE_BF16;
        b.ws = sums;
        e = moe::launch_fp8_input_grad(b, stream);
        if (e != hipSuccess) return hip_status(e, what);
    }
    moe::GemmArgs a = gemm_args(gate_shape(*p));
    a.a = x;
    a.pairs = sorted_pairs;
    a.offsets = expert_offsets;
    a.ws = sums;
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
    moe::GemmArgs d = gemm_args(down_shape(*p));
    d.offsets = expert_offsets;
    d.ws = sums;
    d.out_bf16 = a.out_bf16;
    d.accumulate = a.accumulate;
    d.dout = dy;
    d.a = at<uint16_t>(ws, L.h);
    d.out = dw_down;
    return hip_status(moe::launch_grouped_wgrad(d, stream), what);
}
