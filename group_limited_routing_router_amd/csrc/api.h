// api.h -- what the files of the C ABI share: the last error, argument checks,
// the workspace of the forward pass.
//
// Host side only.  All checks of a call run before its first HIP call, so a
// rejected call enqueues nothing and touches no output.
#pragma once

#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include <string>

#include "fp8_kernels.h"
#include "kernels.h"
#include "moe.h"
#include "moe_gemm.h"

#define MOE_EXPORT extern "C" __attribute__((visibility("default")))

#define MOE_TRY(expr)                      \
    do {                                   \
        const moe_status _s = (expr);      \
        if (_s != MOE_OK) return _s;       \
    } while (0)

namespace moe {
namespace api {

inline thread_local std::string g_last_error;

inline moe_status fail(moe_status s, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    g_last_error = buf;
    return s;
}

inline moe_status ok() {
    g_last_error.clear();
    return MOE_OK;
}

constexpr size_t kAlign = 256;
constexpr int kMaxDim = 65536;  // largest H and I the kernels take
inline size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

struct Layout {
    size_t ids, weights, offsets, sorted, rows, counts, h, total;
};

inline Layout layout_of(const moe_problem& p) {
    const size_t P = static_cast<size_t>(p.T) * static_cast<size_t>(p.k);
    const size_t nb = static_cast<size_t>(moe::permute_blocks(static_cast<int64_t>(P)));
    Layout L{};
    size_t o = 0;
    L.ids = o;     o += align_up(P * 4);
    L.weights = o; o += align_up(P * 4);
    L.offsets = o; o += align_up((static_cast<size_t>(p.E) + 1) * 4);
    L.sorted = o;  o += align_up(P * 4);
    L.rows = o;    o += align_up(P * 4);
    L.counts = o;  o += align_up(nb * static_cast<size_t>(p.E) * 4);
    L.h = o;       o += align_up(P * static_cast<size_t>(p.I) * 2);
    L.total = o;
    return L;
}

// Shape checks shared by every entry point.
inline moe_status check_problem(const moe_problem* p) {
    if (!p) return fail(MOE_ERR_INVALID_ARG, "problem is NULL");
    if (p->T < 0) return fail(MOE_ERR_INVALID_ARG, "T=%lld < 0", (long long)p->T);
    if (p->H <= 0 || p->H % 64 != 0)
        return fail(MOE_ERR_INVALID_ARG, "H=%d must be a positive multiple of 64", p->H);
    if (p->I <= 0 || p->I % 64 != 0)
        return fail(MOE_ERR_INVALID_ARG, "I=%d must be a positive multiple of 64", p->I);
    if (p->E <= 0) return fail(MOE_ERR_INVALID_ARG, "E=%d must be positive", p->E);
    if (p->G <= 0 || p->E % p->G != 0)
        return fail(MOE_ERR_INVALID_ARG, "G=%d must divide E=%d", p->G, p->E);
    if (p->TG < 1 || p->TG > p->G)
        return fail(MOE_ERR_INVALID_ARG, "TG=%d must be in [1, G=%d]", p->TG, p->G);
    const int64_t cand = static_cast<int64_t>(p->TG) * (p->E / p->G);
    if (p->k < 1 || p->k > cand)
        return fail(MOE_ERR_INVALID_ARG, "k=%d must be in [1, TG*E/G=%lld]", p->k, (long long)cand);
    if (!isfinite(p->scale)) return fail(MOE_ERR_INVALID_ARG, "scale is not finite");
    if (p->T > 0x7fffffffLL / p->k)  // T * k itself may pass 64 bits
        return fail(MOE_ERR_INVALID_ARG, "T=%lld times k=%d exceeds int32", (long long)p->T, p->k);
    if (p->E > 256) return fail(MOE_ERR_UNSUPPORTED, "E=%d > 256", p->E);
    if (p->k > 16) return fail(MOE_ERR_UNSUPPORTED, "k=%d > 16", p->k);
    if (p->H % 128 != 0) return fail(MOE_ERR_UNSUPPORTED, "H=%d is not a multiple of 128", p->H);
    // the expert GEMMs form 32-bit byte offsets within one tile's rows of a
    // weight matrix, h or y (at most 256 rows x 65536 x 4 bytes)
    if (p->H > kMaxDim) return fail(MOE_ERR_UNSUPPORTED, "H=%d > %d", p->H, kMaxDim);
    if (p->I > kMaxDim) return fail(MOE_ERR_UNSUPPORTED, "I=%d > %d", p->I, kMaxDim);
    return MOE_OK;
}

inline moe_status check_ptr(const void* ptr, const char* name, bool nullable = false) {
    if (!ptr) {
        if (nullable) return MOE_OK;
        return fail(MOE_ERR_INVALID_ARG, "%s is NULL", name);
    }
    if (reinterpret_cast<uintptr_t>(ptr) % 16 != 0)
        return fail(MOE_ERR_INVALID_ARG, "%s is not 16-byte aligned", name);
    return MOE_OK;
}

inline moe_status check_ws(const moe_problem& p, const void* ws, size_t ws_bytes) {
    const size_t need = layout_of(p).total;
    if (!ws) return fail(MOE_ERR_WORKSPACE, "workspace is NULL (need %zu bytes)", need);
    if (reinterpret_cast<uintptr_t>(ws) % 16 != 0)
        return fail(MOE_ERR_WORKSPACE, "workspace is not 16-byte aligned");
    if (ws_bytes < need)
        return fail(MOE_ERR_WORKSPACE, "workspace has %zu bytes, need %zu", ws_bytes, need);
    return MOE_OK;
}

inline moe::Problem to_internal(const moe_problem& p) {
    return moe::Problem{p.T, p.H, p.I, p.E, p.G, p.TG, p.k, p.scale};
}

inline moe_status hip_status(hipError_t e, const char* what) {
    if (e == hipSuccess) return ok();
    return fail(MOE_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

template <typename T>
T* at(void* ws, size_t off) {
    return reinterpret_cast<T*>(static_cast<char*>(ws) + off);
}

// k_multiple: elements of the operands in 16 bytes.
inline moe_status check_gemm(const moe_gemm_problem* g, int k_multiple) {
    if (!g) return fail(MOE_ERR_INVALID_ARG, "problem is NULL");
    if (g->P < 0 || g->P > 0x7fffffffLL)
        return fail(MOE_ERR_INVALID_ARG, "P=%lld must be in [0, 2^31)", (long long)g->P);
    if (g->S < 0 || g->S > 0x7fffffffLL)
        return fail(MOE_ERR_INVALID_ARG, "S=%lld must be in [0, 2^31)", (long long)g->S);
    if (g->E <= 0) return fail(MOE_ERR_INVALID_ARG, "E=%d must be positive", g->E);
    if (g->k < 1) return fail(MOE_ERR_INVALID_ARG, "k=%d must be positive", g->k);
    if (g->N <= 0 || g->N % 8 != 0)
        return fail(MOE_ERR_INVALID_ARG, "N=%d must be a positive multiple of 8", g->N);
    if (g->K <= 0 || g->K % k_multiple != 0)
        return fail(MOE_ERR_INVALID_ARG, "K=%d must be a positive multiple of %d", g->K, k_multiple);
    if (g->E > 256) return fail(MOE_ERR_UNSUPPORTED, "E=%d > 256", g->E);
    if (g->N > kMaxDim) return fail(MOE_ERR_UNSUPPORTED, "N=%d > %d", g->N, kMaxDim);
    if (g->K > kMaxDim) return fail(MOE_ERR_UNSUPPORTED, "K=%d > %d", g->K, kMaxDim);
    return MOE_OK;
}

// The rows the positions read: every position is its own row without pairs.
inline moe_status check_rows(const moe_gemm_problem& g, const int32_t* sorted_pairs) {
    if (!sorted_pairs && g.S < g.P)
        return fail(MOE_ERR_INVALID_ARG, "S=%lld rows for P=%lld positions without sorted_pairs",
                    (long long)g.S, (long long)g.P);
    if (sorted_pairs && g.P > 0 && g.S < 1)
        return fail(MOE_ERR_INVALID_ARG, "S=%lld rows for P=%lld positions", (long long)g.S, (long long)g.P);
    return check_ptr(sorted_pairs, "sorted_pairs", true);
}

// The outputs of a product of P rows and cols columns.
inline moe_status check_outputs(int64_t P, int64_t cols) {
    if (P * cols > moe::kMaxOutputs)
        return fail(MOE_ERR_UNSUPPORTED, "%lld x %lld outputs > 2^38", (long long)P, (long long)cols);
    return MOE_OK;
}

// The outputs of the experts' products ([P,I] and [P,H]).
inline moe_status check_expert_outputs(const moe_problem& p) {
    MOE_TRY(check_outputs(p.T * p.k, p.I));
    return check_outputs(p.T * p.k, p.H);
}

inline moe_status check_offsets(const moe_gemm_problem& g, const int32_t* expert_offsets) {
    return check_ptr(expert_offsets, "expert_offsets", g.E == 1);
}

inline moe_status check_gemm_out(moe_dtype dtype, int accumulate) {
    if (dtype != MOE_DTYPE_F32 && dtype != MOE_DTYPE_BF16)
        return fail(MOE_ERR_INVALID_ARG, "dtype=%d is not MOE_DTYPE_F32/BF16", (int)dtype);
    if (accumulate && dtype != MOE_DTYPE_F32)
        return fail(MOE_ERR_INVALID_ARG, "accumulate needs an fp32 output");
    return MOE_OK;
}

inline moe_status check_ws_bytes(size_t need, const void* ws, size_t ws_bytes) {
    if (need == 0) return MOE_OK;
    if (!ws) return fail(MOE_ERR_WORKSPACE, "workspace is NULL (need %zu bytes)", need);
    if (reinterpret_cast<uintptr_t>(ws) % 16 != 0)
        return fail(MOE_ERR_WORKSPACE, "workspace is not 16-byte aligned");
    if (ws_bytes < need)
        return fail(MOE_ERR_WORKSPACE, "workspace has %zu bytes, need %zu", ws_bytes, need);
    return MOE_OK;
}

inline moe::GemmArgs gemm_args(const moe_gemm_problem& g) {
    moe::GemmArgs a{};
    a.P = g.P;
    a.S = g.S;
    a.E = g.E;
    a.N = g.N;
    a.K = g.K;
    a.k = g.k;
    // 2^(31 + b) / k rounded up, b = ceil(log2 k): a 32-bit multiplier that
    // gives the exact quotient of every 31-bit dividend
    int b = 0;
    while ((1LL << b) < g.k) ++b;
    a.k_magic = static_cast<uint32_t>((1ULL << (31 + b)) / static_cast<uint64_t>(g.k) + 1);
    a.k_shift = b - 1;
    a.splits = 1;
    return a;
}

inline size_t gemm_ws_bytes(const moe_gemm_problem& g) {
    return moe::grouped_ws_bytes(gemm_args(g));
}

// Scratch of every call on g, those of moe_fp8.h too.  The calls of moe_gemm.h
// ask only for their own part: some shapes split in FP8 alone (2191 rows by 8
// experts, 13744 x 1216), and there they go without a workspace.
inline size_t all_gemm_ws_bytes(const moe_gemm_problem& g) {
    const size_t n = gemm_ws_bytes(g), fp8 = moe::fp8_ws_bytes(g.P, g.E, g.N, g.K);
    return n > fp8 ? n : fp8;
}

inline moe_status check_gemm_ws(const moe_gemm_problem& g, const void* ws, size_t ws_bytes) {
    return check_ws_bytes(gemm_ws_bytes(g), ws, ws_bytes);
}

// ---- the experts on these products ----

inline moe_gemm_problem gate_shape(const moe_problem& p) {  // x -> g, u
    return moe_gemm_problem{p.T * p.k, p.T, p.E, p.I, p.H, p.k};
}

inline moe_gemm_problem down_shape(const moe_problem& p) {  // h -> y
    return moe_gemm_problem{p.T * p.k, p.T * p.k, p.E, p.H, p.I, 1};
}

}  // namespace api
}  // namespace moe
