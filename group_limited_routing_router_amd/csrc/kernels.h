// kernels.h -- internal launchers behind the C ABI (not exported).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

struct Problem {
    int64_t T;
    int H, I, E, G, TG, k;
    float scale;
};

// A grouped product (moe_gemm.h): shape, operands, output.
struct GemmArgs {
    int64_t P;               // sorted positions
    int64_t S;               // rows of a
    int E, N, K;             // w is [E,N,K]
    int k;                   // row(q) = pairs[q] / k
    uint32_t k_magic;        // p / k = umulhi(p, k_magic) >> k_shift for 0 <= p < 2^31
    int k_shift;             // (k = 1: k_shift < 0)
    const void* a;           // activations [S,K]: bf16 or int8 codes
    const void* dout;        // output gradient [P,N] bf16 (the two gradients)
    const void* w;           // weights [E,N,K]: bf16 or int8 codes
    const int32_t* pairs;    // [P], or NULL: row(q) = q
    const int32_t* offsets;  // [E+1], or NULL (E = 1): all P rows
    const float* a_scale;    // int8: [S]
    const float* w_scale;    // int8: [E,N]
    void* out;
    bool out_bf16;           // out is bf16, else fp32
    bool accumulate;         // out += (fp32)
    void* ws;                // sums of a split reduction
    int splits;              // weight gradient: parts of each expert's positions
};

// A launch takes fewer than 2^32 threads along x (the runtime wraps a longer
// grid without an error): workgroups of 256.
constexpr int64_t kMaxWorkgroups = (1LL << 24) - 1;

// A grid of n workgroups (n <= 2^35) of at most 1024 threads, in rows of 2^20
// where one launch dimension does not take them; workgroup i is folded_index(),
// up to a row less one of which are past n.
inline dim3 folded_grid(int64_t n, int threads = 256) {
    constexpr int64_t kRow = 1 << 20;
    return n * threads < (1LL << 32)
               ? dim3(static_cast<unsigned>(n))
               : dim3(static_cast<unsigned>(kRow), static_cast<unsigned>((n + kRow - 1) / kRow));
}

// Outputs of one grouped product, at most (512 GiB of bf16): with P <= 2^31 rows
// of at most 65536 columns over at most 256 experts, the 256 x 256 tiles are at
// most (P / 256 + 257) (cols / 256 + 1) <= 2^22 + 2^23 + 2^16 + 2^9.
constexpr int64_t kMaxOutputs = 1LL << 38;

// Pairs handled by one block of the counting sort.
constexpr int kPermuteChunk = 4096;

inline int64_t permute_blocks(int64_t pairs) {
    return pairs <= 0 ? 1 : (pairs + kPermuteChunk - 1) / kPermuteChunk;
}

hipError_t launch_route(const Problem& p, const uint16_t* x, const uint16_t* w_router,
                        const float* bias, int32_t* ids, float* weights, hipStream_t s);

// The router with device scratch of at least T*E*4 bytes (unused contents):
// for up to 512 tokens the experts are split over workgroups and the scores
// pass through the scratch (the same scores, bit for bit, as launch_route);
// otherwise, or with too little scratch, launch_route.
hipError_t launch_route_scratch(const Problem& p, const uint16_t* x, const uint16_t* w_router,
                                const float* bias, int32_t* ids, float* weights, void* scratch,
                                size_t scratch_bytes, hipStream_t s);

hipError_t launch_permute(const Problem& p, const int32_t* ids, int32_t* offsets,
                          int32_t* sorted_pairs, int32_t* pair_rows, int32_t* block_counts,
                          hipStream_t s);

// sorted_pairs = 0 .. T-1 and offsets = {0, T}: the dispatch of one expert
// that takes every token (a dense layer).
hipError_t launch_identity_dispatch(int64_t T, int32_t* offsets, int32_t* sorted_pairs,
                                    hipStream_t s);

hipError_t launch_expert_ffn(const Problem& p, const uint16_t* x, const int32_t* sorted_pairs,
                             const int32_t* offsets, const uint16_t* w_gate,
                             const uint16_t* w_up, const uint16_t* w_down, uint16_t* h, float* y,
                             hipStream_t s);

// The expert FFN with FP8 E4M3 weights and fp32 per-output-channel scales
// (s_gate/s_up [E,I], s_down [E,H]); x, h and y as in launch_expert_ffn.
hipError_t launch_expert_ffn_fp8(const Problem& p, const uint16_t* x, const int32_t* sorted_pairs,
                                 const int32_t* offsets, const uint8_t* w_gate,
                                 const float* s_gate, const uint8_t* w_up, const float* s_up,
                                 const uint8_t* w_down, const float* s_down, uint16_t* h,
                                 float* y, hipStream_t s);

hipError_t launch_gate_up(const Problem& p, const uint16_t* x, const int32_t* sorted_pairs,
                          const int32_t* offsets, const uint16_t* w_gate, const uint16_t* w_up,
                          uint16_t* h, hipStream_t s);

hipError_t launch_down(const Problem& p, const uint16_t* h, const int32_t* offsets,
                       const uint16_t* w_down, float* y, hipStream_t s);

hipError_t launch_combine(const Problem& p, const float* y, const int32_t* pair_rows,
                          const float* weights, void* out, bool out_bf16, hipStream_t s);

// Combine fused with the post-norm and residual update; the combined row is
// held in registers, at most kResidualMaxChunks float4 chunks per thread of
// 256, i.e. H <= 16384.
constexpr int kResidualMaxChunks = 16;
constexpr int kResidualMaxH = kResidualMaxChunks * 4 * 256;

hipError_t launch_combine_residual(const Problem& p, const float* y, const int32_t* pair_rows,
                                   const float* weights, const float* gain, float eps,
                                   float wa, float wb, float* res, hipStream_t s);

// Scratch the grouped products of this shape need.
size_t grouped_ws_bytes(const GemmArgs& g);

hipError_t launch_grouped_gemm(const GemmArgs& g, hipStream_t s);
hipError_t launch_grouped_dgrad(const GemmArgs& g, hipStream_t s);
hipError_t launch_grouped_wgrad(const GemmArgs& g, hipStream_t s);
hipError_t launch_grouped_int8(const GemmArgs& g, hipStream_t s);

// Rows of bf16 [rows,K] as int8 codes with one fp32 scale each.
hipError_t launch_quantize_rows(int64_t rows, int K, const uint16_t* x, int8_t* codes, float* scales,
                                hipStream_t s);

// h = silu(g) u of the rows that belong to an expert, as int8 codes [P,I] with
// one scale per row [P].
hipError_t launch_swiglu_quantize(const float* g, const float* u, int64_t P, int I, const int32_t* offsets, int E,
                                  int8_t* codes, float* scales, hipStream_t s);

// h = silu(g) u and the gradients of g and u from dh, all rounded to bf16.
hipError_t launch_swiglu_backward(const float* g, const float* u, const float* dh, int64_t values, uint16_t* h,
                                  uint16_t* dg, uint16_t* du, hipStream_t s);

}  // namespace moe
