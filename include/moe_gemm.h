/*
 * moe_gemm.h -- C ABI of libmoe.so: the experts' matrix products by
 * themselves, grouped by expert with ragged sizes, with their two gradients,
 * and in 8-bit integers with a scale for each token and each output channel.
 *
 * The conventions of moe.h hold: device pointers owned by the caller,
 * contiguous, row-major, 16-byte aligned, no output overlapping an input or
 * another output; nothing is allocated, freed or
 * synchronised; every argument is checked on the host before anything is
 * enqueued; no memset, so every call can be captured into a HIP graph; no
 * atomics, so results are the same from run to run.
 *
 * Positions q = 0 .. P-1 are sorted by expert: expert e owns positions
 * expert_offsets[e] .. expert_offsets[e+1]-1 (expert_offsets and sorted_pairs
 * as moe_permute writes them).  Position q reads activation row
 *     row(q) = sorted_pairs[q] / k,   or q where sorted_pairs is NULL.
 * Offsets are clamped to [0, P] and rows to [0, S), so no contents of these
 * arrays make a call read or write out of range.  Positions before
 * expert_offsets[0] or from expert_offsets[E] on belong to no expert: their
 * activations are not read and their output rows keep what they hold.  With
 * E = 1, expert_offsets may be NULL: the one group then takes all P rows (a
 * dense layer).
 *
 * Rows gathered by sorted_pairs from an activation tensor of more than 4 GiB
 * less 1 MiB (S K 2 bytes, S K for int8) run on a simpler kernel: the product
 * about 3.5 times and the weight gradient 6.5 times slower (420000 rows of 5120
 * to 2560 columns: 31 and 83 ms against 9 and 13).
 *
 * A row that holds an infinity or NaN affects its own output row alone (in
 * the weight gradient, its own expert's gradient).
 */
#ifndef MOE_GEMM_H
#define MOE_GEMM_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Shape of a grouped product.
 *   P  sorted positions (>= 0, fits in int32)
 *   S  rows of the activations a (S >= P where sorted_pairs is NULL)
 *   E  experts, 1 <= E <= 256
 *   N, K  the weights are [E,N,K]; multiples of 8 (K of 16 for the int8
 *      product), at most 65536
 *   k  positions per activation row, >= 1: row(q) = sorted_pairs[q] / k
 * The outputs of one call, P N (P K for the input gradient), at most 2^38. */
typedef struct moe_gemm_problem {
    int64_t P, S;
    int32_t E, N, K, k;
} moe_gemm_problem;

/* Bytes of scratch the calls below need in `ws` for problem g (0 if g is
 * invalid, or if none is needed: ws may then be NULL).  One workspace sized
 * by this function serves every call on g; what it holds before a call does
 * not matter.  Calls that overlap need one workspace each. */
size_t moe_gemm_workspace_bytes(const moe_gemm_problem* g);

/* The product: out[q,n] = sum_k a[row(q),k] * w[e,n,k], e the expert that
 * owns q.
 *   a    [S,K] bf16
 *   w    [E,N,K] bf16
 *   out  [P,N] fp32 or bf16 (out_dtype): summed in fp32, rounded once */
moe_status moe_grouped_gemm(const moe_gemm_problem* g, const moe_bf16* a,
                            const int32_t* sorted_pairs, const int32_t* expert_offsets,
                            const moe_bf16* w, void* out, moe_dtype out_dtype, void* ws,
                            size_t ws_bytes, hipStream_t stream);

/* The gradient of the product's input, position by position:
 *     da[q,k] = sum_n dout[q,n] * w[e,n,k]
 *   dout [P,N] bf16 in sorted order
 *   da   [P,K] fp32 or bf16 in sorted order (the sum over the k positions of
 *        one activation row is moe_combine with weights of one)
 *   accumulate  not 0: da += (fp32 only) */
moe_status moe_grouped_gemm_dgrad(const moe_gemm_problem* g, const moe_bf16* dout,
                                  const int32_t* expert_offsets, const moe_bf16* w, void* da,
                                  moe_dtype da_dtype, int accumulate, void* ws, size_t ws_bytes,
                                  hipStream_t stream);

/* The gradient of the product's weights:
 *     dw[e,n,k] = sum over e's positions q of dout[q,n] * a[row(q),k]
 *   dout [P,N] bf16 in sorted order;  a [S,K] bf16
 *   dw   [E,N,K] fp32 or bf16; zero for an expert without positions
 *   accumulate  not 0: dw += (fp32 only)
 * With P = 0, dout, a and sorted_pairs may be NULL; dw is still written. */
moe_status moe_grouped_gemm_wgrad(const moe_gemm_problem* g, const moe_bf16* dout,
                                  const moe_bf16* a, const int32_t* sorted_pairs,
                                  const int32_t* expert_offsets, void* dw, moe_dtype dw_dtype,
                                  int accumulate, void* ws, size_t ws_bytes, hipStream_t stream);

/* Rows of bf16 as 8-bit integers with one fp32 scale each:
 *     amax = max_k |x[r,k]|,  scales[r] = amax / 127,
 *     codes[r,k] = 127 x[r,k] / amax, rounded to the nearest integer (ties to
 *     even)
 * A row of zeros gets the scale 1 and codes 0; so does a row whose amax is
 * below 2^-100.  A row that holds an infinity or NaN gets the scale NaN and
 * codes 0.
 *   x [rows,K] bf16;  codes [rows,K] int8;  scales [rows] fp32
 *   rows >= 0, K a multiple of 16, K <= 65536 */
moe_status moe_quantize_rows_int8(int64_t rows, int32_t K, const moe_bf16* x, int8_t* codes,
                                  float* scales, hipStream_t stream);

/* The product in 8-bit integers:
 *     out[q,n] = (a_scale[row(q)] * w_scale[e,n])
 *                * sum_k a[row(q),k] * w[e,n,k]
 * The sum is exact (int32); the scales multiply it in fp32.
 *   a [S,K] int8 codes, a_scale [S] fp32;  w [E,N,K] int8 codes, w_scale
 *   [E,N] fp32;  out [P,N] fp32 or bf16.  K a multiple of 16. */
moe_status moe_grouped_gemm_int8(const moe_gemm_problem* g, const int8_t* a, const float* a_scale,
                                 const int32_t* sorted_pairs, const int32_t* expert_offsets,
                                 const int8_t* w, const float* w_scale, void* out,
                                 moe_dtype out_dtype, void* ws, size_t ws_bytes,
                                 hipStream_t stream);

/* ---- the experts of moe.h on these products ---- */

/* Experts with int8 weights and activations (moe_expert_ffn, moe_forward).
 * The rows of x are quantised as moe_quantize_rows_int8 does it, g and u are
 * int8 products in fp32, h = silu(g) u in fp32 is quantised by rows in the
 * same way (127 h / amax to the nearest, ties to even), y is an int8 product:
 *     g[n] = sx s_gate[e,n] (xc . w_gate[e,n]),  u likewise,
 *     y[m] = sh s_down[e,m] (hc . w_down[e,m])
 *   w_gate, w_up  [E,I,H] int8 codes;  s_gate, s_up  [E,I] fp32
 *   w_down        [E,H,I] int8 codes;  s_down        [E,H] fp32
 *   ws            moe_int8_workspace_bytes(p) bytes
 * T k I and T k H at most 2^38 (so too for moe_expert_ffn_backward).
 * A token that holds an infinity or NaN has NaN in its own outputs alone.
 * Everything else as moe_expert_ffn / moe_forward. */
size_t moe_int8_workspace_bytes(const moe_problem* p);

moe_status moe_expert_ffn_int8(const moe_problem* p, const moe_bf16* x,
                               const int32_t* sorted_pairs, const int32_t* expert_offsets,
                               const int8_t* w_gate, const float* s_gate, const int8_t* w_up,
                               const float* s_up, const int8_t* w_down, const float* s_down,
                               float* y, void* ws, size_t ws_bytes, hipStream_t stream);

moe_status moe_forward_int8(const moe_problem* p, const moe_bf16* x, const moe_bf16* w_router,
                            const float* bias, const int8_t* w_gate, const float* s_gate,
                            const int8_t* w_up, const float* s_up, const int8_t* w_down,
                            const float* s_down, void* out, moe_dtype out_dtype, int32_t* topk_ids,
                            float* topk_weights, float* y, void* ws, size_t ws_bytes,
                            hipStream_t stream);

/* The gradients of moe_expert_ffn (bf16 weights) from the gradient of y:
 *   x, sorted_pairs, expert_offsets, w_gate, w_up, w_down  as the forward call
 *   dy       [T*k,H] bf16 in sorted order
 *   dx       [T*k,H] fp32 out in sorted order: the gradient of each pair's
 *            row of x (the sum over a token's pairs is moe_combine with
 *            weights and scale of one)
 *   dw_gate, dw_up [E,I,H], dw_down [E,H,I]  out, fp32 or bf16 (dw_dtype);
 *            zero for idle experts;  accumulate not 0: += (fp32 only)
 *   ws       moe_backward_workspace_bytes(p) bytes
 * g, u (the products of the forward pass, computed again) and dh = dy . w_down
 * are fp32; h = silu(g) u, dg = dh u s (1 + g (1 - s)) and du = dh g s, with s
 * = 1 / (1 + exp(-g)), are rounded to bf16 and multiplied:
 *     dw_down = dy^T h, dw_gate = dg^T x, dw_up = du^T x (by expert),
 *     dx = dg . w_gate + du . w_up
 * With T = 0 the weight gradients are still written. */
size_t moe_backward_workspace_bytes(const moe_problem* p);

moe_status moe_expert_ffn_backward(const moe_problem* p, const moe_bf16* x,
                                   const int32_t* sorted_pairs, const int32_t* expert_offsets,
                                   const moe_bf16* w_gate, const moe_bf16* w_up,
                                   const moe_bf16* w_down, const moe_bf16* dy, float* dx,
                                   void* dw_gate, void* dw_up, void* dw_down, moe_dtype dw_dtype,
                                   int accumulate, void* ws, size_t ws_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_GEMM_H */
