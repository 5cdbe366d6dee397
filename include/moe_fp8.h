/*
 * moe_fp8.h -- C ABI of libmoe.so: the experts in 8-bit floating point with a
 * scale for each block of 128: the products by expert on FP8 operands, the
 * gated feed-forward pass on them and its gradients.
 *
 * The conventions of moe.h and moe_gemm.h hold (positions sorted by expert,
 * offsets and rows clamped, rows of no expert neither read nor written, no
 * atomics, no memset, capturable).
 *
 * Format.  Codes are OCP e4m3 (bias 7, no infinities, 0x7f NaN), as in
 * moe_expert_ffn_fp8.  A scale is a power of two held as one byte, its
 * exponent + 127 (OCP e8m0): the matrix instructions of gfx950 take it as an
 * operand.  The scale of a block whose largest magnitude is amax is
 *     2^ceil(log2(amax / 448)),
 * the smallest power of two that keeps the block in range, and a code is value
 * / scale rounded to the nearest e4m3, ties to even.  A block whose amax is
 * below 2^-100 gets the scale 1 and codes 0; one that holds an infinity or NaN
 * the scale 1 and codes NaN (0x7f) throughout.
 *   activations, gradients  [rows,C]: a block is 128 columns of one row.
 *            Scales [rows,SB], SB = moe_fp8_block_scales(C) = ceil(C / 128)
 *            rounded up to a multiple of 4; the bytes behind the last block
 *            are padding.
 *   weights  [E,N,K]: a block is 128 x 128 of one matrix (less at its edges).
 *            Scales [E, ceil(N / 128), ceil(K / 128)].
 * The quantisers write scale bytes 19 to 247.  Operands made otherwise may use 1
 * to 254 (255 is no scale) with dequantised values below 2^127; gate_up and the
 * calls on it 3 to 254.
 *
 * Sums.  The matrix instructions add 8 products of one block at a time, each
 * cut towards zero to a multiple of 2^-13 of the power of two of the largest,
 * and everything else in fp32: a sum is off by at most 7 x 2^-13 of the sum of
 * magnitudes, about 2^-16 of the result for values of mixed signs.
 * gate_up (in the pass, the block and the gradients too) multiplies the same
 * operands as bf16 instead, exactly, and sums in fp32 throughout, where the
 * positions are at most 24 for each expert that can have any (T k / min(E, T k)).
 * A token's g and u then differ in the last bits on either side of that, and
 * with them some codes of h by a step.  As bf16, units of 2^-9 of a block are
 * held from scale byte 3 on, and what the quantisers round up to 2^128 (bf16 from
 * 31/32 of it on) is infinite.  Measured against the definition in 64 bits, in
 * norm, with bf16 outputs: products 1.7e-3 off (their own rounding), y of the
 * pass at most 2.1e-3, dx of the gradients at most 2.7e-3.
 *
 * Rows gathered by sorted_pairs may take at most 4 GiB less 1 MiB of codes
 * (else MOE_ERR_UNSUPPORTED).
 */
#ifndef MOE_FP8_H
#define MOE_FP8_H

#include "moe_gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bytes of a row's scales for C columns (0 for C <= 0). */
int32_t moe_fp8_block_scales(int32_t C);

/* Rows of bf16 [rows,K] as codes [rows,K] and scales [rows,SB] (the padding is
 * written as 127).  K a multiple of 16, K <= 65536. */
moe_status moe_quantize_rows_fp8_block(int64_t rows, int32_t K, const moe_bf16* x, uint8_t* codes,
                                       uint8_t* scales, hipStream_t stream);

/* Weights of bf16 [E,N,K] as codes [E,N,K] and scales [E,NB,KB].  E <= 256; N
 * and K multiples of 16, at most 65536. */
moe_status moe_quantize_weights_fp8_block(int32_t E, int32_t N, int32_t K, const moe_bf16* w,
                                          uint8_t* codes, uint8_t* scales, hipStream_t stream);

/* The product: out[q,n] = sum_k A[row(q),k] W[e,n,k] on the dequantised
 * operands.  N and K multiples of 16.
 *   a [S,K] codes, a_scale [S, scales of K];  w [E,N,K] codes, w_scale
 *   out [P,N] fp32 or bf16
 *   ws moe_gemm_workspace_bytes(g) bytes */
moe_status moe_grouped_gemm_fp8_block(const moe_gemm_problem* g, const uint8_t* a,
                                      const uint8_t* a_scale, const int32_t* sorted_pairs,
                                      const int32_t* expert_offsets, const uint8_t* w,
                                      const uint8_t* w_scale, void* out, moe_dtype out_dtype,
                                      void* ws, size_t ws_bytes, hipStream_t stream);

/* The gradient of the product's input on the same weights, read down their
 * rows: da[q,k] = sum_n D[q,n] W[e,n,k].
 *   dout [P,N] codes in sorted order, dout_scale [P, scales of N]
 *   da   [P,K] fp32 or bf16;  accumulate not 0: da += (fp32 only)
 * The gradient of the weights is moe_grouped_gemm_wgrad on bf16 operands. */
moe_status moe_grouped_gemm_fp8_block_dgrad(const moe_gemm_problem* g, const uint8_t* dout,
                                            const uint8_t* dout_scale,
                                            const int32_t* expert_offsets, const uint8_t* w,
                                            const uint8_t* w_scale, void* da, moe_dtype da_dtype,
                                            int accumulate, void* ws, size_t ws_bytes,
                                            hipStream_t stream);

/* ---- the experts of moe.h on these products ----
 *   w_gate, w_up [E,I,H] codes, s_gate, s_up [E, ceil(I/128), H/128]
 *   w_down       [E,H,I] codes, s_down       [E, H/128, ceil(I/128)]
 * With E = 1 and k = 1 (a dense layer) sorted_pairs and expert_offsets may be
 * NULL: the one expert then takes all T rows in order. */

/* Both projections, the activation, the product and its quantisation in one
 * kernel: h = silu(g) u, g = X . Wgate[e]^T, u = X . Wup[e]^T in fp32, goes out
 * as codes [T*k,I] and scales [T*k, scales of I], without a rounding between.
 *   x [T,H] codes, x_scale [T, scales of H] */
moe_status moe_expert_gate_up_fp8_block(const moe_problem* p, const uint8_t* x,
                                        const uint8_t* x_scale, const int32_t* sorted_pairs,
                                        const int32_t* expert_offsets, const uint8_t* w_gate,
                                        const uint8_t* s_gate, const uint8_t* w_up,
                                        const uint8_t* s_up, uint8_t* h, uint8_t* h_scale,
                                        hipStream_t stream);

/* Bytes of `ws` for the two calls below (0 if p is invalid). */
size_t moe_fp8_block_workspace_bytes(const moe_problem* p);

/* The experts' pass: x is quantised by rows, then gate_up above, then
 *   y[q] = H . Wdown[e]^T, [T*k,H] fp32 or bf16 (y_dtype) in sorted order. */
moe_status moe_expert_ffn_fp8_block(const moe_problem* p, const moe_bf16* x,
                                    const int32_t* sorted_pairs, const int32_t* expert_offsets,
                                    const uint8_t* w_gate, const uint8_t* s_gate,
                                    const uint8_t* w_up, const uint8_t* s_up,
                                    const uint8_t* w_down, const uint8_t* s_down, void* y,
                                    moe_dtype y_dtype, void* ws, size_t ws_bytes,
                                    hipStream_t stream);

/* The whole block with these experts: everything else as moe_forward. */
moe_status moe_forward_fp8_block(const moe_problem* p, const moe_bf16* x, const moe_bf16* w_router,
                                 const float* bias, const uint8_t* w_gate, const uint8_t* s_gate,
                                 const uint8_t* w_up, const uint8_t* s_up, const uint8_t* w_down,
                                 const uint8_t* s_down, void* out, moe_dtype out_dtype,
                                 int32_t* topk_ids, float* topk_weights, float* y, void* ws,
                                 size_t ws_bytes, hipStream_t stream);

/* The gradients of moe_expert_ffn_fp8_block from dy [T*k,H] bf16 in sorted
 * order.  The roundings of the forward pass are passed over (their gradient is
 * taken as one); h, g and u are computed again:
 *   dh = DY . Wdown[e]                  DY: dy quantised by rows
 *   dg = dh u s (1 + g (1 - s)),  du = dh g s,  s = 1 / (1 + exp(-g))   in fp32
 *   dx = DG . Wgate[e] + DU . Wup[e]    DG, DU: dg and du quantised by rows
 *   dw_gate = dg^T x, dw_up = du^T x, dw_down = dy^T h by expert, as
 *   moe_grouped_gemm_wgrad, from x, dy and dg, du, h rounded to bf16: the
 *   weights' gradients sum over tokens, along which the blocks do not lie
 *   dx       [T*k,H] fp32 or bf16 (dx_dtype) in sorted order
 *   dw_gate, dw_up [E,I,H], dw_down [E,H,I]  fp32 or bf16 (dw_dtype); zero for
 *            idle experts;  accumulate not 0: += (fp32 only)
 *   ws       moe_fp8_block_backward_workspace_bytes(p) bytes
 * With T = 0 the weights' gradients are still written. */
size_t moe_fp8_block_backward_workspace_bytes(const moe_problem* p);

moe_status moe_expert_ffn_fp8_block_backward(
    const moe_problem* p, const moe_bf16* x, const int32_t* sorted_pairs,
    const int32_t* expert_offsets, const uint8_t* w_gate, const uint8_t* s_gate,
    const uint8_t* w_up, const uint8_t* s_up, const uint8_t* w_down, const uint8_t* s_down,
    const moe_bf16* dy, void* dx, moe_dtype dx_dtype, void* dw_gate, void* dw_up, void* dw_down,
    moe_dtype dw_dtype, int accumulate, void* ws, size_t ws_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_FP8_H */
