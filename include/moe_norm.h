/*
 * moe_norm.h -- C ABI of libmoe.so: the norm in front of the block and its
 * gradient ("Welcome Beam: a 501B open model you can own, customize, and
 * scale", section "Residual Stream": every sublayer's input is normalised; the
 * norms compute in FP32).  The norm behind it is part of
 * moe_combine_residual.
 *
 * The conventions of moe.h hold.  Rows are contiguous; H is a multiple of 8,
 * at most 16384 (a row stays in registers; else MOE_ERR_UNSUPPORTED).
 *     out[t,i] = (x[t,i] - mean[t]) r[t] weight[i] + bias[i]
 *     r[t] = 1 / sqrt(mean over i of (x[t,i] - mean[t])^2 + eps)
 * center = 0 (RMS norm): mean[t] is taken as 0.  center not 0 (layer norm): the
 * mean of the row; the squares are those of the differences, a second pass
 * over the row's registers, so a mean far above the spread costs no digits.
 * Sums of squares are fp32: magnitudes from about 1e18 on overflow (r = 0).
 */
#ifndef MOE_NORM_H
#define MOE_NORM_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/*   x       [rows,H] fp32 or bf16 (x_dtype)
 *   weight  [H] fp32;  bias [H] fp32 or NULL (0)
 *   eps     > 0
 *   out     [rows,H] fp32 or bf16 (out_dtype), computed in fp32, rounded once;
 *           may be x itself where the types are the same
 *   stats   [rows,2] fp32 out or NULL: mean and r, for the backward call */
moe_status moe_norm(int64_t rows, int32_t H, const void* x, moe_dtype x_dtype, const float* weight,
                    const float* bias, float eps, int center, void* out, moe_dtype out_dtype,
                    float* stats, hipStream_t stream);

/* Bytes of `ws` for the backward call (0 for invalid sizes or no rows). */
size_t moe_norm_workspace_bytes(int64_t rows, int32_t H);

/* With xh = (x - mean) r and d = dy weight:
 *     dx = r (d - xh mean_i(d xh) - mean_i(d))     (the last mean only with
 *     dweight = sum over rows of dy xh              center)
 *     dbias   = sum over rows of dy
 *   dy      [rows,H] fp32 or bf16 (dy_dtype)
 *   x, x_dtype, weight, center  as the forward call;  stats as it wrote them
 *   dx      [rows,H] fp32 or bf16 (dx_dtype); may be dy or x itself where the
 *           types are the same
 *   dweight [H] fp32;  dbias [H] fp32 or NULL
 *   accumulate  not 0: dweight += and dbias +=
 * The sums over rows are fp32 in a fixed order.  With no rows dweight and dbias
 * are still written. */
moe_status moe_norm_backward(int64_t rows, int32_t H, const void* dy, moe_dtype dy_dtype,
                             const void* x, moe_dtype x_dtype, const float* weight,
                             const float* stats, int center, void* dx, moe_dtype dx_dtype,
                             float* dweight, float* dbias, int accumulate, void* ws,
                             size_t ws_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_NORM_H */
