// fp8_kernels.h -- internal launchers of the FP8 products with a scale for each
// block of 128 (not exported).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kernels.h"

namespace moe {

constexpr int kBlock = 128;  // values along a row, and rows of a weight matrix, that share a scale

inline int blocks_of(int n) { return (n + kBlock - 1) / kBlock; }

// Bytes of a row's scales: whole 32-bit words.
inline int scale_pitch(int n) { return (blocks_of(n) + 3) / 4 * 4; }

// A grouped product on FP8 operands (moe_fp8.h).  y are the rows of the
// output, x its columns:
//              y                            x                   reduction
//   product    a [S,K], gathered            w [E,N,K]           K
//   input grad dout [P,N]                   w [E,N,K] (columns) N
//   gate_up    x [S,K], gathered            gate, up [E,N,K]    K
struct Fp8Args {
    int64_t P, S;            // sorted positions, rows of y where they are gathered
    int E, N, K, k;          // the weights are [E,N,K]; row(q) = pairs[q] / k
    const uint8_t* y;        // codes
    int64_t y_cols;          // bytes of a row of y
    const uint8_t* y_scale;  // [rows of y, y_pitch]
    int y_pitch;
    const uint8_t* w[2];        // codes; gate_up: gate, up; input grad: the second
    const uint8_t* w_scale[2];  // follows the first in the reduction (NULL: one only)
    const int32_t* pairs;    // [P], or NULL: row(q) = q
    const int32_t* offsets;  // [E+1], or NULL (E = 1): all P rows
    void* out;               // product, input grad: [P, N or K]
    bool out_bf16;
    bool accumulate;         // out += (fp32)
    void* ws;                // sums of a split reduction
    // gate_up: h = silu(g) u as codes and scales.  With dh: the codes and
    // scales of [dg | du] instead (each part of whole blocks), and h, dg, du
    uint8_t* q;
    int64_t q_cols;
    uint8_t* q_scale;
    int q_pitch;
    const float* dh;
    uint16_t *h, *dg, *du;
};

// Scratch of the product (or the input gradient) of this shape.
size_t fp8_ws_bytes(int64_t P, int E, int N, int K);

// And of the input gradient of two matrices [E,N,K] at once.
size_t fp8_pair_ws_bytes(int64_t P, int E, int N, int K);

// Rows gathered from more bytes than this are refused: the tiles address them
// with 32-bit offsets.
constexpr int64_t kMaxGatherBytes = 0xFFF00000LL;

hipError_t launch_fp8_product(const Fp8Args& g, hipStream_t s);
hipError_t launch_fp8_input_grad(const Fp8Args& g, hipStream_t s);
hipError_t launch_fp8_gate_up(const Fp8Args& g, hipStream_t s);

// Rows of bf16 as e4m3 codes with a scale for each 128 columns.
hipError_t launch_fp8_rows(int64_t rows, int K, const uint16_t* x, uint8_t* codes, uint8_t* scales, hipStream_t s);

// Matrices [E,N,K] of bf16 as e4m3 codes with a scale for each 128 x 128.
hipError_t launch_fp8_weights(int E, int N, int K, const uint16_t* w, uint8_t* codes, uint8_t* scales,
                              hipStream_t s);

}  // namespace moe
