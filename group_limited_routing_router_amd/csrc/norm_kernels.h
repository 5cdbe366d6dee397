// norm_kernels.h -- internal launchers of the norm and its gradient.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace moe {

// A row stays in registers: 2 chunks of 8 values for each of 1024 threads.
constexpr int kNormMaxH = 2 * 8 * 1024;

struct NormArgs {
    int64_t rows;
    int H;
    const void *x, *dy;
    bool x_f32, dy_f32, out_f32;
    const float *weight, *bias;
    float eps;
    bool center;
    void* out;          // the normalised rows, or dx
    float* stats;       // [rows,2]: mean, 1 / sqrt(var + eps)
    float *dweight, *dbias;
    bool accumulate;
    float* ws;          // sums of dweight (and dbias) of each workgroup
};

// Scratch of the gradient.
size_t norm_ws_bytes(int64_t rows, int H);

hipError_t launch_norm(const NormArgs& a, hipStream_t s);
hipError_t launch_norm_backward(const NormArgs& a, hipStream_t s);

}  // namespace moe
