// swiglu.hip -- between the experts' products: the SwiGLU product quantised by
// rows (8-bit experts) and its gradient (training).
//
//   h = silu(g) u,  silu(g) = g s,  s = 1 / (1 + exp(-g))
//   dL/dg = dh u s (1 + g (1 - s)),  dL/du = dh silu(g)
//
// Both are bound by memory: they read fp32 sums of the products and write
// codes or bf16 operands of the next ones.
#include "codes.h"
#include "common.h"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kThreads = 256;

// One row a workgroup: h, its largest magnitude, the codes 127 h / amax (to
// the nearest, ties to even) and the scale amax / 127.  h stays in registers, CHUNKS groups
// of 4 a thread; CHUNKS = 0 computes it twice (I > 16384).  Rows of no expert
// are left out.
template <int CHUNKS>
__global__ __launch_bounds__(kThreads) void swiglu_quantize_kernel(const float* g, const float* u, int64_t P, int I,
                                                                   const int32_t* offsets, int E, int8_t* codes,
                                                                   float* scales) {
    __shared__ float s_max[kThreads / kWave];
    __shared__ int s_bad[kThreads / kWave];
    const int64_t q = folded_index();
    if (q >= P || q < offsets[0] || q >= offsets[E]) return;
    const int tid = threadIdx.x;
    const float* gr = g + q * I;
    const float* ur = u + q * I;
    auto product = [&](int c) {
        const f32x4 a = *reinterpret_cast<const f32x4*>(gr + c), b = *reinterpret_cast<const f32x4*>(ur + c);
        f32x4 h;
#pragma unroll
        // h stays in fp32: the hardware exp2 of silu_f32 is off by 2^-18 at
        // gates of -80
        for (int i = 0; i < 4; ++i) h[i] = a[i] * sigmoid_f32(a[i]) * b[i];
        return h;
    };
    float m = 0.0f;
    int bad = 0;
    auto look = [&](const f32x4& h) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            m = fmaxf(m, fabsf(h[i]));
            bad |= !(fabsf(h[i]) < __builtin_inff());
        }
    };
    f32x4 h[CHUNKS > 0 ? CHUNKS : 1];
    if constexpr (CHUNKS > 0) {
#pragma unroll
        for (int j = 0; j < CHUNKS; ++j) {
            const int c = (j * kThreads + tid) * 4;
            h[j] = c < I ? product(c) : f32x4{0.f, 0.f, 0.f, 0.f};
            look(h[j]);
        }
    } else {
        for (int c = tid * 4; c < I; c += kThreads * 4) look(product(c));
    }
#pragma unroll
    for (int d = 32; d; d >>= 1) {
        m = fmaxf(m, __shfl_xor(m, d, kWave));
        bad |= __shfl_xor(bad, d, kWave);
    }
    if ((tid & 63) == 0) {
        s_max[tid >> 6] = m;
        s_bad[tid >> 6] = bad;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / kWave; ++w) {
        m = fmaxf(m, s_max[w]);
        bad |= s_bad[w];
    }
    // as moe_quantize_rows_int8 treats its rows
    const bool zero = bad || m < 0x1p-100f;
    if (tid == 0) scales[q] = bad ? __builtin_nanf("") : (zero ? 1.0f : m / 127.0f);
    // large rows are scaled down first, since 127 h would overflow
    const float shrink = m > 0x1p100f ? 0x1p-30f : 1.0f, ms = m * shrink, inv = 1.0f / ms;
    auto write = [&](int c, const f32x4& v) {
        uint32_t o = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int code = zero ? 0 : code_of_f32(v[i] * shrink, ms, inv);
            o |= static_cast<uint32_t>(static_cast<uint8_t>(code)) << (8 * i);
        }
        *reinterpret_cast<uint32_t*>(codes + q * I + c) = o;
    };
    if constexpr (CHUNKS > 0) {
#pragma unroll
        for (int j = 0; j < CHUNKS; ++j) {
            const int c = (j * kThreads + tid) * 4;
            if (c < I) write(c, h[j]);
        }
    } else {
        for (int c = tid * 4; c < I; c += kThreads * 4) write(c, product(c));
    }
}

// Four values a thread: h, dg and du as bf16 operands of the next products.
__global__ __launch_bounds__(kThreads) void swiglu_backward_kernel(const float* g, const float* u, const float* dh,
                                                                   int64_t values, uint16_t* h, uint16_t* dg,
                                                                   uint16_t* du) {
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    const int64_t at = (folded_index() * kThreads + threadIdx.x) * 4;
    if (at >= values) return;
    const f32x4 a = *reinterpret_cast<const f32x4*>(g + at), b = *reinterpret_cast<const f32x4*>(u + at),
                d = *reinterpret_cast<const f32x4*>(dh + at);
    f32x4 o0, o1, o2;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float s = sigmoid_f32(a[i]), silu = a[i] * s;
        o0[i] = silu * b[i];
        o1[i] = d[i] * b[i] * (s + silu * (1.0f - s));
        o2[i] = d[i] * silu;
    }
    *reinterpret_cast<u32x2*>(h + at) = u32x2{pack_bf16(o0[0], o0[1]), pack_bf16(o0[2], o0[3])};
    *reinterpret_cast<u32x2*>(dg + at) = u32x2{pack_bf16(o1[0], o1[1]), pack_bf16(o1[2], o1[3])};
    *reinterpret_cast<u32x2*>(du + at) = u32x2{pack_bf16(o2[0], o2[1]), pack_bf16(o2[2], o2[3])};
}

}  // namespace

hipError_t launch_swiglu_quantize(const float* g, const float* u, int64_t P, int I, const int32_t* offsets, int E,
                                  int8_t* codes, float* scales, hipStream_t s) {
    if (P <= 0) return hipSuccess;
    const dim3 grid = folded_grid(P), threads(kThreads);
    if (I <= 4096)
        swiglu_quantize_kernel<4><<<grid, threads, 0, s>>>(g, u, P, I, offsets, E, codes, scales);
    else if (I <= 16384)
        swiglu_quantize_kernel<16><<<grid, threads, 0, s>>>(g, u, P, I, offsets, E, codes, scales);
    else
        swiglu_quantize_kernel<0><<<grid, threads, 0, s>>>(g, u, P, I, offsets, E, codes, scales);
    return hipGetLastError();
}

hipError_t launch_swiglu_backward(const float* g, const float* u, const float* dh, int64_t values, uint16_t* h,
                                  uint16_t* dg, uint16_t* du, hipStream_t s) {
    const int64_t blocks = (values / 4 + kThreads - 1) / kThreads;
    if (blocks <= 0) return hipSuccess;
    swiglu_backward_kernel<<<folded_grid(blocks), dim3(kThreads), 0, s>>>(g, u, dh, values, h, dg, du);
    return hipGetLastError();
}

}  // namespace moe
