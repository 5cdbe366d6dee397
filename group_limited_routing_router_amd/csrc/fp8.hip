// fp8.hip -- FP8 with a scale for each block of 128: quantisation of rows and
// of weights, and the launches of the tiled products (gemm_fp8.h).
#include "common.h"
#include "fp8_plan.h"
#include "gemm_fp8.h"

namespace moe {
namespace {

// The larger of the magnitudes of 8 bf16 values, as fp32 bits: in the order of
// integers infinity and NaN come last.
__device__ __forceinline__ uint32_t top_of(const u32x4& p, uint32_t top) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        top = max(top, (p[i] & 0x7fffu) << 16);
        top = max(top, p[i] & 0x7fff0000u);
    }
    return top;
}

// The codes of 8 bf16 values.
__device__ __forceinline__ u32x2 codes_of(const u32x4& p, uint32_t top, float inverse) {
    u32x2 o;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        f32x4 v;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t w = p[2 * j + i / 2];
            v[i] = __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
        }
        o[j] = block_codes(v, top, inverse);
    }
    return o;
}

// Rows: 16 lanes a block, a wave four of them, whose scales are one word.
__global__ __launch_bounds__(kThreads) void fp8_rows_kernel(const uint16_t* x, int64_t units, int K, int words,
                                                            uint8_t* codes, uint8_t* scales) {
    const int lane = threadIdx.x & 63;
    const int64_t unit = folded_index() * kWaves + (threadIdx.x >> 6);
    if (unit >= units) return;
    const int64_t row = unit / words;
    const int word = static_cast<int>(unit - row * words);
    const int c = word * 4 * kBlock + lane * 8;
    const u32x4 v = c < K ? ld16(x + row * K + c) : u32x4{0, 0, 0, 0};
    uint32_t top = top_of(v, 0);
#pragma unroll
    for (int d = 8; d; d >>= 1) top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), d, kWave)));
    const int scale = fp8_scale_of(top);
    if (c < K)
        *reinterpret_cast<u32x2*>(codes + row * K + c) =
            codes_of(v, top, __uint_as_float(fp8_inverse_bits(scale)));
    uint32_t all = 0;
#pragma unroll
    for (int b = 0; b < 4; ++b) all |= static_cast<uint32_t>(__shfl(scale, b * 16, kWave)) << (8 * b);
    if (lane == 0) *reinterpret_cast<uint32_t*>(scales + (row * words + word) * 4) = all;
}

// Weights: a workgroup takes one 128 x 128 block, 16 lanes a row.
__global__ __launch_bounds__(kThreads) void fp8_weights_kernel(const uint16_t* w, int N, int K, uint8_t* codes,
                                                               uint8_t* scales, int64_t blocks) {
    __shared__ uint32_t s_top[kWaves];
    const int64_t block = folded_index();
    if (block >= blocks) return;
    const int KB = (K + kBlock - 1) / kBlock, NB = (N + kBlock - 1) / kBlock;
    const int kb = static_cast<int>(block % KB), nb = static_cast<int>(block / KB % NB);
    const int64_t matrix = block / KB / NB * N * K;
    const int tid = threadIdx.x, c = kb * kBlock + (tid & 15) * 8, r = nb * kBlock + (tid >> 4);
    u32x4 v[8];
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int rj = r + j * 16;
        v[j] = rj < N && c < K ? ld16(w + matrix + static_cast<int64_t>(rj) * K + c) : u32x4{0, 0, 0, 0};
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) top = top_of(v[j], top);
#pragma unroll
    for (int d = 32; d; d >>= 1) top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), d, kWave)));
    if ((tid & 63) == 0) s_top[tid >> 6] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kWaves; ++i) top = max(top, s_top[i]);
    const int scale = fp8_scale_of(top);
    const float inverse = __uint_as_float(fp8_inverse_bits(scale));
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int rj = r + j * 16;
        if (rj < N && c < K)
            *reinterpret_cast<u32x2*>(codes + matrix + static_cast<int64_t>(rj) * K + c) = codes_of(v[j], top, inverse);
    }
    if (tid == 0) scales[block] = static_cast<uint8_t>(scale);
}

// The parts of a split reduction, [splits][P][cols], added in order; a thread
// adds 4 columns.
__global__ __launch_bounds__(kThreads) void fp8_join_kernel(Fp8Args g, int cols, int splits) {
    const int c = (blockIdx.x * kThreads + threadIdx.x) * 4;
    const int64_t q = blockIdx.y + static_cast<int64_t>(blockIdx.z) * gridDim.y;
    if (c >= cols || q >= g.P) return;
    if (g.offsets && (q < g.offsets[0] || q >= g.offsets[g.E])) return;  // of no expert
    const int64_t at = q * cols + c, step = g.P * cols;
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < splits; ++s) v += *reinterpret_cast<const f32x4*>(static_cast<const float*>(g.ws) + s * step + at);
    if (g.out_bf16) {
        const u32x2 h = {pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
        *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(g.out) + at) = h;
    } else {
        f32x4* o = reinterpret_cast<f32x4*>(static_cast<float*>(g.out) + at);
        if (g.accumulate) v += *o;
        *o = v;
    }
}

size_t sums_bytes(int splits, int64_t P, int cols) {
    return splits > 1 ? static_cast<size_t>(splits) * static_cast<size_t>(P) * static_cast<size_t>(cols) * 4 : 0;
}

template <int MODE>
hipError_t launch(const Fp8Args& g, const TilePlan& p, hipStream_t s) {
    hipError_t err;
    if (p.rows == 256)
        err = launch_tiles<MODE, 256, 256>(g, s, p.splits);
    else if (p.rows == 32)
        err = p.nt ? launch_tiles<MODE, 128, 32, true>(g, s, p.splits) : launch_tiles<MODE, 128, 32>(g, s, p.splits);
    else
        err = p.nt ? launch_tiles<MODE, 128, 128, true>(g, s, p.splits) : launch_tiles<MODE, 128, 128>(g, s, p.splits);
    if (err != hipSuccess || p.splits == 1) return err;
    const int cols = MODE == kF8Product ? g.N : g.K;
    const unsigned y = static_cast<unsigned>(g.P < 32768 ? g.P : 32768);
    fp8_join_kernel<<<dim3((cols / 4 + kThreads - 1) / kThreads, y, static_cast<unsigned>((g.P + y - 1) / y)),
                      dim3(kThreads), 0, s>>>(g, cols, p.splits);
    return hipGetLastError();
}

}  // namespace

size_t fp8_ws_bytes(int64_t P, int E, int N, int K) {
    if (P == 0) return 0;
    const size_t a = sums_bytes(product_plan(P, E, N, K).splits, P, N);
    const size_t b = sums_bytes(input_grad_plan(P, E, N, K).splits, P, K);
    return a > b ? a : b;
}

size_t fp8_pair_ws_bytes(int64_t P, int E, int N, int K) {
    return P == 0 ? 0 : sums_bytes(input_grad_plan(P, E, pair_red(N), K).splits, P, K);
}

hipError_t launch_fp8_product(const Fp8Args& g, hipStream_t s) {
    return launch<kF8Product>(g, product_plan(g.P, g.E, g.N, g.K), s);
}

hipError_t launch_fp8_input_grad(const Fp8Args& g, hipStream_t s) {
    return launch<kF8InputGrad>(g, input_grad_plan(g.P, g.E, g.w[1] ? pair_red(g.N) : g.N, g.K), s);
}

hipError_t launch_fp8_rows(int64_t rows, int K, const uint16_t* x, uint8_t* codes, uint8_t* scales, hipStream_t s) {
    if (rows <= 0) return hipSuccess;
    const int words = scale_pitch(K) / 4;
    const int64_t units = rows * words;
    fp8_rows_kernel<<<folded_grid((units + kWaves - 1) / kWaves), dim3(kThreads), 0, s>>>(x, units, K, words, codes,
                                                                                         scales);
    return hipGetLastError();
}

hipError_t launch_fp8_weights(int E, int N, int K, const uint16_t* w, uint8_t* codes, uint8_t* scales,
                              hipStream_t s) {
    const int64_t blocks = static_cast<int64_t>(E) * blocks_of(N) * blocks_of(K);
    fp8_weights_kernel<<<folded_grid(blocks), dim3(kThreads), 0, s>>>(w, N, K, codes, scales, blocks);
    return hipGetLastError();
}

}  // namespace moe
