// grouped.hip -- the experts' matrix products by themselves: the product, its
// two gradients, and the product in 8-bit integers, grouped by expert over
// the sorted positions.
//
//   product      out[q,n]  = sum_k a[row(q),k] w[e,n,k]
//   input grad   da[q,k]   = sum_n dout[q,n] w[e,n,k]
//   weight grad  dw[e,n,k] = sum_{q of e} dout[q,n] a[row(q),k]
//   int8         out[q,n]  = a_scale[row(q)] w_scale[e,n] sum_k a[row(q),k] w[e,n,k]
#include <math.h>

#include "common.h"
#include "gemm_tile.h"
#include "gemm_wgrad.h"
#include "kernels.h"

namespace moe {
namespace {

// The rows of the sorted order that expert e owns, clamped to [0, P].
__device__ __forceinline__ void expert_rows(const GemmArgs& g, int e, int64_t& first, int64_t& n) {
    int64_t b = 0, t = g.P;
    if (g.offsets) {
        b = g.offsets[e];
        t = g.offsets[e + 1];
        b = b < 0 ? 0 : (b > g.P ? g.P : b);
        t = t < 0 ? 0 : (t > g.P ? g.P : t);
    }
    first = b;
    n = t > b ? t - b : 0;
}

// Activation row of sorted position q, clamped to [0, S).
__device__ __forceinline__ int64_t source_row(const GemmArgs& g, int64_t q) {
    if (!g.pairs) return q;
    int64_t r = g.pairs[q] / g.k;
    return r < 0 ? 0 : (r >= g.S ? g.S - 1 : r);
}

// The plain kernel, for rows gathered from more than 4 GiB (the tiles address
// them with 32-bit offsets): one 64 x 64 tile of the product or the weight
// gradient, the reduction in steps of 64 bytes a row through LDS.  In LDS both operands lie with the reduction
// along the row; an operand whose reduction runs down the rows in memory is
// transposed on the way in.  Grid: (column tiles, row tiles of the fullest
// possible expert or, for the weight gradient, row tiles of N, experts).
template <int MODE, bool I8>
__global__ __launch_bounds__(kThreads) void gemm_plain_kernel(GemmArgs g) {
    static_assert(MODE != kInputGrad, "gathers nothing");
    constexpr int EB = I8 ? 1 : 2;        // bytes per operand element
    constexpr int PER16 = 16 / EB;        // elements per 16 bytes
    constexpr int BK = 64 / EB;           // reduction per step
    constexpr int PITCH = 64 + 16;        // bytes per LDS row
    __shared__ __attribute__((aligned(16))) unsigned char s_y[64 * PITCH];  // output rows
    __shared__ __attribute__((aligned(16))) unsigned char s_x[64 * PITCH];  // output columns
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int e = blockIdx.z;
    int64_t first, n_e;
    expert_rows(g, e, first, n_e);
    // output: rows [r0, rows) x columns [c0, cols); reduction over [0, red)
    const int64_t rows = MODE == kWeightGrad ? g.N : n_e;
    const int cols = MODE == kProduct ? g.N : g.K;
    const int64_t red = MODE == kProduct ? g.K : n_e;
    const int c0 = blockIdx.x * 64;
    const unsigned char* a = static_cast<const unsigned char*>(g.a);
    const unsigned char* w = static_cast<const unsigned char*>(g.w) +
                             static_cast<int64_t>(e) * g.N * g.K * EB;
    for (int64_t r0 = static_cast<int64_t>(blockIdx.y) * 64; r0 < rows;
         r0 += static_cast<int64_t>(gridDim.y) * 64) {
        f32x4 acc[4];
        i32x4 iacc[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            acc[c] = f32x4{0.f, 0.f, 0.f, 0.f};
            iacc[c] = i32x4{0, 0, 0, 0};
        }
        for (int64_t k0 = 0; k0 < red; k0 += BK) {
            const u32x4 zero = {0, 0, 0, 0};
            // one 16-byte piece of each operand a thread
            {
                u32x4 v = zero;
                if constexpr (MODE == kWeightGrad) {  // dout[q, n..n+7]: transposed
                    const int kk = tid >> 3, rr = (tid & 7) * 8;
                    if (k0 + kk < red && r0 + rr < rows)
                        v = ld16(static_cast<const unsigned char*>(g.dout) +
                                 ((first + k0 + kk) * g.N + r0 + rr) * EB);
                    const uint16_t* h = reinterpret_cast<const uint16_t*>(&v);
                    for (int i = 0; i < 8; ++i)
                        *reinterpret_cast<uint16_t*>(&s_y[(rr + i) * PITCH + kk * 2]) = h[i];
                } else {
                    const int rr = tid >> 2, kk = (tid & 3) * PER16;
                    if (r0 + rr < rows && k0 + kk < red) {
                        const int64_t q = first + r0 + rr;
                        v = ld16(a + (source_row(g, q) * g.K + k0 + kk) * EB);
                    }
                    *reinterpret_cast<u32x4*>(&s_y[rr * PITCH + (tid & 3) * 16]) = v;
                }
            }
            {
                u32x4 v = zero;
                if constexpr (MODE == kProduct) {
                    const int cc = tid >> 2, kk = (tid & 3) * PER16;
                    if (c0 + cc < cols && k0 + kk < red)
                        v = ld16(w + (static_cast<int64_t>(c0 + cc) * g.K + k0 + kk) * EB);
                    *reinterpret_cast<u32x4*>(&s_x[cc * PITCH + (tid & 3) * 16]) = v;
                } else {
                    const int kk = tid >> 3, cc = (tid & 7) * 8;
                    if (k0 + kk < red && c0 + cc < cols)
                        v = ld16(a + (source_row(g, first + k0 + kk) * g.K + c0 + cc) * EB);
                    const uint16_t* h = reinterpret_cast<const uint16_t*>(&v);
                    for (int i = 0; i < 8; ++i)
                        *reinterpret_cast<uint16_t*>(&s_x[(cc + i) * PITCH + kk * 2]) = h[i];
                }
            }
            __syncthreads();
            const u32x4 yv = ld16(&s_y[(wave * 16 + (lane & 15)) * PITCH + (lane >> 4) * 16]);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const u32x4 xv = ld16(&s_x[(c * 16 + (lane & 15)) * PITCH + (lane >> 4) * 16]);
                if constexpr (I8)
                    iacc[c] = mfma16_i8(yv, xv, iacc[c]);
                else
                    acc[c] = mfma16(as_bf16x8(yv), as_bf16x8(xv), acc[c]);
            }
            __syncthreads();
        }
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t r = r0 + wave * 16 + 4 * (lane >> 4) + i;
                const int col = c0 + c * 16 + (lane & 15);
                if (r >= rows || col >= cols) continue;
                float v = acc[c][i];
                if constexpr (I8)
                    v = static_cast<float>(iacc[c][i]) *
                        (g.a_scale[source_row(g, first + r)] *
                         g.w_scale[static_cast<int64_t>(e) * g.N + col]);
                const int64_t at = MODE == kWeightGrad
                                       ? (static_cast<int64_t>(e) * g.N + r) * g.K + col
                                       : (first + r) * cols + col;
                if (g.out_bf16)
                    static_cast<uint16_t*>(g.out)[at] = f32_to_bf16_rne(v);
                else if (g.accumulate)
                    static_cast<float*>(g.out)[at] += v;
                else
                    static_cast<float*>(g.out)[at] = v;
            }
    }
}

template <int MODE, bool I8>
hipError_t launch_plain(const GemmArgs& g, hipStream_t s) {
    const int cols = MODE == kProduct ? g.N : g.K;
    const int64_t rows = MODE == kWeightGrad ? g.N : g.P;
    if (rows <= 0) return hipSuccess;
    const int64_t rt = (rows + 63) / 64;
    const dim3 grid((cols + 63) / 64, static_cast<unsigned>(rt < 1024 ? rt : 1024), g.E);
    gemm_plain_kernel<MODE, I8><<<grid, dim3(kThreads), 0, s>>>(g);
    return hipGetLastError();
}

// Workgroups of a tiled launch (an upper bound: the host does not read the
// experts' counts).
template <int MODE>
int64_t tile_grid(const GemmArgs& g, int bx, int by) {
    const int64_t cols = MODE == kProduct ? g.N : g.K;
    const int64_t row_tiles = (g.P + by - 1) / by + (g.E < g.P ? g.E : g.P);
    const int64_t tiles = row_tiles * ((cols + bx - 1) / bx);
    return (tiles + kNumXcd - 1) / kNumXcd * kNumXcd;
}

// splits > 1: the reduction in that many parts, whose sums go to g.ws.
template <int MODE, bool I8, int BX, int BY, bool NT = false>
hipError_t launch_tiles(const GemmArgs& g, hipStream_t s, int splits = 1) {
    const int64_t grid = tile_grid<MODE>(g, BX, BY);
    if (grid <= 0) return hipSuccess;
    if (grid > kMaxWorkgroups) return hipErrorInvalidConfiguration;
    const dim3 blocks(static_cast<unsigned>(grid), splits), threads(kThreads);
    if constexpr (MODE == kProduct) {
        if (g.pairs) {
            gemm_tile_kernel<MODE, I8, BX, BY, true, NT><<<blocks, threads, 0, s>>>(g);
            return hipGetLastError();
        }
    }
    gemm_tile_kernel<MODE, I8, BX, BY, false, NT><<<blocks, threads, 0, s>>>(g);
    return hipGetLastError();
}

// The gathered rows of a, addressed with 32-bit offsets by the tiled kernels.
bool gather_fits(const GemmArgs& g, int bytes) {
    return !g.pairs || g.S * static_cast<int64_t>(g.K) * bytes <= static_cast<int64_t>(kNoRowOffset);
}

// How the product and the input gradient of a shape run.
struct TilePlan {
    int rows;    // tile: 32 x 128, 128 x 128 or 256 x 256
    bool nt;     // weights stream past the caches
    int splits;  // parts of the reduction
};

// Microseconds of `tiles` workgroups over `stages` stages each.  A round holds
// one 256-row tile on each compute unit or two of the smaller ones.  Measured:
// a stage (128 bytes of reduction) takes 1.85 us on 256 rows with the whole
// chip busy, 1.05 with little of it; 0.6 on 128 and 0.22 on 32 rows with a
// compute unit to itself, 1.1 and 0.5 with two on it; a round costs 11, 5.5
// and 4 us beside its stages (first loads, writing out).
float tile_time(int rows, float tiles, float stages) {
    const float slots = rows == 256 ? kNumCu : 2.0f * kNumCu;
    float rounds = tiles / slots;
    // the last round of a few is not full, but then runs faster
    if (rounds <= 2.0f)
        rounds = ceilf(rounds);
    else if (rounds < 4.0f)
        rounds = 0.5f * (rounds + ceilf(rounds));
    if (rows == 256)
        return rounds * ((1.05f + 0.8f * (tiles < kNumCu ? tiles / kNumCu : 1.0f)) * stages + 11.0f);
    const bool alone = tiles <= kNumCu;
    if (rows == 128) return rounds * ((alone ? 0.6f : 1.1f) * stages + 5.5f);
    return rounds * ((alone ? 0.22f : 0.5f) * stages + 4.0f);
}

// The host does not read the experts' counts: a mean expert is taken, with
// half a tile more for the ragged end.
template <int MODE, bool I8>
TilePlan plan_tiles(const GemmArgs& g) {
    const int eb = I8 ? 1 : 2;
    const int cols = MODE == kProduct ? g.N : g.K;
    const int64_t met = g.E < g.P ? g.E : g.P;  // experts that can have rows
    const float experts = static_cast<float>(met);
    const float mean_rows = static_cast<float>(g.P) / experts;
    const bool large = met * g.N * g.K * eb > kStreamBytes;
    const float stages = static_cast<float>(((MODE == kProduct ? g.K : g.N) + 128 / eb - 1) / (128 / eb));
    auto tiles_of = [&](int rows) {
        const float each = met == 1 ? static_cast<float>((g.P + rows - 1) / rows) : mean_rows / rows + 0.45f;
        const int width = rows == 256 ? 256 : 128;
        return experts * (each > 1.0f ? each : 1.0f) * static_cast<float>((cols + width - 1) / width);
    };
    TilePlan p{256, false, 1};
    const bool stream = large && mean_rows <= 32;
    if (stream) {
        // the weight stream is the time: the tile that takes an expert's rows
        // at once and keeps the most loads in flight (256 experts of 2560 x
        // 5120: 4 rows each 0.97 ms on 32, 1.07 on 128 rows; 24 rows each 1.10
        // and 1.09 ms)
        p.rows = mean_rows <= 24 ? 32 : 128;
        // past the caches where rows are whole lines (0.97 against 1.07 ms;
        // rows of 1776 bytes: 452 against 381 us)
        p.nt = g.K * eb % 128 == 0;
    }
    float best = -1.0f;
    // a large weight stream with more rows and tiles for every compute unit:
    // the tile that reads the weights least often (4096 tokens over 256 busy
    // and idle experts: 1.46 against 1.68 ms on 128 rows)
    if (large && !stream && tiles_of(256) >= kNumCu) return p;
    for (int rows : {32, 128, 256}) {
        if (stream && rows != p.rows) continue;
        // more tiles than a launch takes (2^31 - 1 rows of width 8 on 128
        // rows); outputs of up to kMaxOutputs always fit on 256
        if (rows < 256 && tile_grid<MODE>(g, 128, rows) > kMaxWorkgroups) continue;
        for (int splits = 1; splits <= 16; splits *= 2) {
            if (splits > 1 && stages < 4 * splits) break;
            // rows that are not whole lines take more lines a stage, which
            // shows most where the tile's part of a row is short (185 x 4
            // rows, K 2232: 112 us on 128 rows, 76 on 256)
            const float lines = g.K * eb % 128 == 0 ? 1.0f : (rows == 256 ? 1.1f : 1.3f);
            float t = tile_time(rows, tiles_of(rows) * splits, lines * stages / splits);
            // the sums written and read, one more launch, and 5% for the parts'
            // own first loads.  Of 1, 2, 4, 8, 16 parts: 32 rows, 512 x 16384:
            // 58, 36, 24, 19, 19 us, 16 taken; 256 rows, 2048 x 4096: 21, 22,
            // 20, 22, 26, 1 taken; 8192 rows, 5120 x 20480: 1367, 1350, 1446,
            // 1708, 2249, 1 taken; worst of twelve shapes: 8 x 128 rows, 1024 x
            // 4096: 22, 30, 28, 31, 43, 2 taken
            if (splits > 1) t = 1.05f * t + 4.0f + 2.0f * splits * static_cast<float>(g.P) * cols * 4.0f / 5e6f;
            if (best < 0.0f || t < best) {
                best = t;
                p.rows = rows;
                p.splits = splits;
            }
        }
    }
    return p;
}

// The sums of a split reduction: [splits][P][cols] 32-bit values, added in
// order, then the output's scales and rounding.  A thread adds 4 columns.
template <int MODE, bool I8>
__global__ __launch_bounds__(kThreads) void join_splits_kernel(GemmArgs g, int splits) {
    const int cols = MODE == kProduct ? g.N : g.K;
    const int c = (blockIdx.x * kThreads + threadIdx.x) * 4;
    const int64_t q = blockIdx.y + static_cast<int64_t>(blockIdx.z) * gridDim.y;
    if (c >= cols || q >= g.P) return;
    int e = 0;
    if (g.offsets) {
        if (q < g.offsets[0] || q >= g.offsets[g.E]) return;  // of no expert
        if constexpr (I8) {
            int hi = g.E - 1;  // last expert that begins at or before q
            while (e < hi) {
                const int mid = (e + hi + 1) >> 1;
                if (g.offsets[mid] <= q) e = mid; else hi = mid - 1;
            }
        }
    }
    const int64_t at = q * cols + c, step = g.P * cols;
    f32x4 v;
    if constexpr (I8) {
        i32x4 sum = {0, 0, 0, 0};
        for (int s = 0; s < splits; ++s) sum += *reinterpret_cast<const i32x4*>(static_cast<const int32_t*>(g.ws) + s * step + at);
        int64_t r = q;
        if (g.pairs) {
            r = g.pairs[q] / g.k;
            r = r < 0 ? 0 : (r >= g.S ? g.S - 1 : r);
        }
        const float a = g.a_scale[r];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[i] = static_cast<float>(sum[i]) * (a * g.w_scale[static_cast<int64_t>(e) * g.N + c + i]);
    } else {
        v = f32x4{0.f, 0.f, 0.f, 0.f};
        for (int s = 0; s < splits; ++s) v += *reinterpret_cast<const f32x4*>(static_cast<const float*>(g.ws) + s * step + at);
    }
    if (g.out_bf16) {
        u32x2 h;
        h[0] = pack_bf16(v[0], v[1]);
        h[1] = pack_bf16(v[2], v[3]);
        *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(g.out) + at) = h;
    } else {
        f32x4* o = reinterpret_cast<f32x4*>(static_cast<float*>(g.out) + at);
        if (g.accumulate) v += *o;
        *o = v;
    }
}

template <int MODE, bool I8>
hipError_t launch(const GemmArgs& g, hipStream_t s) {
    // the input gradient gathers nothing, whatever pairs its caller has
    if constexpr (MODE == kProduct)
        if (!gather_fits(g, I8 ? 1 : 2)) return launch_plain<MODE, I8>(g, s);
    const TilePlan p = plan_tiles<MODE, I8>(g);
    hipError_t err;
    if (p.rows == 256)
        err = launch_tiles<MODE, I8, 256, 256>(g, s, p.splits);
    else if (p.rows == 32)
        err = p.nt ? launch_tiles<MODE, I8, 128, 32, true>(g, s, p.splits)
                   : launch_tiles<MODE, I8, 128, 32>(g, s, p.splits);
    else
        err = p.nt ? launch_tiles<MODE, I8, 128, 128, true>(g, s, p.splits)
                   : launch_tiles<MODE, I8, 128, 128>(g, s, p.splits);
    if (err != hipSuccess || p.splits == 1) return err;
    const int cols = MODE == kProduct ? g.N : g.K;
    const unsigned y = static_cast<unsigned>(g.P < 32768 ? g.P : 32768);
    join_splits_kernel<MODE, I8><<<dim3((cols / 4 + kThreads - 1) / kThreads, y, static_cast<unsigned>((g.P + y - 1) / y)),
                                   dim3(kThreads), 0, s>>>(g, p.splits);
    return hipGetLastError();
}

// How the weight gradient of a shape runs.
struct WgradPlan {
    bool big;    // 256 x 256 tiles, else 128 x 128
    int splits;  // parts of each expert's positions
};

WgradPlan plan_wgrad(const GemmArgs& g) {
    // 256 x 256 tiles from about two for each compute unit on (256 experts of
    // 2560 x 5120, 256 rows each: 2.6 against 3.5 ms).  Large against small
    // tiles at 256 rows an expert: 320 of them (one expert of 4096 x 5120) 26.0
    // and 21.5 us, 384 (24 of 776 x 1000) 27.9 and 26.1, 512 (32 of these) 29.2
    // and 29.1, 512 (32 of 1024 x 1024) 29.6 and 31.5, 1024 (64 of 776 x 1000)
    // 50.0 and 52.9
    WgradPlan p{static_cast<int64_t>((g.K + 255) / 256) * ((g.N + 255) / 256) * g.E >= 512, 1};
    if (p.big) return p;
    // Parts of the positions, where the sums are long.  Microseconds: a stage
    // of 32 positions takes 0.43 on two tiles to a compute unit, a tile about
    // 16 stages more for its writing; the busiest expert is taken as three
    // times the mean; the parts' sums are written, read and joined.
    const float stages = static_cast<float>(g.P) / g.E / 32.0f;
    const float tiles = static_cast<float>((g.K + 127) / 128) * static_cast<float>((g.N + 127) / 128) * g.E;
    const float bytes = static_cast<float>(g.E) * g.N * g.K * 4.0f;
    float best = -1.0f;
    for (int n = 1; n <= 64 && n * g.E <= kMaxE; n *= 2) {  // kMaxE: the kernel's list of parts
        if (n > 1 && stages < 8.0f * n) break;
        const float all = tiles * (stages + 16.0f * n) / (2 * kNumCu), longest = 3.0f * stages / n + 16.0f;
        float t = 0.43f * (all > longest ? all : longest);
        if (n > 1) t += 4.0f + 2.0f * n * bytes / 5e6f;
        if (best < 0.0f || t < best) {
            best = t;
            p.splits = n;
        }
    }
    return p;
}

// dw (+)= the sums of the parts, in order; a thread adds 4 values.
__global__ __launch_bounds__(kThreads) void join_wgrad_kernel(GemmArgs g, int64_t values, int splits) {
    const int64_t i = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) * 4;
    if (i >= values) return;
    const float* part = static_cast<const float*>(g.ws) + i;
    f32x4 v = *reinterpret_cast<const f32x4*>(part);
    for (int s = 1; s < splits; ++s) v += *reinterpret_cast<const f32x4*>(part + s * values);
    if (g.out_bf16) {
        u32x2 h;
        h[0] = pack_bf16(v[0], v[1]);
        h[1] = pack_bf16(v[2], v[3]);
        *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(g.out) + i) = h;
    } else {
        f32x4* o = reinterpret_cast<f32x4*>(static_cast<float*>(g.out) + i);
        if (g.accumulate) v += *o;
        *o = v;
    }
}

template <int BX, int BY, bool GATHER>
hipError_t launch_wgrad_tiles(const GemmArgs& g, hipStream_t s) {
    const int64_t tiles = static_cast<int64_t>((g.K + BX - 1) / BX) * ((g.N + BY - 1) / BY) * g.E * g.splits;
    const int64_t most = static_cast<int64_t>(kNumCu) * WgradShape<BX, BY, GATHER>::kPerCu;
    const int64_t grid = tiles < most ? (tiles + kNumXcd - 1) / kNumXcd * kNumXcd : most;
    const dim3 blocks(static_cast<unsigned>(grid)), threads(kThreads);
    if (g.out_bf16)
        gemm_wgrad_kernel<BX, BY, GATHER, true, false><<<blocks, threads, 0, s>>>(g);
    else if (g.accumulate)
        gemm_wgrad_kernel<BX, BY, GATHER, false, true><<<blocks, threads, 0, s>>>(g);
    else
        gemm_wgrad_kernel<BX, BY, GATHER, false, false><<<blocks, threads, 0, s>>>(g);
    return hipGetLastError();
}

// The code of x in a row whose largest magnitude is m, 1 / m rounded to fp32:
// 127 x / m to the nearest, ties to even, exactly.  127 x is exact (15 bits),
// the product with 1 / m within one of the code, and the remainder 127 x - r m
// exact, so it tells on which side of the half way point the quotient lies (x
// = m / 2 lies on one).
__device__ __forceinline__ int code_of(float x, float m, float inv) {
    const float y = 127.0f * x;
    float r = rintf(y * inv);
    const float e = fmaf(-r, m, y), e2 = 2.0f * fabsf(e);
    const bool odd = static_cast<int>(r) & 1;
    if (e2 > m || (e2 == m && odd)) r += copysignf(1.0f, e);
    return static_cast<int>(r);
}

// Rows of bf16 as 8-bit codes with one scale each, LANES lanes a row.  A row
// is read once and stays in registers (CHUNKS 16-byte pieces a lane); CHUNKS =
// 0 reads it twice (K > 16384).  Bound by memory: 8192 rows of 5120 (126 MB
// read and written) 32-35 us, 3.6-3.9 TB/s.
template <int LANES, int CHUNKS>
__global__ __launch_bounds__(kThreads) void quantize_rows_kernel(const uint16_t* x, int64_t rows, int K,
                                                                 int8_t* codes, float* scales) {
    __shared__ float s_max[kWaves];
    const int tid = threadIdx.x, lane = tid % LANES;
    const int64_t r = folded_index() * (kThreads / LANES) + tid / LANES;
    if (r >= rows) return;  // whole waves, or the whole workgroup of one row
    const uint16_t* row = x + r * K;
    // magnitudes as integers: in this order infinity and NaN come last
    uint32_t top = 0;
    u32x4 v[CHUNKS > 0 ? CHUNKS : 1];
    auto look = [&](const u32x4& p) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            top = max(top, p[i] & 0x7fffu);
            top = max(top, p[i] >> 16 & 0x7fffu);
        }
    };
    if constexpr (CHUNKS > 0) {
#pragma unroll
        for (int j = 0; j < CHUNKS; ++j) {
            const int c = (j * LANES + lane) * 8;
            v[j] = c < K ? ld16(row + c) : u32x4{0, 0, 0, 0};
        }
#pragma unroll
        for (int j = 0; j < CHUNKS; ++j) look(v[j]);
    } else {
        for (int c = lane * 8; c < K; c += LANES * 8) look(ld16(row + c));
    }
#pragma unroll
    for (int d = 32; d; d >>= 1) top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), d, kWave)));
    float m = bf16_to_f32(static_cast<uint16_t>(top));
    if constexpr (LANES > kWave) {
        if ((tid & 63) == 0) s_max[tid >> 6] = __uint_as_float(top);  // the bits
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWaves; ++w) top = max(top, __float_as_uint(s_max[w]));
        m = bf16_to_f32(static_cast<uint16_t>(top));
    }
    const bool bad = top >= 0x7f80u;
    const bool zero = bad || m < 0x1p-100f;
    if (lane == 0) scales[r] = bad ? __builtin_nanf("") : (zero ? 1.0f : m / 127.0f);
    // large rows are scaled down first, since 127 x would overflow
    const float shrink = m > 0x1p100f ? 0x1p-30f : 1.0f;
    const float ms = m * shrink, inv = 1.0f / ms;
    auto write = [&](int c, const u32x4& p) {
        uint64_t o = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float xi = __uint_as_float(i & 1 ? p[i / 2] & 0xffff0000u : p[i / 2] << 16);
            const int code = zero ? 0 : code_of(xi * shrink, ms, inv);
            o |= static_cast<uint64_t>(static_cast<uint8_t>(code)) << (8 * i);
        }
        *reinterpret_cast<uint64_t*>(codes + r * K + c) = o;
    };
    if constexpr (CHUNKS > 0) {
#pragma unroll
        for (int j = 0; j < CHUNKS; ++j) {
            const int c = (j * LANES + lane) * 8;
            if (c < K) write(c, v[j]);
        }
    } else {
        for (int c = lane * 8; c < K; c += LANES * 8) write(c, ld16(row + c));
    }
}

}  // namespace

size_t grouped_ws_bytes(const GemmArgs& g) {
    if (g.P == 0) return 0;
    size_t most = 0;
    auto need = [&](int splits, int64_t values) {
        const size_t n = splits > 1 ? static_cast<size_t>(splits) * static_cast<size_t>(values) * 4 : 0;
        most = n > most ? n : most;
    };
    need(plan_tiles<kProduct, false>(g).splits, g.P * g.N);
    need(plan_tiles<kProduct, true>(g).splits, g.P * g.N);
    need(plan_tiles<kInputGrad, false>(g).splits, g.P * g.K);
    need(plan_wgrad(g).splits, static_cast<int64_t>(g.E) * g.N * g.K);
    return most;
}

hipError_t launch_grouped_gemm(const GemmArgs& g, hipStream_t s) { return launch<kProduct, false>(g, s); }

hipError_t launch_grouped_dgrad(const GemmArgs& g, hipStream_t s) { return launch<kInputGrad, false>(g, s); }

hipError_t launch_grouped_wgrad(const GemmArgs& g, hipStream_t s) {
    if (!gather_fits(g, 2)) return launch_plain<kWeightGrad, false>(g, s);
    const WgradPlan p = plan_wgrad(g);
    if (p.big) return g.pairs ? launch_wgrad_tiles<256, 256, true>(g, s) : launch_wgrad_tiles<256, 256, false>(g, s);
    if (p.splits == 1)
        return g.pairs ? launch_wgrad_tiles<128, 128, true>(g, s) : launch_wgrad_tiles<128, 128, false>(g, s);
    GemmArgs part = g;
    part.out = g.ws;
    part.out_bf16 = false;
    part.accumulate = false;
    part.splits = p.splits;
    const hipError_t err =
        g.pairs ? launch_wgrad_tiles<128, 128, true>(part, s) : launch_wgrad_tiles<128, 128, false>(part, s);
    if (err != hipSuccess) return err;
    const int64_t values = static_cast<int64_t>(g.E) * g.N * g.K;
    const int64_t blocks = (values / 4 + kThreads - 1) / kThreads;
    join_wgrad_kernel<<<dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, s>>>(g, values, p.splits);
    return hipGetLastError();
}

hipError_t launch_grouped_int8(const GemmArgs& g, hipStream_t s) { return launch<kProduct, true>(g, s); }

hipError_t launch_quantize_rows(int64_t rows, int K, const uint16_t* x, int8_t* codes, float* scales,
                                hipStream_t s) {
    if (rows <= 0) return hipSuccess;
    const dim3 threads(kThreads), whole = folded_grid(rows), waves = folded_grid((rows + 3) / 4);
    // few rows: a workgroup each rather than a wave (rows of 1040: 301 3.0
    // against 5.2 us, 2048 4.6 and 5.5, 4096 6.7 and 7.3, 8192 11.5 and 10.9,
    // 32768 36.7 and 29.5)
    if (rows < 2048 && K > 512 && K <= 2048)
        quantize_rows_kernel<kThreads, 1><<<whole, threads, 0, s>>>(x, rows, K, codes, scales);
    else if (K <= 512)
        quantize_rows_kernel<kWave, 1><<<waves, threads, 0, s>>>(x, rows, K, codes, scales);
    else if (K <= 2048)
        quantize_rows_kernel<kWave, 4><<<waves, threads, 0, s>>>(x, rows, K, codes, scales);
    else if (K <= 8192)
        quantize_rows_kernel<kThreads, 4><<<whole, threads, 0, s>>>(x, rows, K, codes, scales);
    else if (K <= 16384)
        quantize_rows_kernel<kThreads, 8><<<whole, threads, 0, s>>>(x, rows, K, codes, scales);
    else
        quantize_rows_kernel<kThreads, 0><<<whole, threads, 0, s>>>(x, rows, K, codes, scales);
    return hipGetLastError();
}

}  // namespace moe
