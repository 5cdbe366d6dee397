// norm.hip -- the norm of rows and its gradient.
//
//   out = (x - mean) r weight + bias,  r = 1 / sqrt(mean((x - mean)^2) + eps)
//   dx  = r (d - xh mean(d xh) - mean(d)),  d = dy weight,  xh = (x - mean) r
//   dweight = sum over rows of dy xh,  dbias = sum over rows of dy
//
// (the RMS form: mean = 0, and no mean(d)).  Both are bound by memory: a row is
// read once, stays in registers and is written once.  Rows of 5120 in fp32:
// 65536 to bf16 at 5.6-6.0 TB/s, the gradient of 8192 at 4.8 TB/s (a copy of 2 GiB
// moves 4.9 TB/s, a fill 6.8).  A lane holds at most 16 values of a row and
// long rows take workgroups of up to 16 waves: 64 values a lane of 4 waves took
// 213 us for the gradient of 4096 x 16384 in bf16, this 87.
#include <type_traits>

#include "common.h"
#include "kernels.h"
#include "norm_kernels.h"

namespace moe {
namespace {

// Threads of a workgroup: LANES lanes a row, at least 256.
template <int LANES>
constexpr int kThreads = LANES > 256 ? LANES : 256;

struct Eight {
    float v[8];
};

// 8 values at element i of fp32 or bf16 rows.
template <bool F32>
__device__ __forceinline__ Eight load8(const void* p, int64_t i) {
    Eight o;
    if constexpr (F32) {
        const f32x4* q = reinterpret_cast<const f32x4*>(static_cast<const float*>(p) + i);
        const f32x4 a = q[0], b = q[1];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            o.v[j] = a[j];
            o.v[4 + j] = b[j];
        }
    } else {
        const u32x4 a = ld16(static_cast<const uint16_t*>(p) + i);
#pragma unroll
        for (int j = 0; j < 8; ++j) o.v[j] = __uint_as_float(j & 1 ? a[j / 2] & 0xffff0000u : a[j / 2] << 16);
    }
    return o;
}

__device__ __forceinline__ void store8(void* p, int64_t i, bool f32, const Eight& e) {
    if (f32) {
        f32x4* q = reinterpret_cast<f32x4*>(static_cast<float*>(p) + i);
        q[0] = f32x4{e.v[0], e.v[1], e.v[2], e.v[3]};
        q[1] = f32x4{e.v[4], e.v[5], e.v[6], e.v[7]};
    } else {
        *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p) + i) =
            u32x4{pack_bf16(e.v[0], e.v[1]), pack_bf16(e.v[2], e.v[3]), pack_bf16(e.v[4], e.v[5]),
                  pack_bf16(e.v[6], e.v[7])};
    }
}

// The sum over the LANES lanes of a row, the same in each: a wave, or the
// workgroup through s (a place for each wave, that no earlier sum still reads).
template <int LANES>
__device__ __forceinline__ float row_sum(float v, float* s) {
#pragma unroll
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d, kWave);
    if constexpr (LANES > kWave) {
        if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int w = 0; w < LANES / kWave; ++w) v += s[w];
    }
    return v;
}

// LANES lanes a row, CHUNKS times 8 values each.
template <bool F32, int LANES, int CHUNKS>
__global__ __launch_bounds__(kThreads<LANES>) void norm_kernel(NormArgs a) {
    __shared__ float s_sum[2][LANES / kWave];
    const int lane = threadIdx.x % LANES;
    const int64_t r = folded_index() * (kThreads<LANES> / LANES) + threadIdx.x / LANES;
    if (r >= a.rows) return;  // whole waves, or the whole workgroup of one row
    const int64_t at = r * a.H;
    Eight x[CHUNKS];
#pragma unroll
    for (int j = 0; j < CHUNKS; ++j) {
        const int c = (j * LANES + lane) * 8;
        if (c < a.H)
            x[j] = load8<F32>(a.x, at + c);
        else
            x[j] = Eight{};
    }
    float mean = 0.0f;
    if (a.center) {
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < CHUNKS; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) sum += x[j].v[i];
        mean = row_sum<LANES>(sum, s_sum[0]) / static_cast<float>(a.H);
    }
    float square = 0.0f;
#pragma unroll
    for (int j = 0; j < CHUNKS; ++j) {
        const bool inside = (j * LANES + lane) * 8 < a.H;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float d = inside ? x[j].v[i] - mean : 0.0f;
            square += d * d;
        }
    }
    const float inv = 1.0f / sqrtf(row_sum<LANES>(square, s_sum[1]) / static_cast<float>(a.H) + a.eps);
    if (a.stats && lane == 0) {
        a.stats[2 * r] = mean;
        a.stats[2 * r + 1] = inv;
    }
#pragma unroll
    for (int j = 0; j < CHUNKS; ++j) {
        const int c = (j * LANES + lane) * 8;
        if (c >= a.H) continue;
        const Eight w = load8<true>(a.weight, c);
        Eight o, b{};
        if (a.bias) b = load8<true>(a.bias, c);
#pragma unroll
        for (int i = 0; i < 8; ++i) o.v[i] = (x[j].v[i] - mean) * inv * w.v[i] + b.v[i];
        store8(a.out, at + c, a.out_f32, o);
    }
}

// Each group of LANES lanes takes rows r, r + groups, ... and keeps its sums of
// dweight and dbias in registers.  They go to ws, two rows of H for each
// workgroup.
template <bool X32, bool D32, int LANES, int CHUNKS>
__global__ __launch_bounds__(kThreads<LANES>) void norm_backward_kernel(NormArgs a) {
    constexpr int GROUPS = kThreads<LANES> / LANES;  // of a workgroup
    __shared__ float s_sum[2][2][LANES / kWave];
    const int lane = threadIdx.x % LANES;
    const int64_t group = static_cast<int64_t>(blockIdx.x) * GROUPS + threadIdx.x / LANES;
    const int64_t groups = static_cast<int64_t>(gridDim.x) * GROUPS;
    Eight dw[CHUNKS], db[CHUNKS];
#pragma unroll
    for (int j = 0; j < CHUNKS; ++j) dw[j] = db[j] = Eight{};
    const float per = 1.0f / static_cast<float>(a.H);
    int turn = 0;
    for (int64_t r = group; r < a.rows; r += groups, turn ^= 1) {
        const int64_t at = r * a.H;
        Eight x[CHUNKS], d[CHUNKS];
#pragma unroll
        for (int j = 0; j < CHUNKS; ++j) {
            const int c = (j * LANES + lane) * 8;
            x[j] = d[j] = Eight{};
            if (c < a.H) {
                x[j] = load8<X32>(a.x, at + c);
                d[j] = load8<D32>(a.dy, at + c);
            }
        }
        const float mean = a.stats[2 * r], inv = a.stats[2 * r + 1];
        float along = 0.0f, sum = 0.0f;
#pragma unroll
        for (int j = 0; j < CHUNKS; ++j) {
            const int c = (j * LANES + lane) * 8;
            if (c >= a.H) continue;
            const Eight w = load8<true>(a.weight, c);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float xh = (x[j].v[i] - mean) * inv, dy = d[j].v[i], g = dy * w.v[i];
                dw[j].v[i] += dy * xh;
                db[j].v[i] += dy;
                along += g * xh;
                sum += g;
                x[j].v[i] = xh;
                d[j].v[i] = g;
            }
        }
        along = row_sum<LANES>(along, s_sum[turn][0]) * per;
        sum = a.center ? row_sum<LANES>(sum, s_sum[turn][1]) * per : 0.0f;
#pragma unroll
        for (int j = 0; j < CHUNKS; ++j) {
            const int c = (j * LANES + lane) * 8;
            if (c >= a.H) continue;
            Eight o;
#pragma unroll
            for (int i = 0; i < 8; ++i) o.v[i] = (d[j].v[i] - x[j].v[i] * along - sum) * inv;
            store8(a.out, at + c, a.out_f32, o);
        }
    }
    if constexpr (GROUPS > 1) {  // the waves' sums added in order, in the first wave
        __shared__ Eight s_part[2][GROUPS - 1][LANES * CHUNKS];
        const int w = threadIdx.x / LANES;
#pragma unroll
        for (int j = 0; j < CHUNKS; ++j) {
            if (w == 0) continue;
            s_part[0][w - 1][j * LANES + lane] = dw[j];
            s_part[1][w - 1][j * LANES + lane] = db[j];
        }
        __syncthreads();
        if (w) return;
#pragma unroll
        for (int j = 0; j < CHUNKS; ++j)
            for (int k = 0; k < GROUPS - 1; ++k)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    dw[j].v[i] += s_part[0][k][j * LANES + lane].v[i];
                    db[j].v[i] += s_part[1][k][j * LANES + lane].v[i];
                }
    }
    const int64_t at = static_cast<int64_t>(blockIdx.x) * 2 * a.H;
#pragma unroll
    for (int j = 0; j < CHUNKS; ++j) {
        const int c = (j * LANES + lane) * 8;
        if (c >= a.H) continue;
        store8(a.ws, at + c, true, dw[j]);
        if (a.dbias) store8(a.ws, at + a.H + c, true, db[j]);
    }
}

// dweight and dbias (blockIdx.y) from the workgroups' sums, in a fixed order:
// 64 columns, 4 a thread, every 16th sum.
__global__ __launch_bounds__(256) void norm_sums_kernel(NormArgs a, int parts) {
    __shared__ f32x4 s_part[16][16];
    const int quad = threadIdx.x & 15, part = threadIdx.x >> 4;
    const int c = (blockIdx.x * 16 + quad) * 4;
    f32x4 sum = {0.f, 0.f, 0.f, 0.f};
    if (c < a.H) {
        const float* p = a.ws + static_cast<int64_t>(blockIdx.y) * a.H + c;
#pragma unroll 8
        for (int64_t g = part; g < parts; g += 16) sum += *reinterpret_cast<const f32x4*>(p + g * 2 * a.H);
    }
    s_part[part][quad] = sum;
    __syncthreads();
    if (part || c >= a.H) return;
#pragma unroll
    for (int i = 1; i < 16; ++i) sum += s_part[i][quad];
    f32x4* out = reinterpret_cast<f32x4*>((blockIdx.y ? a.dbias : a.dweight) + c);
    *out = a.accumulate ? *out + sum : sum;
}

// Lanes a row and chunks a lane, by the row's length: a wave, then workgroups
// of more and more waves, so that a lane holds at most 16 values of a row.
template <typename F>
hipError_t by_length(int H, F&& f) {
    using std::integral_constant;
    using One = integral_constant<int, 1>;
    using Two = integral_constant<int, 2>;
    if (H <= 512) return f(integral_constant<int, 64>{}, One{});
    if (H <= 2048) return f(integral_constant<int, 256>{}, One{});
    if (H <= 4096) return f(integral_constant<int, 512>{}, One{});
    if (H <= 8192) return f(integral_constant<int, 512>{}, Two{});
    return f(integral_constant<int, 1024>{}, Two{});
}

// Workgroups that share the rows of the gradient: as many as run at once, each
// writing its sums once (65536 x 1280: 512 of them 231 us, 1024 168, 1792 172;
// 8192 x 5120: 256 of them 121, 512 92, 768 110, 1024 118; 4096 x 16384: 256 of
// them 87, 512 92).
int parts_of(int64_t rows, int H) {
    const int64_t most = H <= 512 ? 512 : H <= 2048 ? 1024 : H <= 8192 ? 512 : 256;
    const int64_t want = H <= 512 ? (rows + 3) / 4 : rows;
    return static_cast<int>(want < most ? want : most);
}

}  // namespace

size_t norm_ws_bytes(int64_t rows, int H) {
    return rows <= 0 ? 0 : static_cast<size_t>(parts_of(rows, H)) * 2 * static_cast<size_t>(H) * sizeof(float);
}

hipError_t launch_norm(const NormArgs& a, hipStream_t s) {
    if (a.rows <= 0) return hipSuccess;
    return by_length(a.H, [&](auto lanes, auto chunks) {
        constexpr int L = decltype(lanes)::value, C = decltype(chunks)::value, T = kThreads<L>;
        const dim3 grid = folded_grid((a.rows + T / L - 1) / (T / L), T);
        if (a.x_f32)
            norm_kernel<true, L, C><<<grid, dim3(T), 0, s>>>(a);
        else
            norm_kernel<false, L, C><<<grid, dim3(T), 0, s>>>(a);
        return hipGetLastError();
    });
}

hipError_t launch_norm_backward(const NormArgs& a, hipStream_t s) {
    const int parts = a.rows > 0 ? parts_of(a.rows, a.H) : 0;
    if (parts) {
        const hipError_t e = by_length(a.H, [&](auto lanes, auto chunks) {
            constexpr int L = decltype(lanes)::value, C = decltype(chunks)::value;
            const dim3 grid(static_cast<unsigned>(parts)), threads(kThreads<L>);
            if (a.x_f32 && a.dy_f32)
                norm_backward_kernel<true, true, L, C><<<grid, threads, 0, s>>>(a);
            else if (a.x_f32)
                norm_backward_kernel<true, false, L, C><<<grid, threads, 0, s>>>(a);
            else if (a.dy_f32)
                norm_backward_kernel<false, true, L, C><<<grid, threads, 0, s>>>(a);
            else
                norm_backward_kernel<false, false, L, C><<<grid, threads, 0, s>>>(a);
            return hipGetLastError();
        });
        if (e != hipSuccess) return e;
    }
    norm_sums_kernel<<<dim3((a.H + 63) / 64, a.dbias ? 2 : 1), dim3(256), 0, s>>>(a, parts);
    return hipGetLastError();
}

}  // namespace moe
