// gemm_fp8.h -- the tiled kernel of the FP8 products with a scale for each
// block of 128 (moe_fp8.h).
//
//   out[q,c] = sum over blocks b of 2^(sy[row(q),b] + sx[e,b,c / 128])
//              sum over r in b of y[row(q),r] x[e,r,c]
//
// on e4m3 codes.  Scales are powers of two, so the scaled matrix instruction
// (32x32x64, twice the rate of bf16) applies them to its sums by itself and
// the fp32 accumulators never leave the matrix registers: with fp32 scales
// every block of the reduction would end in 16 multiply-adds a lane for each
// 32 x 32 of output, on registers that the vector unit can reach.
//
// The tile and its LDS layout are those of gemm_tile.h: 4 waves, BY rows of an
// expert by BX columns, operands loaded straight into LDS in stages of 128
// bytes a row.  A stage is one block of the reduction, two matrix
// instructions deep, so a lane needs one scale byte for each of its rows and
// one for its columns a stage.  The rows' scales are read 40 stages at a time
// into registers (LDS is full) and shifted down; the columns' lie one stage
// to a lane and are broadcast.
//
// Sums.  Measured: the matrix instructions add groups of 8 products, each cut
// towards zero to a multiple of 2^-13 of the largest's power of two, and sum
// the groups in fp32.  On normal values the cut is 1.5e-5 of the result, on
// equal signs 8e-5: 200 times below the operands' own rounding (2^-4), and
// below that of a bf16 output (2^-8).  Operands widened to bf16 (WIDE, codes times
// scale, exact) are summed in fp32 throughout, at half the rate.  gate_up does
// that on few rows: what g and u are off moves codes of h by whole steps (one
// row of 20480 x 5120, y after the down product: 2.5e-3 off the exact pass
// instead of 1.7e-3, y's own rounding), and the weight stream hides it (one row
// 54.6 -> 56.8 us, 256 experts of 4 rows 1053 -> 1061).  On more rows it would
// not (64 rows 1287 -> 1507; one matrix of 2 x 2560 x 5120, 512 rows: 42 -> 66),
// nor in the products (one row of 20480 x 5120: 26.6 -> 32).
//
// Three forms:
//   kF8Product    x = w[e] rows along K
//   kF8InputGrad  x = w[e] columns: the stage holds 128 rows of BX codes and
//                 the operand is read with the transposing LDS load
//                 (ds_read_b64_tr_b8: in each group of 16 lanes, lane i reads
//                 8 codes of row i / 2 and receives column i of the 8 x 16
//                 block).  Chunk c of row r lies at place c ^ down_swizzle(r),
//                 so that the 8 rows x 32 bytes of 32 lanes lie on all banks
//                 once.  A second matrix may follow the first in the reduction
//                 (dx = dg . gate + du . up in one pass).
//   kF8GateUp     BX / 2 columns of gate and the same of up, in turn by wave,
//                 so that a lane ends with g and u of the same places; BX / 2
//                 = 128 is a block of h, whose scale needs only its own tile.
#pragma once

#include "fp8_codes.h"
#include "fp8_kernels.h"
#include "gemm_tile.h"
#include "tile_plan.h"

namespace moe {
namespace {

enum Fp8Mode { kF8Product = 0, kF8InputGrad = 1, kF8GateUp = 2, kF8GateUpGrad = 3 };

// A pointer that is the same in every lane, in scalar registers.
__device__ __forceinline__ const uint8_t* uniform(const uint8_t* p) {
    const uint64_t v = reinterpret_cast<uint64_t>(p);
    const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v));
    const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v >> 32));
    return reinterpret_cast<const uint8_t*>(static_cast<uint64_t>(hi) << 32 | lo);
}

typedef int32_t i32x8 __attribute__((ext_vector_type(8)));
typedef int32_t i32x2 __attribute__((ext_vector_type(2)));

// One 32x32x64 step on e4m3 codes: lane l supplies 32 codes of row (or column)
// l % 32, half l / 32 of the 64; any order within the 64, the same for both.
// sa, sb: scale bytes in the low 8 bits.
__device__ __forceinline__ f32x16 mfma32_fp8(const i32x8& a, const i32x8& b, const f32x16& c, int sa, int sb) {
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 0, 0, 0, sa, 0, sb);
}

__device__ __forceinline__ u32x2 lds_read_tr8(const unsigned char* p) {
    return __builtin_bit_cast(
        u32x2, __builtin_amdgcn_ds_read_tr8_b64_v2i32(
                   (__attribute__((address_space(3))) i32x2*)const_cast<unsigned char*>(p)));
}

// Rows of 256 bytes: 8 of them put 32 bytes on each eighth of the banks; rows
// of 128: the parity of the row is one bit of the bank already.
template <int BX>
__device__ __forceinline__ int down_swizzle(int r) {
    return BX >= 256 ? (r & 7) << 1 : ((r >> 1) & 3) << 1;
}

// Four fp32 -> four e4m3 codes (nearest even), the first in the low byte.
__device__ __forceinline__ uint32_t pack_fp8(float a, float b, float c, float d) {
    int v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true));
}

// Codes of four values in a block whose largest magnitude has the bits top
// (without a branch: see the epilogue).
__device__ __forceinline__ uint32_t block_codes(const f32x4& v, uint32_t top, float inverse) {
    const uint32_t keep = top - kTinyBits < kInfBits - kTinyBits ? 0xffffffffu : 0u;
    const uint32_t bad = top >= kInfBits ? 0x7f7f7f7fu : 0u;
    return (pack_fp8(v[0] * inverse, v[1] * inverse, v[2] * inverse, v[3] * inverse) & keep) | bad;
}

__device__ __forceinline__ uint32_t magnitude_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// gemm_tile.h's tiles, and 32 rows of gate and up: two buffers of 36 KB, so
// that two workgroups share a compute unit and one's first loads and writing
// run beside the other's stages (256 experts of 2 x 2560 x 5120, 4 rows each:
// 1051 us, with four buffers and a compute unit to itself 1113).
template <int BX, int BY>
struct Fp8Shape {
    static constexpr int kWavesY = BY >= 64 ? 2 : 1, kWavesX = kWaves / kWavesY;
    static constexpr bool kSmall = BX == 256 && BY == 32;
    static constexpr int kXBufs = BY >= 64 ? 3 : (kSmall ? 2 : 4), kYBufs = BY >= 64 || kSmall ? 2 : 4;
    static constexpr int kXStage = BX * 128, kYStage = BY * 128;
    static constexpr int kArena = kXBufs * kXStage + kYBufs * kYStage;
    static_assert(kArena <= 163840, "LDS budget");
    static constexpr int kPerCu = kArena <= 81920 ? 2 : 1;
};

// 8 codes times their scale as bf16, exactly: codes have 4 significant bits and
// are multiples of 2^-9, so from scale 2^-124 on (byte 3) they are multiples of
// bf16's smallest, 2^-133, which the matrix instruction takes as it is; values
// below 2^128 are finite.
__device__ __forceinline__ bf16x8 widen(uint32_t lo, uint32_t hi, float scale) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true);
    return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// Words of a row's scales held in registers: 40 stages, K = 5120.
constexpr int kScaleWords = 10;

template <int MODE, int BX, int BY, bool GATHER, bool NT, bool WIDE>
__global__ __launch_bounds__(kThreads, (Fp8Shape<BX, BY>::kPerCu)) void fp8_tile_kernel(Fp8Args g) {
    typedef Fp8Shape<BX, BY> Shape;
    constexpr bool TRX = MODE == kF8InputGrad;
    constexpr bool GATED = MODE == kF8GateUp || MODE == kF8GateUpGrad;
    constexpr int PARTS = MODE == kF8Product ? 1 : 2;    // weight matrices
    constexpr int WY = Shape::kWavesY, WX = Shape::kWavesX;
    constexpr int XB = BX / 32 / WX, YB = BY / 32 / WY;  // 32-blocks per wave
    constexpr int COLS = GATED ? BX / 2 : BX;            // output columns of the tile
    constexpr int WCOLS = COLS / WX;                     // and of a wave
    static_assert(WCOLS <= kBlock && kBlock % WCOLS == 0, "a wave's columns lie in one block");
    static_assert(!GATED || (COLS == kBlock && XB % 2 == 0), "a tile is a block of h");
    constexpr int XS = Shape::kXStage, YS = Shape::kYStage;
    constexpr int XBUFS = Shape::kXBufs, YBUFS = Shape::kYBufs;
    // Stages the loads run ahead.  Both operands of a stage are in registers
    // half way through it, so a barrier there (MID) frees an operand's buffer
    // for the loads of the stage after the next where it has only two
    constexpr bool MID = YBUFS == 2, X_LATE = XBUFS == 2;
    constexpr int XA = X_LATE ? 2 : XBUFS - 1, YA = MID ? 2 : YBUFS - 1;
    static_assert(XA == YA && (MID || !X_LATE), "the count of younger loads");
    constexpr int DMA_X = BX / 32, DMA_Y = BY / 32;      // 1 KB loads per wave and stage
    // loads younger than those of the next stage, at a stage's end
    constexpr int YOUNGER = (XA - 1) * (DMA_X + DMA_Y);

    __shared__ __attribute__((aligned(1024))) unsigned char s_arena[Shape::kArena];
    const uint32_t arena = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(s_arena));

    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int cols = MODE == kF8InputGrad ? g.K : g.N;
    const int col_tiles = (cols + COLS - 1) / COLS;

    // Inlined, and in variables of their own, so that the tile is in scalar
    // registers: as a call it came back through scratch, and every branch on it
    // below was a lane mask
    int found[4];
    bool work;
    [[clang::always_inline]] work = find_tile<BY, BY >= 64 ? 64 : 1, kBand>(
        g.offsets, g.P, g.E, col_tiles, reinterpret_cast<int32_t*>(s_arena),
        reinterpret_cast<int32_t*>(s_arena) + (kMaxE + 1), found[0], found[1], found[2], found[3]);
    if (!work) return;
    const int e = __builtin_amdgcn_readfirstlane(found[0]), nt = __builtin_amdgcn_readfirstlane(found[1]);
    const int row0 = __builtin_amdgcn_readfirstlane(found[2]), rows = __builtin_amdgcn_readfirstlane(found[3]);
    __syncthreads();  // everyone is done with the schedule before the arena is reused
    const int c0 = nt * COLS;
    const int64_t orow0 = row0;
    const int nblk = (rows + 31) >> 5;
    const int64_t K = g.K, N = g.N;
    const int NB = (g.N + kBlock - 1) / kBlock, KB = (g.K + kBlock - 1) / kBlock;
    // stages: blocks of the reduction; input grad: those of both matrices
    const int part_stages = TRX ? NB : KB;
    const int nk = TRX && g.w[1] ? 2 * NB : part_stages;
    const int s0 = static_cast<int>(static_cast<int64_t>(nk) * blockIdx.y / gridDim.y);
    const int s1 = static_cast<int>(static_cast<int64_t>(nk) * (blockIdx.y + 1) / gridDim.y);
    const bool split = gridDim.y > 1;

    // ---- loads (gemm_tile.h) ----
    const int64_t matrix = static_cast<int64_t>(e) * N * K + static_cast<int64_t>(c0) * (TRX ? 1 : K);
    const uint8_t* const xbase0 = uniform(g.w[0] + matrix);
    const uint8_t* const xbase1 = PARTS > 1 ? uniform(g.w[1] + matrix) : xbase0;
    const uint8_t* const xscale0 = g.w_scale[0] + static_cast<int64_t>(e) * NB * KB;
    const uint8_t* const xscale1 = PARTS > 1 ? g.w_scale[1] + static_cast<int64_t>(e) * NB * KB : xscale0;
    const uint8_t* ybase = g.y + (GATHER ? 0 : orow0 * g.y_cols);
    uint32_t vx[DMA_X], vy[DMA_Y];
    auto along_row = [&](int j, int per_wave) { return wave * per_wave + j * 8 + (lane >> 3); };
    auto along_chunk = [&](int r) { return (lane & 7) ^ ((r >> 1) & 7); };
    auto gather_row = [&](int r) -> int64_t {  // the row of y of output row r
        const int64_t q = orow0 + min(r, rows - 1);
        if constexpr (!GATHER) return q;
        const int64_t s = g.pairs[q] / g.k;
        return s < 0 ? 0 : (s >= g.S ? g.S - 1 : s);
    };
    // gated: the matrix and column of a stage's row, wave by wave: gate, up.
    // A wave loads of one matrix, or of both, half its loads each
    constexpr int HALF = BX / WX / 2;
    static_assert(!GATED || HALF * 2 == BX / 4 || HALF == BX / 4, "rows of a wave's loads");
    auto x_second = [&](int j) { return GATED && (HALF == BX / 4 ? (wave & 1) != 0 : j >= DMA_X / 2); };
    const uint32_t xbytes = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(min(COLS, cols - c0) * K));
#pragma unroll
    for (int j = 0; j < DMA_X; ++j) {
        if constexpr (TRX) {
            const int r = wave * 32 + j * (1024 / BX) + lane / (BX / 16);
            const int c = (lane % (BX / 16)) ^ down_swizzle<BX>(r);
            vx[j] = static_cast<uint32_t>(r * K + c * 16);
        } else {
            const int r = along_row(j, BX / 4);
            const int col = GATED ? r / (2 * HALF) * HALF + r % HALF : r;
            vx[j] = static_cast<uint32_t>(col * K + along_chunk(r) * 16);
        }
    }
#pragma unroll
    for (int j = 0; j < DMA_Y; ++j) {
        const int r = along_row(j, BY / 4);
        const int c = along_chunk(r);
        if (r >= nblk * 32)
            vy[j] = kNoRowOffset;
        else if constexpr (GATHER)
            vy[j] = static_cast<uint32_t>(gather_row(r) * g.y_cols + c * 16);
        else
            vy[j] = static_cast<uint32_t>(r * g.y_cols + c * 16);
    }
    // chunks of a matrix's last stage that lie inside the reduction (along
    // rows; the rows of y of two matrices are padded to whole blocks)
    const int tail = (TRX ? (g.w[1] ? kBlock : g.N - (NB - 1) * kBlock) : g.K - (KB - 1) * kBlock) / 16;
    auto x_buf = [&](int i) { return arena + i * XS; };
    auto y_buf = [&](int i) { return arena + XBUFS * XS + i * YS; };
    const __amdgpu_buffer_rsrc_t rsrc_y =
        make_rsrc(uniform(ybase), __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(
                                      (GATHER ? g.S : static_cast<int64_t>(rows)) * g.y_cols)));
    auto dma_x = [&](int j, int buf, int kt) {
        const uint32_t at = x_buf(buf) + wave * (XS / 4) + j * 1024;
        if constexpr (TRX) {
            // the buffer starts at the stage's first row and ends with its
            // last row inside the reduction
            const bool second = kt >= part_stages;
            const int kk = second ? kt - part_stages : kt;
            const int valid = min(kBlock, g.N - kk * kBlock);
            dma_load16<NT>(at,
                           make_rsrc(uniform((second ? xbase1 : xbase0) + static_cast<int64_t>(kk) * kBlock * K),
                                     __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(valid * K - c0))),
                           vx[j], 0);
        } else {
            const bool past = kt == nk - 1 && along_chunk(along_row(j, BX / 4)) >= tail;
            dma_load16<NT>(at, make_rsrc(uniform(x_second(j) ? xbase1 : xbase0), xbytes), past ? kNoRowOffset : vx[j],
                           static_cast<uint32_t>(kt * 128));
        }
    };
    auto dma_y = [&](int j, int buf, int kt) {
        const uint32_t at = y_buf(buf) + wave * (YS / 4) + j * 1024;
        const bool past = kt == nk - 1 && along_chunk(along_row(j, BY / 4)) >= tail;
        dma_load16(at, rsrc_y, past ? kNoRowOffset : vy[j], static_cast<uint32_t>(kt * 128));
    };

    const int wy = wave / WX, wx = wave % WX;
    const int r32 = lane & 31, half = lane >> 5;
    int valid_blocks = 0;
#pragma unroll
    for (int m = 0; m < YB; ++m) valid_blocks += (wy + WY * m) < nblk;

    f32x16 acc[YB][XB];
#pragma unroll
    for (int m = 0; m < YB; ++m)
#pragma unroll
        for (int n = 0; n < XB; ++n)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[m][n][i] = 0.0f;

    // ---- scales.  Of this wave's columns: one block ----
    const int xblock = min((c0 + wx * WCOLS) / kBlock, (TRX ? KB : NB) - 1);
    uint32_t ysc[YB][kScaleWords];
    int xsc0, xsc1 = 0;
    const uint8_t* yscale[YB];
    static_for<0, YB>([&](auto mc) {
        constexpr int m = decltype(mc)::value;
        yscale[m] = g.y_scale + gather_row((wy + WY * m) * 32 + r32) * g.y_pitch;
    });
    // from stage `first` (a multiple of 4) on
    auto load_scales = [&](int first) {
        const int t = min(first + lane, nk - 1);
        if constexpr (TRX) {
            const bool second = t >= part_stages;
            xsc0 = (second ? xscale1 : xscale0)[static_cast<int64_t>(second ? t - part_stages : t) * KB + xblock];
        } else {
            xsc0 = xscale0[static_cast<int64_t>(xblock) * KB + t];
            if constexpr (GATED) xsc1 = xscale1[static_cast<int64_t>(xblock) * KB + t];
        }
#pragma unroll
        for (int i = 0; i < kScaleWords; ++i) {
            if (first + 4 * i >= nk) continue;
#pragma unroll
            for (int m = 0; m < YB; ++m)
                ysc[m][i] = *reinterpret_cast<const uint32_t*>(yscale[m] + first + 4 * i);
        }
    };

    // the operand of rows [32 b, 32 b + 32) (along) or columns (down), substep ks
    auto read_along = [&](uint32_t buf, int b, int ks) {
        const int r = b * 32 + r32;
        const unsigned char* row = s_arena + (buf - arena) + r * 128;
        const int c = ks * 4 + half * 2, sw = (r >> 1) & 7;
        const u32x4 lo = *reinterpret_cast<const u32x4*>(row + ((c ^ sw) << 4));
        const u32x4 hi = *reinterpret_cast<const u32x4*>(row + (((c + 1) ^ sw) << 4));
        return i32x8{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
    };
    auto read_down = [&](uint32_t buf, int b, int ks) {
        const int i = lane & 15;
        const int c = b * 2 + ((lane >> 4) & 1);
        i32x8 v;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int r = ks * 64 + half * 32 + j * 8 + (i >> 1);
            const u32x2 t = lds_read_tr8(s_arena + (buf - arena) + r * BX + ((c ^ down_swizzle<BX>(r)) << 4) + (i & 1) * 8);
            v[2 * j] = static_cast<int>(t[0]);
            v[2 * j + 1] = static_cast<int>(t[1]);
        }
        return v;
    };

    // the stages, with NV valid row blocks in this wave
    auto k_loop = [&](auto nv_tag) {
        constexpr int NV = decltype(nv_tag)::value;
        constexpr int NA = NV > 0 ? NV : 1;
        constexpr int MF = NV * XB;  // matrix instructions per substep
        struct Frags {
            i32x8 y[NA];
            i32x8 x[XB];
        };
        constexpr int NP = NV > 0 ? NV + XB : 0;
        int ys[NA], xs0 = 0, xs1 = 0;
        auto load_piece = [&](Frags& f, int yb, int xb, int ks, auto qc) {
            constexpr int q = decltype(qc)::value;
            if constexpr (q < NV) {
                f.y[q] = read_along(y_buf(yb), wy + WY * q, ks);
            } else if constexpr (NV > 0) {
                constexpr int n = q - NV;
                if constexpr (TRX)
                    f.x[n] = read_down(x_buf(xb), wx * XB + n, ks);
                else
                    f.x[n] = read_along(x_buf(xb), wx * XB + n, ks);
            }
        };
        auto load_frags = [&](Frags& f, int yb, int xb, int ks) {
            static_for<0, NP>([&](auto qc) { load_piece(f, yb, xb, ks, qc); });
        };
        auto mfma_one = [&](const Frags& f, auto ic) {
            constexpr int i = decltype(ic)::value;
            if constexpr (NV > 0 && WIDE) {
                constexpr int m = i % NV, n = i / NV;
                const float x = __uint_as_float(static_cast<uint32_t>(GATED && n >= XB / 2 ? xs1 : xs0) << 23);
                const float y = __uint_as_float(static_cast<uint32_t>(ys[m]) << 23);
                f32x16 c = acc[m][n];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    c = mfma32(widen(f.x[n][2 * k], f.x[n][2 * k + 1], x), widen(f.y[m][2 * k], f.y[m][2 * k + 1], y), c);
                acc[m][n] = c;
            } else if constexpr (NV > 0) {
                constexpr int m = i % NV, n = i / NV;
                acc[m][n] = mfma32_fp8(f.x[n], f.y[m], acc[m][n], GATED && n >= XB / 2 ? xs1 : xs0, ys[m]);
            }
        };
        const int last = s1 - 1;
        static_for<0, XA>([&](auto sc) {
            constexpr int st = decltype(sc)::value;
#pragma unroll
            for (int j = 0; j < DMA_X; ++j) dma_x(j, st, min(s0 + st, last));
#pragma unroll
            for (int j = 0; j < DMA_Y; ++j) dma_y(j, st, min(s0 + st, last));
        });
        int held = s0 & ~3;  // the stage whose scales lie in the first place
        int held_x = held;   // and that of lane 0's column scale
        load_scales(held);
        wait_vmcnt<YOUNGER>();
        __syncthreads();
        int ybuf = 0, xbuf = 0;
        Frags f0, f1;
        load_frags(f0, 0, 0, 0);
        for (int kt = s0; kt < s1; ++kt) {
            if (kt - held_x == 4 * kScaleWords) {
                held = held_x = kt;
                load_scales(kt);
            } else if (kt - held == 4) {
                held = kt;
#pragma unroll
                for (int m = 0; m < NA; ++m)
#pragma unroll
                    for (int i = 0; i + 1 < kScaleWords; ++i) ysc[m][i] = ysc[m][i + 1];
            }
            const int shift = 8 * (kt - held);
#pragma unroll
            for (int m = 0; m < NA; ++m) ys[m] = static_cast<int>(ysc[m][0] >> shift) & (WIDE ? 255 : -1);
            xs0 = __builtin_amdgcn_readlane(xsc0, kt - held_x);
            if constexpr (GATED) xs1 = __builtin_amdgcn_readlane(xsc1, kt - held_x);
            // past the end: an idle buffer is filled again
            const int ky = min(kt + YA, last);
            const int kx = min(kt + XA, last);
            const int xnext = X_LATE ? xbuf : (xbuf == 0 ? XBUFS - 1 : xbuf - 1);  // the buffer freed last
            const int ynext = MID ? ybuf : (ybuf == 0 ? YBUFS - 1 : ybuf - 1);
            // The stage's loads are spread over the matrix instructions of its
            // two substeps, the reads of the next substep's operands between
            // them (scheduling fences keep them there).  The barrier sits
            // before the last eighth of the second substep, so the first
            // operands of the next stage are read while those run.
            auto substep = [&](const Frags& f, auto sc, auto lo_c, auto hi_c, Frags& fn, auto kn_c) {
                constexpr int sub = decltype(sc)::value;
                constexpr int LO = decltype(lo_c)::value, HI = decltype(hi_c)::value;
                constexpr int KN = decltype(kn_c)::value;
                constexpr int NM = HI - LO;
                // this substep's loads, x's in the first of two unless its
                // buffer is still read there
                constexpr int NX = (X_LATE ? sub == 1 : sub == 0) ? DMA_X : 0;
                constexpr int NL = NX + (sub == 1 ? DMA_Y : 0);
                constexpr int NPC = KN >= 0 ? NP : 0;
                constexpr int IT0 = NM > NL ? NM : NL;
                constexpr int IT = IT0 > 0 ? IT0 : 1;
                static_for<0, IT>([&](auto ic) {
                    constexpr int i = decltype(ic)::value;
                    static_for<0, NPC>([&](auto qc) {
                        constexpr int q = decltype(qc)::value;
                        if constexpr (q * IT / (NPC > 0 ? NPC : 1) == i) load_piece(fn, ybuf, xbuf, KN, qc);
                    });
                    if constexpr (i < NM) mfma_one(f, std::integral_constant<int, LO + i>{});
                    constexpr int step = NM >= NL ? (NL > 0 ? NM / NL : 1) : 1;
                    if constexpr (NL > 0 && i % step == step - 1 && i / step < NL) {
                        if constexpr (i / step < NX)
                            dma_x(i / step, xnext, kx);
                        else
                            dma_y(i / step - NX, ynext, ky);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                });
            };
            using C0 = std::integral_constant<int, 0>;
            using CM = std::integral_constant<int, MF>;
            using CH = std::integral_constant<int, MF * 7 / 8>;
            using K0 = std::integral_constant<int, 0>;
            using K1 = std::integral_constant<int, 1>;
            using KNone = std::integral_constant<int, -1>;
            substep(f0, K0{}, C0{}, CM{}, f1, K1{});
            if constexpr (MID) __syncthreads();  // nobody reads this stage's y again
            substep(f1, K1{}, C0{}, CH{}, f0, KNone{});
            wait_vmcnt<YOUNGER>();
            __syncthreads();
            ybuf = ybuf == YBUFS - 1 ? 0 : ybuf + 1;
            xbuf = xbuf == XBUFS - 1 ? 0 : xbuf + 1;
            load_frags(f0, ybuf, xbuf, 0);  // after the last stage: read, never used
            __builtin_amdgcn_sched_barrier(0);
            substep(f1, KNone{}, CH{}, CM{}, f0, KNone{});
        }
        wait_vmcnt<0>();
        __syncthreads();
    };
    static_for<0, YB + 1>([&](auto nv_tag) {
        if (valid_blocks == decltype(nv_tag)::value) k_loop(nv_tag);
    });

    // ---- epilogue: through LDS, one block of 32 rows of this wave at a time
    // (a region of its own), so that the stores are 16 bytes a lane over whole
    // rows.  Nothing here runs under a lane mask: on the 256-row tiles nearly
    // all 512 registers hold sums or dh, and the compiler has been seen to move
    // such values inside the mask of a store and to lose those of the other
    // lanes.  Stores past the tile's rows or columns go to an offset past their
    // buffer's end instead, and loads from there give zeros ----
    constexpr int PITCH = WCOLS * 4 + 16;  // 4-byte elements; others: WCOLS * their bytes + 16
    constexpr int REGION = 32 * PITCH;
    static_assert(4 * REGION + BY * WX * 8 <= Shape::kArena, "epilogue region");
    unsigned char* region = s_arena + wave * REGION;
    const int wc0 = c0 + wx * WCOLS;
    // this tile's rows of an output of `width` bytes a row: at most 256 x 65536
    // x 4 bytes, or 256 x 131072
    auto tile_rows = [&](void* out, int64_t width) {
        uint8_t* const first = static_cast<uint8_t*>(out) + orow0 * width;
        return make_rsrc(uniform(first), __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(rows * width)));
    };
    // place of 16 bytes in them: row r of block blk, column c0 + c (in elements)
    // of the columns below `end`
    auto place = [&](int width, int blk, int r, int c0, int c, int end, int bytes) {
        return static_cast<uint32_t>((blk * 32 + r) * width + (c0 + c) * bytes) | (c0 + c < end ? 0u : kNoRowOffset);
    };
    // 32 rows at `from` in LDS to those rows, `width` elements of BYTES each, at
    // column col, columns below `end`
    auto put_rows = [&](auto bytes_c, const unsigned char* from, __amdgpu_buffer_rsrc_t out, int width, int blk, int col,
                        int end) {
        constexpr int BYTES = decltype(bytes_c)::value;
        constexpr int LPR = WCOLS * BYTES / 16;  // lanes per row
        int l = lane;
        asm volatile("" : "+v"(l));  // its places are computed here, not held over the loop in registers
#pragma unroll
        for (int it = 0; it < 32 * LPR / 64; ++it) {
            const int r = it * (64 / LPR) + l / LPR, c = l % LPR * (16 / BYTES);
            const u32x4 v = ld16(from + r * (WCOLS * BYTES + 16) + c * BYTES);
            __builtin_amdgcn_raw_buffer_store_b128(v, out, place(width * BYTES, blk, r, col, c, end, BYTES), 0, 0);
        }
    };
    using B1 = std::integral_constant<int, 1>;
    using B2 = std::integral_constant<int, 2>;

    if constexpr (!GATED) {
        const bool out_bf16 = g.out_bf16 && !split, accumulate = g.accumulate && !split;
        void* const out = split ? static_cast<float*>(g.ws) + static_cast<int64_t>(blockIdx.y) * g.P * cols : g.out;
        const __amdgpu_buffer_rsrc_t rsrc_out = tile_rows(out, static_cast<int64_t>(cols) * (out_bf16 ? 2 : 4));
#pragma unroll
        for (int m = 0; m < YB; ++m) {
            if (m >= valid_blocks) continue;
            const int blk = wy + WY * m;
#pragma unroll
            for (int n = 0; n < XB; ++n)
#pragma unroll
                for (int i4 = 0; i4 < 4; ++i4) {
                    const int col = n * 32 + 8 * i4 + 4 * half;
                    f32x4 v;
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[i] = acc[m][n][4 * i4 + i];
                    if (out_bf16) {
                        const u32x2 b = {pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
                        *reinterpret_cast<u32x2*>(region + r32 * (WCOLS * 2 + 16) + col * 2) = b;
                    } else {
                        *reinterpret_cast<f32x4*>(region + r32 * PITCH + col * 4) = v;
                    }
                }
            wave_lds_fence();
            if (out_bf16) {
                put_rows(B2{}, region, rsrc_out, cols, blk, wc0, cols);
            } else {
                constexpr int LPR = WCOLS / 4;
#pragma unroll
                for (int it = 0; it < 32 * LPR / 64; ++it) {
                    const int r = it * (64 / LPR) + lane / LPR, c = lane % LPR * 4;
                    f32x4 v = *reinterpret_cast<const f32x4*>(region + r * PITCH + c * 4);
                    const uint32_t to = place(cols * 4, blk, r, wc0, c, cols, 4);
                    if (accumulate)
                        v += __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(rsrc_out, to, 0, 0));
                    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), rsrc_out, to, 0, 0);
                }
            }
            wave_lds_fence();
        }
    } else {
        // h = silu(g) u, or dg and du beside it; then the codes of the rows'
        // blocks, whose largest magnitudes the waves of a row exchange
        constexpr bool GRAD = MODE == kF8GateUpGrad;
        constexpr int HB = XB / 2;
        constexpr int CODES = 32 * (WCOLS * 2 + 16);  // the codes' place behind bf16 rows in the region
        static_assert(!GRAD || CODES + 32 * (WCOLS + 16) <= REGION, "both fit");
        uint32_t* const s_top = reinterpret_cast<uint32_t*>(s_arena + 4 * REGION);  // [2][BY][WX]
        // h, dg and du of four places, from the accumulators and dh.  The
        // gradients are computed in both passes below: kept, they would take
        // the place of g and u and spill (256 registers each)
        f32x4 dh[GRAD ? YB : 1][HB][4];  // all asked for at once, held over both passes
        __amdgpu_buffer_rsrc_t rsrc_h, rsrc_dg, rsrc_du;
        const __amdgpu_buffer_rsrc_t rsrc_q = tile_rows(g.q, g.q_cols), rsrc_scale = tile_rows(g.q_scale, g.q_pitch);
        if constexpr (GRAD) {
            rsrc_h = tile_rows(g.h, N * 2);
            rsrc_dg = tile_rows(g.dg, N * 2);
            rsrc_du = tile_rows(g.du, N * 2);
            const __amdgpu_buffer_rsrc_t rsrc_dh = tile_rows(const_cast<float*>(g.dh), N * 4);
#pragma unroll
            for (int m = 0; m < YB; ++m)
#pragma unroll
                for (int n = 0; n < HB; ++n)
#pragma unroll
                    for (int i4 = 0; i4 < 4; ++i4)
                        dh[m][n][i4] = __builtin_bit_cast(
                            f32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                       rsrc_dh, place(cols * 4, wy + WY * m, r32, wc0, n * 32 + 8 * i4 + 4 * half, cols, 4), 0, 0));
        }
        auto four = [&](int m, int n, int i4, f32x4& h, f32x4& dg, f32x4& du) {
            f32x4 d = {0.f, 0.f, 0.f, 0.f};
            if constexpr (GRAD) d = dh[m][n][i4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float a = acc[m][n][4 * i4 + i], b = acc[m][n + HB][4 * i4 + i];
                const float s = sigmoid_f32(a), silu = a * s;
                h[i] = silu * b;
                dg[i] = d[i] * b * (s + silu * (1.0f - s));
                du[i] = d[i] * silu;
            }
        };
#pragma unroll
        for (int m = 0; m < YB; ++m) {
            if (m >= valid_blocks) continue;
            const int blk = wy + WY * m;
            uint32_t top0 = 0, top1 = 0;
#pragma unroll
            for (int n = 0; n < HB; ++n)
#pragma unroll
                for (int i4 = 0; i4 < 4; ++i4) {
                    f32x4 h, dg, du;
                    four(m, n, i4, h, dg, du);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if constexpr (GRAD) {
                            top0 = max(top0, magnitude_bits(dg[i]));
                            top1 = max(top1, magnitude_bits(du[i]));
                        } else {
                            top0 = max(top0, magnitude_bits(h[i]));
                            acc[m][n][4 * i4 + i] = h[i];
                        }
                    }
                    if constexpr (GRAD)
                        *reinterpret_cast<u32x2*>(region + r32 * (WCOLS * 2 + 16) + (n * 32 + 8 * i4 + 4 * half) * 2) =
                            u32x2{pack_bf16(h[0], h[1]), pack_bf16(h[2], h[3])};
                }
            top0 = max(top0, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top0), 32, kWave)));
            if constexpr (GRAD) top1 = max(top1, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top1), 32, kWave)));
            // both halves hold the same and write it to the same place
            s_top[(blk * 32 + r32) * WX + wx] = top0;
            if constexpr (GRAD) s_top[(BY + blk * 32 + r32) * WX + wx] = top1;
            if constexpr (GRAD) {
                wave_lds_fence();
                put_rows(B2{}, region, rsrc_h, cols, blk, wc0, cols);
                wave_lds_fence();
            }
        }
        __syncthreads();
#pragma unroll
        for (int m = 0; m < YB; ++m) {
            if (m >= valid_blocks) continue;
            const int blk = wy + WY * m;
#pragma unroll
            for (int part = 0; part < (GRAD ? 2 : 1); ++part) {
                uint32_t top = 0;
#pragma unroll
                for (int w = 0; w < WX; ++w) top = max(top, s_top[(part * BY + blk * 32 + r32) * WX + w]);
                const int scale = fp8_scale_of(top);
                const float inverse = __uint_as_float(fp8_inverse_bits(scale));
#pragma unroll
                for (int n = 0; n < HB; ++n)
#pragma unroll
                    for (int i4 = 0; i4 < 4; ++i4) {
                        const int col = n * 32 + 8 * i4 + 4 * half;
                        f32x4 v;
                        if constexpr (GRAD) {
                            f32x4 h, dg, du;
                            four(m, n, i4, h, dg, du);
                            v = part ? du : dg;
                            *reinterpret_cast<u32x2*>(region + r32 * (WCOLS * 2 + 16) + col * 2) =
                                u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
                        } else {
#pragma unroll
                            for (int i = 0; i < 4; ++i) v[i] = acc[m][n][4 * i4 + i];
                        }
                        *reinterpret_cast<uint32_t*>(region + (GRAD ? CODES : 0) + r32 * (WCOLS + 16) + col) =
                            block_codes(v, top, inverse);
                    }
                wave_lds_fence();
                if constexpr (GRAD) put_rows(B2{}, region, part ? rsrc_du : rsrc_dg, cols, blk, wc0, cols);
                // [dg | du]: every column of the last block is written, zeros
                // behind the last, since the two parts are one reduction
                const int first = part * col_tiles * kBlock;
                put_rows(B1{}, region + (GRAD ? CODES : 0), rsrc_q, static_cast<int>(g.q_cols), blk, first + wc0,
                         first + (GRAD ? col_tiles * kBlock : cols));
                wave_lds_fence();
                if (wx == 0)
                    __builtin_amdgcn_raw_buffer_store_b8(
                        static_cast<uint8_t>(scale), rsrc_scale,
                        static_cast<uint32_t>((blk * 32 + r32) * g.q_pitch + part * col_tiles + nt) | (half ? kNoRowOffset : 0u),
                        0, 0);
            }
        }
    }
}

template <int MODE, int BX, int BY, bool NT = false, bool WIDE = false>
hipError_t launch_tiles(const Fp8Args& g, hipStream_t s, int splits = 1) {
    constexpr bool kGated = MODE == kF8GateUp || MODE == kF8GateUpGrad;
    const int64_t grid = tile_grid(g.P, g.E, MODE == kF8InputGrad ? g.K : g.N, kGated ? BX / 2 : BX, BY);
    if (grid <= 0) return hipSuccess;
    if (grid > kMaxWorkgroups) return hipErrorInvalidConfiguration;
    const dim3 blocks(static_cast<unsigned>(grid), splits), threads(kThreads);
    if constexpr (MODE != kF8InputGrad) {
        if (g.pairs) {
            fp8_tile_kernel<MODE, BX, BY, true, NT, WIDE><<<blocks, threads, 0, s>>>(g);
            return hipGetLastError();
        }
    }
    fp8_tile_kernel<MODE, BX, BY, false, NT, WIDE><<<blocks, threads, 0, s>>>(g);
    return hipGetLastError();
}

}  // namespace
}  // namespace moe
