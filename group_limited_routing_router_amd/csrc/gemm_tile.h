// gemm_tile.h -- the tiled kernel of the grouped products (moe_gemm.h).
//
// The product and the input gradient (the weight gradient: gemm_wgrad.h).
// A workgroup of 4 waves owns a BY x BX tile of one expert's output: BY
// positions of the expert by BX columns.
// Each wave owns a quarter, 32 x 32 blocks dealt over the two wave rows
// (block b to wave row b % 2), blocks past the tile's last row skipped, so a
// partly filled tile costs matrix time in proportion to its rows.
//
// Operand X supplies the output's columns, operand Y its rows:
//              X (columns)                 Y (rows)
//   product    w[e], reduction along rows  a, reduction along rows (gathered)
//   input grad w[e], reduction down rows   dout, reduction along rows
// X is the first operand of the matrix instruction, so a lane ends with one
// output row and groups of four consecutive columns of it.
//
// Both operands go straight from HBM into LDS (buffer loads with an LDS
// destination, 1 KB an instruction), no staging registers.  A stage is 128
// bytes of reduction (64 bf16, 128 int8):
//  - reduction along the rows in memory: the stage holds 128 bytes of each
//    row, chunk c (16 bytes) of row r at place c ^ ((r >> 1) & 7), so the 16
//    rows of an operand read lie on all 64 banks once;
//  - reduction down the rows: the stage holds 64 rows of BX elements,
//    chunk c of row r at place c ^ tr_swizzle(r), and the operand is read
//    with the transposing LDS load (ds_read_b64_tr_b16: in each group of 16
//    lanes, lane i reads 4 elements of row i / 4 and receives column i of
//    the 4 x 16 block).  The swizzle puts the 4 rows x 64 bytes that 32 lanes
//    read on all 64 banks once.
// Measured with the epilogue: 0-6% of the LDS cycles lost to bank conflicts.
// X is loaded two stages ahead into three buffers, Y one ahead into two; the
// 32-row tile (few rows, where the weight stream is all the time there is)
// loads both three stages ahead into four.
// The compiler does not see these loads: the kernel waits for them (vmcnt)
// before each stage's barrier, and for all of them before it goes on to its
// epilogue.
//
// Reduction tails (K or N not a multiple of the stage): chunks past the end
// are not loaded (an offset past the buffer gives zeros), on both operands,
// so what lies there, NaN included, does not enter the sum.  Columns and rows
// past the output's edge may hold anything; they are not stored.
#pragma once

#include "kernels.h"
#include "tiles.h"

namespace moe {
namespace {

enum Mode { kProduct = 0, kInputGrad = 1, kWeightGrad = 2 };

// Place of chunk c in row r of a stage whose reduction runs down the rows:
// c ^ tr_swizzle(r).
__device__ __forceinline__ int tr_swizzle(int r) { return ((r & 3) << 2) ^ (((r >> 3) & 1) << 1); }

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ u32x2 lds_read_tr(const unsigned char* p) {
    return __builtin_bit_cast(
        u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                   (__attribute__((address_space(3))) s16x4*)const_cast<unsigned char*>(p)));
}

// Row tiles of an expert are visited in bands of this many: the tiles that
// run together on one XCD then form a block of the output about as wide as
// high, which share both operands in its L2.
constexpr int kBand = 8;

template <int BX, int BY>
struct TileShape {
    static constexpr int kWavesY = BY >= 64 ? 2 : 1, kWavesX = kWaves / kWavesY;
    static constexpr int kXBufs = BY >= 64 ? 3 : 4, kYBufs = BY >= 64 ? 2 : 4;
    static constexpr int kXStage = BX * 128, kYStage = BY * 128;
    static constexpr int kArena = kXBufs * kXStage + kYBufs * kYStage;
    static_assert(kArena <= 163840, "LDS budget");
    static constexpr int kPerCu = kArena <= 81920 ? 2 : 1;
};

template <int MODE, bool I8, int BX, int BY, bool GATHER, bool NT>
__global__ __launch_bounds__(kThreads, (TileShape<BX, BY>::kPerCu)) void gemm_tile_kernel(GemmArgs g) {
    typedef TileShape<BX, BY> Shape;
    constexpr bool TRX = MODE == kInputGrad;
    constexpr int EB = I8 ? 1 : 2;             // bytes per operand element
    constexpr int SK = 128 / EB;               // reduction per stage
    constexpr int WY = Shape::kWavesY, WX = Shape::kWavesX;
    constexpr int XB = BX / 32 / WX, YB = BY / 32 / WY;  // 32-blocks per wave
    constexpr int XS = Shape::kXStage, YS = Shape::kYStage;
    constexpr int XBUFS = Shape::kXBufs, YBUFS = Shape::kYBufs;
    constexpr int XA = XBUFS - 1, YA = YBUFS - 1;        // stages the loads run ahead
    constexpr int DMA_X = BX / 32, DMA_Y = BY / 32;      // 1 KB loads per wave and stage
    // loads younger than those of the next stage, at a stage's end: each stage
    // loads Y first, then X
    constexpr int YOUNGER = YA == 1 ? DMA_X : (XA - 1) * (DMA_X + DMA_Y);
    static_assert(YA == 1 ? XA >= 1 : XA == YA, "the count above");
    static_assert(!TRX || !I8, "the transposing load is for 16-bit elements");
    typedef typename std::conditional<I8, i32x16, f32x16>::type Acc;

    __shared__ __attribute__((aligned(1024))) unsigned char s_arena[Shape::kArena];
    const uint32_t arena = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(s_arena));

    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int cols = MODE == kProduct ? g.N : g.K;
    const int col_tiles = (cols + BX - 1) / BX;

    // ---- this workgroup's tile: output rows [row0, row0 + rows), columns
    // from c0; reduction [0, red) ----
    int e, nt, row0, rows;
    {
        int32_t* s_off = reinterpret_cast<int32_t*>(s_arena);
        int32_t* s_tstart = s_off + (kMaxE + 1);
        if (!find_tile<BY, BY >= 64 ? 64 : 1, kBand>(g.offsets, g.P, g.E, col_tiles, s_off, s_tstart, e, nt, row0, rows)) return;
        // the same in every lane: kept in scalar registers
        e = __builtin_amdgcn_readfirstlane(e);
        nt = __builtin_amdgcn_readfirstlane(nt);
        row0 = __builtin_amdgcn_readfirstlane(row0);
        rows = __builtin_amdgcn_readfirstlane(rows);
        __syncthreads();  // everyone is done with the schedule before the arena is reused
    }
    const int c0 = nt * BX;
    const int red = MODE == kProduct ? g.K : g.N;
    const int64_t orow0 = row0;
    const int nblk = (rows + 31) >> 5;
    const int nk = (red + SK - 1) / SK;
    // a split reduction: this workgroup's stages [s0, s1); its sums go to ws
    const int s0 = static_cast<int>(static_cast<int64_t>(nk) * blockIdx.y / gridDim.y);
    const int s1 = static_cast<int>(static_cast<int64_t>(nk) * (blockIdx.y + 1) / gridDim.y);
    const bool split = gridDim.y > 1;

    // ---- loads.  Along rows: wave w fills rows [w R, w R + R) of a stage (R =
    // BX / 4), 8 rows a load; lane L of load j writes row w R + 8 j + L / 8,
    // place L % 8.  Down rows: wave w fills rows [16 w, 16 w + 16), each of
    // BX / 8 chunks. ----
    const unsigned char* xbase;   // uniform
    const unsigned char* ybase;
    uint32_t vx[DMA_X], vy[DMA_Y];
    const int64_t K = g.K, N = g.N;
    const unsigned char* wmat = static_cast<const unsigned char*>(g.w) + static_cast<int64_t>(e) * N * K * EB;
    if constexpr (MODE == kProduct) {
        xbase = wmat + static_cast<int64_t>(c0) * K * EB;
        ybase = static_cast<const unsigned char*>(g.a) + (GATHER ? 0 : orow0 * K * EB);
    } else {
        xbase = wmat + static_cast<int64_t>(c0) * 2;
        ybase = static_cast<const unsigned char*>(g.dout) + orow0 * N * 2;
    }
    auto along_row = [&](int j, int per_wave) { return wave * per_wave + j * 8 + (lane >> 3); };
    auto along_chunk = [&](int r) { return (lane & 7) ^ ((r >> 1) & 7); };
    auto down_row = [&](int j, int chunks) { return wave * 16 + j * (64 / chunks) + lane / chunks; };
#pragma unroll
    for (int j = 0; j < DMA_X; ++j) {
        if constexpr (TRX) {
            const int r = down_row(j, BX / 8);
            const int c = (lane % (BX / 8)) ^ tr_swizzle(r);
            vx[j] = static_cast<uint32_t>(r * K * 2 + c * 16);
        } else {
            const int r = along_row(j, BX / 4);
            vx[j] = static_cast<uint32_t>(r * K * EB + along_chunk(r) * 16);
        }
    }
#pragma unroll
    for (int j = 0; j < DMA_Y; ++j) {
        const int r = along_row(j, BY / 4);
        const int c = along_chunk(r);
        const int64_t ld = MODE == kProduct ? K * EB : N * 2;
        if (r >= nblk * 32) {
            vy[j] = kNoRowOffset;
        } else if (GATHER) {
            int64_t s = g.pairs[orow0 + min(r, rows - 1)] / g.k;
            s = s < 0 ? 0 : (s >= g.S ? g.S - 1 : s);
            vy[j] = static_cast<uint32_t>(s * ld + c * 16);
        } else {
            vy[j] = static_cast<uint32_t>(r * ld + c * 16);
        }
    }
    // chunks of the last stage that lie inside the reduction (along rows)
    const int tail = (red - (nk - 1) * SK) / (16 / EB);
    auto x_buf = [&](int i) { return arena + i * XS; };
    auto y_buf = [&](int i) { return arena + XBUFS * XS + i * YS; };
    const __amdgpu_buffer_rsrc_t rsrc_x0 =
        make_rsrc(xbase, static_cast<uint32_t>(TRX ? 0 : min(BX, cols - c0) * K * EB));
    const __amdgpu_buffer_rsrc_t rsrc_y0 = make_rsrc(
        ybase, static_cast<uint32_t>(MODE == kProduct ? (GATHER ? g.S : rows) * K * EB : rows * N * 2));
    auto dma_x = [&](int j, int buf, int kt) {
        const uint32_t at = x_buf(buf) + wave * (XS / 4) + j * 1024;
        if constexpr (TRX) {
            // the buffer starts at the stage's first row and ends with its
            // last row inside the reduction
            const int valid = min(SK, red - kt * SK);
            dma_load16<NT>(at,
                       make_rsrc(xbase + static_cast<int64_t>(kt) * SK * K * 2,
                                 static_cast<uint32_t>((valid * K - c0) * 2)),
                       vx[j], 0);
        } else {
            const bool past = kt == nk - 1 && along_chunk(along_row(j, BX / 4)) >= tail;
            dma_load16<NT>(at, rsrc_x0, past ? kNoRowOffset : vx[j], static_cast<uint32_t>(kt * 128));
        }
    };
    auto dma_y = [&](int j, int buf, int kt) {
        const uint32_t at = y_buf(buf) + wave * (YS / 4) + j * 1024;
        const bool past = kt == nk - 1 && along_chunk(along_row(j, BY / 4)) >= tail;
        dma_load16(at, rsrc_y0, past ? kNoRowOffset : vy[j], static_cast<uint32_t>(kt * 128));
    };

    const int wy = wave / WX, wx = wave % WX;
    const int r32 = lane & 31, half = lane >> 5;
    int valid_blocks = 0;
#pragma unroll
    for (int m = 0; m < YB; ++m) valid_blocks += (wy + WY * m) < nblk;

    Acc acc[YB][XB];
#pragma unroll
    for (int m = 0; m < YB; ++m)
#pragma unroll
        for (int n = 0; n < XB; ++n)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[m][n][i] = 0;

    // the operand of rows [32 b, 32 b + 32) (along) or columns (down), substep ks
    auto read_along = [&](uint32_t buf, int b, int ks) {
        const int r = b * 32 + r32;
        return *reinterpret_cast<const u32x4*>(s_arena + (buf - arena) + r * 128 +
                                               (((ks * 2 + half) ^ ((r >> 1) & 7)) << 4));
    };
    auto read_down = [&](uint32_t buf, int width, int b, int ks) {
        const int i = lane & 15;
        const int r = ks * 16 + half * 8 + (i >> 2);
        const int c = b * 32 + ((lane >> 4) & 1) * 16 + (i & 3) * 4;
        u32x4 v;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int rj = r + 4 * j;
            const u32x2 t = lds_read_tr(s_arena + (buf - arena) + rj * width * 2 +
                                        (((c >> 3) ^ tr_swizzle(rj)) << 4) + (c & 4) * 2);
            v[2 * j] = t[0];
            v[2 * j + 1] = t[1];
        }
        return v;
    };

    // the stages, with NV valid row blocks in this wave
    auto k_loop = [&](auto nv_tag) {
        constexpr int NV = decltype(nv_tag)::value;
        constexpr int NA = NV > 0 ? NV : 1;
        constexpr int MF = NV * XB;  // matrix instructions per substep
        struct Frags {
            u32x4 y[NA];
            u32x4 x[XB];
        };
        constexpr int NP = NV > 0 ? NV + XB : 0;
        auto load_piece = [&](Frags& f, int yb, int xb, int ks, auto qc) {
            constexpr int q = decltype(qc)::value;
            if constexpr (q < NV) {
                f.y[q] = read_along(y_buf(yb), wy + WY * q, ks);
            } else if constexpr (NV > 0) {
                constexpr int n = q - NV;
                if constexpr (TRX)
                    f.x[n] = read_down(x_buf(xb), BX, wx * XB + n, ks);
                else
                    f.x[n] = read_along(x_buf(xb), wx * XB + n, ks);
            }
        };
        auto load_frags = [&](Frags& f, int yb, int xb, int ks) {
            static_for<0, NP>([&](auto qc) { load_piece(f, yb, xb, ks, qc); });
        };
        auto mfma_one = [&](const Frags& f, auto ic) {
            constexpr int i = decltype(ic)::value;
            if constexpr (NV > 0) {
                constexpr int m = i % NV, n = i / NV;
                if constexpr (I8)
                    acc[m][n] = mfma32_i8(f.x[n], f.y[m], acc[m][n]);
                else
                    acc[m][n] = mfma32(as_bf16x8(f.x[n]), as_bf16x8(f.y[m]), acc[m][n]);
            }
        };
        const int last = s1 - 1;
        static_for<0, XA>([&](auto sc) {
            constexpr int st = decltype(sc)::value;
            if constexpr (st < YA) {
#pragma unroll
                for (int j = 0; j < DMA_Y; ++j) dma_y(j, st, min(s0 + st, last));
            }
#pragma unroll
            for (int j = 0; j < DMA_X; ++j) dma_x(j, st, min(s0 + st, last));
        });
        wait_vmcnt<YOUNGER>();
        __syncthreads();
        int ybuf = 0, xbuf = 0;
        Frags f0, f1;
        load_frags(f0, 0, 0, 0);
        for (int kt = s0; kt < s1; ++kt) {
            // past the end: an idle buffer is filled again
            const int ky = min(kt + YA, last);
            const int kx = min(kt + XA, last);
            const int ynext = ybuf == 0 ? YBUFS - 1 : ybuf - 1;  // the buffer freed last
            const int xnext = xbuf == 0 ? XBUFS - 1 : xbuf - 1;
            // The stage's loads are spread over the matrix instructions of its
            // four substeps, the reads of the next substep's operands between
            // them (scheduling fences keep them there).  The barrier sits
            // before the last eighth of the last substep, so the first
            // operands of the next stage are read while those run.
            constexpr int LOADS = DMA_X + DMA_Y;
            auto substep = [&](const Frags& f, auto sc, auto lo_c, auto hi_c, Frags& fn, auto kn_c) {
                constexpr int sub = decltype(sc)::value;
                constexpr int LO = decltype(lo_c)::value, HI = decltype(hi_c)::value;
                constexpr int KN = decltype(kn_c)::value;
                constexpr int NM = HI - LO;
                // this substep's loads: [L0, L1) of the stage's
                constexpr int L0 = sub >= 0 ? (sub * LOADS + 3) / 4 : 0;
                constexpr int L1 = sub >= 0 ? ((sub + 1) * LOADS + 3) / 4 : 0;
                constexpr int NL = L1 - L0;
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
                        constexpr int j = L0 + i / step;
                        if constexpr (j < DMA_Y)
                            dma_y(j, ynext, ky);
                        else
                            dma_x(j - DMA_Y, xnext, kx);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                });
            };
            using C0 = std::integral_constant<int, 0>;
            using CM = std::integral_constant<int, MF>;
            using CH = std::integral_constant<int, MF * 7 / 8>;
            using K0 = std::integral_constant<int, 0>;
            using K1 = std::integral_constant<int, 1>;
            using K2 = std::integral_constant<int, 2>;
            using K3 = std::integral_constant<int, 3>;
            using KNone = std::integral_constant<int, -1>;
            substep(f0, K0{}, C0{}, CM{}, f1, K1{});
            substep(f1, K1{}, C0{}, CM{}, f0, K2{});
            substep(f0, K2{}, C0{}, CM{}, f1, K3{});
            substep(f1, K3{}, C0{}, CH{}, f0, KNone{});
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
    // (a region of its own, so no barrier), so that the stores are 16 bytes a
    // lane over whole rows.  Written straight from the accumulators they
    // would touch 64 lines an instruction. ----
    constexpr int WCOLS = XB * 32;
    constexpr int PITCH = WCOLS * 4 + 16;  // 4-byte elements; 2-byte ones: WCOLS * 2 + 16
    constexpr int REGION = 32 * PITCH;
    static_assert(4 * REGION <= Shape::kArena, "epilogue region");
    unsigned char* region = s_arena + wave * REGION;
    const int wc0 = c0 + wx * WCOLS;
    const bool out_bf16 = g.out_bf16 && !split, accumulate = g.accumulate && !split;
    void* const out =
        split ? static_cast<float*>(g.ws) + static_cast<int64_t>(blockIdx.y) * g.P * cols : static_cast<float*>(g.out);
    // int8: the scales of this lane's rows, all asked for at once
    float a_sc[YB];
    if constexpr (I8) {
        int64_t src[YB];
#pragma unroll
        for (int m = 0; m < YB; ++m) {
            const int64_t q = orow0 + min((wy + WY * m) * 32 + r32, rows - 1);
            src[m] = GATHER ? g.pairs[q] : q;
        }
#pragma unroll
        for (int m = 0; m < YB; ++m) {
            int64_t s = GATHER ? static_cast<int32_t>(src[m]) / g.k : src[m];
            s = s < 0 ? 0 : (s >= g.S ? g.S - 1 : s);
            a_sc[m] = g.a_scale[s];
        }
    }
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
                if (split) {  // raw sums
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const auto x = acc[m][n][4 * i4 + i];
                        v[i] = __builtin_bit_cast(float, x);
                    }
                } else if constexpr (I8) {
                    const int at = min(wc0 + col, cols - 4);
                    const f32x4 ws = *reinterpret_cast<const f32x4*>(g.w_scale + static_cast<int64_t>(e) * N + at);
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[i] = static_cast<float>(acc[m][n][4 * i4 + i]) * (a_sc[m] * ws[i]);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[i] = acc[m][n][4 * i4 + i];
                }
                if (out_bf16) {
                    u32x2 h;
                    h[0] = pack_bf16(v[0], v[1]);
                    h[1] = pack_bf16(v[2], v[3]);
                    *reinterpret_cast<u32x2*>(region + r32 * (WCOLS * 2 + 16) + col * 2) = h;
                } else {
                    *reinterpret_cast<f32x4*>(region + r32 * PITCH + col * 4) = v;
                }
            }
        wave_lds_fence();
        const int64_t base = (orow0 + blk * 32) * cols + wc0;
        const int left = rows - blk * 32;  // rows of this block inside the tile
        if (out_bf16) {
            constexpr int LPR = WCOLS / 8;  // lanes per row
#pragma unroll
            for (int it = 0; it < 32 * LPR / 64; ++it) {
                const int r = it * (64 / LPR) + lane / LPR, c = lane % LPR * 8;
                const u32x4 v = ld16(region + r * (WCOLS * 2 + 16) + c * 2);
                if (r < left && wc0 + c < cols)
                    *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(out) + base + static_cast<int64_t>(r) * cols + c) = v;
            }
        } else {
            constexpr int LPR = WCOLS / 4;
#pragma unroll
            for (int it = 0; it < 32 * LPR / 64; ++it) {
                const int r = it * (64 / LPR) + lane / LPR, c = lane % LPR * 4;
                f32x4 v = *reinterpret_cast<const f32x4*>(region + r * PITCH + c * 4);
                if (r < left && wc0 + c < cols) {
                    f32x4* o = reinterpret_cast<f32x4*>(static_cast<float*>(out) + base + static_cast<int64_t>(r) * cols + c);
                    if (accumulate) v += *o;
                    *o = v;
                }
            }
        }
        wave_lds_fence();
    }
}

}  // namespace
}  // namespace moe
