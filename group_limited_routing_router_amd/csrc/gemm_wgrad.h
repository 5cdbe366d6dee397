// gemm_wgrad.h -- the weight gradient of the grouped products:
//   dw[e,n,k] = sum over e's positions q of dout[q,n] a[row(q),k].
//
// The sum is short (an expert's rows: a few stages) and the output long (E N K
// values), so what a tile costs around its sum counts: with a workgroup for
// each tile, 8192 tokens over 256 experts of 2560 x 5120 spent more time on
// first loads and on writing out than on the sums (3.7 ms; 1.3 ms of it with
// no rows at all).  So a workgroup stays for many tiles and the loads of the
// next tiles go on while one is written out.
//
// A stage is 32 positions: X = 32 rows of BX columns of a, Y = 32 rows of BY
// columns of dout, both straight from HBM into LDS and read with the
// transposing LDS load (see gemm_tile.h for its layout).  Five stage buffers
// (four where rows are gathered); the loads run four (three) stages ahead,
// over the ends of tiles.  Positions past
// the expert's last row are not loaded (zeros in LDS), so nothing that lies
// there enters the sum.
//
// The results go through LDS, in the part of the stage buffer just consumed
// that this wave itself fills next, so no other wave is concerned; they are
// stored 16 bytes a lane.  Memory operations complete in order, so a wait for
// the loads of the next stages also waits for older stores; the first waits
// after a tile therefore allow for its stores (exactly as many as the store
// instructions, which are issued for every lane; lanes outside the output
// get an offset past its end, which drops them).
#pragma once

#include "gemm_tile.h"

namespace moe {
namespace {

constexpr int kNumCu = 256;

// A tile of the weight gradient: expert, first output column and row, and the
// expert's positions [first, first + red).
struct WgradTile {
    int e, c0, n0, red, nk;
    int64_t first;
};

template <int BX, int BY, bool GATHER>
struct WgradShape {
    static constexpr int kRows = 32;  // positions per stage
    static constexpr int kBufs = GATHER ? 4 : 5;
    static constexpr int kXStage = kRows * BX * 2, kYStage = kRows * BY * 2;
    static constexpr int kStage = kXStage + kYStage;
    static constexpr int kSlots = 8;  // stages of row indexes in LDS, 256 bytes a wave and stage
    static constexpr int kArena = kBufs * kStage + (GATHER ? kSlots * 256 * kWaves : 0);
    static_assert(kArena <= 163840, "LDS budget");
    static constexpr int kPerCu = kArena <= 81920 ? 2 : 1;
};

template <int BX, int BY, bool GATHER, bool BF16, bool ACC>
__global__ __launch_bounds__(kThreads, (WgradShape<BX, BY, GATHER>::kPerCu)) void gemm_wgrad_kernel(GemmArgs g) {
    typedef WgradShape<BX, BY, GATHER> Shape;
    constexpr int SR = Shape::kRows, NBUF = Shape::kBufs;
    constexpr int XB = BX / 64, YB = BY / 64;              // 32-blocks per wave
    constexpr int XS = Shape::kXStage, YS = Shape::kYStage, STAGE = Shape::kStage;
    constexpr int DMA_X = XS / 4096, DMA_Y = YS / 4096;    // 1 KB loads per wave and stage
    constexpr int DMA = DMA_X + DMA_Y + (GATHER ? 1 : 0);  // per wave and stage
    constexpr int AHEAD = NBUF - 1;

    __shared__ __attribute__((aligned(1024))) unsigned char s_arena[Shape::kArena];
    const uint32_t arena = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(s_arena));
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int N = g.N, K = g.K;

    // ---- this workgroup's tiles.  The list goes expert by expert (an
    // expert's tiles in bands of kBand rows); each XCD takes a contiguous run
    // of it, so the tiles that run together on one XCD share an expert's
    // operands in its L2, and the XCD's workgroups take the run's tiles in
    // turn.  The runs are of equal cost, not of equal length: a tile costs its
    // stages and, for what lies around them, kTileCost more (routing with
    // busy and idle experts: 24 experts, 776 x 1000, 4503 rows: 50 us with
    // runs of equal length). ----
    const int col_tiles = (K + BX - 1) / BX, row_tiles = (N + BY - 1) / BY;
    const int per_expert = col_tiles * row_tiles;
    const int xcd = blockIdx.x % kNumXcd, slots = gridDim.x / kNumXcd;
    const bool interleave = g.E % kNumXcd == 0;
    auto expert_at = [&](int pos) {
        return interleave ? (pos % kNumXcd) * (g.E / kNumXcd) + pos / kNumXcd : pos;
    };
    typedef const __attribute__((address_space(4))) int32_t* ConstInts;
    auto expert_span = [&](int e, int64_t& b, int64_t& m) {
        b = 0;
        m = g.P;
        if (g.offsets) {
            b = g.offsets[e];
            m = g.offsets[e + 1];
            b = b < 0 ? 0 : (b > g.P ? g.P : b);
            m = m < 0 ? 0 : (m > g.P ? g.P : m);
        }
        m = m > b ? m - b : 0;
    };
    int l0, run_end;
    const int total = per_expert * g.E;
    if (total <= static_cast<int>(gridDim.x)) {  // one tile a workgroup
        const int per = total / kNumXcd, rem = total % kNumXcd;
        const int begin = xcd * per + min(xcd, rem);
        l0 = begin + blockIdx.x / kNumXcd;
        run_end = begin + per + (xcd < rem ? 1 : 0);
    } else {
        int64_t* s_sum = reinterpret_cast<int64_t*>(s_arena);            // [kWaves]
        int* s_bound = reinterpret_cast<int*>(s_arena + kWaves * 8);     // [kNumXcd + 1]
        constexpr int kTileCost = BF16 ? 8 : 16;
        int64_t cost = 0;
        if (tid < g.E) {
            int64_t b, n;
            expert_span(expert_at(tid), b, n);
            cost = (n + SR - 1) / SR + kTileCost;
        }
        int64_t incl = cost;
#pragma unroll
        for (int d = 1; d < kWave; d <<= 1) {
            const int64_t v = __shfl_up(incl, d, kWave);
            if (lane >= d) incl += v;
        }
        if (lane == kWave - 1) s_sum[wave] = incl;
        __syncthreads();
        int64_t all = 0;
        for (int w = 0; w < kWaves; ++w) {
            if (w < wave) incl += s_sum[w];
            all += s_sum[w];
        }
        // costs of one tile row of experts; a boundary between runs falls at
        // the first tile that begins at or after its share of the whole
        all *= per_expert;
        const int64_t end = incl * per_expert, begin = end - cost * per_expert;
        for (int x = 0; x <= kNumXcd; ++x) {
            const int64_t at = all * x / kNumXcd;
            if (tid < g.E && at >= begin && at < end)
                s_bound[x] = tid * per_expert + static_cast<int>((at - begin + cost - 1) / cost);
        }
        if (tid == 0) s_bound[kNumXcd] = per_expert * g.E;
        __syncthreads();
        l0 = __builtin_amdgcn_readfirstlane(s_bound[xcd]) + blockIdx.x / kNumXcd;
        run_end = __builtin_amdgcn_readfirstlane(s_bound[xcd + 1]);
        __syncthreads();  // before the loads reuse this part of LDS
    }
    auto tile_at = [&](int l) {
        WgradTile t;
        const int pos = l / per_expert, in = l - pos * per_expert;
        t.e = expert_at(pos);
        const int band = in / (kBand * col_tiles), ib = in - band * kBand * col_tiles;
        const int high = min(kBand, row_tiles - band * kBand);
        const int ct = ib / high;
        t.c0 = ct * BX;
        t.n0 = (band * kBand + ib - ct * high) * BY;
        int64_t b = 0, m = g.P;
        if (g.offsets) {
            const ConstInts off = (ConstInts)g.offsets;
            b = off[t.e];
            m = off[t.e + 1];
            b = b < 0 ? 0 : (b > g.P ? g.P : b);
            m = m < 0 ? 0 : (m > g.P ? g.P : m);
        }
        t.first = b;
        t.red = static_cast<int>(m > b ? m - b : 0);
        t.nk = (t.red + SR - 1) / SR;
        return t;
    };
    if (l0 >= run_end) return;

    // ---- loads: wave w fills rows [8 w, 8 w + 8) of a stage ----
    auto down_row = [&](int j, int chunks) { return wave * 8 + j * (64 / chunks) + lane / chunks; };
    uint32_t vx[DMA_X], vy[DMA_Y];
#pragma unroll
    for (int j = 0; j < DMA_X; ++j) {
        const int r = down_row(j, BX / 8);
        const int c = (lane % (BX / 8)) ^ tr_swizzle(r);
        vx[j] = GATHER ? static_cast<uint32_t>(c * 16) : static_cast<uint32_t>(r * K * 2 + c * 16);
    }
#pragma unroll
    for (int j = 0; j < DMA_Y; ++j) {
        const int r = down_row(j, BY / 8);
        vy[j] = static_cast<uint32_t>(r * N * 2 + ((lane % (BY / 8)) ^ tr_swizzle(r)) * 16);
    }
    // A place in this workgroup's stages: tile (list index l), its stage k.
    // Past the last stage it stays there (an idle buffer is filled again).
    struct Cursor {
        WgradTile t;
        int l, k;
    };
    auto next_filled = [&](Cursor& c) {  // from list index c.l on, the first tile with rows
        while (c.t.nk == 0) {
            if (c.l + slots >= run_end) return false;
            c.l += slots;
            c.t = tile_at(c.l);
        }
        return true;
    };
    auto advance = [&](Cursor& c) {
        if (c.k + 1 < c.t.nk) {
            ++c.k;
            return;
        }
        Cursor n = c;
        if (n.l + slots < run_end) {
            n.l += slots;
            n.t = tile_at(n.l);
            n.k = 0;
            if (next_filled(n)) c = n;
        }
    };
    Cursor ld{tile_at(l0), l0, 0};  // the stage loaded next
    const bool any = next_filled(ld);
    // GATHER: the row indexes of a stage come into LDS AHEAD stages before
    // the stage's own loads, each wave its own copy (pairs of the 32
    // positions; the upper lanes fetch the 32 after them, unused).  Every
    // stage issues one such load, so the counts of the waits are fixed.
    Cursor ix = ld;
    int ix_slot = 0, ld_slot = 0;
    const uint32_t index_at = arena + NBUF * STAGE + wave * (Shape::kSlots * 256);
    auto dma_index = [&]() {
        if constexpr (GATHER) {
            const int64_t at = ix.t.first + ix.k * SR;
            const int64_t left = g.P - at < 64 ? g.P - at : 64;
            asm volatile(
                "s_mov_b32 m0, %0\n\t"
                "s_nop 0\n\t"
                "buffer_load_dword %1, %2, 0 offen lds"
                :
                : "s"(__builtin_amdgcn_readfirstlane(index_at + ix_slot * 256)),
                  "v"(static_cast<uint32_t>(lane * 4)), "s"(make_rsrc(g.pairs + at, static_cast<uint32_t>(left * 4)))
                : "memory", "m0");
            ix_slot = (ix_slot + 1) % Shape::kSlots;
            advance(ix);
        }
    };
    // the byte offset of the row this lane fetches a part of in load j; a
    // position past the expert's last gets an offset past the buffer
    uint32_t src[GATHER ? DMA_X : 1];
    auto read_index = [&]() {
        if constexpr (GATHER) {
            const int32_t* idx = reinterpret_cast<const int32_t*>(s_arena + (index_at - arena) + ld_slot * 256);
            const int valid = min(SR, ld.t.red - ld.k * SR);
#pragma unroll
            for (int j = 0; j < DMA_X; ++j) {
                const int r = down_row(j, BX / 8);
                const int p = max(idx[r], 0);
                // p / k, exact for 0 <= p < 2^31
                uint32_t q = g.k_shift < 0 ? p : __umulhi(static_cast<uint32_t>(p), g.k_magic) >> g.k_shift;
                q = min(q, static_cast<uint32_t>(g.S - 1));
                src[j] = r < valid ? q * static_cast<uint32_t>(K * 2) : kNoRowOffset;
            }
        }
    };
    auto ld_next = [&]() {
        ld_slot = (ld_slot + 1) % Shape::kSlots;
        advance(ld);
    };
    auto dma_x = [&](int j, uint32_t buf) {
        const uint32_t at = buf + wave * (XS / 4) + j * 1024;
        const unsigned char* a = static_cast<const unsigned char*>(g.a) + static_cast<int64_t>(ld.t.c0) * 2;
        const int valid = min(SR, ld.t.red - ld.k * SR);
        if constexpr (GATHER) {
            dma_load16(at, make_rsrc(a, static_cast<uint32_t>((g.S * K - ld.t.c0) * 2)), src[j] + vx[j], 0);
        } else {
            dma_load16(at, make_rsrc(a + (ld.t.first + ld.k * SR) * K * 2,
                                     static_cast<uint32_t>((valid * K - ld.t.c0) * 2)),
                       vx[j], 0);
        }
    };
    auto dma_y = [&](int j, uint32_t buf) {
        const int valid = min(SR, ld.t.red - ld.k * SR);
        dma_load16(buf + XS + wave * (YS / 4) + j * 1024,
                   make_rsrc(static_cast<const unsigned char*>(g.dout) +
                                 ((ld.t.first + ld.k * SR) * N + ld.t.n0) * 2,
                             static_cast<uint32_t>((valid * N - ld.t.n0) * 2)),
                   vy[j], 0);
    };

    const int wy = wave >> 1, wx = wave & 1;
    const int r32 = lane & 31, half = lane >> 5;
    // Operand reads.  X's columns reach the matrix instruction in the order
    // that leaves each lane 8 consecutive ones (bits 2 and 3 of the place in
    // the block swapped).
    auto read_down = [&](uint32_t buf, int width, int b, int ks, bool x) {
        const int i = lane & 15;
        const int r = ks * 16 + half * 8 + (i >> 2);
        const int cg = x ? ((i & 1) << 1) | ((i >> 1) & 1) : i & 3;
        const int c = b * 32 + ((lane >> 4) & 1) * 16 + cg * 4;
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
    struct Frags {
        u32x4 y[YB], x[XB];
    };
    constexpr int NP = YB + XB, MF = YB * XB;
    auto load_piece = [&](Frags& f, uint32_t buf, int ks, auto qc) {
        constexpr int q = decltype(qc)::value;
        if constexpr (q < YB)
            f.y[q] = read_down(buf + XS, BY, wy * YB + q, ks, false);
        else
            f.x[q - YB] = read_down(buf, BX, wx * XB + q - YB, ks, true);
    };
    f32x16 acc[YB][XB];
    auto clear = [&]() {
#pragma unroll
        for (int m = 0; m < YB; ++m)
#pragma unroll
            for (int n = 0; n < XB; ++n)
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[m][n][i] = 0.0f;
    };
    auto mfma_one = [&](const Frags& f, auto ic) {
        constexpr int i = decltype(ic)::value;
        constexpr int m = i % YB, n = i / YB;
        acc[m][n] = mfma32(as_bf16x8(f.x[n]), as_bf16x8(f.y[m]), acc[m][n]);
    };

    Frags f0, f1;
    int cur = 0;  // ring place of the stage to compute next
    auto place = [&](int i) { return arena + i * STAGE; };
    if (any) {
        if constexpr (GATHER) {
            for (int s = 0; s < AHEAD; ++s) dma_index();
            wait_vmcnt<0>();
        }
#pragma unroll
        for (int s = 0; s < AHEAD; ++s) {
            read_index();
            dma_index();
#pragma unroll
            for (int j = 0; j < DMA_Y; ++j) dma_y(j, place(s));
#pragma unroll
            for (int j = 0; j < DMA_X; ++j) dma_x(j, place(s));
            ld_next();
        }
        wait_vmcnt<(AHEAD - 1) * DMA>();
        __syncthreads();
        static_for<0, NP>([&](auto qc) { load_piece(f0, place(0), 0, qc); });
    }

    // stores of one tile, per wave
    constexpr int OB = BF16 ? 2 : 4;
    constexpr int STORES = ACC ? 0 : BX / 2 * (BY / 2) * OB / 1024;
    constexpr int RELAXED = (AHEAD - 1) * DMA + STORES < 63 ? (AHEAD - 1) * DMA + STORES : 63;
    int since = AHEAD;  // stages since the last stores

    for (int l = l0; l < run_end; l += slots) {
        const WgradTile t = tile_at(l);
        clear();
        for (int kt = 0; kt < t.nk; ++kt) {
            const uint32_t buf = place(cur);
            const uint32_t into = place(cur == 0 ? NBUF - 1 : cur - 1);
            read_index();
            dma_index();
            // two substeps; the stage's loads and the next operands' reads
            // spread over their matrix instructions
            auto substep = [&](const Frags& f, auto lo_c, auto hi_c, auto first_load, auto num_loads, auto reads) {
                constexpr int LO = decltype(lo_c)::value, HI = decltype(hi_c)::value;
                constexpr int L0 = decltype(first_load)::value, NL = decltype(num_loads)::value;
                constexpr int NPC = decltype(reads)::value ? NP : 0;
                constexpr int NM = HI - LO;
                static_for<0, NM>([&](auto ic) {
                    constexpr int i = decltype(ic)::value;
                    static_for<0, NPC>([&](auto qc) {
                        constexpr int q = decltype(qc)::value;
                        if constexpr (q * NM / NP == i) load_piece(f1, buf, 1, qc);
                    });
                    mfma_one(f, std::integral_constant<int, LO + i>{});
                    static_for<0, NL>([&](auto jc) {
                        constexpr int j = decltype(jc)::value;
                        if constexpr ((j + 1) * NM / NL - 1 == i || (NM < NL && j * NM / NL == i)) {
                            if constexpr (L0 + j < DMA_Y)
                                dma_y(L0 + j, into);
                            else
                                dma_x(L0 + j - DMA_Y, into);
                        }
                    });
                    __builtin_amdgcn_sched_barrier(0);
                });
            };
            static_assert(MF * 3 / 4 >= DMA_X && MF >= DMA_Y, "loads spread over the matrix instructions");
            using C0 = std::integral_constant<int, 0>;
            using CM = std::integral_constant<int, MF>;
            using CH = std::integral_constant<int, MF * 3 / 4>;
            using LY = std::integral_constant<int, DMA_Y>;
            using LX = std::integral_constant<int, DMA_X>;
            substep(f0, C0{}, CM{}, C0{}, LY{}, std::true_type{});
            substep(f1, C0{}, CH{}, LY{}, LX{}, std::false_type{});
            ld_next();
            if (since < AHEAD - 1)
                wait_vmcnt<RELAXED>();
            else
                wait_vmcnt<(AHEAD - 1) * DMA>();
            ++since;
            __syncthreads();
            cur = cur == NBUF - 1 ? 0 : cur + 1;
            static_for<0, NP>([&](auto qc) { load_piece(f0, place(cur), 0, qc); });
            __builtin_amdgcn_sched_barrier(0);
            substep(f1, CH{}, CM{}, C0{}, C0{}, std::false_type{});
        }
        if (ACC && t.nk == 0) continue;

        // ---- write the tile: 32 rows x PITCH bytes at a time through this
        // wave's part of the idle buffer, X's and Y's in turn ----
        const uint32_t idle = place(cur == 0 ? NBUF - 1 : cur - 1);
        constexpr int PITCH = (BX < BY ? BX : BY) / 2;
        constexpr int PASS_COLS = PITCH / OB;
        constexpr int CPR = PITCH / 16;        // chunks per row
        constexpr int PASSES = XB * 32 / PASS_COLS;
        const int rows = min(BY, N - t.n0), cols = K - t.c0;
        const int64_t at0 = ((static_cast<int64_t>(t.e) * N + t.n0) * K + t.c0) * OB;
        const __amdgpu_buffer_rsrc_t rsrc =
            make_rsrc(static_cast<unsigned char*>(g.out) + at0,
                      static_cast<uint32_t>(((rows - 1) * static_cast<int64_t>(K) + min(BX, cols)) * OB));
        // chunk c of row r sits at place c ^ (bits of r), so that 16 lanes
        // (16 rows of one chunk) lie on all banks
        auto chunk_at = [&](int r, int c) {
            return r * PITCH + ((c ^ (CPR == 8 ? (r >> 1) & 7 : (r >> 2) & 3)) << 4);
        };
        static_for<0, YB>([&](auto mc) {
            constexpr int m = decltype(mc)::value;
            static_for<0, PASSES>([&](auto pc) {
                constexpr int p = decltype(pc)::value;
                unsigned char* region = s_arena + (idle - arena) +
                                        ((m * PASSES + p) & 1 ? XS + wave * (YS / 4) : wave * (XS / 4));
                static_for<0, PASS_COLS / 16>([&](auto cc) {
                    // 16 columns: this lane's 8 (chunks of 16 bytes: one of
                    // bf16, two of fp32)
                    constexpr int c16 = decltype(cc)::value;
                    constexpr int col = p * PASS_COLS + c16 * 16;
                    constexpr int n = col / 32, i0 = (col % 32) / 2;
                    const f32x16 v = acc[m][n];
                    if constexpr (BF16) {
                        u32x4 h;
#pragma unroll
                        for (int i = 0; i < 4; ++i) h[i] = pack_bf16(v[i0 + 2 * i], v[i0 + 2 * i + 1]);
                        *reinterpret_cast<u32x4*>(region + chunk_at(r32, c16 * 2 + half)) = h;
                    } else {
#pragma unroll
                        for (int d = 0; d < 2; ++d) {
                            f32x4 h;
#pragma unroll
                            for (int i = 0; i < 4; ++i) h[i] = v[i0 + 4 * d + i];
                            *reinterpret_cast<f32x4*>(region + chunk_at(r32, c16 * 4 + half * 2 + d)) = h;
                        }
                    }
                });
                wave_lds_fence();
#pragma unroll
                for (int it = 0; it < 32 * CPR / 64; ++it) {
                    const int r = it * (64 / CPR) + lane / CPR, c = lane % CPR;
                    u32x4 v = ld16(region + chunk_at(r, c));
                    const int orow = (wy * YB + m) * 32 + r;
                    const int ocol = wx * XB * 32 + p * PASS_COLS + c * (16 / OB);
                    const bool in = orow < rows && ocol < cols;
                    const uint32_t off = static_cast<uint32_t>((orow * static_cast<int64_t>(K) + ocol) * OB);
                    if constexpr (ACC) {
                        if (in) {
                            f32x4* o = reinterpret_cast<f32x4*>(static_cast<unsigned char*>(g.out) + at0 + off);
                            *o = *o + __builtin_bit_cast(f32x4, v);
                        }
                    } else {
                        __builtin_amdgcn_raw_buffer_store_b128(v, rsrc, in ? off : kNoRowOffset, 0, 0);
                    }
                }
                wave_lds_fence();
            });
        });
        since = 0;
    }
    wait_vmcnt<0>();
}

}  // namespace
}  // namespace moe
