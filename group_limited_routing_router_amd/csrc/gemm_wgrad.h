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
//
// 8192 tokens, 256 experts of 2560 x 5120, bf16: 2.65 ms, 9.0 GB moved (6.7 of
// them the output), the matrix units busy 31% of it, a fifth of the LDS cycles
// lost to bank conflicts.  With accumulate a tile's values are read one load
// at a time, each waited for: 128 tokens, 2.4 ms written and 9.9 ms added to.
#pragma once

#include "gemm_tile.h"

namespace moe {
namespace {

constexpr int kNumCu = 256;

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
    // With splits > 1 the positions of an expert come in that many parts, each
    // a list entry of its own whose output is the part's own array (part s of
    // expert e: array s * E + e of out).
    const int parts = g.E * g.splits;
    const bool interleave = parts % kNumXcd == 0;
    auto expert_at = [&](int pos) {
        return interleave ? (pos % kNumXcd) * (parts / kNumXcd) + pos / kNumXcd : pos;
    };
    auto part_of = [&](int e, int64_t& b, int64_t& n) {  // positions of part e / E, from the expert's
        if (g.splits > 1) {
            const int64_t each = (n + g.splits * SR - 1) / (g.splits * SR) * SR, skip = each * (e / g.E);
            b += skip < n ? skip : n;
            n = skip < n ? (n - skip < each ? n - skip : each) : 0;
        }
    };
    typedef const __attribute__((address_space(4))) int32_t* ConstInts;
    auto expert_span = [&](int e, int64_t& b, int64_t& m) {
        b = 0;
        m = g.P;
        if (g.offsets) {
            b = g.offsets[e % g.E];
            m = g.offsets[e % g.E + 1];
            b = b < 0 ? 0 : (b > g.P ? g.P : b);
            m = m < 0 ? 0 : (m > g.P ? g.P : m);
        }
        m = m > b ? m - b : 0;
        part_of(e, b, m);
    };
    int l0, run_end;
    const int total = per_expert * parts;
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
        if (tid < parts) {
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
            if (tid < parts && at >= begin && at < end)
                s_bound[x] = tid * per_expert + static_cast<int>((at - begin + cost - 1) / cost);
        }
        if (tid == 0) s_bound[kNumXcd] = total;
        __syncthreads();
        l0 = __builtin_amdgcn_readfirstlane(s_bound[xcd]) + blockIdx.x / kNumXcd;
        run_end = __builtin_amdgcn_readfirstlane(s_bound[xcd + 1]);
        __syncthreads();  // before the loads reuse this part of LDS
    }
    // A place in this workgroup's stages: tile `l` of the list (tile `in` of
    // the expert at position pos), its stage k.  Steps go from the tile before,
    // without divisions, and read the offsets only where the expert changes.
    struct Cursor {
        int l, pos, in, k;
        int e, red, nk;  // expert, its positions [first, first + red), stages
        int64_t first;
        int c0, n0;      // first output column and row
    };
    auto enter_expert = [&](Cursor& c) {
        c.e = expert_at(c.pos);
        int64_t b = 0, m = g.P;
        if (g.offsets) {
            const ConstInts off = (ConstInts)g.offsets;
            const int e = g.splits > 1 ? c.e % g.E : c.e;
            b = off[e];
            m = off[e + 1];
            b = b < 0 ? 0 : (b > g.P ? g.P : b);
            m = m < 0 ? 0 : (m > g.P ? g.P : m);
        }
        m = m > b ? m - b : 0;
        part_of(c.e, b, m);
        // the same in every lane (P < 2^31): kept in scalar registers
        c.first = __builtin_amdgcn_readfirstlane(static_cast<int>(b));
        c.red = __builtin_amdgcn_readfirstlane(static_cast<int>(m));
        c.nk = row_tiles_of(c.red, SR);
    };
    auto enter_tile = [&](Cursor& c) {
        const int band_tiles = kBand * col_tiles;
        const int band = row_tiles > kBand ? c.in / band_tiles : 0;
        const int ib = c.in - band * band_tiles;
        const int high = min(kBand, row_tiles - band * kBand);
        const int ct = high == kBand ? ib / kBand : ib / high;
        c.c0 = ct * BX;
        c.n0 = (band * kBand + ib - ct * high) * BY;
        c.k = 0;
    };
    auto step = [&](Cursor& c) {  // to the next tile, which has to be in the run
        c.l += slots;
        c.in += slots;
        if (c.in >= per_expert) {
            do {
                c.in -= per_expert;
                ++c.pos;
            } while (c.in >= per_expert);
            enter_expert(c);
        }
        enter_tile(c);
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
    auto next_filled = [&](Cursor& c) {  // from tile c on, the first with rows
        while (c.nk == 0) {
            if (c.l + slots >= run_end) return false;
            step(c);
        }
        return true;
    };
    // past the last stage a cursor stays there (an idle buffer is filled again)
    auto advance = [&](Cursor& c) {
        if (c.k + 1 < c.nk) {
            ++c.k;
            return;
        }
        Cursor n = c;
        if (n.l + slots < run_end) {
            step(n);
            if (next_filled(n)) c = n;
        }
    };
    Cursor now;  // the tile computed
    now.l = l0;
    now.pos = l0 / per_expert;
    now.in = l0 - now.pos * per_expert;
    enter_expert(now);
    enter_tile(now);
    Cursor ld = now;  // the stage loaded next
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
            const int64_t at = ix.first + ix.k * SR;
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
            const int valid = min(SR, ld.red - ld.k * SR);
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
        const unsigned char* a = static_cast<const unsigned char*>(g.a) + static_cast<int64_t>(ld.c0) * 2;
        const int valid = min(SR, ld.red - ld.k * SR);
        if constexpr (GATHER) {
            dma_load16(at, make_rsrc(a, static_cast<uint32_t>((g.S * K - ld.c0) * 2)), src[j] + vx[j], 0);
        } else {
            dma_load16(at, make_rsrc(a + (ld.first + ld.k * SR) * K * 2,
                                     static_cast<uint32_t>((valid * K - ld.c0) * 2)),
                       vx[j], 0);
        }
    };
    auto dma_y = [&](int j, uint32_t buf) {
        const int valid = min(SR, ld.red - ld.k * SR);
        dma_load16(buf + XS + wave * (YS / 4) + j * 1024,
                   make_rsrc(static_cast<const unsigned char*>(g.dout) +
                                 ((ld.first + ld.k * SR) * N + ld.n0) * 2,
                             static_cast<uint32_t>((valid * N - ld.n0) * 2)),
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
    // onto_zero: a tile's first products
    auto mfma_one = [&](const Frags& f, auto ic, auto onto_zero) {
        constexpr int i = decltype(ic)::value;
        constexpr int m = i % YB, n = i / YB;
        if constexpr (decltype(onto_zero)::value) {
            const f32x16 zero = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            acc[m][n] = mfma32(as_bf16x8(f.x[n]), as_bf16x8(f.y[m]), zero);
        } else {
            acc[m][n] = mfma32(as_bf16x8(f.x[n]), as_bf16x8(f.y[m]), acc[m][n]);
        }
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

    while (true) {
        const Cursor t = now;
        auto stage = [&](auto first_c) {
            constexpr bool FIRST = decltype(first_c)::value;
            const uint32_t buf = place(cur);
            const uint32_t into = place(cur == 0 ? NBUF - 1 : cur - 1);
            read_index();
            dma_index();
            // two substeps; the stage's loads and the next operands' reads
            // spread over their matrix instructions
            auto substep = [&](const Frags& f, auto lo_c, auto hi_c, auto first_load, auto num_loads, auto reads,
                               auto onto_zero) {
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
                    mfma_one(f, std::integral_constant<int, LO + i>{}, onto_zero);
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
            substep(f0, C0{}, CM{}, C0{}, LY{}, std::true_type{}, std::integral_constant<bool, FIRST>{});
            substep(f1, C0{}, CH{}, LY{}, LX{}, std::false_type{}, std::false_type{});
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
            substep(f1, CH{}, CM{}, C0{}, C0{}, std::false_type{}, std::false_type{});
        };
        if (t.nk > 0) {
            stage(std::true_type{});
            for (int kt = 1; kt < t.nk; ++kt) stage(std::false_type{});
        } else {
            clear();
        }

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
        constexpr int UNITS = YB * PASSES, PER_UNIT = 32 * CPR / 64;
        auto region = [&](int u) {
            return s_arena + (idle - arena) + (u & 1 ? XS + wave * (YS / 4) : wave * (XS / 4));
        };
        auto put = [&](auto uc) {
            constexpr int u = decltype(uc)::value, m = u / PASSES, p = u % PASSES;
            static_for<0, PASS_COLS / 16>([&](auto cc) {
                // 16 columns: this lane's 8 (chunks of 16 bytes: one of bf16,
                // two of fp32)
                constexpr int c16 = decltype(cc)::value;
                constexpr int col = p * PASS_COLS + c16 * 16;
                constexpr int n = col / 32, i0 = (col % 32) / 2;
                const f32x16 v = acc[m][n];
                if constexpr (BF16) {
                    u32x4 h;
#pragma unroll
                    for (int i = 0; i < 4; ++i) h[i] = pack_bf16(v[i0 + 2 * i], v[i0 + 2 * i + 1]);
                    *reinterpret_cast<u32x4*>(region(u) + chunk_at(r32, c16 * 2 + half)) = h;
                } else {
#pragma unroll
                    for (int d = 0; d < 2; ++d) {
                        f32x4 h;
#pragma unroll
                        for (int i = 0; i < 4; ++i) h[i] = v[i0 + 4 * d + i];
                        *reinterpret_cast<f32x4*>(region(u) + chunk_at(r32, c16 * 4 + half * 2 + d)) = h;
                    }
                }
            });
        };
        u32x4 v[2][PER_UNIT];
        auto fetch = [&](auto uc) {
            constexpr int u = decltype(uc)::value;
#pragma unroll
            for (int it = 0; it < PER_UNIT; ++it)
                v[u & 1][it] = ld16(region(u) + chunk_at(it * (64 / CPR) + lane / CPR, lane % CPR));
        };
        const int64_t row_bytes = static_cast<int64_t>(K) * OB;
        auto send = [&](auto uc) {
            constexpr int u = decltype(uc)::value, m = u / PASSES, p = u % PASSES;
            const int ocol = wx * XB * 32 + p * PASS_COLS + lane % CPR * (16 / OB);
#pragma unroll
            for (int it = 0; it < PER_UNIT; ++it) {
                const int orow = (wy * YB + m) * 32 + it * (64 / CPR) + lane / CPR;
                const bool in = orow < rows && ocol < cols;
                const uint32_t off = static_cast<uint32_t>(orow * row_bytes + ocol * OB);
                if constexpr (ACC) {
                    if (in && t.nk > 0) {
                        f32x4* o = reinterpret_cast<f32x4*>(static_cast<unsigned char*>(g.out) + at0 + off);
                        *o = *o + __builtin_bit_cast(f32x4, v[u & 1][it]);
                    }
                } else {
                    __builtin_amdgcn_raw_buffer_store_b128(v[u & 1][it], rsrc, in ? off : kNoRowOffset, 0, 0);
                }
            }
        };
        // unit u + 1 goes into LDS while unit u comes back
        put(std::integral_constant<int, 0>{});
        static_for<0, UNITS>([&](auto uc) {
            constexpr int u = decltype(uc)::value;
            wave_lds_fence();
            if constexpr (u + 1 < UNITS) put(std::integral_constant<int, u + 1>{});
            fetch(uc);
            wave_lds_fence();
            if constexpr (u > 0) send(std::integral_constant<int, u - 1>{});
        });
        send(std::integral_constant<int, UNITS - 1>{});
        since = 0;
        if (now.l + slots >= run_end) break;
        step(now);
    }
    wait_vmcnt<0>();
}

}  // namespace
}  // namespace moe
