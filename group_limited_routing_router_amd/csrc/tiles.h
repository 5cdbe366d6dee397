// tiles.h -- device-side helpers of the grouped GEMMs: the tile schedule over
// the experts' rows, buffer resources, loads from HBM straight into LDS.
#pragma once

#include <type_traits>

#include "common.h"
#include "schedule.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kMaxE = 256;

// Raw buffer resource over [base, base + bytes): 32-bit offsets from one
// scalar base; loads past `bytes` return zero.  Third dword: gfx9 default.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* base, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), static_cast<short>(0),
                                             static_cast<int>(bytes), 0x00020000);
}

// Compile-time loop: f(std::integral_constant<int, I>) for I in [B, E).
template <int B, int E, typename F>
__device__ __forceinline__ void static_for(F&& f) {
    if constexpr (B < E) {
        f(std::integral_constant<int, B>{});
        static_for<B + 1, E>(f);
    }
}

// The large tile reads its operands through buffer resources with 32-bit
// offsets.  A stage row past the tile's last 32-row block gets this offset,
// which lies past the end of any operand the kernel takes (x of at most
// kNoRowOffset bytes, so up to 4 GiB less 1 MiB) and cannot wrap when a
// stage's K offset is added, so its loads fetch nothing.
constexpr uint32_t kNoRowOffset = 0xFFF00000u;

// Map this workgroup to a tile (expert e, column tile nt, row range
// [row0, row0 + rows)).  Every workgroup rebuilds the prefix sum of per-expert
// row tiles from expert_offsets in LDS (no host read-back); an expert with n
// rows gets ceil(n / BM) row tiles.  The tile list is ordered
// by expert position, then column tile, then row tile; workgroup b runs on
// XCD b % 8 and XCD x takes the x-th contiguous run of the list, so the row
// tiles that share a weight tile are neighbours on one XCD.  Expert positions
// interleave the experts (position i holds expert (i % 8) * (E / 8) + i / 8
// when 8 divides E), so each XCD's run draws on every group of consecutive
// experts and a few heavily routed neighbours do not land on one XCD.
// GRAN = 1 splits an expert's rows evenly over its row tiles; GRAN > 1 gives
// every row tile but the last the same multiple of GRAN rows (for the large
// tile, whose two row waves take alternate 32-row blocks: 64-row multiples
// keep them equally busy).  BAND > 0 orders an expert's tiles in bands of that
// many row tiles (column by column inside a band) instead of all row tiles of
// a column.  offsets may be NULL: one expert with all P rows.  Returns false
// for surplus workgroups (uniform
// over the workgroup).  s_off holds kMaxE + 1 entries, s_tstart
// kMaxE + 1 + kWaves.
template <int BM, int GRAN = 1, int BAND = 0>
__device__ bool find_tile(const int32_t* offsets, int64_t P, int E, int ncol_tiles, int32_t* s_off,
                          int32_t* s_tstart, int& e_out, int& nt_out, int& row0_out, int& rows_out) {
    const int tid = threadIdx.x;
    for (int e = tid; e <= E; e += kThreads) {
        int64_t o = offsets ? offsets[e] : (e == 0 ? 0 : P);
        o = o < 0 ? 0 : (o > P ? P : o);
        s_off[e] = static_cast<int32_t>(o);
    }
    __syncthreads();
    // expert at list position i
    const bool interleave = E % kNumXcd == 0;
    auto expert_at = [&](int i) { return interleave ? (i % kNumXcd) * (E / kNumXcd) + i / kNumXcd : i; };
    int cnt = 0;
    if (tid < E) {
        const int ex = expert_at(tid);
        const int n = s_off[ex + 1] - s_off[ex];
        cnt = row_tiles_of(n, BM);
    }
    // inclusive prefix sum over positions (kThreads == kMaxE): within each
    // wave by shuffles, then the totals of the waves before it
    const int lane = tid & (kWave - 1), wave = tid / kWave;
    int incl = cnt;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
        const int v = __shfl_up(incl, d, kWave);
        if (lane >= d) incl += v;
    }
    int32_t* s_wave_total = s_tstart + (kMaxE + 1);
    if (lane == kWave - 1) s_wave_total[wave] = incl;
    __syncthreads();
    for (int w = 0; w < wave; ++w) incl += s_wave_total[w];
    s_tstart[tid + 1] = incl;  // exclusive prefix over positions; s_tstart[E] = total row tiles
    if (tid == 0) s_tstart[0] = 0;
    __syncthreads();
    const int64_t total = static_cast<int64_t>(s_tstart[E]) * ncol_tiles;
    const int xcd = blockIdx.x % kNumXcd;
    const int64_t local = blockIdx.x / kNumXcd;
    const int64_t per = total / kNumXcd, rem = total % kNumXcd;
    if (local >= per + (xcd < rem ? 1 : 0)) return false;
    const int64_t L = xcd * per + (xcd < rem ? xcd : rem) + local;
    int lo = 0, hi = E - 1;  // last position i with s_tstart[i] * ncol_tiles <= L
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (static_cast<int64_t>(s_tstart[mid]) * ncol_tiles <= L) lo = mid; else hi = mid - 1;
    }
    const int pos = lo;
    const int e = expert_at(pos);
    const int tiles_e = s_tstart[pos + 1] - s_tstart[pos];  // >= 1 for the position found
    const int64_t rel = L - static_cast<int64_t>(s_tstart[pos]) * ncol_tiles;
    int nt, mt;
    if constexpr (BAND > 0) {
        const int64_t per_band = static_cast<int64_t>(BAND) * ncol_tiles;
        const int band = static_cast<int>(rel / per_band);
        const int in = static_cast<int>(rel - band * per_band);
        const int high = min(BAND, tiles_e - band * BAND);
        nt = in / high;
        mt = band * BAND + in % high;
    } else {
        nt = static_cast<int>(rel / tiles_e);
        mt = static_cast<int>(rel - static_cast<int64_t>(nt) * tiles_e);
    }
    const int n_e = s_off[e + 1] - s_off[e];
    e_out = e;
    nt_out = nt;
    if constexpr (GRAN == 1) {
        const int base = n_e / tiles_e, extra = n_e % tiles_e;
        row0_out = s_off[e] + mt * base + (mt < extra ? mt : extra);
        rows_out = base + (mt < extra ? 1 : 0);
    } else {
        static_assert(BM % GRAN == 0, "granule divides the tile");
        const int per = rows_per_tile(n_e, tiles_e, GRAN);
        row0_out = s_off[e] + mt * per;
        rows_out = min(per, n_e - mt * per);
    }
    return true;
}

// One wave's 64 x 16 bytes from the buffer straight into LDS at lds_byte_addr
// (contiguous, lane order); voffset is the lane's byte offset, soffset a
// uniform one.  The compiler does not see the load: the caller waits for it
// with wait_vmcnt.
// NT streams past the caches.
template <bool NT = false>
__device__ __forceinline__ void dma_load16(uint32_t lds_byte_addr, __amdgpu_buffer_rsrc_t rsrc,
                                           uint32_t voffset, uint32_t soffset) {
    if constexpr (NT)
        asm volatile(
        "s_mov_b32 m0, %0\n\t"
        "s_nop 0\n\t"
        "buffer_load_dwordx4 %1, %2, %3 offen nt lds"
        :
        : "s"(__builtin_amdgcn_readfirstlane(lds_byte_addr)), "v"(voffset), "s"(rsrc),
          "s"(__builtin_amdgcn_readfirstlane(soffset))
        : "memory", "m0");
    else
        asm volatile(
        "s_mov_b32 m0, %0\n\t"
        "s_nop 0\n\t"
        "buffer_load_dwordx4 %1, %2, %3 offen lds"
        :
        : "s"(__builtin_amdgcn_readfirstlane(lds_byte_addr)), "v"(voffset), "s"(rsrc),
          "s"(__builtin_amdgcn_readfirstlane(soffset))
        : "memory", "m0");
}

template <int N>
__device__ __forceinline__ void wait_vmcnt() {
    static_assert(N >= 0 && N < 64, "vmcnt range");
    asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory");
}

}  // namespace
}  // namespace moe
