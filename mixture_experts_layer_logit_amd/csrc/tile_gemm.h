// Output tiles of a product of two row-major operands, W rows times A rows along
// K (gfx950): LDS stages of 128 bytes of K of every row, and the K loop that keeps
// the matrix cores fed from them.  The kernels that use it bring the element type
// (an Op with the matrix instruction), the loads and the epilogue.
#pragma once

#include <type_traits>

#include "common.h"
#include "gemm_common.h"

namespace moe {

// Block tile BM x BN, WM x WN wavefronts, S stages.  The BN rows of W are two halves;
// a wavefront takes the same rows of both, so that a gate and an up value of a hidden
// column meet in one lane.  GM: m-tiles of a group that share W's columns (decode_tile).
// SCALES: the operands have scales, 8 bytes for the 128 of a row and slice, which lie behind
// the stages, those of two slices in two places in turn.
template <int BM_, int WM_, int WN_, int S_, int GM_, int BN_, int PER_CU_, bool SCALES_>
struct TileShape {
    static constexpr int BM = BM_, BN = BN_, kHalf = BN / 2, kPerCu = PER_CU_;
    static constexpr int WM = WM_, WN = WN_, S = S_, GM = GM_, RB = 128;
    static constexpr bool kScales = SCALES_;
    static constexpr int kWaves = WM * WN, kThreads = kWaves * kWave;
    static constexpr int kWavesPerSimd = kWaves / 4 * kPerCu;
    static constexpr int kWaveM = BM / WM, kWaveN = BN / WN;
    static constexpr int kFM = kWaveM / 32, kFN = kWaveN / 32;
    static constexpr int kHalfN = kWaveN / 2, kHalfF = kFN / 2;
    static constexpr int kRows = 1024 / RB;  // tile rows of a 1 KB load
    static constexpr int kLdsA = BM * RB, kLdsW = BN * RB;
    // a load of scales takes 16 bytes, two slices' of a row, a lane
    static constexpr int kSclGroups = kScales ? (BM + BN) / 64 : 0, kBlkS = (kSclGroups + kWaves - 1) / kWaves;
    static constexpr int kSclUnit = kSclGroups * 1024;
    static constexpr int kStage = kLdsA + kLdsW, kLds = S * kStage + 2 * kSclUnit;
    static constexpr int kBlkA = BM / kRows / kWaves, kBlkW = BN / kRows / kWaves;  // loads per wavefront and stage
    static constexpr int kLoads = kBlkA + kBlkW;
    static constexpr int kTileFloats = BM * BN;
    static_assert(kFN % 2 == 0, "a wavefront takes rows of both halves of W");
    static_assert(kWaves % 4 == 0 && BM % (kRows * kWaves) == 0, "loads split evenly");
    static_assert(kBlkW % 2 == 0, "a load lies in one half of W");
    static_assert(!kScales || (BM % 64 == 0 && BN % 64 == 0 && kSclGroups % kWaves == 0), "scale loads split evenly");
    static_assert(S >= 2 && (S - 1) * kLoads <= 63, "vmcnt range");
};

// LDS offset of 16-byte chunk c of tile row `row`: the chunk index XOR-ed with the
// row pair's number (two rows fill the 64 banks once), so that one chunk of 16
// consecutive rows touches every bank once.
__device__ __forceinline__ int tile_swz(int row) { return (row >> 1) & 7; }
__device__ __forceinline__ uint32_t tile_at(int row, int c) { return row * 128 + ((c ^ tile_swz(row)) << 4); }

// dma16 for a wavefront whose lanes are all active, where `on` is all ones, or, where it is 0,
// nothing: a condition without a branch, which would split a loop that is scheduled as a
// whole.
__device__ __forceinline__ void dma16_if(uint32_t on, const i32x4& rsrc, uint32_t lds, uint32_t voff, uint32_t soff)
{
    const uint32_t m0 = __builtin_amdgcn_readfirstlane(lds), mask = __builtin_amdgcn_readfirstlane(on);
    uint32_t so = __builtin_amdgcn_readfirstlane(soff);
    __asm__("" : "+s"(so));
    __asm__ volatile("s_mov_b32 exec_lo, %4\n\ts_mov_b32 exec_hi, %4\n\ts_mov_b32 m0, %0\n\t"
                     "buffer_load_dwordx4 %1, %2, %3 offen lds\n\ts_mov_b64 exec, -1"
                     :
                     : "s"(m0), "v"(voff), "s"(rsrc), "s"(so), "s"(mask)
                     : "memory");
}

// The K loop over slices [k0, k1) (k0 even where there are scales) (each 128 bytes of K) for a wavefront whose first L
// row fragments hold rows that count (the others are neither read nor multiplied).
// issue(q, st, n0, n1) starts loads [n0, n1) of the kLoads of slice q into stage st,
// W's first; scales(q, place, on) those of the scales from slice q on, if on; keep(q) is a mask that
// clears the scales of what is missing of slice q (only of the last one).
//
// Lane l of a 32-row fragment reads the chunks 4 (l / 32) .. + 3 of its row, one per
// matrix instruction: two chunks in each of a slice's two k-steps.  Which values of K
// meet in an instruction is free as long as both operands agree, and this way a lane
// takes four neighbouring scales, one dword of which every instruction selects a byte.
//
// In a slice's first k-step the second's fragments are read as fast as the LDS gives
// them; behind a barrier the stage is free then and takes the loads of slice kt + S.
// Between the two k-steps slice kt + 1 has to be there (a second barrier), so a load
// has 1 1/4 slices (S = 2) to arrive.
template <typename S, typename Op, int L, typename Loads>
__device__ __forceinline__ void tile_kloop(f32x16 (&acc)[S::kFM][S::kFN], const uint8_t* lds, int wm, int wn, int k0,
                                           int k1, const Loads& loads)
{
    constexpr int kHalfF = S::kHalfF;
    constexpr int NI = L * S::kFN, kNI = NI > 0 ? NI : 1, NM = 2 * NI, NR = L > 0 ? 2 * (L + S::kFN) : 0;
    const int lane = lane_id();
    const uint32_t rdA = tile_at(wm * S::kWaveM + (lane & 31), 4 * (lane >> 5));
    const uint32_t rdW = S::kLdsA + tile_at(wn * S::kHalfN + (lane & 31), 4 * (lane >> 5));
    const uint32_t scl = S::S * S::kStage + 16 * (lane & 31) + 4 * (lane >> 5);
    const uint32_t scA = scl + 16 * wm * S::kWaveM, scW = scl + 16 * (S::BM + wn * S::kHalfN);
    auto scales_at = [&](int q) { return (q >> 1 & 1) * S::kSclUnit + (q & 1) * 8; };  // where slice q's lie
    struct Frags {
        i32x4 w[2][S::kFN], a[2][S::kFM];
    };
    Frags f0, f1;
    int sa[S::kFM] = {}, sw[S::kFN] = {}, swn[S::kFN] = {};
    auto read = [&](int r, Frags& nx, uint32_t st, int kk) {
        const int n = r / 2, h = r % 2;  // fragment, chunk
        const uint32_t x = (uint32_t)(kk * 32) ^ (uint32_t)(h * 16);
        const i32x4 v = *reinterpret_cast<const i32x4*>(
            lds + st + (n < S::kFN ? (rdW ^ x) + ((n / kHalfF) * S::kHalf + (n % kHalfF) * 32) * S::RB
                                   : (rdA ^ x) + (n - S::kFN) * 32 * S::RB));
        if (n < S::kFN)
            nx.w[h][n] = v;
        else
            nx.a[h][n - S::kFN] = v;
    };
    auto read_a_scale = [&](int i, uint32_t at) {
        if constexpr (S::kScales)
            sa[i] = *reinterpret_cast<const int*>(lds + at + scA + i * 512);
    };
    auto read_w_scales = [&](uint32_t at) {
        if constexpr (S::kScales)
#pragma unroll
            for (int j = 0; j < S::kFN; ++j)
                swn[j] = *reinterpret_cast<const int*>(lds + at + scW +
                                                       16 * ((j / kHalfF) * S::kHalf + (j % kHalfF) * 32));
    };
    auto cut_scales = [&](int q) {
        if constexpr (S::kScales) {
            const int keep = loads.keep(q);
#pragma unroll
            for (int i = 0; i < L; ++i)
                sa[i] &= keep;
#pragma unroll
            for (int j = 0; j < S::kFN; ++j)
                sw[j] &= keep;
        }
    };
    // One k-step: the matrix instructions on the fragments in f, and between them the
    // LDS reads of the next k-step's fragments into nx (k-step kk of stage st) and,
    // where LAST, the scales of slice q + 1 (at sc); where LOADS, the loads of slice q + S
    // into stage lst, and of scales.  A matrix instruction runs for 32 cycles, in which its wavefront can
    // issue the few instructions that follow it.
    // In the second k-step of an odd slice q its own scales, the last of their place, have
    // been read by every wavefront: the place takes those of slices q + 3 and q + 4, which are
    // read more than S - 1 slices' loads later, behind a wait that leaves fewer than those in
    // flight.  Behind the last slice nothing is read.
    auto next_scales = [&](int q) {
        if constexpr (S::kScales)
            loads.scales(q + 3, (q + 3) >> 1 & 1, -(uint32_t)(q & 1));
    };
    constexpr int kEarly = S::kBlkW;  // loads issued in a slice's first k-step: W's
    constexpr int kFree = NM >= 16 ? 6 : NM > 2 ? NM / 2 : NM;     // instructions behind which its reads are spread
    constexpr int kBar = NM >= 16 ? 6 : NM > 0 ? kFree - 1 : 0;    // the one behind which the stage is free
    auto kstep = [&](const Frags& f, Frags& nx, uint32_t st, int kk, uint32_t sc, auto last, auto more, int q, int lst) {
        constexpr bool LAST = decltype(last)::value, LOADS = decltype(more)::value;
        constexpr int kOver = LAST ? NM : kFree;
        constexpr int kPer = kOver > 0 && (NR + kOver - 1) / kOver > 1 ? (NR + kOver - 1) / kOver : 1;
        if constexpr (NM == 0) {
            if (!LAST && LOADS)
                lds_barrier();
            if (LOADS)
                loads.issue(q + S::S, lst, LAST ? kEarly : 0, LAST ? S::kLoads : kEarly);
            if constexpr (LAST && LOADS)
                next_scales(q);
        }
#pragma unroll
        for (int m = 0; m < NM; ++m) {
            const int h = m / kNI, i = m % kNI / S::kFN, j = m % S::kFN;
            acc[i][j] = h == 0 ? Op::template mma<LAST ? 2 : 0>(f.w[0][j], f.a[0][i], acc[i][j], sw[j], sa[i])
                               : Op::template mma<LAST ? 3 : 1>(f.w[1][j], f.a[1][i], acc[i][j], sw[j], sa[i]);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int r = 0; r < NR; ++r)
                if (r / kPer == m)
                    read(r, nx, st, kk);
            if constexpr (LAST) {
                if (h == 1 && j == S::kFN - 1)
                    read_a_scale(i, sc);
                if (m == 0)
                    read_w_scales(sc);
                if constexpr (LOADS)
                    if (m == 1)
                        next_scales(q);
                constexpr int kLate = S::kLoads - kEarly, kSafe = NM > 0 ? NM : 1;
                if constexpr (LOADS)
                    loads.issue(q + S::S, lst, kEarly + m * kLate / kSafe, kEarly + (m + 1) * kLate / kSafe);
            } else if constexpr (LOADS) {
                // every wavefront's reads of the stage are done: it is free
                if (m == kBar)
                    lds_barrier();
                if (m >= kBar) {
                    constexpr int kLeft = NM - kBar > 0 ? NM - kBar : 1;
                    loads.issue(q + S::S, lst, (m - kBar) * kEarly / kLeft, (m - kBar + 1) * kEarly / kLeft);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    constexpr std::integral_constant<bool, false> no{};
    constexpr std::integral_constant<bool, true> yes{};
    // in the order of the loop's own reads: the waits at its head are the stricter
    // of the two
#pragma unroll
    for (int m = 0; m < NM; ++m) {
        constexpr int kPer = (NR + NM - 1) / (NM > 0 ? NM : 1) > 1 ? (NR + NM - 1) / (NM > 0 ? NM : 1) : 1;
#pragma unroll
        for (int r = 0; r < NR; ++r)
            if (r / kPer == m)
                read(r, f0, 0, 0);
        if (m >= NI && m % S::kFN == S::kFN - 1)
            read_a_scale(m % kNI / S::kFN, scales_at(k0));
        if (m == 0)
            read_w_scales(scales_at(k0));
        __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int j = 0; j < S::kFN; ++j)
        sw[j] = swn[j];
    int cur = 0;  // stage of slice kt
    auto slice = [&](int kt, auto more) {
        constexpr bool LOADS = decltype(more)::value;
        const int nxt = cur + 1 == S::S ? 0 : cur + 1;
        if constexpr (!LOADS)
            cut_scales(kt);
        kstep(f0, f1, cur * S::kStage, 1, 0, no, more, kt, cur);
        // slice kt + 1 has to be there (scales among the newer loads only make the wait
        // stricter)
        wait_vmcnt<LOADS ? (S::S - 2) * S::kLoads + kEarly : 0>();
        lds_barrier();
        kstep(f1, f0, nxt * S::kStage, 0, scales_at(kt + 1), yes, more, kt, cur);
#pragma unroll
        for (int j = 0; j < S::kFN; ++j)
            sw[j] = swn[j];
        cur = nxt;
    };
    int kt = k0;
    for (; kt + S::S < k1; ++kt)
        slice(kt, yes);
    for (; kt < k1; ++kt)  // nothing is left to load
        slice(kt, no);
}

// All of a tile's K: the first stages' loads, and the loop for the `live` row
// fragments of this wavefront (a copy of it for each count).  Every earlier access to
// the stages has to be behind a barrier.
template <typename S, typename Op, typename Loads>
__device__ __forceinline__ void tile_product(f32x16 (&acc)[S::kFM][S::kFN], const uint8_t* lds, int wm, int wn,
                                             int live, int k0, int k1, const Loads& loads)
{
#pragma unroll
    for (int i = 0; i < S::kFM; ++i)
#pragma unroll
        for (int j = 0; j < S::kFN; ++j)
#pragma unroll
            for (int v = 0; v < 16; ++v)
                acc[i][j][v] = 0.0f;
    if constexpr (S::kScales)
#pragma unroll
        for (int u = 0; u < 2; ++u)
            loads.scales(k0 + 2 * u, ((k0 >> 1) + u) & 1, k0 + 2 * u < k1 ? ~0u : 0u);
#pragma unroll
    for (int q = 0; q < S::S; ++q)
        if (k0 + q < k1)
            loads.issue(k0 + q, q, 0, S::kLoads);
    if (k1 - k0 >= S::S)
        wait_vmcnt<(S::S - 1) * S::kLoads>();
    else
        wait_vmcnt<0>();
    lds_barrier();
    if (S::kFM == 1 || live >= S::kFM)
        tile_kloop<S, Op, S::kFM>(acc, lds, wm, wn, k0, k1, loads);
    else if (S::kFM > 3 && live == 3)
        tile_kloop<S, Op, (S::kFM > 3 ? 3 : 1)>(acc, lds, wm, wn, k0, k1, loads);
    else if (S::kFM > 2 && live == 2)
        tile_kloop<S, Op, (S::kFM > 2 ? 2 : 1)>(acc, lds, wm, wn, k0, k1, loads);
    else if (live == 1)
        tile_kloop<S, Op, 1>(acc, lds, wm, wn, k0, k1, loads);
    else
        tile_kloop<S, Op, 0>(acc, lds, wm, wn, k0, k1, loads);
    lds_barrier();
}

}  // namespace moe
