// Building blocks shared by the grouped GEMM kernels (gfx950): the scan of the
// per-expert tile counts, the tile order, buffer resources, direct loads from
// memory into LDS, and the waits and barriers that order them.
#pragma once

#include "common.h"

namespace moe {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kGemmMaxE = 1024;

// Rows of expert e, with the offsets clamped into [0, max_rows] and made
// non-decreasing, so that no offsets array can send a tile out of bounds.
// offsets == NULL: one segment of all max_rows rows (a dense layer, E = 1).
__device__ __forceinline__ void seg_bounds(const int32_t* __restrict__ offsets, int e, int max_rows, int& lo,
                                           int& rows)
{
    if (offsets == nullptr) {
        lo = 0;
        rows = max_rows;
        return;
    }
    lo = min(max(offsets[e], 0), max_rows);
    const int hi = min(max(offsets[e + 1], lo), max_rows);
    rows = hi - lo;
}

// Exclusive scan of per-expert tile counts into s_pref[0..E] (s_pref[E] = total).
template <int kThreads>
__device__ void tile_prefix(const int32_t* __restrict__ offsets, int E, int max_rows, int BM, int ntn,
                            int32_t* s_pref, int32_t* s_wsum)
{
    constexpr int kPerThread = (kGemmMaxE + kThreads - 1) / kThreads;
    const int tid = threadIdx.x;
    int vals[kPerThread];
    int local = 0;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        const int e = tid * kPerThread + i;
        int v = 0;
        if (e < E) {
            int lo, rows;
            seg_bounds(offsets, e, max_rows, lo, rows);
            v = ((rows + BM - 1) / BM) * ntn;
        }
        vals[i] = v;
        local += v;
    }
    const int lane = lane_id(), wave = tid / kWave;
    int incl = local;
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
        const int n = __shfl_up(incl, o);
        if (lane >= o)
            incl += n;
    }
    if (lane == kWave - 1)
        s_wsum[wave] = incl;
    __syncthreads();
    int base = 0;
    for (int w = 0; w < wave; ++w)
        base += s_wsum[w];
    int run = base + incl - local;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        const int e = tid * kPerThread + i;
        if (e < E)
            s_pref[e] = run;
        run += vals[i];
    }
    if (tid == kThreads - 1)
        s_pref[E] = run;
    __syncthreads();
}

// One output tile: expert, first row and row count, first output column.
struct TileDec {
    int e, row0, rows, n0;
};

template <typename S>
__device__ __forceinline__ TileDec decode_tile(int tile, const int32_t* s_pref, const int32_t* __restrict__ offsets,
                                               int E, int max_rows, int ntn, int tile_cols)
{
    int lo = 0, hi = E;  // largest e with s_pref[e] <= tile
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_pref[mid] <= tile)
            lo = mid;
        else
            hi = mid;
    }
    TileDec t;
    t.e = lo;
    int seg0, seg_rows;
    seg_bounds(offsets, t.e, max_rows, seg0, seg_rows);
    const int mt_e = (seg_rows + S::BM - 1) / S::BM;
    // (m-group, n-tile, m-tile within group) order inside the expert
    const int local = tile - s_pref[t.e];
    const int g = local / (S::GM * ntn);
    const int within = local - g * S::GM * ntn;
    const int gs = min(S::GM, mt_e - g * S::GM);
    const int nt = within / gs;
    const int mt = g * S::GM + within % gs;
    t.row0 = seg0 + mt * S::BM;
    t.rows = min(S::BM, seg_rows - mt * S::BM);
    t.n0 = nt * tile_cols;
    return t;
}

typedef __attribute__((address_space(3))) void* lds_ptr_t;

// Raw buffer resource over [base, base + bytes): loads past the end return 0.
__device__ __forceinline__ i32x4 make_rsrc(const void* base, uint32_t bytes)
{
    const uint64_t a = reinterpret_cast<uint64_t>(base);
    i32x4 r;
    r[0] = __builtin_amdgcn_readfirstlane((int)(uint32_t)a);
    r[1] = __builtin_amdgcn_readfirstlane((int)(uint32_t)(a >> 32));  // stride 0: raw buffer
    r[2] = __builtin_amdgcn_readfirstlane((int)bytes);                 // num_records, in bytes
    r[3] = 0x00020000;                                                 // gfx9 raw-buffer descriptor word 3
    return r;
}

// Byte address of a shared-memory object in the LDS address space.
__device__ __forceinline__ uint32_t lds_addr(const void* p)
{
    return (uint32_t)(uintptr_t)(lds_ptr_t)p;
}

// 16 bytes per lane from buffer `rsrc` at voff + soff straight into LDS at
// byte address lds + 16 * lane (buffer_load_dwordx4 ... lds; M0 holds the
// LDS base).
// Issued from asm so that the compiler does not track the LDS writes: they
// are ordered by the kernel's own vmcnt waits and barriers (the compiler
// would otherwise make LDS reads wait for all loads in flight).  The
// instruction has no destination register; its address operands are read at
// issue.
__device__ __forceinline__ void dma16(const i32x4& rsrc, uint32_t lds, uint32_t voff, uint32_t soff)
{
    // scalar operands: wave-uniform by construction; readfirstlane makes the
    // compiler place them in SGPRs (and keeps the offset off the immediate field)
    const uint32_t m0 = __builtin_amdgcn_readfirstlane(lds);
    uint32_t so = __builtin_amdgcn_readfirstlane(soff);
    __asm__("" : "+s"(so));
    __asm__ volatile("s_mov_b32 m0, %0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                     :
                     : "s"(m0), "v"(voff), "s"(rsrc), "s"(so)
                     : "memory");
}

// Workgroup barrier for the K loop.  __syncthreads() (and any workgroup
// fence that covers LDS) waits for every outstanding load, DMA loads into LDS
// included, which would drain the load pipeline at each K slice.  Here the
// ordering is explicit instead: before the barrier each wave waits (vmcnt)
// for its own loads of the slice about to be read and (lgkmcnt) for its own
// LDS reads of the slice about to be overwritten; the asm statement's memory
// clobber keeps the compiler from moving memory accesses across it.
__device__ __forceinline__ void lds_barrier()
{
    __builtin_amdgcn_s_waitcnt((0x3f & 0xf) | ((0x3f >> 4) << 14) | (0x7 << 4) | (0 << 8));  // lgkmcnt(0)
    __asm__ volatile("s_barrier" ::: "memory");
}

// s_waitcnt with vmcnt(n) and no wait on the other counters (gfx9 encoding).
template <int N>
__device__ __forceinline__ void wait_vmcnt()
{
    static_assert(N >= 0 && N <= 63, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((N & 0xf) | ((N >> 4) << 14) | (0x7 << 4) | (0xf << 8));
}

}  // namespace moe
