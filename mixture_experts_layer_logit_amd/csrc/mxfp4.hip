// MXFP4 experts (gfx950): quantisation to E2M1 codes with a scale for each block
// of 32 values, its inverse, and the grouped GEMMs of the two expert layers on
// such codes.
//
// The experts' weights and the rows that meet them carry one E8M0 scale per 32
// consecutive values of K (a byte b stands for 2^(b - 127)):
//   u[r, n] = sum_b 2^(sA[r, b] + sW[n, b] - 254) sum_{k in block b} a[r, k] w[n, k]
#include <algorithm>
#include <cmath>

#include "common.h"
#include "gemm_common.h"
#include "mxfp4.h"
#include "tile_gemm.h"

namespace moe {

// ---------------------------------------------------------------- quantisation
// The most workgroups of a launch (a launch has fewer than 2^32 threads).
constexpr long long kMxGrid = 1 << 23;

// 4 lanes of 8 values each per block, the blocks of all rows in one run (K is a
// multiple of 32): every lane's access is one wide load or store, the maximum takes two
// exchanges between neighbours, and no row's length matters.  Bound by HBM: 28672 x 4096
// fp32 values take 106 us (5.0 TB/s read and written), their way back to bf16 64 us (4.6
// TB/s); a copy of 4 GiB runs at 4.8.  A few rows take the launch (1.3 to 2.5 us).
template <typename ET>
__global__ __launch_bounds__(256) void moe_mxfp4_quantize_kernel(const typename ET::storage* __restrict__ src,
                                                                 long long blocks, uint8_t* __restrict__ codes,
                                                                 uint8_t* __restrict__ scales)
{
    const long long b = (long long)blockIdx.x * 64 + threadIdx.x / 4;
    if (b >= blocks)
        return;
    const size_t at = (size_t)b * kMxBlk + 8 * (threadIdx.x % 4);
    float f[8];
    uint32_t amax = 0;
    load8(src + at, f);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        amax = max(amax, abs_bits(f[i]));
    amax = max(amax, (uint32_t)__shfl_xor((int)amax, 1));
    amax = max(amax, (uint32_t)__shfl_xor((int)amax, 2));
    const uint32_t s = mx_scale_byte(amax);
    *reinterpret_cast<uint32_t*>(codes + at / 2) = e2m1_encode8(f, s);
    if (threadIdx.x % 4 == 0)
        scales[b] = (uint8_t)s;
}

template <typename ET>
__global__ __launch_bounds__(256) void moe_mxfp4_dequantize_kernel(const uint8_t* __restrict__ codes,
                                                                   const uint8_t* __restrict__ scales,
                                                                   long long blocks,
                                                                   typename ET::storage* __restrict__ dst)
{
    const long long b = (long long)blockIdx.x * 64 + threadIdx.x / 4;
    if (b >= blocks)
        return;
    const size_t at = (size_t)b * kMxBlk + 8 * (threadIdx.x % 4);
    float f[8];
    e2m1_decode8(*reinterpret_cast<const uint32_t*>(codes + at / 2), scales[b], f);
    store8(dst + at, f);
}

// ---------------------------------------------------------------- grouped GEMM
// Rows of expert e's segment times its weight matrix, in tiles of tile_gemm.h: a
// slice is 256 values of K (128 bytes of codes and 8 scales of a row).  For SwiGLU the
// two halves of a tile's weight rows are the gate rows and the matching up rows of
// 128 hidden columns, else consecutive rows.
//
// MFMA 32x32x64 f8f6f4 with E2M1 operands: lane l holds 32 values (a block) of operand
// row l % 32 and the byte that scales them, so the matrix core applies both scales of
// a block itself.  The weight tile is its first operand, the activation tile its
// second: a lane's accumulators are 4 consecutive columns of one row, and a 32 x 32
// fragment holds whole blocks of h.
//
// Few rows are bound by the weights' bytes (33 rows of 8 experts, 14336 wide: 49 us, 5.1
// TB/s), many by the loads' arrival: 8192 rows of 8 experts with 4096 x 14336 weights take
// 542 us up (SwiGLU, 3.55 PFLOP/s) and 240 + 12 us down, with the matrix cores busy 46 and
// 52 % of the cycles at the 1.86 GHz that the card holds.  Without its LDS reads the first
// is 5 % faster, with half of its matrix instructions 15 %, without the loop's loads 27 %.
// Four wavefronts of 128 x 128, which read a third less LDS, are 8 to 19 % slower; m-groups
// of 4 and 16, other places of the barriers and wave priorities make no difference.  8
// bytes of scales a row and slice, a slice at a time, cost 18 % (each touches a cache line
// of its own); 16 for two slices half of that.
enum { MXEPI_NONE = 0, MXEPI_RELU = 1, MXEPI_SWIGLU = 2, MXEPI_F32 = 3 };  // bf16 rows, hidden codes (2), fp32 rows

constexpr int kMxSlice = 256;       // values of K of a slice
constexpr int kMxMaxParts = 16;     // K parts of a tail tile
constexpr int kMxSplitSlots = 256;  // partial tiles the workspace holds
constexpr int kMxMinPart = 4;       // slices of a part

// 256 x 256 with 8 wavefronts, or 128 x 128 with 4 and two blocks a CU, which hide each
// other's waits.
typedef TileShape<256, 2, 4, 2, 8, 256, 1, true> LargeShape;
typedef TileShape<128, 2, 2, 2, 4, 128, 2, true> PairShape;

struct MxOp {
    template <int BYTE>
    static __device__ __forceinline__ f32x16 mma(const i32x4& w, const i32x4& a, const f32x16& c, int sw, int sa)
    {
        const i32x8 wv = __builtin_shufflevector(w, w, 0, 1, 2, 3, -1, -1, -1, -1);
        const i32x8 av = __builtin_shufflevector(a, a, 0, 1, 2, 3, -1, -1, -1, -1);
        return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wv, av, c, 4, 4, BYTE, sw, BYTE, sa);
    }
};

struct MxGemmArgs {
    const uint8_t* A;       // codes of the activation rows [.][K / 2]
    const uint8_t* As;      // their scales [.][K / 32]
    const int32_t* gather;  // nullable: row r is A's row gather[r] of gather_rows
    int gather_rows;
    const uint8_t* W;   // [E][Nw][K / 2]
    const uint8_t* Ws;  // [E][Nw][K / 32]
    uint8_t* Hq;        // codes of the hidden rows [.][Nout / 2] (activation epilogues)
    uint8_t* Hs;        // their scales [.][Nout / 32]
    void* Y;            // bf16 or fp32 rows [.][Nout] (plain epilogues)
    const int32_t* offsets;
    int E, K, Nw, Nout, F, max_rows;
    float* partial;  // nullable: no K split
};

__device__ __forceinline__ int mx_parts(int total, int G, int nk, bool enabled)
{
    const int tail = total % G;
    if (!enabled || tail == 0)
        return 1;
    return max(1, min(min(kMxMaxParts, min(G, kMxSplitSlots) / tail), nk / kMxMinPart));
}

// silu(u) v, silu(u) = u / (1 + e^-u).  The exponent is rounded to fp32, which costs
// the exponential |u| 1.3 of 2^-24, and it and the reciprocal are a step or so off
// themselves: (1.3 |u| + 8) 2^-24 of the result where u is negative, 8 of 2^-24 where it is
// positive; below about -87, where e^-u leaves fp32's range, the result is 0.  A value or
// a block's maximum that lies this close to a border can take the code on its other side.
__device__ __forceinline__ float mx_glu(float u, float v)
{
    return u * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(u * -1.44269504088896341f)) * v;
}

// Hidden rows of row fragment i: every 32 x 32 fragment holds one block of each of its
// rows, 16 of the values in lane l and 16 in lane l ^ 32, which are quantised as they
// are (fp32, no rounding to bf16 in between).  The two lanes swap halves of their codes
// so that each stores 8 consecutive bytes.
template <typename S, int EPI>
__device__ __forceinline__ void mx_store_hidden(const f32x16 (&acc)[S::kFN], int i, const TileDec& t,
                                                const MxGemmArgs& g)
{
    constexpr bool kGlu = EPI == MXEPI_SWIGLU;
    const int lane = lane_id(), wave = threadIdx.x / kWave, half = lane >> 5;
    const int wm = wave / S::WN, wn = wave % S::WN;
    const int m = wm * S::kWaveM + i * 32 + (lane & 31);
#pragma unroll
    for (int j = 0; j < (kGlu ? S::kHalfF : S::kFN); ++j) {
        const int n = t.n0 + (j / S::kHalfF) * S::kHalf + wn * S::kHalfN + (j % S::kHalfF) * 32;
        float h[16];
        uint32_t amax = 0;
#pragma unroll
        for (int v = 0; v < 16; ++v) {
            const float u = acc[j][v];
            if constexpr (kGlu)
                h[v] = mx_glu(u, acc[j + S::kHalfF][v]);
            else
                h[v] = u <= 0.0f ? 0.0f : u;  // a NaN stays one
            amax = max(amax, abs_bits(h[v]));
        }
        amax = max(amax, (uint32_t)__shfl_xor((int)amax, 32));
        const uint32_t s = mx_scale_byte(amax);
        // 16 bits of codes for each 4 columns 8 q + 4 half ..: this lane's of q = 0, 1 in
        // c0, of q = 2, 3 in c1
        const uint32_t c0 = e2m1_encode8(h, s), c1 = e2m1_encode8(h + 8, s);
        const uint32_t got = (uint32_t)__shfl_xor((int)(half ? c0 : c1), 32), own = half ? c1 : c0;
        const uint32_t lo = half ? got : own, hi = half ? own : got;  // of columns 8 q, and 8 q + 4
        if (m < t.rows && n < g.Nout) {
            const size_t at = (size_t)(t.row0 + m) * (g.Nout / kMxBlk) + n / kMxBlk;
            *reinterpret_cast<uint2*>(g.Hq + at * 16 + 8 * half) =
                make_uint2((lo & 0xffffu) | (hi << 16), (lo >> 16) | (hi & 0xffff0000u));
            if (half == 0)
                g.Hs[at] = (uint8_t)s;
        }
    }
}

// Plain rows of row fragment i of every wavefront (WM bands of 32 rows): staged in LDS
// as [band row][column] (16-byte chunks XOR-swizzled by the row), then stored row by
// row.
template <typename S, int EPI>
__device__ __forceinline__ void mx_store_rows(const f32x16 (&acc)[S::kFN], int i, const TileDec& t, uint8_t* buf,
                                              const MxGemmArgs& g)
{
    constexpr int kEl = EPI == MXEPI_F32 ? 4 : 2;
    constexpr int kRows = S::WM * 32, kRowBytes = S::BN * kEl;
    constexpr int kSwz = kRowBytes / 16 - 1 < 31 ? kRowBytes / 16 - 1 : 31;
    int tid = threadIdx.x;
    __asm__ volatile("" : "+v"(tid));
    const int lane = tid & (kWave - 1), wave = tid / kWave;
    const int wm = wave / S::WN, wn = wave % S::WN;
    const int r = wm * 32 + (lane & 31);
#pragma unroll
    for (int j = 0; j < S::kFN; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int col = (j / S::kHalfF) * S::kHalf + wn * S::kHalfN + (j % S::kHalfF) * 32 + 8 * q + 4 * (lane >> 5);
            const f32x4 v = {acc[j][4 * q], acc[j][4 * q + 1], acc[j][4 * q + 2], acc[j][4 * q + 3]};
            const int byte = col * kEl;
            uint8_t* dst = buf + r * kRowBytes + (((byte >> 4) ^ (r & kSwz)) << 4) + (byte & 15);
            if constexpr (kEl == 2) {
                typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
                *reinterpret_cast<bf16x4*>(dst) = __builtin_convertvector(v, bf16x4);
            } else {
                *reinterpret_cast<f32x4*>(dst) = v;
            }
        }
    lds_barrier();
    constexpr int kChunks = kRowBytes / 16, kPer = 16 / kEl;
#pragma unroll
    for (int it = 0; it < kRows * kChunks / S::kThreads; ++it) {
        const int c = tid + it * S::kThreads;
        const int rr = c / kChunks, q = c % kChunks;
        const int m = (rr / 32) * S::kWaveM + i * 32 + (rr % 32);
        if (m < t.rows && t.n0 + q * kPer < g.Nout)
            *reinterpret_cast<uint4*>(static_cast<uint8_t*>(g.Y) +
                                      ((size_t)(t.row0 + m) * g.Nout + t.n0 + q * kPer) * kEl) =
                *reinterpret_cast<const uint4*>(buf + rr * kRowBytes + ((q ^ (rr & kSwz)) << 4));
    }
}

template <typename S, int EPI>
__global__ __launch_bounds__(S::kThreads) __attribute__((amdgpu_waves_per_eu(S::kWavesPerSimd, S::kWavesPerSimd)))
void moe_mxfp4_gemm_kernel(MxGemmArgs g)
{
#if defined(__HIP_DEVICE_COMPILE__)  // the body uses device-only types; the host pass needs the stub only
    static_assert((S::kFM > 1 ? 2 : 1) * (S::WM * 32) * S::BN * 4 <= S::S * S::kStage, "staged row fragments fit");
    __shared__ __attribute__((aligned(1024))) uint8_t lds[S::kLds];
    __shared__ int32_t s_pref[kGemmMaxE + 1];
    __shared__ int32_t s_wsum[S::kWaves];
    const int tid = threadIdx.x;
    const int lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int wm = wave / S::WN, wn = wave % S::WN;
    const int pitch = g.K / 2, spitch = g.K / kMxBlk;  // bytes of a row's codes and scales
    const int nk = (g.K + kMxSlice - 1) / kMxSlice;
    const int ragged = g.K % kMxSlice ? nk - 1 : -1;  // the slice of which only the first half is there
    const uint32_t lds0 = lds_addr(lds);

    const int tile_cols = EPI == MXEPI_SWIGLU ? S::kHalf : S::BN;
    const int ntn = (g.Nout + tile_cols - 1) / tile_cols;
    tile_prefix<S::kThreads>(g.offsets, g.E, g.max_rows, S::BM, ntn, s_pref, s_wsum);
    const int total = s_pref[g.E];
    const int G = gridDim.x;
    const int parts = mx_parts(total, G, nk, g.partial != nullptr);
    const int full = parts > 1 ? total - total % G : total;
    const int tail = total - full;
    const int items = full + tail * parts;

    for (int base = 0; base < items; base += G) {
        const int b = blockIdx.x;
        // an XCD's blocks side by side; with two blocks a CU a round that is not full
        // is spread over all XCDs
        const int each = S::kPerCu > 1 ? (min(G, items - base) + 7) / 8 : G / 8;
        const int item = (G % 8 == 0) ? base + (b % 8) * each + b / 8 : base + b;
        if (item >= items || (S::kPerCu > 1 && G % 8 == 0 && b / 8 >= each))
            continue;
        int tile = item, k0 = 0, k1 = nk, slot = -1;
        if (item >= full) {
            const int j = item - full, part = j / tail;
            tile = full + j % tail;
            k0 = part * nk / parts / 2 * 2;
            k1 = part + 1 < parts ? (part + 1) * nk / parts / 2 * 2 : nk;
            slot = (j % tail) * parts + part;
        }
        const TileDec t = decode_tile<S>(tile, s_pref, g.offsets, g.E, g.max_rows, ntn, tile_cols);

        // lane's place in a 1 KB load of kRows rows: row lane / 8, physical chunk
        // lane % 8; the swizzle term is the same in all of a wavefront's loads (their
        // row blocks all have the parity of its number)
        const int lrow = S::kRows * wave + lane / 8;
        const int chunk = (lane % 8) ^ tile_swz(lrow);
        const uint32_t lchunk = (uint32_t)chunk * 16;
        // the missing half of a ragged slice reads behind the buffer: zeros
        const uint32_t cutHalf = chunk >= 4 ? 0xf0000000u : 0;
        // first rows of the two halves of the weight tile; the second, or its end, may
        // lie behind the matrix
        const uint32_t half1 = EPI == MXEPI_SWIGLU ? (uint32_t)(g.F + t.n0) : (uint32_t)(t.n0 + S::kHalf);
        const bool second = EPI == MXEPI_SWIGLU || (int)half1 < g.Nw;
        uint32_t voffA[S::kBlkA];
        auto source = [&](int r) {  // the row of A of tile row r, -1 for none
            if (r >= t.rows)
                return -1;
            if (!g.gather)
                return r;
            const int src = g.gather[t.row0 + r];
            return src < g.gather_rows ? src : -1;
        };
        const size_t rowA = g.gather ? 0 : t.row0;
        const uint32_t rowsA = g.gather ? g.gather_rows : t.rows;
        const i32x4 rsA = make_rsrc(g.A + rowA * pitch, rowsA * (uint32_t)pitch);
#pragma unroll
        for (int i = 0; i < S::kBlkA; ++i) {
            const int src = source(lrow + S::kRows * S::kWaves * i);
            voffA[i] = src >= 0 ? (uint32_t)src * (uint32_t)pitch + lchunk : 0xf0000000u;
        }
        const i32x4 rsW = make_rsrc(g.W + (size_t)t.e * g.Nw * pitch, (uint32_t)g.Nw * (uint32_t)pitch);
        const uint32_t voffW = (uint32_t)lrow * (uint32_t)pitch + lchunk;
        const uint32_t voffW1 = second ? voffW : 0xf0000000u, row0 = (uint32_t)t.n0 * (uint32_t)pitch;
        const uint32_t row1 = second ? half1 * (uint32_t)pitch : 0, step = S::kRows * S::kWaves * (uint32_t)pitch;
        // this wavefront's loads of scales: 64 rows of A, or of the tile's rows of W
        uint32_t voffS[S::kBlkS];
        i32x4 rsS[S::kBlkS];
#pragma unroll
        for (int q = 0; q < S::kBlkS; ++q) {
            const int group = wave + q * S::kWaves;
            const bool a = group * 64 < S::BM;
            const int r = group * 64 + lane - (a ? 0 : S::BM);
            const uint8_t* base = a ? g.As + rowA * spitch : g.Ws + (size_t)t.e * g.Nw * spitch;
            rsS[q] = make_rsrc(base, (a ? rowsA : (uint32_t)g.Nw) * (uint32_t)spitch);
            int src = a ? source(r) : r < S::kHalf ? t.n0 + r : (int)half1 + r - S::kHalf;
            if (!a && src >= g.Nw)
                src = -1;
            voffS[q] = src >= 0 ? (uint32_t)src * (uint32_t)spitch : 0xf0000000u;
        }
        // Two blocks a CU, which stream weights where rows are few: every tile of columns
        // starts at another slice, so that blocks which read rows a power of two apart at a
        // time do not meet in few of the memory's channels.  The tile decides, so the sums
        // keep their order from run to run.  The first slice follows the last behind an odd
        // one.
        constexpr bool kRotate = S::kPerCu > 1;
        int rot = 0;
        if (kRotate && pitch >= 4096 && pitch % 2048 == 0)
            rot = (t.n0 / tile_cols * 5) % (k1 - k0);
        if ((k1 - rot) % 2)
            rot ^= rot > 0;

        struct Loads {
            const i32x4 &rsA, &rsW;
            const i32x4 (&rsS)[S::kBlkS];
            const uint32_t (&voffA)[S::kBlkA], (&voffS)[S::kBlkS];
            uint32_t voffW, voffW1, row0, row1, step, lds0, cutHalf;
            int keepS, wave, k0, k1, rot, last;
            __device__ __forceinline__ int slice_of(int q) const
            {
                if constexpr (S::kPerCu > 1)
                    return q + rot >= k1 ? q + rot - (k1 - k0) : q + rot;
                return q;
            }
            __device__ __forceinline__ void issue(int q, int st, int n0, int n1) const
            {
                const uint32_t dst = lds0 + st * S::kStage + wave * 1024;
                const int kb = slice_of(q);
                const uint32_t soff = (uint32_t)kb * S::RB, cut = kb == last ? cutHalf : 0;
#pragma unroll
                for (int p = 0; p < S::kLoads; ++p) {
                    if (p < n0 || p >= n1)
                        continue;
                    if (p < S::kBlkW / 2)
                        dma16(rsW, dst + S::kLdsA + S::kWaves * p * 1024, voffW | cut, soff + row0 + p * step);
                    else if (p < S::kBlkW)
                        dma16(rsW, dst + S::kLdsA + S::kWaves * p * 1024, (EPI == MXEPI_SWIGLU ? voffW : voffW1) | cut,
                              soff + row1 + (p - S::kBlkW / 2) * step);
                    else
                        dma16(rsA, dst + S::kWaves * (p - S::kBlkW) * 1024, voffA[p - S::kBlkW] | cut, soff);
                }
            }
            __device__ __forceinline__ void scales(int q0, int place, uint32_t on) const
            {
                const uint32_t dst = lds0 + S::S * S::kStage + place * S::kSclUnit;
                // in the lane's offset: what lies behind the operand's end reads as zeros
                const uint32_t at = (uint32_t)slice_of(q0) * 8;
#pragma unroll
                for (int q = 0; q < S::kBlkS; ++q)
                    dma16_if(on, rsS[q], dst + (wave + q * S::kWaves) * 1024, voffS[q] + at, 0);
            }
            // the last slice's second half may be missing: its codes are zeros, and its
            // scales, whatever lies there, must not be NaN.  (No row that is rotated
            // ends in half a slice: the last one stays the last.)
            __device__ __forceinline__ int keep(int q) const { return q == last ? keepS : -1; }
        };
        const Loads loads = {rsA,  rsW,  rsS,  voffA, voffS, voffW, voffW1, row0, row1, step, lds0,
                             cutHalf, (lane >> 5) - 1, wave, k0, k1, rot, ragged};

        wait_vmcnt<0>();  // the previous tile's stores are out of the count
        __syncthreads();  // and every wave is done with its LDS
        f32x16 acc[S::kFM][S::kFN];
        const int live = min(max((t.rows - wm * S::kWaveM + 31) / 32, 0), S::kFM);
        tile_product<S, MxOp>(acc, lds, wm, wn, live, k0, k1, loads);
        if (slot < 0) {
#pragma unroll
            for (int i = 0; i < S::kFM; ++i) {
                if constexpr (EPI == MXEPI_NONE || EPI == MXEPI_F32) {
                    if (i * 32 < t.rows)
                        mx_store_rows<S, EPI>(acc[i], i, t, lds + (i & 1) * (S::WM * 32 * S::BN * 4), g);
                } else if (i < live) {
                    mx_store_hidden<S, EPI>(acc[i], i, t, g);
                }
            }
        } else {
            // rows past the segment's end stay unwritten
            float* dst = g.partial + (size_t)slot * S::kTileFloats;
#pragma unroll
            for (int i = 0; i < S::kFM; ++i)
                if (wm * S::kWaveM + i * 32 + (lane & 31) < t.rows)
#pragma unroll
                    for (int j = 0; j < S::kFN; ++j)
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            *reinterpret_cast<float4*>(
                                dst + ((((size_t)i * S::kWaves + wave) * S::kFN + j) * 4 + q) * 256 + lane * 4) =
                                make_float4(acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2],
                                            acc[i][j][4 * q + 3]);
        }
    }
#endif
}

// Second pass of the K split: block (split tile, row fragment) adds the parts in part
// order and runs the epilogue.  The loads of four parts leave together (one token of two
// experts, 64 tiles in four parts: 6.4 -> 5.1 us, a launch alone takes 2 to 3).  512 slots
// for 128 x 128 tiles, with twice the parts, were slower (one token's layers 50 -> 54 us).
template <typename S, int EPI>
__global__ __launch_bounds__(S::kThreads) void moe_mxfp4_tail_kernel(MxGemmArgs g, int G)
{
#if defined(__HIP_DEVICE_COMPILE__)
    __shared__ __attribute__((aligned(1024))) uint8_t buf[S::WM * 32 * S::BN * 4];
    __shared__ int32_t s_pref[kGemmMaxE + 1];
    __shared__ int32_t s_wsum[S::kWaves];
    const int lane = lane_id(), wave = threadIdx.x / kWave;
    const int tile_cols = EPI == MXEPI_SWIGLU ? S::kHalf : S::BN;
    const int ntn = (g.Nout + tile_cols - 1) / tile_cols;
    tile_prefix<S::kThreads>(g.offsets, g.E, g.max_rows, S::BM, ntn, s_pref, s_wsum);
    const int total = s_pref[g.E];
    const int parts = mx_parts(total, G, (g.K + kMxSlice - 1) / kMxSlice, true);
    if (parts <= 1)
        return;
    const int tail = total % G, full = total - tail;
    const int j = blockIdx.x / S::kFM, i = blockIdx.x % S::kFM;
    if (j >= tail)
        return;
    const TileDec t = decode_tile<S>(full + j, s_pref, g.offsets, g.E, g.max_rows, ntn, tile_cols);
    if (i * 32 >= t.rows)
        return;
    const bool live = (wave / S::WN) * S::kWaveM + i * 32 + (lane & 31) < t.rows;
    f32x16 acc[S::kFN];
#pragma unroll
    for (int n = 0; n < S::kFN; ++n)
#pragma unroll
        for (int v = 0; v < 16; ++v)
            acc[n][v] = 0.0f;
#pragma unroll 4
    for (int part = 0; part < (live ? parts : 0); ++part) {
        const float* src = g.partial + (size_t)(j * parts + part) * S::kTileFloats +
                           (size_t)(i * S::kWaves + wave) * S::kFN * 1024 + lane * 4;
#pragma unroll
        for (int n = 0; n < S::kFN; ++n)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float4 p = *reinterpret_cast<const float4*>(src + (n * 4 + q) * 256);
                acc[n][4 * q] += p.x;
                acc[n][4 * q + 1] += p.y;
                acc[n][4 * q + 2] += p.z;
                acc[n][4 * q + 3] += p.w;
            }
    }
    if constexpr (EPI == MXEPI_NONE || EPI == MXEPI_F32)
        mx_store_rows<S, EPI>(acc, i, t, buf, g);
    else
        mx_store_hidden<S, EPI>(acc, i, t, g);
#endif
}

}  // namespace moe

namespace {
using namespace moe;

constexpr int kMxCus = 256;  // of gfx950

// How a product is run: its tiles, and whether the last, partly filled round of them is
// split along K.
struct MxChoice {
    bool large, split;
    double us;
};

// Time in us on tiles of one shape, fitted to 118 sizes (1 to 2048 rows of 1 to 256 experts,
// K 512 to 14336, both kinds of layer).  A tile takes 3.5 or 7 us and, a slice, 0.45 to 1.32
// us (128 x 128) or 0.9 to 2.03 (256 x 256) with the share of its rows that exist and of
// the blocks that run at a time (where some CUs run two, they set the time); a split round
// takes 7 us more for its second launch; and no size is faster than its weights at 5.9
// TB/s.  Experts hold about max(1, mean / BM +
// 1/2) tiles of rows, for their rows are seldom even.  Measured, 128 x 128 / 256 x 256:
//   SwiGLU, 8 experts, 4096 x 4096     1 row  24 /  25    96  28 / 30    256  55 / 71    512   98 / 100   2048  359 / 305
//   plain, 8 experts, 14336 x 4096     8      41 /  48    96  53 / 61    256 108 / 112   512  178 / 183   2048  631 / 484
//   SwiGLU, 8 experts, 14336 x 4096    1      89 /  94    128 149 / 111  256 208 / 222   512  352 / 285
//   plain, 256 experts, 1024 x 512     8      17 /  19    96  24 / 27    256  42 /  45
// 64-, 96- and 128-row tiles of 256 columns were at best 10 % faster than the better of the
// two, at most sizes slower.
template <typename S>
MxChoice estimate(int E, int K, int Nout, bool glu, int max_rows, int mean_rows, bool split)
{
    const bool large = S::BM == 256;
    const int nk = (K + kMxSlice - 1) / kMxSlice, cols = glu ? S::kHalf : S::BN, busy = std::min(E, max_rows);
    const double mean = std::max(1, mean_rows);
    const double mt = busy == 1 ? (max_rows + S::BM - 1) / S::BM : mean < 0.8 * S::BM ? 1.0 : mean / S::BM + 0.5;
    const double tiles = busy * mt * ((Nout + cols - 1) / cols), slots = kMxCus * S::kPerCu, rows = std::min(1.0, mean / S::BM);
    auto time = [&](double slices, double blocks) {
        const double f = (blocks > kMxCus ? 1.0 : blocks / slots) * rows;
        return large ? 7.0 + slices * (0.9 + 1.13 * f) : 3.5 + slices * (0.45 + 0.87 * f);
    };
    const double rounds = std::floor(tiles / slots), rest = tiles - rounds * slots;
    double tail = rest > 0.5 ? time(nk, rest) : 0.0;
    const int parts = rest > 0.5 ? std::min(std::min(kMxMaxParts, (int)(kMxSplitSlots / rest)), nk / kMxMinPart) : 1;
    MxChoice c = {large, false, 0.0};
    if (split && parts > 1) {
        const double t = 7.0 + time((double)nk / parts, rest * parts);
        if (t < tail)
            tail = t, c.split = true;
    }
    const double weights = (double)busy * (glu ? 2 : 1) * Nout * K * (0.5 + 1.0 / kMxBlk);
    c.us = std::max(rounds * time(nk, slots) + tail, weights / 5.9e6);
    return c;
}

MxChoice choose(int E, int K, int Nout, bool glu, int max_rows, int mean_rows, bool split)
{
    const MxChoice l = estimate<LargeShape>(E, K, Nout, glu, max_rows, mean_rows, split);
    const MxChoice p = estimate<PairShape>(E, K, Nout, glu, max_rows, mean_rows, split);
    return l.us < 0.98 * p.us ? l : p;
}

template <typename S, int EPI>
hipError_t launch_shape(const MxGemmArgs& g, int ncu, hipStream_t stream)
{
    const int tile_cols = EPI == MXEPI_SWIGLU ? S::kHalf : S::BN;
    const long long ntn = (g.Nout + tile_cols - 1) / tile_cols;
    // upper bound on m-tiles: whole tiles plus one partial per expert
    const long long mt = g.max_rows / S::BM + (long long)std::min(g.E, g.max_rows);
    long long grid = ncu * S::kPerCu;
    if (mt * ntn < grid && g.partial == nullptr)
        grid = (mt * ntn + 7) / 8 * 8;
    moe_mxfp4_gemm_kernel<S, EPI><<<dim3((unsigned)grid), dim3(S::kThreads), 0, stream>>>(g);
    hipError_t err = hipGetLastError();
    if (err != hipSuccess || g.partial == nullptr)
        return err;
    moe_mxfp4_tail_kernel<S, EPI>
        <<<dim3(kMxSplitSlots / 2 * S::kFM), dim3(S::kThreads), 0, stream>>>(g, (int)grid);
    return hipGetLastError();
}

template <typename S>
hipError_t launch_epi(int epi, const MxGemmArgs& g, int ncu, hipStream_t s)
{
    if (epi == MXEPI_SWIGLU)
        return launch_shape<S, MXEPI_SWIGLU>(g, ncu, s);
    if (epi == MXEPI_RELU)
        return launch_shape<S, MXEPI_RELU>(g, ncu, s);
    return epi == MXEPI_F32 ? launch_shape<S, MXEPI_F32>(g, ncu, s) : launch_shape<S, MXEPI_NONE>(g, ncu, s);
}

template <typename ET>
void launch_quantize(const void* src, long long blocks, uint8_t* codes, uint8_t* scales, hipStream_t s)
{
    typedef typename ET::storage T;
    for (long long b = 0; b < blocks; b += 64 * kMxGrid) {
        const long long n = std::min(blocks - b, 64 * kMxGrid);
        moe_mxfp4_quantize_kernel<ET><<<dim3((unsigned)((n + 63) / 64)), dim3(256), 0, s>>>(
            (const T*)src + b * kMxBlk, n, codes + b * (kMxBlk / 2), scales + b);
    }
}

template <typename ET>
void launch_dequantize(const uint8_t* codes, const uint8_t* scales, long long blocks, void* dst, hipStream_t s)
{
    typedef typename ET::storage T;
    for (long long b = 0; b < blocks; b += 64 * kMxGrid) {
        const long long n = std::min(blocks - b, 64 * kMxGrid);
        moe_mxfp4_dequantize_kernel<ET><<<dim3((unsigned)((n + 63) / 64)), dim3(256), 0, s>>>(
            codes + b * (kMxBlk / 2), scales + b, n, (T*)dst + b * kMxBlk);
    }
}
}  // namespace

// src: blocks runs of 32 values (dtype 0 fp32, 1 bf16).
extern "C" hipError_t moe_launch_mxfp4_quantize(int dtype, const void* src, long long blocks, uint8_t* codes,
                                                uint8_t* scales, hipStream_t stream)
{
    if (blocks <= 0)
        return hipSuccess;
    dtype == 0 ? launch_quantize<f32_t>(src, blocks, codes, scales, stream)
               : launch_quantize<bf16_t>(src, blocks, codes, scales, stream);
    return hipGetLastError();
}

extern "C" hipError_t moe_launch_mxfp4_dequantize(int dtype, const uint8_t* codes, const uint8_t* scales,
                                                  long long blocks, void* dst, hipStream_t stream)
{
    if (blocks <= 0)
        return hipSuccess;
    dtype == 0 ? launch_dequantize<f32_t>(codes, scales, blocks, dst, stream)
               : launch_dequantize<bf16_t>(codes, scales, blocks, dst, stream);
    return hipGetLastError();
}

// Bytes of the partial tiles of a product whose last round is split along K (0: it is not).
// moe_launch_mxfp4_gemm chooses by the same sizes.
extern "C" size_t moe_mxfp4_gemm_partial_bytes(int E, int K, int Nout, int glu, int max_rows, int mean_rows)
{
    if (max_rows <= 0)
        return 0;
    const MxChoice c = choose(E, K, Nout, glu, max_rows, mean_rows, true);
    return c.split ? (size_t)kMxSplitSlots * 4 * (c.large ? LargeShape::kTileFloats : PairShape::kTileFloats) : 0;
}

// epi 0: Y = bf16 rows, 3: Y = fp32 rows; 1 ReLU, 2 SwiGLU: Hq, Hs.  mean_rows:
// expected rows per expert.  partial (nullable): the K split's workspace,
// moe_mxfp4_gemm_partial_bytes bytes.
extern "C" hipError_t moe_launch_mxfp4_gemm(int epi, const uint8_t* A, const uint8_t* As, const int32_t* gather,
                                            int gather_rows, const uint8_t* W, const uint8_t* Ws, uint8_t* Hq,
                                            uint8_t* Hs, void* Y, const int32_t* offsets, int E, int K, int Nw,
                                            int Nout, int F, int max_rows, int mean_rows, int ncu, float* partial,
                                            hipStream_t stream)
{
    const MxChoice c = choose(E, K, Nout, epi == MXEPI_SWIGLU, max_rows, mean_rows, partial != nullptr);
    const MxGemmArgs g = {A, As, gather, gather_rows, W, Ws, Hq, Hs, Y, offsets, E, K, Nw, Nout, F,
                          max_rows, c.split ? partial : nullptr};
    return c.large ? launch_epi<LargeShape>(epi, g, ncu, stream) : launch_epi<PairShape>(epi, g, ncu, stream);
}
