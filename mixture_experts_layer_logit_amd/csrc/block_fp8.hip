// Block-scaled FP8 experts (gfx950): quantisation to E4M3 codes with a scale
// for each block of 128 values, and the grouped GEMMs of the two expert
// layers on such codes.
//
// FP8 experts (Skywork-MoE model card: an FP8 checkpoint; news item
// "4090推理": FP8-quantised inference; Megatron-Core page, "关键特性": FP8
// among the coming features).  Activations carry one scale per 1 x 128 block
// of a row, weights one per 128 x 128 block of a matrix:
//   u[r, n] = sum_b sA[r, b] sW[n / 128, b] sum_{k in block b} a[r, k] w[n, k]
// Activation scales are E8M0 bytes (b stands for 2^(b - 127)); weight scales
// are E8M0 bytes or fp32 numbers.
#include <algorithm>
#include <type_traits>

#include "common.h"
#include "fp8.h"
#include "gemm_common.h"

namespace moe {

constexpr int kBlk = 128;  // values of K that share a scale, and rows of a weight block

// ---------------------------------------------------------------- quantisation
// Each block gets the smallest power-of-two scale s with max|block| <= 448 s,
// at least 2^-127 (s = 1 for an all-zero block), and each value the E4M3 code
// nearest to v / s (ties to even); v / s is exact, so every code is decided
// exactly.

// One scale as the E8M0 byte or the fp32 number.
template <bool F32>
__device__ __forceinline__ void store_scale(void* scales, size_t i, int e)
{
    if constexpr (F32)
        static_cast<float*>(scales)[i] = ldexpf(1.0f, e);
    else
        static_cast<uint8_t*>(scales)[i] = (uint8_t)(e + 127);
}

// The most workgroups of a quantising launch (a launch has fewer than 2^32
// threads); larger inputs take several.
constexpr long long kQuantGrid = 1 << 23;

// 1 x 128 blocks: 16 lanes of 8 values each per block, the blocks of all rows
// in one run (K is a multiple of 128).  Bound by memory: 8192 x 4608 bf16 in
// 21 us, 5.4 TB/s, and the 8 x 4096 of a decoding batch by its launch.
template <typename ET, bool F32>
__global__ __launch_bounds__(256) void moe_quantize_rows_kernel(const typename ET::storage* __restrict__ src,
                                                                long long blocks, uint8_t* __restrict__ codes,
                                                                void* __restrict__ scales)
{
    const long long b = (long long)blockIdx.x * 16 + threadIdx.x / 16;
    if (b >= blocks)
        return;
    const size_t at = (size_t)b * kBlk + 8 * (threadIdx.x % 16);
    float f[8], amax = 0.0f;
    load8(src + at, f);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        amax = fmaxf(amax, fabsf(f[i]));
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1)
        amax = fmaxf(amax, __shfl_xor(amax, o));
    const int e = fp8_block_scale_exp(amax);
    *reinterpret_cast<uint2*>(codes + at) = e4m3_encode8(f, e);
    if (threadIdx.x % 16 == 0)
        store_scale<F32>(scales, (size_t)b, e);
}

// 128 x 128 blocks, one per workgroup (the last block row may be shorter):
// thread t takes 8 columns of rows t / 16, t / 16 + 16, ..., held in registers
// between the maximum and the codes, so memory is crossed once (57344 x 4096
// fp32 in 200 us, 5.9 TB/s).
template <typename ET, bool F32>
__global__ __launch_bounds__(256) void moe_quantize_tiles_kernel(const typename ET::storage* __restrict__ src,
                                                                 long long R, int K, uint8_t* __restrict__ codes,
                                                                 void* __restrict__ scales)
{
    __shared__ float s_max[4];
    const int nkb = K / kBlk;
    const long long br = blockIdx.x / nkb;
    const int bc = blockIdx.x % nkb;
    const long long r0 = br * kBlk;
    const size_t col = (size_t)bc * kBlk + 8 * (threadIdx.x % 16);
    float f[8][8], amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const long long r = r0 + threadIdx.x / 16 + 16 * i;
        load8(src + (size_t)min(r, R - 1) * K + col, f[i]);
#pragma unroll
        for (int q = 0; q < 8; ++q)
            amax = fmaxf(amax, r < R ? fabsf(f[i][q]) : 0.0f);
    }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1)
        amax = fmaxf(amax, __shfl_xor(amax, o));
    if (lane_id() == 0)
        s_max[threadIdx.x / kWave] = amax;
    __syncthreads();
    amax = fmaxf(fmaxf(s_max[0], s_max[1]), fmaxf(s_max[2], s_max[3]));
    const int e = fp8_block_scale_exp(amax);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const long long r = r0 + threadIdx.x / 16 + 16 * i;
        if (r < R)
            *reinterpret_cast<uint2*>(codes + (size_t)r * K + col) = e4m3_encode8(f[i], e);
    }
    if (threadIdx.x == 0)
        store_scale<F32>(scales, (size_t)blockIdx.x, e);
}

// ---------------------------------------------------------------- grouped GEMM
// Rows of expert e's segment times its weight matrix.  Block tile BM x BN, WM x WN
// wavefronts, K in slices of 128 values (one scale block), each slice loaded from
// memory straight into one of S LDS stages.  The 256 weight rows of a tile are two
// halves of 128: for SwiGLU the gate rows and the matching up rows of 128 hidden
// columns, else 256 consecutive rows; each half lies in one row of weight blocks,
// so a tile has two weight scales per slice.  A wavefront takes the same rows of
// both halves, so the gate and up values of a hidden column meet in one lane.
// (Where tiles are few, 128 weight rows, two halves of 64 under one scale.)
//
// MFMA 32x32x64 f8f6f4 with block scales: lane l holds 32 consecutive K
// values of operand row l % 32 (the half l / 32 of the 64) and the E8M0 byte
// that scales them, so the matrix core applies both scales of a block to the
// products itself.  The weight tile is its first operand, the activation tile
// its second: a lane's accumulators are 4 consecutive columns of one row.
enum { BEPI_NONE = 0, BEPI_RELU = 1, BEPI_SWIGLU = 2, BEPI_F32 = 3 };  // bf16 rows, hidden codes (2), fp32 rows

constexpr int kBlkMaxParts = 16;     // K parts of a tail tile
constexpr int kBlkSplitSlots = 256;  // partial tiles the workspace holds
constexpr int kBlkMinPart = 4;       // K slices of a part
[[maybe_unused]] constexpr int kBlkMaxSlices = 512;   // K <= 65536

template <int BM_, int WM_, int WN_, int S_, int GM_, int BN_ = 256, int PER_CU_ = 1>
struct BlockShape {
    static constexpr int BM = BM_, BN = BN_, kHalf = BN / 2, kPerCu = PER_CU_;
    static constexpr int WM = WM_, WN = WN_, S = S_, GM = GM_, RB = 128;
    static constexpr int kWaves = WM * WN, kThreads = kWaves * kWave;
    static constexpr int kWavesPerSimd = kWaves / 4 * kPerCu;
    static constexpr int kWaveM = BM / WM, kWaveN = BN / WN;
    static constexpr int kFM = kWaveM / 32, kFN = kWaveN / 32;
    static constexpr int kRows = 1024 / RB;  // tile rows of a 1 KB load
    static constexpr int kLdsA = BM * RB, kLdsW = BN * RB;
    // Scales of the stage's activation rows, a dword each.  Each wavefront loads 64
    // rows' (none behind row BM); where two blocks have to fit a CU, the others
    // load the same rows' into the same place (as the 256-row tile's second four
    // wavefronts that would cost 4 %).
    static constexpr int kSclWaves = kPerCu > 1 ? BM / kWave : kWaves;
    static constexpr int kScl = kSclWaves * kWave * 4;
    static constexpr int kStage = kLdsA + kLdsW + kScl;
    static constexpr int kBlkA = BM / kRows / kWaves, kBlkW = BN / kRows / kWaves;  // loads per wavefront and stage
    static constexpr int kLoads = kBlkA + kBlkW + 1;
    static constexpr int kTileFloats = BM * BN;
    static_assert(kFN % 2 == 0, "a wavefront takes rows of both weight halves");
    static_assert(kWaves % 4 == 0 && BM % (kRows * kWaves) == 0 && kThreads >= BM, "loads split evenly");
    static_assert(kBlkW % 2 == 0, "a load lies in one weight half");
    static_assert(S >= 2 && (S - 1) * kLoads <= 63, "vmcnt range");
    static_assert(2 * (WM * 32) * BN * 4 <= S * kStage, "two staged row fragments fit the stages");
};

struct BlockGemmArgs {
    const uint8_t* A;       // codes of the activation rows [.][K]
    const uint8_t* As;      // their scales [.][K / 128]
    const int32_t* gather;  // nullable: row r is A's row gather[r] of gather_rows
    int gather_rows;
    const uint8_t* W;  // [E][Nw][K]
    const void* Ws;    // [E][Nw / 128][K / 128]
    uint8_t* Hq;       // codes of the hidden rows [.][Nout] (activation epilogues)
    uint8_t* Hs;       // their scales [.][Nout / 128]
    void* Y;           // bf16 or fp32 rows [.][Nout] (plain epilogues)
    const int32_t* offsets;
    int E, K, Nw, Nout, F, max_rows;
    float* partial;  // nullable: no K split
};

// LDS offset of 16-byte chunk c of tile row `row`: the chunk index XOR-ed with
// the row pair's number (two rows fill the 64 banks once), so that one chunk of
// 16 consecutive rows touches every bank once.
template <typename S>
__device__ __forceinline__ int bswz_term(int row)
{
    return (row >> 1) & 7;
}
template <typename S>
__device__ __forceinline__ uint32_t bswz(int row, int c)
{
    return row * S::RB + ((c ^ bswz_term<S>(row)) << 4);
}

// One dword per lane from a byte of buffer `rsrc` at voff + soff, zero
// extended, into LDS at byte address lds + 4 * lane (see dma16).
__device__ __forceinline__ void dma_byte(const i32x4& rsrc, uint32_t lds, uint32_t voff, uint32_t soff)
{
    const uint32_t m0 = __builtin_amdgcn_readfirstlane(lds);
    uint32_t so = __builtin_amdgcn_readfirstlane(soff);
    __asm__("" : "+s"(so));
    __asm__ volatile("s_mov_b32 m0, %0\n\tbuffer_load_ubyte %1, %2, %3 offen lds"
                     :
                     : "s"(m0), "v"(voff), "s"(rsrc), "s"(so)
                     : "memory");
}

__device__ __forceinline__ int block_parts(int total, int G, int nk, bool enabled)
{
    const int tail = total % G;
    if (!enabled || tail == 0)
        return 1;
    return max(1, min(min(kBlkMaxParts, min(G, kBlkSplitSlots) / tail), nk / kBlkMinPart));
}

// silu(u) v, silu(u) = u / (1 + e^-u); the exponential and the reciprocal to
// within a step or two of fp32, which the E4M3 code behind them does not see.
__device__ __forceinline__ float glu(float u, float v)
{
    return u * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(u * -1.44269504088896341f)) * v;
}

// Epilogue of row fragment i of every wavefront (WM bands of 32 rows), whose
// accumulators are acc[0 .. kFN): staged in LDS as [band row][column] (16-byte
// chunks XOR-swizzled by the row), then taken row by row.  Activation
// epilogues: fp32 h is quantised as it is, without a rounding to bf16 in
// between, block by block; a block's 128 values are spread over a few lanes of
// one wavefront.
template <typename S, int EPI>
__device__ __forceinline__ void block_store(const f32x16 (&acc)[S::kFN], int i, const TileDec& t, uint8_t* buf,
                                            const BlockGemmArgs& g)
{
    constexpr bool kGlu = EPI == BEPI_SWIGLU;
    constexpr bool kRows32 = EPI == BEPI_F32, kPlain = EPI == BEPI_NONE || kRows32;
    static_assert(S::BN == 256 || !kGlu, "h is stored by whole blocks");
    constexpr int HC = kGlu ? 128 : S::BN;  // output columns of the tile
    constexpr int kRows = S::WM * 32;
    constexpr int kEl = EPI == BEPI_NONE ? 2 : 4;
    constexpr int kRowBytes = HC * kEl;
    constexpr int kSwz = kRowBytes / 16 - 1 < 31 ? kRowBytes / 16 - 1 : 31;
    int tid = threadIdx.x;
    __asm__ volatile("" : "+v"(tid));
    const int lane = tid & (kWave - 1), wave = tid / kWave;
    const int wm = wave / S::WN, wn = wave % S::WN;
    const int r = wm * 32 + (lane & 31);
#pragma unroll
    for (int j = 0; j < (kGlu ? S::kFN / 2 : S::kFN); ++j)
#pragma unroll
        for (int g4 = 0; g4 < 4; ++g4) {
            constexpr int kHalfN = S::kWaveN / 2, kHalfF = S::kFN / 2;
            const int col = (j / kHalfF) * S::kHalf + wn * kHalfN + (j % kHalfF) * 32 + 8 * g4 + 4 * (lane >> 5);
            float v[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float u = acc[j][4 * g4 + q];
                if constexpr (kGlu)
                    v[q] = glu(u, acc[j + kHalfF][4 * g4 + q]);
                else if constexpr (EPI == BEPI_RELU)
                    v[q] = u <= 0.0f ? 0.0f : u;  // a NaN stays one
                else
                    v[q] = u;
            }
            const int byte = col * kEl;
            uint8_t* dst = buf + r * kRowBytes + (((byte >> 4) ^ (r & kSwz)) << 4) + (byte & 15);
            if constexpr (kEl == 2) {
                typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
                *reinterpret_cast<bf16x4*>(dst) = __builtin_convertvector(f32x4{v[0], v[1], v[2], v[3]}, bf16x4);
            } else {
                *reinterpret_cast<float4*>(dst) = make_float4(v[0], v[1], v[2], v[3]);
            }
        }
    lds_barrier();
    if constexpr (kPlain) {
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
    } else {
        constexpr int kPer = S::kThreads / kRows;  // threads of a row
        constexpr int V = HC / kPer;               // consecutive values of a thread
        constexpr int kLanes = kBlk / V;           // lanes of a block
        const int rr = tid / kPer, part = tid % kPer;
        const int m = (rr / 32) * S::kWaveM + i * 32 + (rr % 32);
        const int n = t.n0 + part * V;
        float f[V], amax = 0.0f;
#pragma unroll
        for (int c = 0; c < V / 4; ++c) {
            const int q = part * (V / 4) + c;
            const float4 x = *reinterpret_cast<const float4*>(buf + rr * kRowBytes + ((q ^ (rr & kSwz)) << 4));
            f[4 * c] = x.x;
            f[4 * c + 1] = x.y;
            f[4 * c + 2] = x.z;
            f[4 * c + 3] = x.w;
            amax = fmaxf(fmaxf(amax, fmaxf(fabsf(x.x), fabsf(x.y))), fmaxf(fabsf(x.z), fabsf(x.w)));
        }
#pragma unroll
        for (int o = kLanes / 2; o >= 1; o >>= 1)
            amax = fmaxf(amax, __shfl_xor(amax, o));
        const int e = fp8_block_scale_exp(amax);
        if (m < t.rows && n < g.Nout) {
            uint8_t* out = g.Hq + (size_t)(t.row0 + m) * g.Nout + n;
#pragma unroll
            for (int c = 0; c < V / 16; ++c) {
                const uint2 lo = e4m3_encode8(f + 16 * c, e), hi = e4m3_encode8(f + 16 * c + 8, e);
                *reinterpret_cast<uint4*>(out + 16 * c) = make_uint4(lo.x, lo.y, hi.x, hi.y);
            }
            if (part % kLanes == 0)
                g.Hs[(size_t)(t.row0 + m) * (g.Nout / kBlk) + n / kBlk] = (uint8_t)(e + 127);
        }
    }
}

template <typename S, int EPI, bool WF32>
__global__ __launch_bounds__(S::kThreads) __attribute__((amdgpu_waves_per_eu(S::kWavesPerSimd, S::kWavesPerSimd)))
void moe_block_gemm_kernel(BlockGemmArgs g)
{
#if defined(__HIP_DEVICE_COMPILE__)  // the body uses device-only types; the host pass needs the stub only
    __shared__ __attribute__((aligned(1024))) uint8_t lds[S::S * S::kStage];
    __shared__ uint32_t s_ws[S::BN / kBlk][kBlkMaxSlices];  // the tile's weight scales
    __shared__ int32_t s_pref[kGemmMaxE + 1];
    __shared__ int32_t s_wsum[S::kWaves];
    const int tid = threadIdx.x;
    const int lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int wm = wave / S::WN, wn = wave % S::WN;
    const int K = g.K, nk = K / kBlk;
    const uint32_t lds0 = lds_addr(lds);
    constexpr int kHalfN = S::kWaveN / 2, kHalfF = S::kFN / 2;
    // LDS offsets of this lane's first fragments in a stage; the k-step and the
    // 16-byte half flip single bits of them, fragments 32 rows apart keep their
    // swizzle
    const uint32_t rdA = bswz<S>(wm * S::kWaveM + (lane & 31), 2 * (lane >> 5));
    const uint32_t rdW = S::kLdsA + bswz<S>(wn * kHalfN + (lane & 31), 2 * (lane >> 5));
    const uint32_t rdS = S::kLdsA + S::kLdsW + 4 * (wm * S::kWaveM + (lane & 31));

    const int tile_cols = EPI == BEPI_SWIGLU ? 128 : S::BN;
    const int ntn = (g.Nout + tile_cols - 1) / tile_cols;
    tile_prefix<S::kThreads>(g.offsets, g.E, g.max_rows, S::BM, ntn, s_pref, s_wsum);
    const int total = s_pref[g.E];
    const int G = gridDim.x;
    const int parts = block_parts(total, G, nk, g.partial != nullptr);
    const int full = parts > 1 ? total - total % G : total;
    const int tail = total - full;
    const int items = full + tail * parts;

    for (int base = 0; base < items; base += G) {
        const int b = blockIdx.x;
        // an XCD's blocks side by side; with two blocks a CU a round that is not
        // full is spread over all XCDs (half a round 39.5 -> 25.7 us; with one block
        // a CU no difference, and scalar registers that the 256-row tile lacks)
        const int each = S::kPerCu > 1 ? (min(G, items - base) + 7) / 8 : G / 8;
        const int item = (G % 8 == 0) ? base + (b % 8) * each + b / 8 : base + b;
        if (item >= items || (S::kPerCu > 1 && G % 8 == 0 && b / 8 >= each))
            continue;
        int tile = item, k0 = 0, k1 = nk, slot = -1;
        if (item >= full) {
            const int j = item - full, part = j / tail;
            tile = full + j % tail;
            k0 = part * nk / parts;
            k1 = (part + 1) * nk / parts;
            slot = (j % tail) * parts + part;
        }
        const TileDec t = decode_tile<S>(tile, s_pref, g.offsets, g.E, g.max_rows, ntn, tile_cols);

        // lane's place in a 1 KB load of kRows rows: row lane / kCh, physical
        // chunk lane % kCh; the swizzle term is the same in all of a
        // wavefront's loads (their row blocks all have the parity of its number)
        constexpr int kCh = S::RB / 16;
        const int lrow = S::kRows * wave + lane / kCh;
        const uint32_t lchunk = (uint32_t)((lane % kCh) ^ bswz_term<S>(lrow)) * 16;
        i32x4 rsA, rsS;
        uint32_t voffA[S::kBlkA], voffS;
        const int srow = wave % S::kSclWaves * kWave + lane;  // the tile row whose scale this lane loads
        if (g.gather) {
            rsA = make_rsrc(g.A, (uint32_t)g.gather_rows * (uint32_t)K);
            rsS = make_rsrc(g.As, (uint32_t)g.gather_rows * (uint32_t)nk);
            auto source = [&](int r) {
                const int src = r < t.rows ? g.gather[t.row0 + r] : -1;
                return src < g.gather_rows ? src : -1;
            };
#pragma unroll
            for (int i = 0; i < S::kBlkA; ++i) {
                const int src = source(lrow + S::kRows * S::kWaves * i);
                voffA[i] = src >= 0 ? (uint32_t)src * (uint32_t)K + lchunk : 0xf0000000u;
            }
            const int src = source(srow);
            voffS = src >= 0 ? (uint32_t)src * (uint32_t)nk : 0xf0000000u;
        } else {
            rsA = make_rsrc(g.A + (size_t)t.row0 * K, (uint32_t)t.rows * (uint32_t)K);
            rsS = make_rsrc(g.As + (size_t)t.row0 * nk, (uint32_t)t.rows * (uint32_t)nk);
#pragma unroll
            for (int i = 0; i < S::kBlkA; ++i)
                voffA[i] = (uint32_t)(lrow + S::kRows * S::kWaves * i) * (uint32_t)K + lchunk;
            voffS = srow < t.rows ? (uint32_t)srow * (uint32_t)nk : 0xf0000000u;
        }
        // the weight rows' offsets: one lane part, and a scalar part per load;
        // the second half of the last tile may lie behind the matrix
        const i32x4 rsW = make_rsrc(g.W + (size_t)t.e * g.Nw * K, (uint32_t)g.Nw * (uint32_t)K);
        const uint32_t voffW = (uint32_t)lrow * (uint32_t)K + lchunk;
        const uint32_t half1 = EPI == BEPI_SWIGLU ? (uint32_t)(g.F + t.n0) : (uint32_t)(t.n0 + S::kHalf);
        const bool second = EPI == BEPI_SWIGLU || (int)half1 < g.Nw;
        const uint32_t voffW1 = second ? voffW : 0xf0000000u, row0 = (uint32_t)t.n0 * (uint32_t)K;
        const uint32_t row1 = second ? half1 * (uint32_t)K : 0, step = S::kRows * S::kWaves * (uint32_t)K;
        // Small tiles, which stream weights: every tile of columns starts at
        // another slice.  Where rows lie a multiple of 2048 bytes apart, blocks
        // that all read the same slice at a time meet in few of the memory's
        // channels (weights 4096 wide, 8 experts, 16 rows: 202 -> 166 us, 4.65 ->
        // 5.67 TB/s; 6144, 8192 and 12288 wide 13 to 30 % faster; 14336 wide no
        // difference; 2048, 2560 and 3584 wide 3 to 6 % slower, left alone).  The
        // tile decides, so the sums keep their order from run to run.
        constexpr bool kRotate = S::kWaves == 4;
        int rot = 0;
        if (kRotate && K >= 4096 && K % 2048 == 0)
            rot = (t.n0 / tile_cols * 5) % (k1 - k0);
        auto slice_of = [&](int q) {
            if constexpr (kRotate)
                return q + rot >= k1 ? q + rot - (k1 - k0) : q + rot;
            else
                return q;
        };

        // Loads [n0, n1) of the kLoads of slice number q into LDS stage st.
        // Weights, which come from farthest away, then scales, then activations;
        // the half behind the matrix's last row reads behind the buffer: zeros.
        auto issue = [&](int q, int st, int n0, int n1) {
            const uint32_t at = lds0 + st * S::kStage, dst = at + wave * 1024;
            const uint32_t kb = (uint32_t)slice_of(q), soff = kb * S::RB;
#pragma unroll
            for (int p = 0; p < S::kLoads; ++p) {
                if (p < n0 || p >= n1)
                    continue;
                if (p < S::kBlkW / 2)
                    dma16(rsW, dst + S::kLdsA + S::kWaves * p * 1024, voffW, soff + row0 + p * step);
                else if (p < S::kBlkW)
                    dma16(rsW, dst + S::kLdsA + S::kWaves * p * 1024, EPI == BEPI_SWIGLU ? voffW : voffW1,
                          soff + row1 + (p - S::kBlkW / 2) * step);
                else if (p == S::kBlkW)
                    dma_byte(rsS, at + S::kLdsA + S::kLdsW + wave % S::kSclWaves * 256, voffS, kb);
                else
                    dma16(rsA, dst + S::kWaves * (p - S::kBlkW - 1) * 1024, voffA[p > S::kBlkW ? p - S::kBlkW - 1 : 0],
                          soff);
            }
        };
        auto load_weight_scales = [&]() {
            const size_t brow = (size_t)t.e * (g.Nw / kBlk);
            const int c0 = t.n0 / kBlk;
            const int c1 = EPI == BEPI_SWIGLU ? (g.F + t.n0) / kBlk : min((t.n0 + S::kHalf) / kBlk, g.Nw / kBlk - 1);
            for (int q = tid; q < S::BN / kBlk * (k1 - k0); q += S::kThreads) {
                const int h = q >= k1 - k0, kb = k0 + q - (h ? k1 - k0 : 0);
                const size_t at = (brow + (h ? c1 : c0)) * nk + kb;
                if constexpr (WF32)
                    s_ws[h][kb] = __float_as_uint(static_cast<const float*>(g.Ws)[at]);
                else
                    s_ws[h][kb] = static_cast<const uint8_t*>(g.Ws)[at];
            }
        };

        f32x16 acc[S::kFM][S::kFN];
#pragma unroll
        for (int i = 0; i < S::kFM; ++i)
#pragma unroll
            for (int j = 0; j < S::kFN; ++j)
#pragma unroll
                for (int v = 0; v < 16; ++v)
                    acc[i][j][v] = 0.0f;

        wait_vmcnt<0>();  // the previous tile's stores are out of the count
        __syncthreads();  // and every wave is done with its LDS
        load_weight_scales();
#pragma unroll
        for (int q = 0; q < S::S; ++q)
            if (k0 + q < k1)
                issue(k0 + q, q, 0, S::kLoads);
        if (k1 - k0 >= S::S)
            wait_vmcnt<(S::S - 1) * S::kLoads>();
        else
            wait_vmcnt<0>();
        lds_barrier();

        struct Frags {
            i32x8 w[S::kFN], a[S::kFM];
        };
        // The K loop for a wavefront whose first L row fragments hold rows of the
        // segment (the others are neither read nor multiplied).  A slice takes two
        // k-steps of 64 values.  In the first, the second's fragments are read as
        // fast as the LDS gives them; behind a barrier the stage is free then and
        // takes the loads of slice kt + S, weights first.  Between the two k-steps
        // slice kt + 1 has to be there (a second barrier).  So a load has 1 1/4
        // slices (S = 2) to arrive.  Against one barrier between the k-steps and a
        // load time of one slice, 8 wavefronts of 128 x 64 each, same card: 16
        // experts of 512 rows 915 -> 845 us, one of 8192 rows 790 -> 793 us (4096 x
        // 28672 weights; the weights of one expert stay in the caches).  Loads
        // spread over fewer MFMAs, all behind the second barrier or half of them in
        // the next slice, 64-byte slices in four stages, and touching the weight
        // lines two slices ahead were slower by 2 to 15 %; so were flags in LDS in
        // place of the barriers, and 4 wavefronts of 128 x 128 each.
        auto kloop = [&](auto lc) {
            constexpr int L = decltype(lc)::value;
            constexpr int NM = L * S::kFN, NR = L > 0 ? 2 * (L + S::kFN) : 0;
            Frags f0, f1;
            int sa[S::kFM], sw[2], swn[2];
            auto read = [&](int r, Frags& nx, uint32_t st, int kk) {
                const int n = r / 2, h = r % 2;  // fragment, 16-byte half
                const uint32_t x = (uint32_t)(kk * 64) ^ (uint32_t)(h * 16);
                const i32x4 v = *reinterpret_cast<const i32x4*>(
                    lds + st + (n < S::kFN ? (rdW ^ x) + ((n / kHalfF) * S::kHalf + (n % kHalfF) * 32) * S::RB
                                           : (rdA ^ x) + (n - S::kFN) * 32 * S::RB));
                i32x8& dst = n < S::kFN ? nx.w[n] : nx.a[n - S::kFN];
                if (h)
                    dst.hi = v;
                else
                    dst.lo = v;
            };
            auto read_scale = [&](int i, uint32_t st) {
                sa[i] = *reinterpret_cast<const int*>(lds + st + rdS + i * 128);
            };
            // One k-step (64 values of K): the MFMAs on the fragments in f, and
            // between them the LDS reads of the next k-step's fragments into nx
            // (k-step kk of stage st) and, where LAST, the row scales of the next
            // slice; where LOADS, the loads of slice q into stage lst.  An MFMA runs
            // for 64 cycles, in which its wavefront can issue the few instructions
            // that follow it.
            constexpr int kEarly = S::kBlkW;                       // loads issued in a slice's first k-step: the weights'
            constexpr int kFree = NM >= 8 ? 3 : NM > 2 ? NM / 2 : NM;  // MFMAs behind which its reads are spread
            constexpr int kBar = NM >= 8 ? 3 : NM > 0 ? kFree - 1 : 0;  // the one behind which the stage is free
            auto kstep = [&](const Frags& f, Frags& nx, uint32_t st, int kk, auto last, auto loads, int q, int lst) {
                constexpr bool LAST = decltype(last)::value, LOADS = decltype(loads)::value;
                // reads behind an MFMA
                constexpr int kOver = LAST ? NM : kFree;
                constexpr int kPer = kOver > 0 && (NR + kOver - 1) / kOver > 2 ? (NR + kOver - 1) / kOver : 2;
                if constexpr (NM == 0) {
                    if (!LAST && LOADS)
                        lds_barrier();
                    if (LOADS)
                        issue(q, lst, LAST ? kEarly : 0, LAST ? S::kLoads : kEarly);
                }
#pragma unroll
                for (int m = 0; m < NM; ++m) {
                    const int i = m / S::kFN, j = m % S::kFN;
                    if constexpr (WF32) {
                        f32x16 z = {0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
                        z = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(f.w[j], f.a[i], z, 0, 0, 0, 127, 0, sa[i]);
                        const float s = __int_as_float(sw[j / kHalfF]);
#pragma unroll
                        for (int v = 0; v < 16; ++v)
                            acc[i][j][v] = fmaf(s, z[v], acc[i][j][v]);
                    } else {
                        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(f.w[j], f.a[i], acc[i][j], 0, 0,
                                                                                    0, sw[j / kHalfF], 0, sa[i]);
                    }
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int r = 0; r < NR; ++r)
                        if (r / kPer == m)
                            read(r, nx, st, kk);
                    if constexpr (LAST) {
                        if (j == S::kFN - 1)
                            read_scale(i, st);
                        constexpr int kLate = S::kLoads - kEarly, kSafe = NM > 0 ? NM : 1;
                        if constexpr (LOADS)
                            issue(q, lst, kEarly + m * kLate / kSafe, kEarly + (m + 1) * kLate / kSafe);
                    } else if constexpr (LOADS) {
                        // every wavefront's reads of the stage are done: it is free
                        if (m == kBar)
                            lds_barrier();
                        if (m >= kBar) {
                            constexpr int kLeft = NM - kBar > 0 ? NM - kBar : 1;
                            issue(q, lst, (m - kBar) * kEarly / kLeft, (m - kBar + 1) * kEarly / kLeft);
                        }
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
            };
            constexpr std::integral_constant<bool, false> no{};
            constexpr std::integral_constant<bool, true> yes{};
            // in the order of the loop's own reads: the waits at its head are the
            // stricter of the two
            sw[0] = s_ws[0][slice_of(k0)];
            sw[1] = s_ws[S::BN / kBlk - 1][slice_of(k0)];
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int m = 0; m < NM; ++m) {
                constexpr int kPer = (NR + NM - 1) / (NM > 0 ? NM : 1) > 2 ? (NR + NM - 1) / (NM > 0 ? NM : 1) : 2;
#pragma unroll
                for (int r = 0; r < NR; ++r)
                    if (r / kPer == m)
                        read(r, f0, 0, 0);
                if (m % S::kFN == S::kFN - 1)
                    read_scale(m / S::kFN, 0);
                __builtin_amdgcn_sched_barrier(0);
            }
            int cur = 0;  // stage of slice kt
            auto slice = [&](int kt, auto loads) {
                constexpr bool LOADS = decltype(loads)::value;
                const int nxt = cur + 1 == S::S ? 0 : cur + 1;
                kstep(f0, f1, cur * S::kStage, 1, no, loads, kt + S::S, cur);
                // slice kt + 1 has to be there
                wait_vmcnt<LOADS ? (S::S - 2) * S::kLoads + kEarly : 0>();
                lds_barrier();
                const int sn = slice_of(min(kt + 1, k1 - 1));
                swn[0] = s_ws[0][sn];
                swn[1] = s_ws[S::BN / kBlk - 1][sn];
                kstep(f1, f0, nxt * S::kStage, 0, yes, loads, kt + S::S, cur);
                sw[0] = swn[0];
                sw[1] = swn[1];
                cur = nxt;
            };
            int kt = k0;
            for (; kt + S::S < k1; ++kt)
                slice(kt, yes);
            for (; kt < k1; ++kt)  // nothing is left to load
                slice(kt, no);
        };
        // rows past the segment's end are not stored: a wavefront leaves out the
        // fragments that hold none (a copy of the loop for each count)
        const int live = min(max((t.rows - wm * S::kWaveM + 31) / 32, 0), S::kFM);
        if (S::kFM == 1 || live == S::kFM)
            kloop(std::integral_constant<int, S::kFM>{});
        else if (S::kFM > 3 && live == 3)
            kloop(std::integral_constant<int, (S::kFM > 3 ? 3 : 1)>{});
        else if (S::kFM > 2 && live == 2)
            kloop(std::integral_constant<int, (S::kFM > 2 ? 2 : 1)>{});
        else if (live == 1)
            kloop(std::integral_constant<int, 1>{});
        else
            kloop(std::integral_constant<int, 0>{});
        lds_barrier();
        if (slot < 0) {
#pragma unroll
            for (int i = 0; i < S::kFM; ++i)
                if (i * 32 < t.rows)
                    block_store<S, EPI>(acc[i], i, t, lds + (i & 1) * (S::WM * 32 * S::BN * 4), g);
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

// Second pass of the K split: block (split tile, row fragment) adds the parts
// in part order and runs the epilogue.
template <typename S, int EPI>
__global__ __launch_bounds__(S::kThreads) void moe_block_tail_kernel(BlockGemmArgs g, int G)
{
#if defined(__HIP_DEVICE_COMPILE__)
    __shared__ __attribute__((aligned(1024))) uint8_t buf[S::WM * 32 * S::BN * 4];
    __shared__ int32_t s_pref[kGemmMaxE + 1];
    __shared__ int32_t s_wsum[S::kWaves];
    const int lane = lane_id(), wave = threadIdx.x / kWave;
    const int tile_cols = EPI == BEPI_SWIGLU ? 128 : S::BN;
    const int ntn = (g.Nout + tile_cols - 1) / tile_cols;
    tile_prefix<S::kThreads>(g.offsets, g.E, g.max_rows, S::BM, ntn, s_pref, s_wsum);
    const int total = s_pref[g.E];
    const int parts = block_parts(total, G, g.K / kBlk, true);
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
    for (int part = 0; live && part < parts; ++part) {
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
    block_store<S, EPI>(acc, i, t, buf, g);
#endif
}

// ---------------------------------------------------------------- combine
// y[t] = sum over the kept choices j, in order, of topk_w[t,j] * rows[slot[t,j]]
// in fp32, rounded to bf16 once: the layer keeps the expert outputs in fp32, so
// that y has one rounding (rounded to bf16 on the way they put its error at 1.55
// times that; the rows' traffic is 2 % of a prompt layer's time).  A thread takes
// 8 columns of a token; the loads of all its choices leave together.  Slots
// outside [0, max_rows) are dropped choices.
template <int KMAX>
__global__ __launch_bounds__(256) void moe_combine_rows_kernel(const float* __restrict__ rows,
                                                               const int32_t* __restrict__ slot,
                                                               const float* __restrict__ topk_w, int T, int d, int k,
                                                               int max_rows, uint16_t* __restrict__ y)
{
    const long long at = (long long)blockIdx.x * 256 + threadIdx.x;
    const int per = d / 8;
    const int t = (int)(at / per), c = (int)(at % per) * 8;
    if (t >= T)
        return;
    float f[KMAX][8], w[KMAX];
#pragma unroll
    for (int j = 0; j < KMAX; ++j) {
        const int s = j < k ? slot[(size_t)t * k + j] : -1;
        const bool kept = s >= 0 && s < max_rows;
        w[j] = kept ? topk_w[(size_t)t * k + j] : 0.0f;
        if (kept) {
            load8(rows + (size_t)s * d + c, f[j]);
        } else {
#pragma unroll
            for (int q = 0; q < 8; ++q)
                f[j][q] = 0.0f;
        }
    }
    float acc[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        acc[q] = 0.0f;
#pragma unroll
        for (int j = 0; j < KMAX; ++j)
            acc[q] = fmaf(w[j], f[j][q], acc[q]);
    }
    store8(y + (size_t)t * d + c, acc);
}

}  // namespace moe

namespace {
using namespace moe;

// Tiles, picked by the mean rows per expert, which the host knows without
// reading the offsets (16 experts, SwiGLU 4096 x 4096, up / down in us):
//   rows     64-row tile   96-row      128-row     256-row
//     40       104 / 56   105 / 57    134 / 69    137 / 71
//     72       124 / 68   109 / 60    133 / 71    139 / 73
//    160       173 / 89   144 / 76    152 / 80    148 / 79
//    256       255 / 131  199 / 101   187 / 106   179 / 112
//    512       456 / 221  355 / 177   323 / 165   270 / 148
// The 96-row tile below 192 rows, the 256-row one from there on, but the 96-row or
// else the 128-row one where all of its tiles, however the rows are spread, find
// a CU each (SwiGLU, one expert of 2048 rows, 2048 x 1024: 16 us against 35; 4 of
// 256, 2048 x 2048: 19 against 34; plain, one of 4096, 2048 x 2048: 22 with 128
// rows against 41; spread over two rounds they lose up to 19 %).  Where 96-row
// tiles leave CUs without one, the 64-row tile (16 experts, ReLU 1024 x 2048, 88
// rows each: 13 / 14 us against 16 / 16).  fp32 weight scales need a product of
// their own for each block before it is added, registers that the 256-row tile
// does not have: 128 rows there.  32-row tiles and weights loaded straight into
// the operands' registers, without LDS, were slower or equal at every size (32-row
// tiles also with two blocks a CU).
//
// Where 64 x 128 tiles are few, NarrowShape: two blocks a CU hide each other's
// waits.  Not for SwiGLU, whose tile has to hold a block of 128 hidden columns of
// both halves.  Down, E8M0 / fp32 scales, us, against the shapes above:
//   tiles  rows     K        above        64 x 128
//      64   256  1024   15.6 / 13.4     7.1 /  8.6
//     128  1024  4096   37.6 / 30.0    18.0 / 20.8
//     256     8 14336   88.3 / 89.1    81.5 / 82.3
//     256    75  2048   18.9 / 22.5    11.9 / 14.2
//     256   256  4096   34.1 / 29.3    28.6 / 29.8
//     512     1   512    9.9 / 10.9     8.8 /  9.4
//     512    75  1024   13.0 / 16.6    12.5 / 13.1
//     512    25  2048   27.7 / 28.3    29.2 / 29.6
//     512    75  4096   35.5 / 43.9    40.6 / 41.7
//     512  2048  4096   39.2 / 35.6    29.1 / 31.0
//    1024   256  1024   21.8 / 29.3    23.7 / 26.6
//    2048     8  1024   56.9 / 58.8    54.0 / 53.9
//    2048    32  1024   62.2 / 65.4    58.7 / 57.9
//    2048    64  1024   69.3 / 76.3    72.6 / 70.9
//    2048   128  1024   45.9 / 69.8    50.5 / 52.1
// so (narrow_pays) up to a tile a CU; up to two where K is below 2048, where the
// choice would be the 256-row tile, or with fp32 scales from 64 rows on; and any
// number below 192 rows for K below 2048 with fp32 scales or few rows.  With fp32
// scales, 192 rows or more and more than two tiles a CU the 128-row tile is the
// better one at most sizes (K 512 to 1920, time of 64 x 128 over its time): 1.1 to 1.4
// for 1024 to 4096 tiles of 256, 512 or 2048 rows each, 0.97 to 1.3 for ragged
// segments of about 200, 300 and 512; but 0.87 to 0.94 where 8 or 16 experts of about
// 256 rows leave it a second, nearly empty round (the table's fp32 line), and 0.73 to
// 0.91 where 640 columns end inside its last 256.
typedef BlockShape<256, 2, 4, 2, 8> LargeShape;
typedef BlockShape<128, 2, 4, 3, 8> Shape128;
typedef BlockShape<96, 1, 4, 3, 4> MediumShape;
typedef BlockShape<64, 1, 4, 3, 4> SmallShape;
typedef BlockShape<64, 2, 2, 3, 4, 128, 2> NarrowShape;
constexpr int kLargeRows = 192;

// Whether the last round (at most kBlkSplitSlots / 2 tiles of it) is split along K.
// The split costs a second launch (about 4 us), so it is left out where K is short,
// and where the tiles expected (rows spread evenly over min(rows, E) experts) fill
// more than half of the only round: one token of two experts, 224 tiles of 256 CUs,
// 54.9 -> 51.8 us without.
template <typename S>
bool split_pays(const BlockGemmArgs& g, long long ntn, int blocks)
{
    if (g.K < 2048)
        return false;
    const long long busy = std::min(g.E, g.max_rows);
    const long long tiles = busy * std::max(1ll, (g.max_rows / busy + S::BM - 1) / S::BM) * ntn;
    return tiles <= std::min(blocks, kBlkSplitSlots) / 2 || tiles > blocks;
}

bool narrow_pays(int mean_rows, long long tiles, int K, bool wf32, int ncu)
{
    if (tiles <= ncu)
        return true;
    if (mean_rows >= kLargeRows)
        return tiles <= 2 * ncu;
    if (K < 2048)
        return wf32 || mean_rows <= 32 || tiles <= 2 * ncu;
    return wf32 && mean_rows >= 64 && tiles <= 2 * ncu;
}

template <typename S, int EPI, bool WF32>
hipError_t launch_shape(BlockGemmArgs g, int ncu, hipStream_t stream)
{
    const int tile_cols = EPI == BEPI_SWIGLU ? 128 : S::BN;
    const long long ntn = (g.Nout + tile_cols - 1) / tile_cols;
    // upper bound on m-tiles: whole tiles plus one partial per expert
    const long long mt = g.max_rows / S::BM + (long long)std::min(g.E, g.max_rows);
    ncu *= S::kPerCu;
    if (!split_pays<S>(g, ntn, ncu))
        g.partial = nullptr;
    long long grid = ncu;
    if (mt * ntn < grid && g.partial == nullptr)
        grid = (mt * ntn + 7) / 8 * 8;
    moe_block_gemm_kernel<S, EPI, WF32><<<dim3((unsigned)grid), dim3(S::kThreads), 0, stream>>>(g);
    hipError_t err = hipGetLastError();
    if (err != hipSuccess || g.partial == nullptr)
        return err;
    moe_block_tail_kernel<S, EPI>
        <<<dim3(kBlkSplitSlots / 2 * S::kFM), dim3(S::kThreads), 0, stream>>>(g, (int)grid);
    return hipGetLastError();
}

template <typename S, bool WF32>
hipError_t launch_narrow(int epi, const BlockGemmArgs& g, int ncu, hipStream_t s)
{
    if (epi == BEPI_RELU)
        return launch_shape<S, BEPI_RELU, WF32>(g, ncu, s);
    return epi == BEPI_F32 ? launch_shape<S, BEPI_F32, WF32>(g, ncu, s) : launch_shape<S, BEPI_NONE, WF32>(g, ncu, s);
}

template <typename S, bool WF32>
hipError_t launch_epi(int epi, const BlockGemmArgs& g, int ncu, hipStream_t s)
{
    if (epi == BEPI_SWIGLU)
        return launch_shape<S, BEPI_SWIGLU, WF32>(g, ncu, s);
    return launch_narrow<S, WF32>(epi, g, ncu, s);
}

template <typename ET, bool F32>
void launch_quantize(const void* src, long long R, int K, int block_rows, uint8_t* codes, void* scales, hipStream_t s)
{
    typedef typename ET::storage T;
    constexpr size_t kScaleBytes = F32 ? 4 : 1;
    if (block_rows == 1) {
        const long long blocks = R * (K / kBlk);
        for (long long b = 0; b < blocks; b += 16 * kQuantGrid) {
            const long long n = std::min(blocks - b, 16 * kQuantGrid);
            moe_quantize_rows_kernel<ET, F32><<<dim3((unsigned)((n + 15) / 16)), dim3(256), 0, s>>>(
                (const T*)src + b * kBlk, n, codes + b * kBlk, (uint8_t*)scales + b * kScaleBytes);
        }
    } else {
        const long long nkb = K / kBlk, most = kQuantGrid / nkb;  // block rows of a launch
        for (long long b = 0; b * kBlk < R; b += most) {
            const long long r = std::min(R - b * kBlk, most * kBlk);
            moe_quantize_tiles_kernel<ET, F32><<<dim3((unsigned)((r + kBlk - 1) / kBlk * nkb)), dim3(256), 0, s>>>(
                (const T*)src + b * kBlk * K, r, K, codes + b * kBlk * K, (uint8_t*)scales + b * nkb * kScaleBytes);
        }
    }
}
}  // namespace

// src: R rows of K values (dtype 0 fp32, 1 bf16), K a multiple of 128;
// block_rows 1 or 128; scales fp32 numbers (f32) or E8M0 bytes.
extern "C" hipError_t moe_launch_quantize_block(int dtype, const void* src, long long R, int K, int block_rows,
                                                int f32, uint8_t* codes, void* scales, hipStream_t stream)
{
    if (R <= 0)
        return hipSuccess;
    if (dtype == 0)
        f32 ? launch_quantize<f32_t, true>(src, R, K, block_rows, codes, scales, stream)
            : launch_quantize<f32_t, false>(src, R, K, block_rows, codes, scales, stream);
    else
        f32 ? launch_quantize<bf16_t, true>(src, R, K, block_rows, codes, scales, stream)
            : launch_quantize<bf16_t, false>(src, R, K, block_rows, codes, scales, stream);
    return hipGetLastError();
}

// Bytes of the K split's partial tiles for this mean number of rows per expert.
extern "C" size_t moe_block_gemm_partial_bytes(int mean_rows)
{
    return (size_t)kBlkSplitSlots * 4 * (mean_rows >= kLargeRows ? LargeShape::kTileFloats : MediumShape::kTileFloats);
}

// epi 0: Y = bf16 rows, 3: Y = fp32 rows; 1 ReLU, 2 SwiGLU: Hq, Hs.  wf32: fp32 weight scales.
// mean_rows: expected rows per expert.  partial (nullable): the K split's
// workspace, moe_block_gemm_partial_bytes bytes.
extern "C" hipError_t moe_launch_block_gemm(int epi, int wf32, const uint8_t* A, const uint8_t* As,
                                            const int32_t* gather, int gather_rows, const uint8_t* W, const void* Ws,
                                            uint8_t* Hq, uint8_t* Hs, void* Y, const int32_t* offsets, int E, int K,
                                            int Nw, int Nout, int F, int max_rows, int mean_rows, int ncu,
                                            float* partial, hipStream_t stream)
{
    const BlockGemmArgs g = {A, As, gather, gather_rows, W, Ws, Hq, Hs, Y, offsets, E, K, Nw, Nout, F,
                             max_rows, partial};
    const long long narrow = (long long)std::min(E, max_rows) * std::max(1, (mean_rows + 63) / 64) * (Nout / 128);
    if (epi != BEPI_SWIGLU && narrow_pays(mean_rows, narrow, K, wf32, ncu))
        return wf32 ? launch_narrow<NarrowShape, true>(epi, g, ncu, stream)
                    : launch_narrow<NarrowShape, false>(epi, g, ncu, stream);
    const int tile_cols = epi == BEPI_SWIGLU ? 128 : 256;
    const long long ntn = (Nout + tile_cols - 1) / tile_cols, busy = std::min(E, max_rows);
    if (mean_rows >= kLargeRows) {
        auto most = [&](int bm) { return (busy == 1 ? (max_rows + bm - 1) / bm : max_rows / bm + busy) * ntn; };
        if (wf32)
            return launch_epi<Shape128, true>(epi, g, ncu, stream);
        if (most(MediumShape::BM) <= ncu)
            return launch_epi<MediumShape, false>(epi, g, ncu, stream);
        if (most(Shape128::BM) <= ncu)
            return launch_epi<Shape128, false>(epi, g, ncu, stream);
        return launch_epi<LargeShape, false>(epi, g, ncu, stream);
    }
    const long long tiles = busy * ((mean_rows + 95) / 96 + (mean_rows == 0)) * ntn;
    if (tiles < ncu)
        return wf32 ? launch_epi<SmallShape, true>(epi, g, ncu, stream)
                    : launch_epi<SmallShape, false>(epi, g, ncu, stream);
    return wf32 ? launch_epi<MediumShape, true>(epi, g, ncu, stream)
                : launch_epi<MediumShape, false>(epi, g, ncu, stream);
}

// rows: fp32 [max_rows][d]; d a multiple of 8, k <= 8.
extern "C" hipError_t moe_launch_combine_rows(const float* rows, const int32_t* slot, const float* topk_w, int T,
                                              int d, int k, int max_rows, void* y, hipStream_t stream)
{
    using namespace moe;
    const long long threads = (long long)T * (d / 8);
    const dim3 grid((unsigned)((threads + 255) / 256)), block(256);
    uint16_t* out = (uint16_t*)y;
    if (k == 1)
        moe_combine_rows_kernel<1><<<grid, block, 0, stream>>>(rows, slot, topk_w, T, d, k, max_rows, out);
    else if (k == 2)
        moe_combine_rows_kernel<2><<<grid, block, 0, stream>>>(rows, slot, topk_w, T, d, k, max_rows, out);
    else if (k <= 4)
        moe_combine_rows_kernel<4><<<grid, block, 0, stream>>>(rows, slot, topk_w, T, d, k, max_rows, out);
    else
        moe_combine_rows_kernel<8><<<grid, block, 0, stream>>>(rows, slot, topk_w, T, d, k, max_rows, out);
    return hipGetLastError();
}
