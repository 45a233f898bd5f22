// MXFP4 experts (gfx950): quantisation to E2M1 codes with a scale for each block
// of 32 values, its inverse, and the grouped GEMMs of the two expert layers on
// such codes.
//
// The experts' weights and the rows that meet them carry one E8M0 scale per 32
// consecutive values of K (a byte b stands for 2^(b - 127)):
//   u[r, n] = sum_b 2^(sA[r, b] + sW[n, b] - 254) sum_{k in block b} a[r, k] w[n, k]
#include <algorithm>

#include "common.h"
#include "gemm_common.h"
#include "mxfp4.h"

namespace moe {

// ---------------------------------------------------------------- quantisation
// The most workgroups of a launch (a launch has fewer than 2^32 threads).
constexpr long long kMxGrid = 1 << 23;

// 4 lanes of 8 values each per block, the blocks of all rows in one run (K is a
// multiple of 32).
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
enum { MXEPI_NONE = 0, MXEPI_RELU = 1, MXEPI_SWIGLU = 2, MXEPI_F32 = 3 };  // bf16 rows, hidden codes (2), fp32 rows

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
};

// One wavefront per 32 rows x 32 columns (SwiGLU: the gate and up rows of 32
// hidden columns), fragments from memory.  MFMA 32x32x64 f8f6f4 with E2M1
// operands: lane l holds block l / 32 of operand row l % 32 and its scale byte.
struct MxTile {
    static constexpr int BM = 32, GM = 8;
};
template <int EPI>
__global__ __launch_bounds__(256) void moe_mxfp4_gemm_kernel(MxGemmArgs g)
{
#if defined(__HIP_DEVICE_COMPILE__)
    __shared__ int32_t s_pref[kGemmMaxE + 1];
    __shared__ int32_t s_wsum[4];
    const int lane = lane_id(), wave = threadIdx.x / kWave, half = lane >> 5;
    const int ntn = (g.Nout + 31) / 32, nkb = g.K / kMxBlk;
    tile_prefix<256>(g.offsets, g.E, g.max_rows, 32, ntn, s_pref, s_wsum);
    const int total = s_pref[g.E];
    for (int tile = blockIdx.x * 4 + wave; tile < total; tile += gridDim.x * 4) {
        const TileDec t = decode_tile<MxTile>(tile, s_pref, g.offsets, g.E, g.max_rows, ntn, 32);
        const int r = min(lane & 31, t.rows - 1);
        int row = t.row0 + r;
        if (g.gather)
            row = min(max(g.gather[row], 0), g.gather_rows - 1);
        const size_t n = (size_t)t.e * g.Nw + t.n0 + (lane & 31);
        f32x16 acc[2] = {};
        for (int b = half; b < nkb; b += 2) {
            const uint4 a = *reinterpret_cast<const uint4*>(g.A + ((size_t)row * nkb + b) * 16);
            const i32x8 av = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
            const int as = g.As[(size_t)row * nkb + b];
#pragma unroll
            for (int j = 0; j < (EPI == MXEPI_SWIGLU ? 2 : 1); ++j) {
                const size_t at = (n + (size_t)j * g.F) * nkb + b;
                const uint4 w = *reinterpret_cast<const uint4*>(g.W + at * 16);
                const i32x8 wv = {(int)w.x, (int)w.y, (int)w.z, (int)w.w, 0, 0, 0, 0};
                acc[j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wv, av, acc[j], 4, 4, 0, (int)g.Ws[at], 0, as);
            }
        }
        float h[16];
        uint32_t amax = 0;
#pragma unroll
        for (int v = 0; v < 16; ++v) {
            const float u = acc[0][v];
            h[v] = EPI == MXEPI_SWIGLU ? u / (1.0f + expf(-u)) * acc[1][v] : EPI == MXEPI_RELU && u <= 0.0f ? 0.0f : u;
            amax = max(amax, abs_bits(h[v]));
        }
        if constexpr (EPI == MXEPI_NONE || EPI == MXEPI_F32) {
            if ((lane & 31) < t.rows)
#pragma unroll
                for (int v = 0; v < 16; ++v) {
                    const size_t at = (size_t)(t.row0 + r) * g.Nout + t.n0 + 8 * (v / 4) + 4 * half + v % 4;
                    if constexpr (EPI == MXEPI_F32)
                        static_cast<float*>(g.Y)[at] = h[v];
                    else
                        static_cast<uint16_t*>(g.Y)[at] = (uint16_t)f32_to_bf16_bits(h[v]);
                }
        } else {
            amax = max(amax, (uint32_t)__shfl_xor((int)amax, 32));
            const uint32_t s = mx_scale_byte(amax);
            if ((lane & 31) < t.rows) {
                const size_t out = (size_t)(t.row0 + r) * (g.Nout / kMxBlk) + t.n0 / kMxBlk;
                const uint32_t lo = e2m1_encode8(h, s), hi = e2m1_encode8(h + 8, s);
                uint16_t* dst = reinterpret_cast<uint16_t*>(g.Hq + out * 16) + half;
                dst[0] = (uint16_t)lo;
                dst[2] = (uint16_t)(lo >> 16);
                dst[4] = (uint16_t)hi;
                dst[6] = (uint16_t)(hi >> 16);
                if (half == 0)
                    g.Hs[out] = (uint8_t)s;
            }
        }
    }
#endif
}

}  // namespace moe

namespace {
using namespace moe;

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

// Bytes of the K split's partial tiles for this mean number of rows per expert.
extern "C" size_t moe_mxfp4_gemm_partial_bytes(int mean_rows)
{
    return 0;
}

// epi 0: Y = bf16 rows, 3: Y = fp32 rows; 1 ReLU, 2 SwiGLU: Hq, Hs.
extern "C" hipError_t moe_launch_mxfp4_gemm(int epi, const uint8_t* A, const uint8_t* As, const int32_t* gather,
                                            int gather_rows, const uint8_t* W, const uint8_t* Ws, uint8_t* Hq,
                                            uint8_t* Hs, void* Y, const int32_t* offsets, int E, int K, int Nw,
                                            int Nout, int F, int max_rows, int mean_rows, int ncu, float* partial,
                                            hipStream_t stream)
{
    const MxGemmArgs g = {A, As, gather, gather_rows, W, Ws, Hq, Hs, Y, offsets, E, K, Nw, Nout, F, max_rows};
    const dim3 grid(4 * ncu), block(256);
    if (epi == MXEPI_NONE)
        moe_mxfp4_gemm_kernel<MXEPI_NONE><<<grid, block, 0, stream>>>(g);
    else if (epi == MXEPI_RELU)
        moe_mxfp4_gemm_kernel<MXEPI_RELU><<<grid, block, 0, stream>>>(g);
    else if (epi == MXEPI_SWIGLU)
        moe_mxfp4_gemm_kernel<MXEPI_SWIGLU><<<grid, block, 0, stream>>>(g);
    else
        moe_mxfp4_gemm_kernel<MXEPI_F32><<<grid, block, 0, stream>>>(g);
    return hipGetLastError();
}
