// Orthogonalised updates (gfx950): momentum and Newton-Schulz products of a batch
// of gradient matrices.
//
// The quintic iteration of the Muon optimiser (K. Jordan et al., "Muon: an
// optimizer for hidden layers in neural networks", 2024) brings the singular
// values of X = U / |U|_F towards 1 and leaves the singular vectors:
//   A = X X^T,   X <- a X + (b A + c A^2) X,   (a, b, c) = (3.4445, -4.7750, 2.0315)
// on the orientation of X whose rows m are the fewer; n >= m columns.
//
// Numbers.  The products run on the fp16 matrix cores (fp32 sums): X, A and B = b A
// + c A^2 are rounded to fp16 as operands, scaled by powers of two so that nothing
// leaves fp16's normal range (singular values stay below 1.21, the entries of A
// below 1.5, those of B below 2.9).  A small singular value grows by a = 3.44 a step,
// and with it every rounding that lands on its vectors.  Two of them are kept off:
//   * a X is added from an fp32 X (rounded to fp16 it put the result of a gradient
//     of low rank 2e-2 off, now 5e-4);
//   * the diagonals of A and B, which outweigh the rest of their rows, stay in
//     fp32: X' = a X + diag(B) X + offdiag(B) X.  In the second term X is the fp16
//     operand, so that the rounding of X meets one B as a whole, whose product with
//     it is small where A is; in the last two steps, whose errors no longer grow,
//     it is the fp32 X (Gaussian 512 x 1024: 1.6e-3 -> 7e-4).
// With bf16 iterates the same gradients are 1e-2 to 2e-1 off.
#include <algorithm>
#include <cmath>

#include "common.h"
#include "gemm_common.h"
#include "tile_gemm.h"

namespace moe {

constexpr float kNsA = 3.4445f, kNsB = -4.7750f, kNsC = 2.0315f;
constexpr float kNsScale = 16384.0f;  // of the fp16 A and B
constexpr int kNsPad = 64;            // rows of fp16 operands are padded to whole slices
constexpr int kNsSums = 256;          // partial sums of squares of a matrix, at most

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));

// One batch: matrices of m x n (m <= n), X^T where the source is tall.
struct NsArgs {
    const void* grad;
    float* momentum;  // nullable
    uint16_t* out;    // bf16
    _Float16* x;      // [count][m][np], scaled by sx
    _Float16* xt;     // [2][count][n][mp]
    float* x32;       // [count][np / 32][mp / 32] fragments of X^T, see ns_frag
    _Float16* a;      // [count][m][mp], scaled by kNsScale, zero diagonal
    _Float16* b;      // [count][m][mp]
    float* da;        // [count][mp] diagonal of A
    float* db;        // [count][mp] of B
    double* sums;     // [count][kNsSums]
    float beta, sx;
    int src_dtype, nesterov, count, rows, cols, m, n, mp, np, parts;
};

__device__ __forceinline__ float ns_grad(const NsArgs& g, size_t at)
{
    return g.src_dtype == 0 ? static_cast<const float*>(g.grad)[at]
                            : bf16_bits_to_f32(static_cast<const uint16_t*>(g.grad)[at]);
}

// U at an element, from the gradient and the momentum of this step.
__device__ __forceinline__ float ns_update(const NsArgs& g, size_t at)
{
    if (!g.momentum)
        return ns_grad(g, at);
    return g.nesterov ? fmaf(g.beta, g.momentum[at], ns_grad(g, at)) : g.momentum[at];
}

// Momentum, and sums of squares of U in fp64: block (part, matrix).
__global__ __launch_bounds__(256) void moe_ns_sums_kernel(NsArgs g)
{
    __shared__ double s_sum[256];
    const size_t each = (size_t)g.rows * g.cols, base = (size_t)blockIdx.y * each;
    double sum = 0.0;
    for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < each; i += (size_t)g.parts * 256) {
        if (g.momentum)
            g.momentum[base + i] = fmaf(g.beta, g.momentum[base + i], ns_grad(g, base + i));
        const double u = ns_update(g, base + i);
        sum += u * u;
    }
    s_sum[threadIdx.x] = sum;
    __syncthreads();
    for (int o = 128; o >= 1; o >>= 1) {
        if ((int)threadIdx.x < o)
            s_sum[threadIdx.x] += s_sum[threadIdx.x + o];
        __syncthreads();
    }
    if (threadIdx.x == 0)
        g.sums[(size_t)blockIdx.y * kNsSums + blockIdx.x] = s_sum[0];
}

// First value of the 32 x 32 fragment of X^T at row 32 fi, column 32 fj: 4 groups of
// columns 8 q .., of which lane l holds the 4 from 4 (l / 32) on of row l % 32, as the
// matrix cores leave them.
__device__ __forceinline__ size_t ns_frag(const NsArgs& g, size_t mat, int fi, int fj)
{
    return ((mat * (g.np / 32) + fi) * (g.mp / 32) + fj) * 1024;
}

// X = U / |U|_F in both orientations, and the padding of every operand: block
// (tile of 32 x 32 of the padded X, matrix).
__global__ __launch_bounds__(256) void moe_ns_init_kernel(NsArgs g)
{
    __shared__ float tile[32][33];
    const int tn = g.np / 32;
    const int i0 = blockIdx.x / tn * 32, j0 = blockIdx.x % tn * 32;
    const size_t mat = blockIdx.y;
    double sum = 0.0;
    for (int p = 0; p < g.parts; ++p)
        sum += g.sums[mat * kNsSums + p];
    // 1 / |U|: U is zero where the sum is
    const double inv = sum > 0.0 || sum != sum ? 1.0 / sqrt(sum) : 0.0;
    const size_t base = mat * g.rows * g.cols;
    const int tx = threadIdx.x % 32, ty = threadIdx.x / 32;
    const bool tall = g.rows > g.cols;
#pragma unroll
    for (int k = 0; k < 32; k += 8) {
        const int u = ty + k;  // source rows one after another
        const int i = tall ? i0 + tx : i0 + u, j = tall ? j0 + u : j0 + tx;
        float v = 0.0f;
        if (i < g.m && j < g.n)
            v = (float)(ns_update(g, base + (tall ? (size_t)j * g.cols + i : (size_t)i * g.cols + j)) * inv);
        tile[tall ? tx : u][tall ? u : tx] = v;
    }
    __syncthreads();
    const size_t cells = (size_t)g.count * g.n * g.mp;
    float* frag = g.x32 + ns_frag(g, mat, j0 / 32, i0 / 32);
#pragma unroll
    for (int k = 0; k < 32; k += 8) {
        int i = i0 + ty + k, j = j0 + tx;
        if (i < g.m)
            g.x[(mat * g.m + i) * g.np + j] = (_Float16)(tile[ty + k][tx] * g.sx);
        i = i0 + tx, j = j0 + ty + k;
        const float v = tile[tx][ty + k];
        frag[((tx / 8) * 64 + (tx / 4 % 2) * 32 + ty + k) * 4 + tx % 4] = v;
        if (j < g.n) {
            const size_t at = (mat * g.n + j) * g.mp + i;
            g.xt[at] = (_Float16)(v * g.sx);
            if (i >= g.m)
                g.xt[cells + at] = (_Float16)0.0f;
        }
    }
    if (j0 == 0 && threadIdx.x < 32) {
        g.da[mat * g.mp + i0 + threadIdx.x] = 0.0f;
        g.db[mat * g.mp + i0 + threadIdx.x] = 0.0f;
    }
}

// ---------------------------------------------------------------- the products
enum { NS_GRAM = 0, NS_POLY = 1, NS_UPDATE = 2 };

struct NsOp {
    template <int>
    static __device__ __forceinline__ f32x16 mma(const i32x4& w, const i32x4& a, const f32x16& c, int, int)
    {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, w), __builtin_bit_cast(f16x8, a), c, 0,
                                                      0, 0);
    }
};

typedef TileShape<256, 2, 4, 2, 4, 256, 1, false> NsLarge;
typedef TileShape<128, 2, 2, 2, 8, 128, 2, false> NsSmall;

// Tile `tile` of the lower triangle of T x T tiles: groups of GM rows, in a group column
// by column.
__device__ __forceinline__ void ns_triangle(int tile, int T, int GM, int& ti, int& tj)
{
    int first = 0;
    for (;;) {
        const int R = min(GM, T - first), all = first * R + R * (R + 1) / 2;
        if (tile < all || first + R >= T) {
            if (tile < first * R) {
                tj = tile / R;
                ti = first + tile % R;
                return;
            }
            int left = tile - first * R;
            for (tj = first; left >= first + R - tj; ++tj)
                left -= first + R - tj;
            ti = tj + left;
            return;
        }
        tile -= all;
        first += R;
    }
}

// Where 16-byte chunk c of row `row` of the staged output tile lies: chunks XOR-ed with
// the row so that neither 32 rows at one chunk nor every eighth row at one column meet in
// few banks.
template <typename S>
__device__ __forceinline__ int ns_staged(int row, int c)
{
    return row * S::BN * 2 + ((c ^ ((row ^ (row >> 3)) & (S::BN / 8 - 1))) << 4);
}

// 8 values to row `row`, columns col .. col + 7 of a matrix of `rows` rows of `cols`
// values, `pitch` apart: what lies inside.
__device__ __forceinline__ void ns_put(uint16_t* dst, const uint4& v, int row, int col, int rows, int cols,
                                       size_t pitch, bool wide)
{
    if (row >= rows || col >= cols)
        return;
    uint16_t* at = dst + (size_t)row * pitch + col;
    if (wide && col + 8 <= cols) {
        *reinterpret_cast<uint4*>(at) = v;
        return;
    }
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int q = 0; q < 8; ++q)
        if (col + q < cols)
            at[q] = (uint16_t)(w[q / 2] >> (16 * (q % 2)));
}

// The staged tile to rows i0 .., columns j0 .. of dst (direct) or, transposed, to rows
// j0 .., columns i0 ...
template <typename S, bool TRANSPOSED>
__device__ __forceinline__ void ns_write(const uint8_t* lds, uint16_t* dst, int i0, int j0, int rows, int cols,
                                         size_t pitch, bool wide)
{
    constexpr int kChunks = (TRANSPOSED ? S::BM : S::BN) / 8, kRows = TRANSPOSED ? S::BN : S::BM;
    for (int it = threadIdx.x; it < kRows * kChunks; it += S::kThreads) {
        const int r = it / kChunks, c = it % kChunks;
        uint4 v;
        if constexpr (TRANSPOSED) {
            uint32_t e[8];
#pragma unroll
            for (int q = 0; q < 8; ++q)
                e[q] = *reinterpret_cast<const uint16_t*>(lds + ns_staged<S>(8 * c + q, r / 8) + (r % 8) * 2);
            v = make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
            ns_put(dst, v, j0 + r, i0 + 8 * c, rows, cols, pitch, wide);
        } else {
            v = *reinterpret_cast<const uint4*>(lds + ns_staged<S>(r, c));
            ns_put(dst, v, i0 + r, j0 + 8 * c, rows, cols, pitch, wide);
        }
    }
}

// One output tile of a product per block:
//   GRAM    A = X X^T      POLY    B = b A + c A^2      UPDATE    X^T <- a X^T + X^T B
// A and B are symmetric: only tiles on and below the diagonal are computed, and stored
// on both sides of it.
template <typename S, int MODE>
__global__ __launch_bounds__(S::kThreads) __attribute__((amdgpu_waves_per_eu(S::kWavesPerSimd, S::kWavesPerSimd)))
void moe_ns_product_kernel(NsArgs g, int tiles, int src, bool fine, bool last, bool wide)
{
#if defined(__HIP_DEVICE_COMPILE__)
    static_assert(S::BM * S::BN * 2 <= S::S * S::kStage, "the staged output tile fits the stages");
    __shared__ __attribute__((aligned(1024))) uint8_t lds[S::S * S::kStage];
    // an XCD's blocks take neighbouring tiles
    const int total = tiles * g.count, each = (total + 7) / 8;
    const int item = blockIdx.x % 8 * each + blockIdx.x / 8;
    if (item >= total)
        return;
    const size_t mat = item / tiles;
    const int tile = item % tiles;
    const int M = MODE == NS_UPDATE ? g.n : g.m, pitch = 2 * (MODE == NS_GRAM ? g.np : g.mp);
    int ti, tj;
    if constexpr (MODE == NS_UPDATE) {
        const int tn = (g.m + S::BN - 1) / S::BN, tm = (g.n + S::BM - 1) / S::BM;
        const int group = tile / (S::GM * tn), within = tile - group * S::GM * tn, gs = min(S::GM, tm - group * S::GM);
        ti = group * S::GM + within % gs;
        tj = within / gs;
    } else {
        ns_triangle(tile, (g.m + S::BN - 1) / S::BN, S::GM, ti, tj);
    }
    const int i0 = ti * S::BM, j0 = tj * S::BN;
    const _Float16* A = MODE == NS_GRAM ? g.x + mat * g.m * g.np
                        : MODE == NS_POLY ? g.a + mat * g.m * g.mp
                                          : g.xt + ((size_t)src * g.count + mat) * g.n * g.mp;
    const _Float16* W = MODE == NS_UPDATE ? g.b + mat * g.m * g.mp : A;

    int tid = threadIdx.x;
    const int lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int wm = wave / S::WN, wn = wave % S::WN;
    const uint32_t lds0 = lds_addr(lds);
    const int rowsA = min(S::BM, M - i0), rowsW = min(S::BN, g.m - j0);
    const i32x4 rsA = make_rsrc(reinterpret_cast<const uint8_t*>(A) + (size_t)i0 * pitch, (uint32_t)rowsA * pitch);
    const i32x4 rsW = make_rsrc(reinterpret_cast<const uint8_t*>(W) + (size_t)j0 * pitch, (uint32_t)rowsW * pitch);
    // lane's place in a 1 KB load of 8 rows; rows behind the last read zeros
    const int lrow = S::kRows * wave + lane / 8;
    const uint32_t lchunk = (uint32_t)((lane % 8) ^ tile_swz(lrow)) * 16;
    uint32_t voffA[S::kBlkA], voffW[S::kBlkW];
#pragma unroll
    for (int i = 0; i < S::kBlkA; ++i) {
        const int r = lrow + S::kRows * S::kWaves * i;
        voffA[i] = r < rowsA ? (uint32_t)r * (uint32_t)pitch + lchunk : 0xf0000000u;
    }
#pragma unroll
    for (int i = 0; i < S::kBlkW; ++i) {
        const int r = lrow + S::kRows * S::kWaves * i;
        voffW[i] = r < rowsW ? (uint32_t)r * (uint32_t)pitch + lchunk : 0xf0000000u;
    }
    auto issue = [&](int q, int st, int n0, int n1) {
        const uint32_t dst = lds0 + st * S::kStage + wave * 1024, soff = (uint32_t)q * S::RB;
#pragma unroll
        for (int p = 0; p < S::kLoads; ++p) {
            if (p < n0 || p >= n1)
                continue;
            if (p < S::kBlkW)
                dma16(rsW, dst + S::kLdsA + S::kWaves * p * 1024, voffW[p], soff);
            else
                dma16(rsA, dst + S::kWaves * (p - S::kBlkW) * 1024, voffA[p - S::kBlkW], soff);
        }
    };
    f32x16 acc[S::kFM][S::kFN];
    const int live = min(max((rowsA - wm * S::kWaveM + 31) / 32, 0), S::kFM);
    tile_product<S, NsOp>(acc, lds, wm, wn, live, 0, pitch / S::RB, issue);

    // Epilogue: the values that the next product reads, staged as 16-bit numbers
    __asm__ volatile("" : "+v"(tid));
#pragma unroll
    for (int fi = 0; fi < S::kFM; ++fi)
#pragma unroll
        for (int fj = 0; fj < S::kFN; ++fj) {
            const int r = wm * S::kWaveM + fi * 32 + (lane & 31), i = i0 + r;
            const int c0 = (fj / S::kHalfF) * S::kHalf + wn * S::kHalfN + (fj % S::kHalfF) * 32, f0 = j0 + c0;
            const bool held = f0 < g.mp && i - (lane & 31) < (MODE == NS_UPDATE ? g.np : g.mp);
            const size_t frag = MODE == NS_UPDATE && held ? ns_frag(g, mat, (i0 + wm * S::kWaveM) / 32 + fi, f0 / 32) : 0;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int c = c0 + 8 * q + 4 * (lane >> 5), j = j0 + c;
                f32x4 v = {acc[fi][fj][4 * q], acc[fi][fj][4 * q + 1], acc[fi][fj][4 * q + 2], acc[fi][fj][4 * q + 3]};
                f16x4 o = {0, 0, 0, 0};
                if constexpr (MODE == NS_GRAM) {
                    const f32x4 s = v * (1.0f / (g.sx * g.sx));
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if (j + e == i && i < g.m)
                            g.da[mat * g.mp + i] = s[e];
                        o[e] = (_Float16)(j + e == i ? 0.0f : s[e] * kNsScale);
                    }
                } else if constexpr (MODE == NS_POLY) {
                    if (held && i < g.m) {
                        const float di = g.da[mat * g.mp + i];
                        const f32x4 dj = *reinterpret_cast<const f32x4*>(g.da + mat * g.mp + j);
                        const f16x4 a = *reinterpret_cast<const f16x4*>(g.a + (mat * g.m + i) * g.mp + j);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float off = (float)a[e] * (1.0f / kNsScale);
                            const float sq = v[e] * (1.0f / (kNsScale * kNsScale));
                            if (j + e == i)
                                g.db[mat * g.mp + i] = fmaf(kNsC, fmaf(di, di, sq), kNsB * di);
                            const float b = fmaf(kNsC, fmaf(di + dj[e], off, sq), kNsB * off);
                            o[e] = (_Float16)(j + e == i ? 0.0f : b * kNsScale);
                        }
                    }
                } else if (held) {
                    float* at = g.x32 + frag + q * 256 + lane * 4;
                    const f32x4 x = *reinterpret_cast<const f32x4*>(at);
                    const f32x4 db = *reinterpret_cast<const f32x4*>(g.db + mat * g.mp + j);
                    f32x4 y;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float xr = fine ? x[e] : (float)(_Float16)(x[e] * g.sx) * (1.0f / g.sx);
                        y[e] = fmaf(kNsA, x[e], fmaf(db[e], xr, v[e] * (1.0f / (kNsScale * g.sx))));
                    }
                    if (last) {
                        typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
                        o = __builtin_bit_cast(f16x4, __builtin_convertvector(y, bf16x4));
                    } else {
                        *reinterpret_cast<f32x4*>(at) = y;
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            o[e] = (_Float16)(y[e] * g.sx);
                    }
                }
                *reinterpret_cast<f16x4*>(lds + ns_staged<S>(r, c / 8) + (c % 8) * 2) = o;
            }
        }
    __syncthreads();
    if constexpr (MODE != NS_UPDATE) {
        uint16_t* dst = reinterpret_cast<uint16_t*>(MODE == NS_GRAM ? g.a : g.b) + mat * g.m * g.mp;
        ns_write<S, false>(lds, dst, i0, j0, g.m, g.mp, g.mp, true);
        if (ti != tj)
            ns_write<S, true>(lds, dst, i0, j0, g.m, g.mp, g.mp, true);
    } else if (last) {
        uint16_t* dst = g.out + mat * g.rows * g.cols;
        if (g.rows > g.cols)
            ns_write<S, false>(lds, dst, i0, j0, g.n, g.m, g.m, wide);
        else
            ns_write<S, true>(lds, dst, i0, j0, g.m, g.n, g.n, wide);
    } else {
        uint16_t* xt = reinterpret_cast<uint16_t*>(g.xt) + ((size_t)(src ^ 1) * g.count + mat) * g.n * g.mp;
        ns_write<S, false>(lds, xt, i0, j0, g.n, g.mp, g.mp, true);
        ns_write<S, true>(lds, reinterpret_cast<uint16_t*>(g.x) + mat * g.m * g.np, i0, j0, g.m, g.np, g.np, true);
    }
#endif
}

}  // namespace moe

namespace {
using namespace moe;

size_t ns_round(size_t v) { return (v + 255) / 256 * 256; }

// The workspace's pieces; returns its size.
size_t ns_layout(NsArgs& g, char* ws)
{
    size_t off = 0;
    auto take = [&](size_t bytes) {
        char* at = ws + off;
        off += ns_round(bytes);
        return at;
    };
    const size_t c = g.count, cells = c * g.n * g.mp, square = c * g.m * g.mp;
    g.x = (_Float16*)take(2 * c * g.m * g.np);
    g.xt = (_Float16*)take(4 * cells);
    g.x32 = (float*)take(4 * c * g.np * g.mp);
    g.a = (_Float16*)take(2 * square);
    g.b = (_Float16*)take(2 * square);
    g.da = (float*)take(4 * c * g.mp);
    g.db = (float*)take(4 * c * g.mp);
    g.sums = (double*)take(8 * c * kNsSums);
    return off;
}

NsArgs ns_args(int count, int rows, int cols)
{
    NsArgs g = {};
    g.count = count, g.rows = rows, g.cols = cols;
    g.m = std::min(rows, cols), g.n = std::max(rows, cols);
    g.mp = (g.m + kNsPad - 1) / kNsPad * kNsPad;
    g.np = (g.n + kNsPad - 1) / kNsPad * kNsPad;
    // entries of a matrix with orthonormal rows are 1 / sqrt(n) in the mean
    int e = 0;
    frexp(std::sqrt((double)g.n), &e);
    g.sx = (float)std::ldexp(1.0, e - 1);
    g.parts = (int)std::min<size_t>(kNsSums, ((size_t)rows * cols + 4095) / 4096);
    return g;
}

template <typename S>
hipError_t launch_steps(const NsArgs& g, int steps, hipStream_t stream)
{
    const long long tm = (g.m + S::BN - 1) / S::BN, tn = (g.n + S::BM - 1) / S::BM;
    const int square = (int)(tm * (tm + 1) / 2), update = (int)(tm * tn);
    // rows of the output that 16-byte stores fit
    const bool wide = g.cols % 8 == 0 && reinterpret_cast<uintptr_t>(g.out) % 16 == 0;
    auto grid = [&](int tiles) { return dim3((unsigned)(((long long)tiles * g.count + 7) / 8 * 8)); };
    const dim3 block(S::kThreads);
    for (int s = 0; s < steps; ++s) {
        const bool fine = s >= steps - 2, last = s == steps - 1;
        moe_ns_product_kernel<S, NS_GRAM><<<grid(square), block, 0, stream>>>(g, square, s & 1, fine, last, wide);
        moe_ns_product_kernel<S, NS_POLY><<<grid(square), block, 0, stream>>>(g, square, s & 1, fine, last, wide);
        moe_ns_product_kernel<S, NS_UPDATE><<<grid(update), block, 0, stream>>>(g, update, s & 1, fine, last, wide);
    }
    return hipGetLastError();
}
}  // namespace

extern "C" size_t moe_orthogonalize_scratch_bytes(int count, int rows, int cols)
{
    NsArgs g = ns_args(count, rows, cols);
    return ns_layout(g, nullptr);
}

// dtype 0 fp32, 1 bf16 gradients [count][rows][cols]; momentum (nullable) fp32; out bf16.
extern "C" hipError_t moe_launch_orthogonalize(int dtype, const void* grad, float* momentum, float beta, int nesterov,
                                               int count, int rows, int cols, int steps, void* out, void* ws,
                                               int ncu, hipStream_t stream)
{
    NsArgs g = ns_args(count, rows, cols);
    ns_layout(g, (char*)ws);
    g.grad = grad, g.momentum = momentum, g.out = (uint16_t*)out;
    g.beta = beta, g.src_dtype = dtype, g.nesterov = nesterov;
    moe_ns_sums_kernel<<<dim3(g.parts, count), dim3(256), 0, stream>>>(g);
    moe_ns_init_kernel<<<dim3(g.mp / 32 * (g.np / 32), count), dim3(256), 0, stream>>>(g);
    const long long large = (long long)count * ((g.m + 255) / 256) * ((g.n + 255) / 256);
    return large >= ncu ? launch_steps<NsLarge>(g, steps, stream) : launch_steps<NsSmall>(g, steps, stream);
}
