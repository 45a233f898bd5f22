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
//   * a X is added from an X of 22 bits, an fp16 number and an fp16 remainder (rounded
//     to fp16 it put the result of a gradient of low rank 2e-2 off, now 5e-4);
//   * the diagonals of A and B, which outweigh the rest of their rows, stay in
//     fp32: X' = a X + diag(B) X + offdiag(B) X.  In the second term X is the fp16
//     operand, so that the rounding of X meets one B as a whole, whose product with
//     it is small where A is; in the last two steps, whose errors go through one
//     more step at most, it is the whole X (Gaussian 512 x 1024: 1.6e-3 -> 7e-4).
// With bf16 iterates the same gradients are 1e-2 to 2e-1 off.  The roundings of A and
// B to 11 bits stay, and the quintic's slope (3.44 at zero, 3.97 at 1.2) carries them on:
// where many entries are equal they fall the same way and add up (4 blocks of ones, 130 x
// 1001: 1.1e-2 at 5 steps), and longer runs gather more of them (Gaussian 200 x 300: 9e-4
// at 5 steps, 2e-3 at 8, 5e-3 at 40).  Directions of a zero singular value last as long as
// 3.44^steps times an fp32 rounding is small.
#include <algorithm>
#include <cmath>

#include "common.h"
#include "gemm_common.h"
#include "tile_gemm.h"

namespace moe {

[[maybe_unused]] constexpr float kNsA = 3.4445f, kNsB = -4.7750f, kNsC = 2.0315f;
[[maybe_unused]] constexpr float kNsScale = 16384.0f;  // of the fp16 A and B
[[maybe_unused]] constexpr float kNsLow = 2048.0f;     // of the remainder of X: fp16 keeps 11 bits before it
constexpr int kNsPad = 64;    // rows of fp16 operands are padded to whole slices
constexpr int kNsSums = 512;  // partial sums of squares of a matrix, at most

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));

// One batch: X of m x n (m <= n), which is U, or U^T where the source is tall.
struct NsArgs {
    const void* grad;
    float* momentum;  // nullable
    uint16_t* out;    // bf16
    _Float16* x;      // [count][m][np] X, scaled by sx
    _Float16* xt;     // [2][count][n][mp] X^T, scaled by sx
    _Float16* low;    // [count][np / 32][mp / 32] fragments of the remainder of X^T, scaled by sx kNsLow, see ns_frag
    _Float16* a;      // [count][m][mp] A, scaled by kNsScale, zero diagonal
    _Float16* b;      // [count][m][mp] B, the same
    float* da;        // [count][mp] diagonal of A
    float* db;        // [count][mp] of B
    double* sums;     // [count][kNsSums]
    float* partial;   // partial tiles of split products
    float beta, sx;
    int src_dtype, nesterov, count, rows, cols, m, n, mp, np, parts;
    bool vec;  // four neighbouring values of the sources can be loaded at once
};

// Four values of the gradient from element `at` on, of which the first `held` are there.
__device__ __forceinline__ f32x4 ns_load_grad(const NsArgs& g, size_t at, int held)
{
    f32x4 v = {0, 0, 0, 0};
    if (g.src_dtype == 0) {
        const float* p = static_cast<const float*>(g.grad) + at;
        if (g.vec && held == 4)
            return *reinterpret_cast<const f32x4*>(p);
        for (int q = 0; q < held; ++q)
            v[q] = p[q];
    } else {
        const uint16_t* p = static_cast<const uint16_t*>(g.grad) + at;
        if (g.vec && held == 4) {
            const uint2 w = *reinterpret_cast<const uint2*>(p);
            return f32x4{__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                         __uint_as_float(w.y & 0xffff0000u)};
        }
        for (int q = 0; q < held; ++q)
            v[q] = bf16_bits_to_f32(p[q]);
    }
    return v;
}

__device__ __forceinline__ f32x4 ns_load_momentum(const NsArgs& g, size_t at, int held)
{
    const float* p = g.momentum + at;
    if (g.vec && held == 4)
        return *reinterpret_cast<const f32x4*>(p);
    f32x4 v = {0, 0, 0, 0};
    for (int q = 0; q < held; ++q)
        v[q] = p[q];
    return v;
}

// Four values of U once the momentum is this step's.
__device__ __forceinline__ f32x4 ns_load_update(const NsArgs& g, size_t at, int held)
{
    if (!g.momentum)
        return ns_load_grad(g, at, held);
    f32x4 m = ns_load_momentum(g, at, held);
    if (g.nesterov) {
        const f32x4 v = ns_load_grad(g, at, held);
#pragma unroll
        for (int q = 0; q < 4; ++q)
            m[q] = fmaf(g.beta, m[q], v[q]);
    }
    return m;
}

// Momentum and sums of squares of U in fp64: block (part, matrix), its partial sum in a
// place of its own, so that the order is fixed.  Bound by HBM: two 4096 x 14336 fp32
// gradients with momentum, 1.4 GB read and written, take 237 us (5.9 TB/s).
__global__ __launch_bounds__(256) void moe_ns_sums_kernel(NsArgs g)
{
    __shared__ double s_sum[4];
    const size_t each = (size_t)g.rows * g.cols, base = (size_t)blockIdx.y * each;
    double sum = 0.0;
    for (size_t i = ((size_t)blockIdx.x * 256 + threadIdx.x) * 4; i < each; i += (size_t)g.parts * 1024) {
        const int held = (int)min((size_t)4, each - i);
        f32x4 u = ns_load_grad(g, base + i, held);
        if (g.momentum) {
            f32x4 m = ns_load_momentum(g, base + i, held);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                m[q] = fmaf(g.beta, m[q], u[q]);
                u[q] = g.nesterov ? fmaf(g.beta, m[q], u[q]) : m[q];
            }
            float* p = g.momentum + base + i;
            if (g.vec && held == 4)
                *reinterpret_cast<f32x4*>(p) = m;
            else
                for (int q = 0; q < held; ++q)
                    p[q] = m[q];
        }
#pragma unroll
        for (int q = 0; q < 4; ++q)
            sum += (double)u[q] * u[q];
    }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1)
        sum += __shfl_xor(sum, o);
    if (lane_id() == 0)
        s_sum[threadIdx.x / kWave] = sum;
    __syncthreads();
    if (threadIdx.x == 0)
        g.sums[(size_t)blockIdx.y * kNsSums + blockIdx.x] = (s_sum[0] + s_sum[1]) + (s_sum[2] + s_sum[3]);
}

// First value of the 32 x 32 fragment of X^T at row 32 fi, column 32 fj: 4 groups of
// columns 8 q .., of which lane l holds the 4 from 4 (l / 32) on of row l % 32, as the
// matrix cores leave them.
__device__ __forceinline__ size_t ns_frag(const NsArgs& g, size_t mat, int fi, int fj)
{
    return ((mat * (g.np / 32) + fi) * (g.mp / 32) + fj) * 1024;
}

// X = U / |U|_F in all its forms: block (64 x 64 of the padded X, matrix).  Bound by HBM:
// the same gradients with Nesterov momentum, 8 bytes read and 6 written a value, take 335
// us (4.9 TB/s).
__global__ __launch_bounds__(256) void moe_ns_init_kernel(NsArgs g)
{
    __shared__ float tile[64][65];
    __shared__ double s_sum[4];
    const int tn = g.np / 64, tid = threadIdx.x, lane = lane_id();
    const int i0 = blockIdx.x / tn * 64, j0 = blockIdx.x % tn * 64;
    const size_t mat = blockIdx.y, base = mat * g.rows * g.cols;
    const bool tall = g.rows > g.cols;
    const int r0 = tall ? j0 : i0, c0 = tall ? i0 : j0;  // of the source
    f32x4 u[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int r = r0 + tid / 16 + 16 * k, c = c0 + tid % 16 * 4;
        u[k] = f32x4{0, 0, 0, 0};
        if (r < g.rows && c < g.cols)
            u[k] = ns_load_update(g, base + (size_t)r * g.cols + c, min(4, g.cols - c));
    }
    double sum = 0.0;
    for (int p = tid; p < g.parts; p += 256)
        sum += g.sums[mat * kNsSums + p];
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1)
        sum += __shfl_xor(sum, o);
    if (lane == 0)
        s_sum[tid / kWave] = sum;
    __syncthreads();
    sum = (s_sum[0] + s_sum[1]) + (s_sum[2] + s_sum[3]);
    // zeros stay zeros; a NaN or an infinity anywhere makes the matrix NaN
    const double inv = sum == 0.0 ? 0.0 : sum * 0.0 + g.sx / sqrt(sum);
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int r = tid / 16 + 16 * k, c = tid % 16 * 4 + q;
            tile[tall ? c : r][tall ? r : c] = (float)(u[k][q] * inv);
        }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int r = tid / 8 + 32 * k, c = tid % 8 * 8;
        f16x8 v, w;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            v[q] = (_Float16)tile[r][c + q];
            w[q] = (_Float16)tile[c + q][r];
        }
        if (i0 + r < g.m)
            *reinterpret_cast<f16x8*>(g.x + (mat * g.m + i0 + r) * g.np + j0 + c) = v;
        if (j0 + r < g.n)
            *reinterpret_cast<f16x8*>(g.xt + (mat * g.n + j0 + r) * g.mp + i0 + c) = w;
    }
    const int fi = tid / 128, fj = tid / 64 % 2;
    _Float16* low = g.low + ns_frag(g, mat, j0 / 32 + fi, i0 / 32 + fj);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        f16x4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float f = tile[fj * 32 + 8 * q + 4 * (lane >> 5) + e][fi * 32 + (lane & 31)];
            v[e] = (_Float16)((f - (float)(_Float16)f) * kNsLow);
        }
        *reinterpret_cast<f16x4*>(low + q * 256 + lane * 4) = v;
    }
    if (j0 == 0 && tid < 64) {
        g.da[mat * g.mp + i0 + tid] = 0.0f;
        g.db[mat * g.mp + i0 + tid] = 0.0f;
    }
}

// ---------------------------------------------------------------- the products
// One output tile of a product per block:
//   GRAM    A = X X^T      POLY    B = b A + c A^2      UPDATE    X^T <- a X^T + X^T B
// A and B are symmetric: only tiles on and below the diagonal are computed, and stored
// on both sides of it.  X and X^T are both kept, since both products want K along the row.
//
// Two matrices of 4096 x 14336, in us a step: A 398 + 14 for its split tiles (matrix cores
// busy 76 % of the cycles, at 1.60 GHz: the card's power), B 139 + 10 (54 % at 1.84), X'
// 885 (60 % at 1.72: 10 bytes a value come and go before and behind the K loop, in which
// memory is idle).  64 of 1024 x 512: A 36, B 29, X' 88 to 92, of 8 or 16 slices a tile.
// All the remainder's loads ahead of the epilogue spill (+5 %).
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

// The tiles of a product: `full` of them in one piece, the others, fewer than blocks run
// at a time, in `parts` parts along K, whose sums moe_ns_tail_kernel adds.
struct NsPlan {
    int tiles;  // of a matrix
    int full, tail, parts;
};

struct NsStep {
    int src;           // which of the two X^T is this step's
    bool fine, last;   // of the last two steps, the last one
    bool wide;         // 16-byte stores to the output are aligned
};

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

template <typename S, int MODE>
__device__ __forceinline__ void ns_tile(const NsArgs& g, int tile, int& ti, int& tj)
{
    const int tn = (g.m + S::BN - 1) / S::BN;
    if constexpr (MODE == NS_UPDATE) {
        const int tm = (g.n + S::BM - 1) / S::BM;
        const int group = tile / (S::GM * tn), within = tile - group * S::GM * tn, gs = min(S::GM, tm - group * S::GM);
        ti = group * S::GM + within % gs;
        tj = within / gs;
    } else {
        ns_triangle(tile, tn, S::GM, ti, tj);
    }
}

// Where 16-byte chunk c of row `row` of a staged tile lies: chunks XOR-ed with the row so
// that neither 32 rows at one chunk nor every eighth row at one column meet in few banks.
template <typename S>
__device__ __forceinline__ int ns_staged_chunk(int row, int c)
{
    return c ^ ((row ^ (row >> 3)) & (S::BN / 8 - 1));
}
template <typename S>
__device__ __forceinline__ int ns_staged(int row, int col)
{
    return row * S::BN * 2 + (ns_staged_chunk<S>(row, col / 8) << 4) + col % 8 * 2;
}

// 8 values to row `row`, columns col .. col + 7 of a matrix of `rows` rows of `cols`
// values: what lies inside.
__device__ __forceinline__ void ns_put(uint16_t* dst, const uint4& v, int row, int col, int rows, int cols, bool wide)
{
    if (row >= rows || col >= cols)
        return;
    uint16_t* at = dst + (size_t)row * cols + col;
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

// The tile row of row sr of a staged band: all of a tile's rows are staged, or (ONE)
// those of row fragment f of every wavefront.
template <typename S, bool ONE>
__device__ __forceinline__ int ns_tile_row(int sr, int f)
{
    return ONE ? sr / 32 * S::kWaveM + f * 32 + sr % 32 : sr;
}

// The staged rows to rows i0 .., columns j0 .. of dst.
template <typename S, bool ONE>
__device__ __forceinline__ void ns_write(const uint8_t* lds, uint16_t* dst, int f, int i0, int j0, int rows, int cols,
                                         bool wide)
{
    constexpr int kChunks = S::BN / 8, kRows = ONE ? S::WM * 32 : S::BM;
#pragma unroll 4
    for (int it = threadIdx.x; it < kRows * kChunks; it += S::kThreads) {
        const int r = it / kChunks, c = it % kChunks;
        const uint4 v = *reinterpret_cast<const uint4*>(lds + ns_staged<S>(r, 8 * c));
        ns_put(dst, v, i0 + ns_tile_row<S, ONE>(r, f), j0 + 8 * c, rows, cols, wide);
    }
}

// The staged rows, transposed, to rows j0 .., columns i0 .. of dst: a thread takes 8 rows
// of 4 columns.
template <typename S, bool ONE>
__device__ __forceinline__ void ns_write_transposed(const uint8_t* lds, uint16_t* dst, int f, int i0, int j0, int rows,
                                                    int cols, bool wide)
{
    constexpr int kChunks = (ONE ? S::WM * 32 : S::BM) / 8;
#pragma unroll 2
    for (int it = threadIdx.x; it < S::BN / 4 * kChunks; it += S::kThreads) {
        const int r = 8 * (it % kChunks), c = 4 * (it / kChunks);
        uint2 e[8];
#pragma unroll
        for (int q = 0; q < 8; ++q)
            e[q] = *reinterpret_cast<const uint2*>(lds + ns_staged<S>(r + q, c));
        const int col = i0 + ns_tile_row<S, ONE>(r, f);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            uint32_t w[4];
#pragma unroll
            for (int p = 0; p < 4; ++p)
                w[p] = __builtin_amdgcn_perm(q < 2 ? e[2 * p + 1].x : e[2 * p + 1].y, q < 2 ? e[2 * p].x : e[2 * p].y,
                                             q % 2 ? 0x07060302u : 0x05040100u);
            ns_put(dst, make_uint4(w[0], w[1], w[2], w[3]), j0 + c + q, col, rows, cols, wide);
        }
    }
}

// What the epilogue needs of a row-major operand at the output tile's place (A of POLY, X^T
// of UPDATE), into LDS in the staged order; it is replaced there by the output.
template <typename S, bool ONE>
__device__ __forceinline__ void ns_fetch(uint8_t* lds, const _Float16* src, int f, int i0, int j0, int rows, int cols)
{
    constexpr int kRows = ONE ? S::WM * 32 : S::BM, kChunks = S::BN / 8, kLoadRows = 64 / kChunks;
    static_assert(kRows % (kLoadRows * S::kWaves) == 0, "loads split evenly");
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = lane_id();
    const i32x4 rs = make_rsrc(src + (size_t)i0 * cols, (uint32_t)min(S::BM, rows - i0) * (uint32_t)cols * 2);
#pragma unroll
    for (int p = 0; p < kRows / (kLoadRows * S::kWaves); ++p) {
        const int first = (p * S::kWaves + wave) * kLoadRows, sr = first + lane / kChunks;
        const int r = ns_tile_row<S, ONE>(sr, f), c = j0 + 8 * ns_staged_chunk<S>(sr, lane % kChunks);
        const uint32_t voff = i0 + r < rows && c < cols ? ((uint32_t)r * (uint32_t)cols + c) * 2 : 0xf0000000u;
        dma16(rs, lds_addr(lds) + first * S::BN * 2, voff, 0);
    }
}

// Epilogue of the row fragments f0 .. f0 + N - 1 of every wavefront, whose sums are acc
// [0 .. N): the values that the next product reads.  `lds` is free.
template <typename S, int MODE, int N>
__device__ __forceinline__ void ns_store(const NsArgs& g, const NsStep& st, size_t mat, int ti, int tj, int f0,
                                         const f32x16 (&acc)[N][S::kFN], uint8_t* lds)
{
    constexpr bool ONE = N != S::kFM;
    const int i0 = ti * S::BM, j0 = tj * S::BN;
    int tid = threadIdx.x;
    __asm__ volatile("" : "+v"(tid));
    const int lane = tid & (kWave - 1), wave = tid / kWave;
    const int wm = wave / S::WN, wn = wave % S::WN;
    if constexpr (MODE == NS_POLY)
        ns_fetch<S, ONE>(lds, g.a + mat * g.m * g.mp, f0, i0, j0, g.m, g.mp);
    if constexpr (MODE == NS_UPDATE)
        ns_fetch<S, ONE>(lds, g.xt + ((size_t)st.src * g.count + mat) * g.n * g.mp, f0, i0, j0, g.n, g.mp);
    // what the columns of this lane need: c dA + b, or the diagonal of B
    f32x4 dj[S::kFN][4];
    if constexpr (MODE != NS_GRAM) {
        const float* d = (MODE == NS_POLY ? g.da : g.db) + mat * g.mp;
#pragma unroll
        for (int fj = 0; fj < S::kFN; ++fj)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int j = j0 + (fj / S::kHalfF) * S::kHalf + wn * S::kHalfN + (fj % S::kHalfF) * 32 + 8 * q + 4 * (lane >> 5);
                dj[fj][q] = *reinterpret_cast<const f32x4*>(d + min(j, g.mp - 4));
                if constexpr (MODE == NS_POLY)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        dj[fj][q][e] = fmaf(kNsC, dj[fj][q][e], kNsB);
            }
    }
    const float inv = 1.0f / g.sx;  // powers of two
    bool ready = false;
#pragma unroll
    for (int fi = 0; fi < N; ++fi) {
        const int sr = ONE ? wm * 32 + (lane & 31) : wm * S::kWaveM + fi * 32 + (lane & 31);
        const int ib = i0 + wm * S::kWaveM + (f0 + fi) * 32, i = ib + (lane & 31);
        const bool held_i = ib < (MODE == NS_UPDATE ? g.np : g.mp);
        // a fragment row's loads leave together: a store in between would hold them back
        f16x4 low[S::kFN][4];
        float di = 0.0f;
        if constexpr (MODE == NS_POLY)
            di = g.da[mat * g.mp + min(i, g.mp - 1)];
        if constexpr (MODE == NS_UPDATE)
#pragma unroll
            for (int fj = 0; fj < S::kFN; ++fj) {
                const int jb = j0 + (fj / S::kHalfF) * S::kHalf + wn * S::kHalfN + (fj % S::kHalfF) * 32;
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    low[fj][q] = held_i && jb < g.mp ? *reinterpret_cast<const f16x4*>(
                                                           g.low + ns_frag(g, mat, ib / 32, jb / 32) + q * 256 + lane * 4)
                                                     : f16x4{0, 0, 0, 0};
            }
        if (!ready) {  // the fetched tile has to be there
            wait_vmcnt<0>();
            lds_barrier();
            ready = true;
        }
#pragma unroll
        for (int fj = 0; fj < S::kFN; ++fj) {
            const int c0 = (fj / S::kHalfF) * S::kHalf + wn * S::kHalfN + (fj % S::kHalfF) * 32;
            if (!held_i || j0 + c0 >= g.mp)
                continue;
            const bool diagonal = MODE != NS_UPDATE && ib == j0 + c0;  // runs through this fragment
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int c = c0 + 8 * q + 4 * (lane >> 5), j = j0 + c;
                const f32x4 v = {acc[fi][fj][4 * q], acc[fi][fj][4 * q + 1], acc[fi][fj][4 * q + 2],
                                 acc[fi][fj][4 * q + 3]};
                f16x4* at = reinterpret_cast<f16x4*>(lds + ns_staged<S>(sr, c));
                f16x4 o;
                if constexpr (MODE == NS_GRAM) {
                    o = __builtin_convertvector(v * (inv * inv * kNsScale), f16x4);
                    if (diagonal)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (j + e == i) {
                                if (i < g.m)
                                    g.da[mat * g.mp + i] = v[e] * (inv * inv);
                                o[e] = (_Float16)0.0f;
                            }
                } else if constexpr (MODE == NS_POLY) {
                    // c (A A)_ij with A = O + diag: the square of O, and twice O's entry
                    const f16x4 a = *at;
                    f32x4 b;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        b[e] = fmaf(fmaf(kNsC, di, dj[fj][q][e]), (float)a[e], v[e] * (kNsC / kNsScale));
                    o = __builtin_convertvector(b, f16x4);
                    if (diagonal)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (j + e == i) {
                                if (i < g.m)
                                    g.db[mat * g.mp + i] =
                                        fmaf(kNsC, fmaf(di, di, v[e] * (1.0f / (kNsScale * kNsScale))), kNsB * di);
                                o[e] = (_Float16)0.0f;
                            }
                } else {
                    const f16x4 hi = *at;
                    f32x4 y;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float h = (float)hi[e], x = fmaf((float)low[fj][q][e], 1.0f / kNsLow, h);
                        y[e] = fmaf(kNsA, x, fmaf(dj[fj][q][e], st.fine ? x : h, v[e] * (1.0f / kNsScale)));
                    }
                    if (st.last) {
                        typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
                        o = __builtin_bit_cast(f16x4, __builtin_convertvector(y * inv, bf16x4));
                    } else {
                        f16x4 l;
                        o = __builtin_convertvector(y, f16x4);
                        l = __builtin_convertvector((y - __builtin_convertvector(o, f32x4)) * kNsLow, f16x4);
                        *reinterpret_cast<f16x4*>(g.low + ns_frag(g, mat, ib / 32, (j0 + c0) / 32) + q * 256 + lane * 4) = l;
                    }
                }
                *at = o;
            }
        }
    }
    lds_barrier();
    if constexpr (MODE != NS_UPDATE) {
        uint16_t* dst = reinterpret_cast<uint16_t*>(MODE == NS_GRAM ? g.a : g.b) + mat * g.m * g.mp;
        ns_write<S, ONE>(lds, dst, f0, i0, j0, g.m, g.mp, true);
        if (ti != tj)
            ns_write_transposed<S, ONE>(lds, dst, f0, i0, j0, g.m, g.mp, true);
    } else if (st.last) {
        uint16_t* dst = g.out + mat * g.rows * g.cols;
        if (g.rows > g.cols)
            ns_write<S, ONE>(lds, dst, f0, i0, j0, g.n, g.m, st.wide);
        else
            ns_write_transposed<S, ONE>(lds, dst, f0, i0, j0, g.m, g.n, st.wide);
    } else {
        uint16_t* xt = reinterpret_cast<uint16_t*>(g.xt) + ((size_t)(st.src ^ 1) * g.count + mat) * g.n * g.mp;
        ns_write<S, ONE>(lds, xt, f0, i0, j0, g.n, g.mp, true);
        ns_write_transposed<S, ONE>(lds, reinterpret_cast<uint16_t*>(g.x) + mat * g.m * g.np, f0, i0, j0, g.m, g.np,
                                    true);
    }
}

template <typename S, int MODE>
__global__ __launch_bounds__(S::kThreads) __attribute__((amdgpu_waves_per_eu(S::kWavesPerSimd, S::kWavesPerSimd)))
void moe_ns_product_kernel(NsArgs g, NsPlan plan, NsStep st)
{
#if defined(__HIP_DEVICE_COMPILE__)
    static_assert(S::BM * S::BN * 2 <= S::S * S::kStage, "the staged output tile fits the stages");
    __shared__ __attribute__((aligned(1024))) uint8_t lds[S::kLds];
    const int M = MODE == NS_UPDATE ? g.n : g.m, pitch = 2 * (MODE == NS_GRAM ? g.np : g.mp), nk = pitch / S::RB;
    // an XCD's blocks take neighbouring tiles; the parts of split ones come last
    int item = blockIdx.x, k0 = 0, k1 = nk, slot = -1;
    if (item < (plan.full + 7) / 8 * 8) {
        item = item % 8 * ((plan.full + 7) / 8) + item / 8;
        if (item >= plan.full)
            return;
    } else {
        item -= (plan.full + 7) / 8 * 8;
        const int part = item / plan.tail;
        if (part >= plan.parts)
            return;
        item %= plan.tail;
        slot = item * plan.parts + part;
        item += plan.full;
        k0 = part * nk / plan.parts;
        k1 = (part + 1) * nk / plan.parts;
    }
    const size_t mat = item / plan.tiles;
    int ti, tj;
    ns_tile<S, MODE>(g, item % plan.tiles, ti, tj);
    const int i0 = ti * S::BM, j0 = tj * S::BN;
    const _Float16* A = MODE == NS_GRAM ? g.x + mat * g.m * g.np
                        : MODE == NS_POLY ? g.a + mat * g.m * g.mp
                                          : g.xt + ((size_t)st.src * g.count + mat) * g.n * g.mp;
    const _Float16* W = MODE == NS_UPDATE ? g.b + mat * g.m * g.mp : A;

    const int lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
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
    struct Loads {
        const i32x4 &rsA, &rsW;
        const uint32_t (&voffA)[S::kBlkA], (&voffW)[S::kBlkW];
        uint32_t lds0;
        __device__ __forceinline__ void issue(int q, int stage, int n0, int n1) const
        {
            const uint32_t dst = lds0 + stage * S::kStage, soff = (uint32_t)q * S::RB;
#pragma unroll
            for (int p = 0; p < S::kLoads; ++p) {
                if (p < n0 || p >= n1)
                    continue;
                if (p < S::kBlkW)
                    dma16(rsW, dst + S::kLdsA + S::kWaves * p * 1024, voffW[p], soff);
                else
                    dma16(rsA, dst + S::kWaves * (p - S::kBlkW) * 1024, voffA[p - S::kBlkW], soff);
            }
        }
    };
    const Loads loads = {rsA, rsW, voffA, voffW, lds0 + wave * 1024};
    f32x16 acc[S::kFM][S::kFN];
    const int live = min(max((rowsA - wm * S::kWaveM + 31) / 32, 0), S::kFM);
    tile_product<S, NsOp>(acc, lds, wm, wn, live, k0, k1, loads);
    if (slot < 0) {
        ns_store<S, MODE, S::kFM>(g, st, mat, ti, tj, 0, acc, lds);
        return;
    }
    float* dst = g.partial + (size_t)slot * S::kTileFloats;
#pragma unroll
    for (int i = 0; i < S::kFM; ++i)
#pragma unroll
        for (int j = 0; j < S::kFN; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                *reinterpret_cast<f32x4*>(dst + ((((size_t)i * S::kWaves + wave) * S::kFN + j) * 4 + q) * 256 + lane * 4) =
                    f32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
#endif
}

// The split tiles' parts added in their order, and the epilogue: block (tile, row
// fragment).
template <typename S, int MODE>
__global__ __launch_bounds__(S::kThreads) void moe_ns_tail_kernel(NsArgs g, NsPlan plan, NsStep st)
{
#if defined(__HIP_DEVICE_COMPILE__)
    __shared__ __attribute__((aligned(1024))) uint8_t lds[S::WM * 32 * S::BN * 2];
    const int lane = lane_id(), wave = threadIdx.x / kWave;
    const int t = blockIdx.x / S::kFM, f = blockIdx.x % S::kFM, item = plan.full + t;
    const size_t mat = item / plan.tiles;
    int ti, tj;
    ns_tile<S, MODE>(g, item % plan.tiles, ti, tj);
    // none of the wavefronts' rows is there (those that only pad the transposed output are)
    if (ti * S::BM + f * 32 >= (MODE == NS_UPDATE ? g.np : g.mp))
        return;
    f32x16 acc[1][S::kFN];
#pragma unroll
    for (int j = 0; j < S::kFN; ++j)
#pragma unroll
        for (int v = 0; v < 16; ++v)
            acc[0][j][v] = 0.0f;
    const float* src = g.partial + (size_t)t * plan.parts * S::kTileFloats + (size_t)(f * S::kWaves + wave) * S::kFN * 1024 +
                       lane * 4;
    for (int part = 0; part < plan.parts; ++part, src += S::kTileFloats)
#pragma unroll
        for (int j = 0; j < S::kFN; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const f32x4 p = *reinterpret_cast<const f32x4*>(src + (j * 4 + q) * 256);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    acc[0][j][4 * q + e] += p[e];
            }
    ns_store<S, MODE, 1>(g, st, mat, ti, tj, f, acc, lds);
#endif
}

// ---------------------------------------------------------------- few rows
// Up to 64 rows the m x m side is small enough for 64 bits and for one workgroup.  Every
// iterate is a polynomial in A_0 = X X^T times X, and A_k goes along without X:
//   Q = a + b A + c A^2,   P <- Q P,   A <- Q A Q       (all commute, all symmetric)
// so the gradient is read twice (A_0, then P X) and the steps in between touch nothing
// else: three launches in place of 2 + 3 or more a step.  P grows to 3.44^steps where a
// singular value is close to zero, and an error of A_0 with it: A_0 and P are held in fp64
// (fp64 matrix cores; A_0's products of fp32 numbers are exact), and P X is an fp32
// product.  A singular value of zero stays one only as long as the
// roundings of P, of 3.44^steps 2^-24, stay small (after 13 steps a gradient of rank 3 had
// grown to 4e3), so longer runs take the tiles, whose X is rounded anew in every step and
// cannot outgrow the iteration's range.
constexpr int kFewRows = 64;
constexpr int kFewSteps = 7;
constexpr int kSlab = 64;         // columns of X at a time
constexpr int kSlabPitch = 68;    // of a slab in LDS, [column][row]: neither operand order meets in few banks
constexpr int kFewBytes = 1 << 19;  // partial sums of A_0 that one workgroup adds, at most

typedef double f64x4 __attribute__((ext_vector_type(4)));

struct NsFew {
    double* partial;  // [count][chunks][mt (mt + 1) / 2][256] partial A_0, tiles on and below the diagonal
    float* p;         // [count][16 mt][16 mt] P
    double* inv;      // [count] 1 / |U|
    int mt, chunks;   // 16-row tiles, workgroups a matrix in the first pass
};

// Columns k0 .. k0 + 63 of U into LDS; with the momentum's step where FIRST.
template <bool FIRST>
__device__ __forceinline__ void ns_load_slab(const NsArgs& g, size_t base, int k0, double scale, float* slab)
{
    const bool tall = g.rows > g.cols;
    const int tid = threadIdx.x;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        const int r = (tall ? k0 : 0) + tid / 16 + 16 * s, c = (tall ? 0 : k0) + tid % 16 * 4;
        f32x4 u = {0, 0, 0, 0};
        if (r < g.rows && c < g.cols) {
            const size_t at = base + (size_t)r * g.cols + c;
            const int held = min(4, g.cols - c);
            if constexpr (FIRST) {
                u = ns_load_grad(g, at, held);
                if (g.momentum) {
                    f32x4 m = ns_load_momentum(g, at, held);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        m[q] = fmaf(g.beta, m[q], u[q]);
                        u[q] = g.nesterov ? fmaf(g.beta, m[q], u[q]) : m[q];
                    }
                    if (g.vec && held == 4)
                        *reinterpret_cast<f32x4*>(g.momentum + at) = m;
                    else
                        for (int q = 0; q < held; ++q)
                            g.momentum[at + q] = m[q];
                }
            } else {
                u = ns_load_update(g, at, held);
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    u[q] = (float)(u[q] * scale);
            }
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int k = tall ? tid / 16 + 16 * s : tid % 16 * 4 + q, i = tall ? tid % 16 * 4 + q : tid / 16 + 16 * s;
            slab[k * kSlabPitch + i] = u[q];
        }
    }
}

// The tile on or below the diagonal with number t.
__device__ __forceinline__ void ns_few_tile(int t, int& ti, int& tj)
{
    ti = t < 1 ? 0 : t < 3 ? 1 : t < 6 ? 2 : 3;
    tj = t - ti * (ti + 1) / 2;
}

// Momentum and partial A_0: block (chunk of the columns, matrix).
__global__ __launch_bounds__(256) void moe_ns_few_gram_kernel(NsArgs g, NsFew w)
{
#if defined(__HIP_DEVICE_COMPILE__)
    __shared__ float slab[kSlab * kSlabPitch];
    const int lane = lane_id(), wave = threadIdx.x / kWave;
    const size_t mat = blockIdx.y, base = mat * g.rows * g.cols;
    const int tiles = w.mt * (w.mt + 1) / 2;
    f64x4 acc[3] = {};  // tiles wave, wave + 4, wave + 8
    for (int k0 = blockIdx.x * kSlab; k0 < g.n; k0 += w.chunks * kSlab) {
        __syncthreads();
        ns_load_slab<true>(g, base, k0, 1.0, slab);
        __syncthreads();
#pragma unroll
        for (int q = 0; q < 3; ++q) {
            const int t = wave + 4 * q;
            if (t >= tiles)
                continue;
            int ti, tj;
            ns_few_tile(t, ti, tj);
            const float* a = slab + (lane / 16) * kSlabPitch + ti * 16 + lane % 16;
            const float* b = slab + (lane / 16) * kSlabPitch + tj * 16 + lane % 16;
#pragma unroll 8
            for (int k = 0; k < kSlab; k += 4)
                acc[q] = __builtin_amdgcn_mfma_f64_16x16x4f64(a[k * kSlabPitch], b[k * kSlabPitch], acc[q], 0, 0, 0);
        }
    }
#pragma unroll
    for (int q = 0; q < 3; ++q)
        if (wave + 4 * q < tiles)
#pragma unroll
            for (int v = 0; v < 4; ++v)
                w.partial[((mat * w.chunks + blockIdx.x) * tiles + wave + 4 * q) * 256 + v * 64 + lane] = acc[q][v];
#endif
}

// The steps on A_0 in one workgroup per matrix, a wavefront per 16 x 16 tile on or below
// the diagonal, which it stores on both sides.
__global__ __launch_bounds__(640) void moe_ns_few_steps_kernel(NsArgs g, NsFew w, int steps)
{
#if defined(__HIP_DEVICE_COMPILE__)
    __shared__ double A[kFewRows][kFewRows], P[kFewRows][kFewRows], Q[kFewRows][kFewRows], T[kFewRows][kFewRows];
    const int lane = lane_id(), wave = threadIdx.x / kWave, M = 16 * w.mt, tiles = w.mt * (w.mt + 1) / 2;
    const size_t mat = blockIdx.x;
    int ti, tj;
    ns_few_tile(wave, ti, tj);
    // this lane's 4 elements of the tile: rows i0 + 4 v, column j
    const int i0 = ti * 16 + lane / 16, j = tj * 16 + lane % 16;
    auto store = [&](double (&x)[kFewRows][kFewRows], const f64x4& v) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            x[i0 + 4 * q][j] = v[q];
            if (ti != tj)
                x[j][i0 + 4 * q] = v[q];
        }
    };
    const double* src = w.partial + (mat * w.chunks * tiles + wave) * 256 + lane;
    f64x4 sum = {0, 0, 0, 0};
#pragma unroll 8
    for (int c = 0; c < w.chunks; ++c)
#pragma unroll
        for (int v = 0; v < 4; ++v)
            sum[v] += src[(size_t)c * tiles * 256 + v * 64];
    store(A, sum);
    __syncthreads();
    double trace = 0.0;
    for (int i = 0; i < g.m; ++i)
        trace += A[i][i];
    // zeros stay zeros; a NaN or an infinity anywhere makes the matrix NaN
    const double inv = trace == 0.0 ? 0.0 : trace * 0.0 + 1.0 / trace;
    if (threadIdx.x == 0)
        w.inv[mat] = trace == 0.0 ? 0.0 : trace * 0.0 + 1.0 / sqrt(trace);
    __syncthreads();
    store(A, sum * inv);
    __syncthreads();
    auto product = [&](const double (&x)[kFewRows][kFewRows], const double (&y)[kFewRows][kFewRows]) {
        f64x4 acc = {0, 0, 0, 0};
        for (int k = 0; k < M; k += 16)  // x is symmetric
#pragma unroll
            for (int q = lane / 16, n = 0; n < 4; ++n, q += 4)
                acc = __builtin_amdgcn_mfma_f64_16x16x4f64(x[k + q][ti * 16 + lane % 16], y[k + q][j], acc, 0, 0, 0);
        return acc;
    };
    for (int s = 0; s < steps; ++s) {
        f64x4 q = product(A, A);
#pragma unroll
        for (int v = 0; v < 4; ++v)
            q[v] = (double)kNsC * q[v] + (double)kNsB * A[i0 + 4 * v][j] + (i0 + 4 * v == j ? (double)kNsA : 0.0);
        store(Q, q);
        __syncthreads();
        f64x4 p = q;
        if (s > 0)
            p = product(Q, P);
        if (s + 1 < steps) {
            store(T, product(Q, A));
            __syncthreads();
            store(A, product(Q, T));  // T and Q are read only, and A no longer
        } else {
            __syncthreads();
        }
        store(P, p);
        __syncthreads();
    }
    for (int q = threadIdx.x; q < M * M; q += blockDim.x)
        w.p[mat * M * M + q] = (float)P[q / M][q % M];
#endif
}

// out = P X: block (chunk of the columns, matrix).
__global__ __launch_bounds__(256) void moe_ns_few_apply_kernel(NsArgs g, NsFew w)
{
#if defined(__HIP_DEVICE_COMPILE__)
    __shared__ float slab[kSlab * kSlabPitch];
    __shared__ float P[kFewRows * kSlabPitch];
    const int lane = lane_id(), wave = threadIdx.x / kWave, M = 16 * w.mt;
    const size_t mat = blockIdx.y, base = mat * g.rows * g.cols;
    for (int q = threadIdx.x; q < M * M; q += 256)
        P[q / M * kSlabPitch + q % M] = w.p[mat * M * M + q];
    const double inv = w.inv[mat];
    const bool tall = g.rows > g.cols;
    for (int k0 = blockIdx.x * kSlab; k0 < g.n; k0 += gridDim.x * kSlab) {
        __syncthreads();
        ns_load_slab<false>(g, base, k0, inv, slab);
        __syncthreads();
        // wavefront w: columns 16 w .. of the slab, 16 rows at a time
        for (int t = 0; t < w.mt; ++t) {
            f32x4 acc = {0, 0, 0, 0};
            const float* x = slab + (wave * 16 + lane % 16) * kSlabPitch + lane / 16;
            const float* p = P + (t * 16 + lane % 16) * kSlabPitch + lane / 16;
            for (int j = 0; j < M; j += 4)
                acc = __builtin_amdgcn_mfma_f32_16x16x4f32(p[j], x[j], acc, 0, 0, 0);
            const int k = k0 + wave * 16 + lane % 16;
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const int i = t * 16 + 4 * (lane / 16) + v;
                if (i < g.m && k < g.n)
                    g.out[base + (tall ? (size_t)k * g.cols + i : (size_t)i * g.cols + k)] =
                        (uint16_t)f32_to_bf16_bits(acc[v]);
            }
        }
    }
#endif
}

}  // namespace moe

namespace {
using namespace moe;

constexpr int kNsCus = 256;      // of gfx950
constexpr int kNsMaxParts = 16;  // K parts of a split tile
constexpr int kNsMinPart = 4;    // slices of a part
constexpr size_t kTilePart = size_t(1) << 30;  // bytes of the matrices of few rows that take the tiles at a time

size_t ns_round(size_t v) { return (v + 255) / 256 * 256; }

// A product's plan on tiles of one shape and its time in us, fitted to traces of 512 to
// 4096 rows, 512 to 14336 columns and 1 to 64 matrices (within a fifth; 128 x 128 tiles
// two to a CU).  With f the share of the blocks that run at a time:
//   a slice                        256: 0.95 + 0.75 f      128: 0.43 + 0.57 f
//   launch, first loads, epilogue  256: 15 (UPDATE 20 + 8 f)  128: 8 (UPDATE 10 + 5 f)
//   in parts: the tail kernel and the partial tiles' traffic in place of the epilogue
// Whole rounds of tiles stay in one piece; the rest goes in the number of parts along K
// that is the fastest.  Measured, 256 x 256 / split, 128 x 128 / split:
//   A of 1 of 500 x 6000     99 / 29   46 / 22     X of 64 of 1024 x 512   90 / 90   102 / 103
//   A of 16 of 1024 x 512    28 / 30   15 / 25     X of 16 of 1024 x 512   30 / 52    22 / 24
//   A of 1 of 2048 x 2048    44 / 40   22 / 25     X of 1 of 4096 x 4096  131 / 131  148 / 148
template <typename S>
double ns_plan(const NsArgs& g, int mode, NsPlan& p)
{
    const bool big = S::BM == 256;
    const long long tn = (g.m + S::BN - 1) / S::BN, tm = (g.n + S::BM - 1) / S::BM;
    p.tiles = (int)(mode == NS_UPDATE ? tm * tn : tn * (tn + 1) / 2);
    const int total = p.tiles * g.count, slots = kNsCus * S::kPerCu, nk = (mode == NS_GRAM ? g.np : g.mp) / 64;
    auto slice = [&](double f) { return big ? 0.95 + 0.75 * f : 0.43 + 0.57 * f; };
    auto round = [&](double f) {
        return (mode == NS_UPDATE ? (big ? 20 + 8 * f : 10 + 5 * f) : big ? 15.0 : 8.0) + nk * slice(f);
    };
    const int rest = total % slots;
    double time = total / slots * round(1.0), best = rest ? round((double)rest / slots) : 0.0;
    p.parts = 1;
    for (int parts = 2; rest && parts <= std::min(std::min(kNsMaxParts, slots / rest), nk / kNsMinPart); ++parts) {
        const double blocks = (double)rest * parts, mb = blocks * S::kTileFloats * 4e-6;
        const double t = (big ? 15.0 : 10.0) + (nk + parts - 1) / parts * slice(blocks / slots) + 0.5 * parts + 0.25 * mb;
        if (t < best)
            best = t, p.parts = parts;
    }
    p.tail = p.parts > 1 ? rest : 0;
    p.full = total - p.tail;
    return time + best;
}

// Whether a product takes the 256 x 256 tiles, and its plan.
bool ns_large(const NsArgs& g, int mode, NsPlan& p)
{
    NsPlan large, small;
    const bool is = ns_plan<NsLarge>(g, mode, large) <= ns_plan<NsSmall>(g, mode, small);
    p = is ? large : small;
    return is;
}

// Workgroups a matrix of the first pass over few rows: enough for every CU, as long as
// there are columns and the sums of one matrix are not too much for the workgroup that
// adds them.
NsFew few_plan(const NsArgs& g)
{
    NsFew w = {};
    w.mt = (g.m + 15) / 16;
    const int slabs = (g.n + kSlab - 1) / kSlab, most = kFewBytes / (w.mt * (w.mt + 1) / 2 * 256 * 8);
    w.chunks = std::min(std::min(slabs, most), std::max(1, 2 * kNsCus / g.count));
    return w;
}

size_t few_layout(NsFew& w, const NsArgs& g, char* ws)
{
    const size_t c = g.count, partial = ns_round(8 * c * w.chunks * (w.mt * (w.mt + 1) / 2) * 256);
    const size_t p = ns_round(4 * c * 256 * w.mt * w.mt);
    w.partial = (double*)ws;
    w.p = (float*)(ws + partial);
    w.inv = (double*)(ws + partial + p);
    return partial + p + ns_round(8 * c);
}

hipError_t launch_few(const NsArgs& g, int steps, char* ws, hipStream_t stream)
{
    NsFew w = few_plan(g);
    few_layout(w, g, ws);
    const int slabs = (g.n + kSlab - 1) / kSlab;
    moe_ns_few_gram_kernel<<<dim3(w.chunks, g.count), dim3(256), 0, stream>>>(g, w);
    moe_ns_few_steps_kernel<<<dim3(g.count), dim3(64 * (w.mt * (w.mt + 1) / 2)), 0, stream>>>(g, w, steps);
    moe_ns_few_apply_kernel<<<dim3(std::min(slabs, std::max(1, 8 * kNsCus / g.count)), g.count), dim3(256), 0, stream>>>(
        g, w);
    return hipGetLastError();
}

// The pieces of the workspace that grow with the number of matrices; returns their size.
size_t ns_pieces(NsArgs& g, char* ws)
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
    g.low = (_Float16*)take(2 * c * g.np * g.mp);
    g.a = (_Float16*)take(2 * square);
    g.b = (_Float16*)take(2 * square);
    g.da = (float*)take(4 * c * g.mp);
    g.db = (float*)take(4 * c * g.mp);
    g.sums = (double*)take(8 * c * kNsSums);
    return off;
}

// All of the tiles' workspace; returns its size.
size_t ns_layout(NsArgs& g, char* ws)
{
    const size_t off = ns_pieces(g, ws);
    size_t partial = 0;
    for (int mode : {NS_GRAM, NS_POLY, NS_UPDATE}) {
        NsPlan p;
        const int floats = ns_large(g, mode, p) ? NsLarge::kTileFloats : NsSmall::kTileFloats;
        partial = std::max(partial, (size_t)p.tail * p.parts * floats * 4);
    }
    g.partial = (float*)(ws + off);
    return off + ns_round(partial);
}

// Matrices that take the tiles at a time.  Up to 64 rows only runs of more than kFewSteps
// steps take them, on rows padded to 64, with up to a thousand times the bytes of the
// three kernels that the usual steps take.  The workspace, whose size does not know the
// steps, holds a part of such a batch: kTilePart bytes, or one matrix.  Eight steps in
// ms, the batch at once / in parts of 1 GiB / of 512 / of 256 MiB:
//   200 of 8 x 65536 (5.0 GB at once)    17.6 / 18.5 / 21.1 / 21.4
//   100 of 32 x 65536 (2.8 GB)            9.5 / 10.4 / 11.8 / 12.9
//   200 of 64 x 16384 (1.6 GB)            5.7 /  5.8 /  6.5 /  6.6
//   32768 of 32 x 32 (1.0 GB)             8.7 /  8.8 /  8.7 /  8.1
int tile_batch(const NsArgs& g)
{
    if (g.m > kFewRows || g.count == 0)
        return g.count;
    NsArgs one = g;
    one.count = 1;
    const size_t most = std::max<size_t>(1, kTilePart / ns_pieces(one, nullptr));
    const int parts = (int)((g.count + most - 1) / most);
    return (g.count + parts - 1) / parts;
}

// Bytes of the tiles' workspace: of a whole part of the batch, and of what is left.
size_t tile_bytes(NsArgs g)
{
    const int count = g.count;
    g.count = tile_batch(g);
    const int rest = count % g.count;
    size_t bytes = ns_layout(g, nullptr);
    if (rest) {
        g.count = rest;
        bytes = std::max(bytes, ns_layout(g, nullptr));
    }
    return bytes;
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

template <typename S, int MODE>
void launch_shape(const NsArgs& g, const NsPlan& p, const NsStep& st, hipStream_t stream)
{
    const dim3 grid((unsigned)((p.full + 7) / 8 * 8 + p.tail * p.parts)), block(S::kThreads);
    moe_ns_product_kernel<S, MODE><<<grid, block, 0, stream>>>(g, p, st);
    if (p.tail)
        moe_ns_tail_kernel<S, MODE><<<dim3((unsigned)(p.tail * S::kFM)), block, 0, stream>>>(g, p, st);
}

// How each of a step's products is run, the same in every step.
struct NsChoice {
    bool large;
    NsPlan plan;
};

template <int MODE>
void launch_product(const NsArgs& g, const NsChoice& c, const NsStep& st, hipStream_t stream)
{
    c.large ? launch_shape<NsLarge, MODE>(g, c.plan, st, stream) : launch_shape<NsSmall, MODE>(g, c.plan, st, stream);
}

// Momentum and start, and the steps' products.
void launch_tiles(NsArgs& g, int steps, char* ws, hipStream_t stream)
{
    ns_layout(g, ws);
    moe_ns_sums_kernel<<<dim3(g.parts, g.count), dim3(256), 0, stream>>>(g);
    moe_ns_init_kernel<<<dim3(g.mp / 64 * (g.np / 64), g.count), dim3(256), 0, stream>>>(g);
    NsChoice c[3];
    for (int mode : {NS_GRAM, NS_POLY, NS_UPDATE})
        c[mode].large = ns_large(g, mode, c[mode].plan);
    const bool wide = g.cols % 8 == 0 && reinterpret_cast<uintptr_t>(g.out) % 16 == 0;
    for (int s = 0; s < steps; ++s) {
        const NsStep st = {s & 1, s >= steps - 2, s == steps - 1, wide};
        launch_product<NS_GRAM>(g, c[NS_GRAM], st, stream);
        launch_product<NS_POLY>(g, c[NS_POLY], st, stream);
        launch_product<NS_UPDATE>(g, c[NS_UPDATE], st, stream);
    }
}
}  // namespace

extern "C" size_t moe_orthogonalize_scratch_bytes(int count, int rows, int cols)
{
    NsArgs g = ns_args(count, rows, cols);
    if (count == 0)
        return 0;
    size_t few = 0;
    if (g.m <= kFewRows) {  // the number of steps, which is not known here, decides
        NsFew w = few_plan(g);
        few = few_layout(w, g, nullptr);
    }
    return std::max(few, tile_bytes(g));
}

// dtype 0 fp32, 1 bf16 gradients [count][rows][cols]; momentum (nullable) fp32; out bf16.
extern "C" hipError_t moe_launch_orthogonalize(int dtype, const void* grad, float* momentum, float beta, int nesterov,
                                               int count, int rows, int cols, int steps, void* out, void* ws,
                                               hipStream_t stream)
{
    NsArgs g = ns_args(count, rows, cols);
    g.grad = grad, g.momentum = momentum, g.out = (uint16_t*)out;
    g.beta = beta, g.src_dtype = dtype, g.nesterov = nesterov;
    auto aligned = [](const void* p, size_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; };
    g.vec = cols % 4 == 0 && aligned(grad, dtype == 0 ? 16 : 8) && aligned(momentum, 16);
    if (g.m <= kFewRows && steps <= kFewSteps)
        return launch_few(g, steps, (char*)ws, stream);
    const size_t each = (size_t)rows * cols;
    for (int first = 0, part = tile_batch(g); first < count; first += part) {
        NsArgs p = g;
        p.count = std::min(part, count - first);
        p.grad = (const char*)grad + first * each * (dtype == 0 ? 4 : 2);
        p.momentum = momentum ? momentum + first * each : nullptr;
        p.out = g.out + first * each;
        launch_tiles(p, steps, (char*)ws, stream);
    }
    return hipGetLastError();
}
