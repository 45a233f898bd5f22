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
    float* x32;       // [count][n][mp]
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
#pragma unroll
    for (int k = 0; k < 32; k += 8) {
        int i = i0 + ty + k, j = j0 + tx;
        if (i < g.m)
            g.x[(mat * g.m + i) * g.np + j] = (_Float16)(tile[ty + k][tx] * g.sx);
        i = i0 + tx, j = j0 + ty + k;
        if (j < g.n && i < g.mp) {
            const size_t at = (mat * g.n + j) * g.mp + i;
            const float v = tile[tx][ty + k];
            g.x32[at] = v;
            g.xt[at] = (_Float16)(v * g.sx);
            if (i >= g.m)
                g.xt[cells + at] = (_Float16)0.0f;
        }
    }
    if (j0 == 0)  // the padded columns of A and B
        for (int q = threadIdx.x; q < 32 * (g.mp - g.m); q += 256) {
            const int i = i0 + q % 32;
            if (i < g.m) {
                const size_t at = (mat * g.m + i) * g.mp + g.m + q / 32;
                g.a[at] = (_Float16)0.0f;
                g.b[at] = (_Float16)0.0f;
            }
        }
}

// ---------------------------------------------------------------- the products
enum { NS_GRAM = 0, NS_POLY = 1, NS_UPDATE = 2 };

// Epilogue of 4 consecutive columns j.. of row i of a product, one column a time
// where they end behind the last.
template <int MODE>
__device__ __forceinline__ void ns_store(const NsArgs& g, size_t mat, int i, int j, const float* acc, int src,
                                         bool fine, bool last)
{
    for (int q = 0; q < 4 && j + q < g.m; ++q) {
        const int c = j + q;
        const float v = acc[q];
        if constexpr (MODE == NS_GRAM) {
            const float s = v / (g.sx * g.sx);
            g.a[(mat * g.m + i) * g.mp + c] = (_Float16)(c == i ? 0.0f : s * kNsScale);
            if (c == i)
                g.da[mat * g.mp + i] = s;
        } else if constexpr (MODE == NS_POLY) {
            const float di = g.da[mat * g.mp + i], dj = g.da[mat * g.mp + c];
            const float o = (float)g.a[(mat * g.m + i) * g.mp + c] / kNsScale;
            const float sq = v / (kNsScale * kNsScale);
            if (c == i)
                g.db[mat * g.mp + i] = fmaf(kNsC, fmaf(di, di, sq), kNsB * di);
            const float b = fmaf(kNsC, fmaf(di + dj, o, sq), kNsB * o);
            g.b[(mat * g.m + i) * g.mp + c] = (_Float16)(c == i ? 0.0f : b * kNsScale);
        } else {
            const size_t at = (mat * g.n + i) * g.mp + c;
            const float x = g.x32[at];
            const float xr = fine ? x : (float)(_Float16)(x * g.sx) / g.sx;
            const float y = fmaf(kNsA, x, fmaf(g.db[mat * g.mp + c], xr, v / (kNsScale * g.sx)));
            if (last) {
                const bool tall = g.rows > g.cols;
                g.out[mat * g.rows * g.cols + (tall ? (size_t)i * g.cols + c : (size_t)c * g.cols + i)] =
                    (uint16_t)f32_to_bf16_bits(y);
            } else {
                const size_t cells = (size_t)g.count * g.n * g.mp;
                g.x32[at] = y;
                g.xt[(src ^ 1) * cells + at] = (_Float16)(y * g.sx);
                g.x[(mat * g.m + c) * g.np + i] = (_Float16)(y * g.sx);
            }
        }
    }
}

// One wavefront per 32 x 32 tile, fragments from memory: block (4 tiles, matrix).
template <int MODE>
__global__ __launch_bounds__(256) void moe_ns_product_kernel(NsArgs g, int src, bool fine, bool last)
{
#if defined(__HIP_DEVICE_COMPILE__)
    const int lane = lane_id(), wave = threadIdx.x / kWave, half = lane >> 5;
    const int M = MODE == NS_UPDATE ? g.n : g.m, K = MODE == NS_GRAM ? g.np : g.mp;
    const int tn = (g.m + 31) / 32, tm = (M + 31) / 32;
    const int tile = blockIdx.x * 4 + wave;
    if (tile >= tn * tm)
        return;
    const size_t mat = blockIdx.y;
    const int i = tile / tn * 32 + (lane & 31), j0 = tile % tn * 32;
    const _Float16* A = MODE == NS_GRAM ? g.x + mat * g.m * g.np
                        : MODE == NS_POLY ? g.a + mat * g.m * g.mp
                                          : g.xt + ((size_t)src * g.count + mat) * g.n * g.mp;
    const _Float16* W = MODE == NS_UPDATE ? g.b + mat * g.m * g.mp : A;
    A += (size_t)min(i, M - 1) * K + 8 * half;
    W += (size_t)min(j0 + (lane & 31), g.m - 1) * K + 8 * half;
    f32x16 acc = {};
    for (int k = 0; k < K; k += 16)
        acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(*reinterpret_cast<const f16x8*>(W + k),
                                                     *reinterpret_cast<const f16x8*>(A + k), acc, 0, 0, 0);
    if (i < M)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float v[4] = {acc[4 * q], acc[4 * q + 1], acc[4 * q + 2], acc[4 * q + 3]};
            ns_store<MODE>(g, mat, i, j0 + 8 * q + 4 * half, v, src, fine, last);
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
    g.x32 = (float*)take(4 * cells);
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
    const int tm = (g.m + 31) / 32, tn = (g.n + 31) / 32;
    moe_ns_init_kernel<<<dim3(g.mp / 32 * (g.np / 32), count), dim3(256), 0, stream>>>(g);
    for (int s = 0; s < steps; ++s) {
        const bool fine = s >= steps - 2, last = s == steps - 1;
        const dim3 sq((tm * tm + 3) / 4, count), up((tm * tn + 3) / 4, count), block(256);
        moe_ns_product_kernel<NS_GRAM><<<sq, block, 0, stream>>>(g, s & 1, fine, last);
        moe_ns_product_kernel<NS_POLY><<<sq, block, 0, stream>>>(g, s & 1, fine, last);
        moe_ns_product_kernel<NS_UPDATE><<<up, block, 0, stream>>>(g, s & 1, fine, last);
    }
    return hipGetLastError();
}
