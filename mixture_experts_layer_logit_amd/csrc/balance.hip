// Balance loss of a batch of sequences, with per-expert counts and the
// gradient of the logits (gfx950).
//
// An auxiliary loss pushes experts towards equal loads (Megatron-Core page,
// "MoE负载均衡的挑战与应对"; Skywork-MoE news item, 技术创新 2) and the Z-loss
// (Megatron-Core page, "关键特性") bounds the logits.  Here the loads are those
// of one sequence each: sequence s holds the n_s tokens offsets[s] ..
// offsets[s + 1] - 1, S+ sequences hold any and N tokens lie in one.
//   f[s,e] = counts[s,e] / (n_s k), counts[s,e] = #{(t,j): topk_idx[t,j] = e}
//   aux = 1/S+ sum_s E sum_e f[s,e] (1/n_s) sum_t p[t,e]
//   Z   = 1/N sum_t lse(z_t)^2
// f is piecewise constant, so with p = softmax(s), s = z or its
// standardisation lambda zh, zh = (z - mu) / sigma:
//   ds = p (f - <p,f>), dz = ds or (lambda / sigma)(ds - mean ds - zh mean(ds zh))
//   dlogits = aux_coef E / (S+ n_s) dz + z_coef (2 / N) lse softmax(z)
// <p,f> is the token's term of aux too, so one pass over the logits gives the
// losses and the gradient.
#include "common.h"

namespace moe {

// Work split: four launches.  One clears the counts and finds S+ and N.  One
// counts: a block takes a run of tokens; a run inside one sequence is added in
// an LDS histogram and flushed, one with a border in it goes to memory
// directly, both with integer atomics, whose order does not change the counts.
// One does the rest: G lanes take a token, lane l the values 4 (l + G r) .. + 3
// of its row, so a row is read and written in 16-byte pieces and its sums stay
// in a few lanes (DPP steps up to 16 lanes); each block adds its tokens' terms
// in fp64 in a fixed order.  A last launch adds the blocks in a fixed order, so
// the sums have the same bits on every run (a ticket by which the last block to
// finish would do that needs a release fence in every block, which writes the
// gradients back from the XCDs' caches first: the launch took 42 us with it, 12
// without, for 65536 tokens of 64 experts; the launch it spares takes 4).
// A small batch takes one block that does all of it in one launch.
constexpr int kBalanceBlocks = 2048;
constexpr int kCountChunk = 256;      // tokens of a counting block
constexpr int kSeqTable = 1024;       // sequences whose borders are kept in LDS
constexpr int kMaxChoices = 8;        // k
constexpr int kSmallCells = 4096;     // counts the one-block form holds in LDS
constexpr int kSmallWork = 1 << 15;   // T * E up to which the one-block form is taken

struct BalanceArgs {
    const float* logits;
    const int32_t* topk_idx;
    const int32_t* offsets;  // nullable: one sequence
    int S, T, E, k, normalize;
    float lambda, aux_coef, z_coef;
    int32_t* counts;
    float* losses;
    float* dlogits;   // nullable
    int32_t* head;    // {S+, N}
    double* partial;  // [blocks][2]
};

// offsets[s] clamped into [0, T].
__device__ __forceinline__ int seq_at(const BalanceArgs& g, int s)
{
    if (g.offsets == nullptr)
        return s == 0 ? 0 : g.T;
    return min(max(g.offsets[s], 0), g.T);
}

// The clamped borders, from LDS where they fit.
struct Borders {
    const BalanceArgs& g;
    const int* table;
    __device__ __forceinline__ int operator()(int s) const { return g.S <= kSeqTable ? table[s] : seq_at(g, s); }
};
// Fills the table; a barrier has to follow.
__device__ __forceinline__ void load_borders(const BalanceArgs& g, int* table)
{
    if (g.S <= kSeqTable)
        for (int s = threadIdx.x; s <= g.S; s += blockDim.x)
            table[s] = seq_at(g, s);
}

// Largest s in [0, S) with border s <= t (0 if there is none).
__device__ __forceinline__ int seq_of(const Borders& at, int t)
{
    int lo = 0, hi = at.g.S;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (at(mid) <= t)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// {S+, N} by the threads of one block; the result on every thread.
template <int THREADS>
__device__ void seq_totals(const BalanceArgs& g, int& some, int& total)
{
    __shared__ int s_some[THREADS / kWave], s_total[THREADS / kWave];
    some = total = 0;
    for (int s = threadIdx.x; s < g.S; s += THREADS) {
        const int n = seq_at(g, s + 1) - seq_at(g, s);
        some += n > 0;
        total += max(n, 0);
    }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) {
        some += __shfl_xor(some, o);
        total += __shfl_xor(total, o);
    }
    if (lane_id() == 0) {
        s_some[threadIdx.x / kWave] = some;
        s_total[threadIdx.x / kWave] = total;
    }
    __syncthreads();
    some = total = 0;
    for (int w = 0; w < THREADS / kWave; ++w) {
        some += s_some[w];
        total += s_total[w];
    }
}

__global__ __launch_bounds__(256) void moe_balance_clear_kernel(BalanceArgs g)
{
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < (long long)g.S * g.E; i += 256ll * gridDim.x)
        g.counts[i] = 0;
    if (blockIdx.x != 0)
        return;
    int some, total;
    seq_totals<256>(g, some, total);
    if (threadIdx.x == 0) {
        g.head[0] = some;
        g.head[1] = total;
    }
}

__global__ __launch_bounds__(kCountChunk) void moe_balance_count_kernel(BalanceArgs g)
{
    __shared__ int s_hist[1024], s_table[kSeqTable + 1];
    const Borders at{g, s_table};
    const int t0 = blockIdx.x * kCountChunk, last = min(t0 + kCountChunk, g.T) - 1, t = t0 + threadIdx.x;
    int ids[kMaxChoices];  // loaded while the borders are
#pragma unroll
    for (int j = 0; j < kMaxChoices; ++j)
        ids[j] = j < g.k && t <= last ? g.topk_idx[(size_t)t * g.k + j] : -1;
    load_borders(g, s_table);
    for (int e = threadIdx.x; e < g.E; e += kCountChunk)
        s_hist[e] = 0;
    __syncthreads();
    const int s0 = seq_of(at, t0);
    if (at(s0) <= t0 && last < at(s0 + 1)) {  // the whole run lies in one sequence
#pragma unroll
        for (int j = 0; j < kMaxChoices; ++j)
            if (ids[j] >= 0 && ids[j] < g.E)
                atomicAdd(s_hist + ids[j], 1);
        __syncthreads();
        for (int e = threadIdx.x; e < g.E; e += kCountChunk)
            if (s_hist[e])
                atomicAdd(g.counts + (size_t)s0 * g.E + e, s_hist[e]);
        return;
    }
    const int s = seq_of(at, t);
    if (t < at(s) || t >= at(s + 1))
        return;
#pragma unroll
    for (int j = 0; j < kMaxChoices; ++j)
        if (ids[j] >= 0 && ids[j] < g.E)
            atomicAdd(g.counts + (size_t)s * g.E + ids[j], 1);
}

// Reductions over aligned groups of G lanes (1 .. 64); every lane gets the
// result.  Up to 16 lanes by DPP: partners i ^ 1, i ^ 2, then 7 - i and 15 - i,
// whose halves already agree.
template <int CTRL>
__device__ __forceinline__ float dpp(float v)
{
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, false));
}
template <int G, typename Op>
__device__ __forceinline__ float group_all(float v, Op op)
{
    if constexpr (G >= 2)
        v = op(v, dpp<0xb1>(v));
    if constexpr (G >= 4)
        v = op(v, dpp<0x4e>(v));
    if constexpr (G >= 8)
        v = op(v, dpp<0x141>(v));
    if constexpr (G >= 16)
        v = op(v, dpp<0x140>(v));
    if constexpr (G >= 32)
        v = op(v, __shfl_xor(v, 16));
    if constexpr (G >= 64)
        v = op(v, __shfl_xor(v, 32));
    return v;
}
template <int G>
__device__ __forceinline__ float group_sum(float v)
{
    return group_all<G>(v, [](float a, float b) { return a + b; });
}
template <int G>
__device__ __forceinline__ float group_top(float v)
{
    return group_all<G>(v, [](float a, float b) { return fmaxf(a, b); });
}

// Losses and gradients of the tokens first, first + step, ... below end, for
// one group of G lanes, lane li; every lane's aux and zl get the tokens' terms.
// VEC: rows are whole 16-byte pieces (E a multiple of 4, aligned pointers).
// All differences are taken from the row's largest logit first, so that a
// common offset of the logits costs no precision; the fp32 exponentials carry a
// relative error of about |difference| * 2^-23.
// The next token's row is loaded before the present one is worked on, the first
// one's before `ready()`, which makes the borders and the counts valid.
template <int G, int R, bool VEC, typename Ready>
__device__ __forceinline__ void balance_tokens(const BalanceArgs& g, const Borders& at, const int32_t* counts,
                                               const int& some, const int& total, int first, int step, int end,
                                               int li, double& aux, double& zl, Ready ready)
{
    constexpr int N = 4 * R;
    constexpr float kLog2e = 1.44269504088896341f;
    const int E = g.E;
    float zn[N];
    auto load_row = [&](int t) {
        const float* zt = g.logits + (size_t)min(t, g.T - 1) * E;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int e = 4 * (li + G * r);
            if constexpr (VEC) {
                const float4 v = *reinterpret_cast<const float4*>(zt + min(e, E - 4));
                zn[4 * r] = v.x, zn[4 * r + 1] = v.y, zn[4 * r + 2] = v.z, zn[4 * r + 3] = v.w;
            } else {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    zn[4 * r + q] = zt[min(e + q, E - 1)];
            }
        }
    };
    if (g.T > 0)
        load_row(first);
    ready();
    // reciprocals to within a step of fp32
    auto over = [](int n) { return __builtin_amdgcn_rcpf((float)max(n, 1)); };
    const float inv_e = over(E), inv_k = over(g.k);
    const float aux_all = g.aux_coef * (float)E * over(some), cz = 2.0f * g.z_coef * over(total);
    int s = seq_of(at, first), lo = at(s), hi = at(s + 1);
    float inv_n = over(hi - lo);
    for (int t = first; t < end; t += step) {
        float z[N], f[N];
#pragma unroll
        for (int i = 0; i < N; ++i)
            z[i] = zn[i];
        if (t + step < end)
            load_row(t + step);
        if (t >= hi && s + 1 < g.S) {
            do {
                ++s;
                lo = at(s);
                hi = at(s + 1);
            } while (t >= hi && s + 1 < g.S);
            inv_n = over(hi - lo);
        }
        if (t < lo || t >= hi)
            continue;  // in no sequence: the same on all lanes of the group
        const int32_t* ct = counts + (size_t)s * E;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int e = 4 * (li + G * r);
            if constexpr (VEC) {
                const int4 c = *reinterpret_cast<const int4*>(ct + min(e, E - 4));
                f[4 * r] = c.x, f[4 * r + 1] = c.y, f[4 * r + 2] = c.z, f[4 * r + 3] = c.w;
            } else {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    f[4 * r + q] = ct[min(e + q, E - 1)];
            }
        }
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const bool in = 4 * (li + G * (i / 4)) + i % 4 < E;
            z[i] = in ? z[i] : -INFINITY;
            f[i] = in ? f[i] * (inv_n * inv_k) : 0.0f;
            top = fmaxf(top, z[i]);
        }
        top = group_top<G>(top);
        const bool any = top > -INFINITY;  // a row of -inf alone adds nothing, one of NaN and -inf is NaN
        float q[N], sum = 0.0f, m = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            z[i] -= any ? top : 0.0f;
            q[i] = __builtin_amdgcn_exp2f(z[i] * kLog2e);
            sum += q[i];
            m += 4 * (li + G * (i / 4)) + i % 4 < E ? z[i] : 0.0f;
        }
        sum = group_sum<G>(sum);
        constexpr float kLn2 = 0.693147180559945309f;
        const float lse = any ? top + __builtin_amdgcn_logf(sum) * kLn2 : sum;  // sum: 0 or NaN
        const float inv = any ? __builtin_amdgcn_rcpf(sum) : sum;
        float p[N], inner = 0.0f, c = 1.0f;
        if (g.normalize) {
            // the differences by a power of two near their mean's, so that the
            // variance of very close logits does not underflow
            m = group_sum<G>(m) * inv_e;
            const int ex = __builtin_amdgcn_frexp_expf(m);
            float v = 0.0f;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                z[i] = 4 * (li + G * (i / 4)) + i % 4 < E ? ldexpf(z[i] - m, -ex) : 0.0f;
                v += z[i] * z[i];
            }
            v = group_sum<G>(v) * inv_e;
            const float rs = v > 0.0f ? __builtin_amdgcn_rsqf(v) : 0.0f;
            const float a = g.lambda * rs * kLog2e, high = ldexpf(-m, -ex) * a;  // the largest logit stands at -m
            sum = 0.0f;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                p[i] = 4 * (li + G * (i / 4)) + i % 4 < E ? __builtin_amdgcn_exp2f(z[i] * a - high) : 0.0f;
                z[i] *= rs;
                sum += p[i];
                inner += p[i] * f[i];
            }
            const float ip = __builtin_amdgcn_rcpf(group_sum<G>(sum));
            inner = group_sum<G>(inner) * ip;
#pragma unroll
            for (int i = 0; i < N; ++i)
                p[i] *= ip;
            c = g.lambda * ldexpf(rs, -ex);  // lambda / sigma
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                p[i] = q[i] * inv;
                inner += p[i] * f[i];
            }
            inner = group_sum<G>(inner);
        }
        aux += (double)(inner * inv_n);
        zl += (double)lse * lse;
        if (!g.dlogits)
            continue;
        float b = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            p[i] *= f[i] - inner;
            b += p[i] * z[i];
        }
        const float ca = aux_all * inv_n * c;
        if (g.normalize) {  // mean ds is zero: ds sums to <p,f> - <p,f>
            b = group_sum<G>(b) * inv_e;
#pragma unroll
            for (int i = 0; i < N; ++i)
                p[i] -= z[i] * b;
        }
        const float cq = cz * lse * inv;
        float* dt = g.dlogits + (size_t)t * E;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int e = 4 * (li + G * r);
            float d[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                d[i] = ca * p[4 * r + i] + cq * q[4 * r + i];
            if constexpr (VEC) {
                if (e < E)
                    *reinterpret_cast<float4*>(dt + e) = make_float4(d[0], d[1], d[2], d[3]);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (e + i < E)
                        dt[e + i] = d[i];
            }
        }
    }
}

// Sum over the block's groups of G lanes (each lane of a group holds the same
// pair) in a fixed order; the result on thread 0.
template <int G, int THREADS>
__device__ __forceinline__ void block_pair(double& a, double& b)
{
    __shared__ double s_pair[THREADS / kWave][2];
#pragma unroll
    for (int o = G; o < kWave; o <<= 1) {
        a += __shfl_xor(a, o);
        b += __shfl_xor(b, o);
    }
    if (lane_id() == 0) {
        s_pair[threadIdx.x / kWave][0] = a;
        s_pair[threadIdx.x / kWave][1] = b;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        a = b = 0.0;
        for (int w = 0; w < THREADS / kWave; ++w) {
            a += s_pair[w][0];
            b += s_pair[w][1];
        }
    }
}

__device__ __forceinline__ void store_losses(const BalanceArgs& g, double aux, double zl, int some, int total)
{
    g.losses[0] = some > 0 ? (float)(aux * g.E / some) : 0.0f;
    g.losses[1] = total > 0 ? (float)(zl / total) : 0.0f;
}

template <int G, int R, bool VEC>
__global__ __launch_bounds__(256) void moe_balance_kernel(BalanceArgs g)
{
    __shared__ int s_table[kSeqTable + 1];
    constexpr int kGroups = 256 / G;
    const Borders at{g, s_table};
    int some = 1, total = 1;
    // a run of consecutive tokens per block, so a group passes few sequences
    const int per = ((g.T + (int)gridDim.x - 1) / (int)gridDim.x + kGroups - 1) / kGroups * kGroups;
    const int t0 = min((long long)blockIdx.x * per, (long long)g.T), t1 = min(t0 + per, g.T);
    double aux = 0.0, zl = 0.0;
    balance_tokens<G, R, VEC>(g, at, g.counts, some, total, t0 + (int)threadIdx.x / G, kGroups, t1, threadIdx.x % G,
                              aux, zl, [&] {
                                  load_borders(g, s_table);
                                  some = g.head[0];
                                  total = g.head[1];
                                  __syncthreads();
                              });
    block_pair<G, 256>(aux, zl);
    if (threadIdx.x == 0) {
        g.partial[2 * blockIdx.x] = aux;
        g.partial[2 * blockIdx.x + 1] = zl;
    }
}

__global__ __launch_bounds__(1024) void moe_balance_final_kernel(BalanceArgs g, int blocks)
{
    double aux = 0.0, zl = 0.0;
#pragma unroll
    for (int i = 0; i < kBalanceBlocks / 1024; ++i) {
        const int b = threadIdx.x + 1024 * i;
        if (b < blocks) {
            const double2 v = reinterpret_cast<const double2*>(g.partial)[b];
            aux += v.x;
            zl += v.y;
        }
    }
    block_pair<1, 1024>(aux, zl);
    if (threadIdx.x == 0)
        store_losses(g, aux, zl, g.head[0], g.head[1]);
}

// The whole batch in one block.
template <int G, int R, bool VEC>
__global__ __launch_bounds__(1024) void moe_balance_small_kernel(BalanceArgs g)
{
    __shared__ __attribute__((aligned(16))) int s_counts[kSmallCells];
    __shared__ int s_table[kSeqTable + 1];
    const Borders at{g, s_table};
    int some, total;
    double aux = 0.0, zl = 0.0;
    auto count = [&] {
        load_borders(g, s_table);
        const int cells = g.S * g.E;
        for (int i = threadIdx.x; i < cells; i += 1024)
            s_counts[i] = 0;
        seq_totals<1024>(g, some, total);  // holds a barrier behind the clearing and the table
        for (int t = threadIdx.x; t < g.T; t += 1024) {
            const int s = seq_of(at, t);
            if (t < at(s) || t >= at(s + 1))
                continue;
            for (int j = 0; j < g.k; ++j) {
                const int e = g.topk_idx[(size_t)t * g.k + j];
                if (e >= 0 && e < g.E)
                    atomicAdd(s_counts + s * g.E + e, 1);
            }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < cells; i += 1024)
            g.counts[i] = s_counts[i];
    };
    balance_tokens<G, R, VEC>(g, at, s_counts, some, total, (int)threadIdx.x / G, 1024 / G, g.T, threadIdx.x % G, aux,
                              zl, count);
    block_pair<G, 1024>(aux, zl);
    if (threadIdx.x == 0)
        store_losses(g, aux, zl, some, total);
}

template <int G, int R, bool VEC>
void launch_balance(const BalanceArgs& g, hipStream_t stream)
{
    const long long cells = (long long)g.S * g.E;
    if ((long long)g.T * g.E <= kSmallWork && g.T <= kSmallWork / 4 && cells <= kSmallCells) {
        moe_balance_small_kernel<G, R, VEC><<<dim3(1), dim3(1024), 0, stream>>>(g);
        return;
    }
    const int clear = (int)(cells < 256ll * 1024 ? (cells + 255) / 256 : 1024);
    moe_balance_clear_kernel<<<dim3(clear), dim3(256), 0, stream>>>(g);
    if (g.T > 0)
        moe_balance_count_kernel<<<dim3((g.T + kCountChunk - 1) / kCountChunk), dim3(256), 0, stream>>>(g);
    const long long want = ((long long)g.T * G + 255) / 256;
    const int blocks = (int)(want < kBalanceBlocks ? want : kBalanceBlocks);
    if (blocks > 0)
        moe_balance_kernel<G, R, VEC><<<dim3(blocks), dim3(256), 0, stream>>>(g);
    moe_balance_final_kernel<<<dim3(1), dim3(1024), 0, stream>>>(g, blocks);
}

// The lanes of a token: as few as hold E values in 16 each (in 32 each from 257
// experts on), since each lane more costs the steps of the token's five sums.
template <bool VEC>
void pick_balance(const BalanceArgs& g, hipStream_t s)
{
    if (g.E <= 4)
        launch_balance<1, 1, VEC>(g, s);
    else if (g.E <= 8)
        launch_balance<1, 2, VEC>(g, s);
    else if (g.E <= 16)
        launch_balance<1, 4, VEC>(g, s);
    else if (g.E <= 32)
        launch_balance<2, 4, VEC>(g, s);
    else if (g.E <= 64)
        launch_balance<4, 4, VEC>(g, s);
    else if (g.E <= 128)
        launch_balance<8, 4, VEC>(g, s);
    else if (g.E <= 256)
        launch_balance<16, 4, VEC>(g, s);
    else if (g.E <= 512)
        launch_balance<16, 8, VEC>(g, s);
    else
        launch_balance<32, 8, VEC>(g, s);
}

}  // namespace moe

extern "C" size_t moe_balance_scratch_bytes(void)
{
    return 256 + sizeof(double) * 2 * moe::kBalanceBlocks;
}

// offsets (nullable: one sequence of all T tokens) holds S + 1 entries;
// dlogits nullable.  scratch: moe_balance_scratch_bytes bytes.  T >= 0.
extern "C" hipError_t moe_launch_balance(const float* logits, const int32_t* topk_idx, const int32_t* offsets, int S,
                                         int T, int E, int k, int normalize, float lambda, float aux_coef,
                                         float z_coef, int32_t* counts, float* losses, float* dlogits, void* scratch,
                                         hipStream_t stream)
{
    using namespace moe;
    const BalanceArgs g = {logits, topk_idx, offsets, S, T, E, k, normalize, lambda, aux_coef, z_coef, counts, losses,
                           dlogits, static_cast<int32_t*>(scratch),
                           reinterpret_cast<double*>(static_cast<char*>(scratch) + 256)};
    const uintptr_t at = (uintptr_t)logits | (uintptr_t)dlogits | (uintptr_t)counts;
    if (E % 4 == 0 && at % 16 == 0)
        pick_balance<true>(g, stream);
    else
        pick_balance<false>(g, stream);
    return hipGetLastError();
}
