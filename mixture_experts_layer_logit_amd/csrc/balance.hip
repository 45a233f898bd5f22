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

constexpr int kBalanceBlocks = 1024;

// offsets[s] clamped into [0, T].
__device__ __forceinline__ int seq_at(const int32_t* __restrict__ offsets, int S, int s, int T)
{
    if (offsets == nullptr)
        return s == 0 ? 0 : T;
    return min(max(offsets[s], 0), T);
}

// The sequence of token t, or -1.
__device__ __forceinline__ int seq_of(const int32_t* __restrict__ offsets, int S, int t, int T)
{
    int lo = 0, hi = S;  // largest s with offsets[s] <= t
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (seq_at(offsets, S, mid, T) <= t)
            lo = mid;
        else
            hi = mid;
    }
    return seq_at(offsets, S, lo, T) <= t && t < seq_at(offsets, S, lo + 1, T) ? lo : -1;
}

// counts = 0; head = {S+, N}.
__global__ __launch_bounds__(256) void moe_balance_clear_kernel(const int32_t* __restrict__ offsets, int S, int T,
                                                                int E, int32_t* __restrict__ counts,
                                                                int32_t* __restrict__ head)
{
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < (long long)S * E; i += 256ll * gridDim.x)
        counts[i] = 0;
    if (blockIdx.x != 0)
        return;
    __shared__ int s_some[256], s_total[256];
    int some = 0, total = 0;
    for (int s = threadIdx.x; s < S; s += 256) {
        const int n = seq_at(offsets, S, s + 1, T) - seq_at(offsets, S, s, T);
        some += n > 0;
        total += max(n, 0);
    }
    s_some[threadIdx.x] = some;
    s_total[threadIdx.x] = total;
    __syncthreads();
    for (int o = 128; o >= 1; o >>= 1) {
        if ((int)threadIdx.x < o) {
            s_some[threadIdx.x] += s_some[threadIdx.x + o];
            s_total[threadIdx.x] += s_total[threadIdx.x + o];
        }
        __syncthreads();
    }
    if (threadIdx.x == 0) {
        head[0] = s_some[0];
        head[1] = s_total[0];
    }
}

__global__ __launch_bounds__(256) void moe_balance_count_kernel(const int32_t* __restrict__ topk_idx,
                                                                const int32_t* __restrict__ offsets, int S, int T,
                                                                int E, int k, int32_t* __restrict__ counts)
{
    const int t = blockIdx.x * 256 + threadIdx.x;
    if (t >= T)
        return;
    const int s = seq_of(offsets, S, t, T);
    if (s < 0)
        return;
    for (int j = 0; j < k; ++j) {
        const int e = topk_idx[(size_t)t * k + j];
        if (e >= 0 && e < E)
            atomicAdd(counts + (size_t)s * E + e, 1);
    }
}

template <typename T>
__device__ __forceinline__ T wave_add(T v)
{
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1)
        v += __shfl_xor(v, o);
    return v;
}

__device__ __forceinline__ float wave_top(float v)
{
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1)
        v = fmaxf(v, __shfl_xor(v, o));
    return v;
}

template <int VPL>
__global__ __launch_bounds__(256) void moe_balance_kernel(const float* __restrict__ logits,
                                                          const int32_t* __restrict__ offsets, int S, int T, int E,
                                                          int k, int normalize, float lambda, float aux_coef,
                                                          float z_coef, const int32_t* __restrict__ counts,
                                                          const int32_t* __restrict__ head,
                                                          float* __restrict__ dlogits, double* __restrict__ partial)
{
    __shared__ double s_sum[4][2];
    const int lane = lane_id(), wave = threadIdx.x / kWave;
    const double some = head[0], total = head[1];
    double aux = 0.0, zl = 0.0;
    for (int t = blockIdx.x * 4 + wave; t < T; t += 4 * gridDim.x) {
        const int s = seq_of(offsets, S, t, T);
        if (s < 0)
            continue;
        const int n = seq_at(offsets, S, s + 1, T) - seq_at(offsets, S, s, T);
        const float* zt = logits + (size_t)t * E;
        float z[VPL], f[VPL], p[VPL], q[VPL];
        const float share = (float)(1.0 / ((double)n * k));
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const int e = lane + kWave * i;
            z[i] = e < E ? zt[e] : -INFINITY;
            f[i] = e < E ? (float)counts[(size_t)s * E + e] * share : 0.0f;
            top = fmaxf(top, z[i]);
        }
        top = wave_top(top);
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            q[i] = z[i] > -INFINITY ? expf(z[i] - top) : 0.0f;
            sum += q[i];
        }
        sum = wave_add(sum);
        const bool any = top > -INFINITY;  // a row of -inf alone adds nothing
        const float lse = any ? top + logf(sum) : 0.0f;
        const float inv = any ? 1.0f / sum : 0.0f;
        double mu = 0.0, sigma = 0.0;
        if (normalize) {
            double m = 0.0;
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                m += lane + kWave * i < E ? (double)z[i] : 0.0;
            mu = wave_add(m) / E;
            m = 0.0;
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                m += lane + kWave * i < E ? ((double)z[i] - mu) * ((double)z[i] - mu) : 0.0;
            sigma = sqrt(wave_add(m) / E);
            const double r = sigma > 0.0 ? lambda / sigma : 0.0;
            const float high = (float)(((double)top - mu) * r);
            sum = 0.0f;
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                p[i] = lane + kWave * i < E ? expf((float)(((double)z[i] - mu) * r) - high) : 0.0f;
                sum += p[i];
            }
            sum = 1.0f / wave_add(sum);
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                p[i] *= sum;
        } else {
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                p[i] = q[i] * inv;
        }
        float inner = 0.0f;
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            inner += p[i] * f[i];
        inner = wave_add(inner);
        aux += (double)inner / n;
        zl += (double)lse * lse;
        if (!dlogits)
            continue;
        float ds[VPL];
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            ds[i] = p[i] * (f[i] - inner);
        if (normalize) {
            const double r = sigma > 0.0 ? 1.0 / sigma : 0.0;
            float a = 0.0f, b = 0.0f, zh[VPL];
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                zh[i] = lane + kWave * i < E ? (float)(((double)z[i] - mu) * r) : 0.0f;
                a += ds[i];
                b += ds[i] * zh[i];
            }
            a = wave_add(a) / E;
            b = wave_add(b) / E;
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                ds[i] = (float)(lambda * r) * (ds[i] - a - zh[i] * b);
        }
        const float ca = (float)((double)aux_coef * E / (some * n)), cz = (float)(2.0 * z_coef / total) * lse * inv;
        float* dt = dlogits + (size_t)t * E;
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (lane + kWave * i < E)
                dt[lane + kWave * i] = ca * ds[i] + cz * q[i];
    }
    if (lane == 0) {
        s_sum[wave][0] = aux;
        s_sum[wave][1] = zl;
    }
    __syncthreads();
    if (threadIdx.x < 2)
        partial[2 * blockIdx.x + threadIdx.x] =
            ((s_sum[0][threadIdx.x] + s_sum[1][threadIdx.x]) + s_sum[2][threadIdx.x]) + s_sum[3][threadIdx.x];
}

__global__ __launch_bounds__(128) void moe_balance_final_kernel(const double* __restrict__ partial, int blocks, int E,
                                                                const int32_t* __restrict__ head,
                                                                float* __restrict__ losses)
{
    const int which = threadIdx.x / kWave;
    double sum = 0.0;
    for (int b = lane_id(); b < blocks; b += kWave)
        sum += partial[2 * b + which];
    sum = wave_add(sum);
    if (lane_id() == 0) {
        const double n = head[which];
        losses[which] = n > 0.0 ? (float)(which ? sum / n : sum * E / n) : 0.0f;
    }
}

}  // namespace moe

extern "C" size_t moe_balance_scratch_bytes(int T, int S)
{
    (void)T;
    (void)S;
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
    int32_t* head = static_cast<int32_t*>(scratch);
    double* partial = reinterpret_cast<double*>(static_cast<char*>(scratch) + 256);
    const long long cells = (long long)S * E;
    const int clear = (int)(cells + 255 < 256ll * 1024 ? (cells + 255) / 256 : 1024);
    moe_balance_clear_kernel<<<dim3(clear), dim3(256), 0, stream>>>(offsets, S, T, E, counts, head);
    const int blocks = T < 4 * kBalanceBlocks ? (T + 3) / 4 : kBalanceBlocks;
    if (T > 0) {
        moe_balance_count_kernel<<<dim3((T + 255) / 256), dim3(256), 0, stream>>>(topk_idx, offsets, S, T, E, k,
                                                                                 counts);
#define GO(V)                                                                                                        \
    moe_balance_kernel<V><<<dim3(blocks), dim3(256), 0, stream>>>(logits, offsets, S, T, E, k, normalize, lambda,    \
                                                                  aux_coef, z_coef, counts, head, dlogits, partial)
        if (E <= 64)
            GO(1);
        else if (E <= 128)
            GO(2);
        else if (E <= 256)
            GO(4);
        else if (E <= 512)
            GO(8);
        else
            GO(16);
#undef GO
    }
    moe_balance_final_kernel<<<dim3(1), dim3(128), 0, stream>>>(partial, blocks, E, head, losses);
    return hipGetLastError();
}
