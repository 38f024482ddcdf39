// The router's balance loss and its gradient.
//
// Over the n tokens that count (all of them, or those `valid` marks), with
// p_te = softmax_e(l_t) and c_e the number of their choices that name expert e:
//
//   P_e  = 1/n sum_t p_te,   f_e = E c_e / (k n),   loss = sum_e f_e P_e
//   d loss / d l_te = p_te (f_e - sum_j f_j p_tj) / n
//
// (f comes from the choices, which have no gradient.)  The loss is 1 when
// choices and probabilities are uniform.
//
// Forward: a warp takes one row of logits at a time, holds it in registers
// (E <= 1024, at most 32 values a lane) for maximum, exponentials and sum, and
// adds the probabilities to its own columns' registers; choices go to a
// shared-memory histogram.  A CTA's column sums meet the other CTAs' in a fixed
// order: within one thread-block cluster through distributed shared memory
// when at most 8 CTAs have work (one launch), else through the workspace in a
// second launch.  No floating-point atomics: results are reproducible bit for
// bit.  All sums are fp32.
// Backward: the row is read again and its softmax recomputed, which costs a
// read of the logits but no saved tensor as large as they are.
// Both are bound by the latency of their launches and of a row's two warp
// reductions at the sizes of a training micro-batch (8,192 x 512 bf16, whose 8.4 MB
// stay in L2: forward 10.0 us in two launches, backward 6.8 us), by launch latency
// at decode sizes (64 x 64 fp32: 4.2 and 2.1 us); 65,536 x 512: 29.9 and 30.5 us,
// 2.2 and 4.4 TB/s.  (Two rows of a warp at a time: 9.9 and 29.2 us forward, but 0.2 us
// more up to 2,048 tokens.)
#include <algorithm>

#include "op_common.cuh"

namespace moe {
namespace {

using namespace op;

constexpr int kBalWarps = 16, kBalThreads = 32 * kBalWarps;
constexpr int kBalCluster = 8;      // CTAs of the cluster that adds the column sums
constexpr int kBalMaxCtas = 148;    // CTAs with partial sums in the workspace
constexpr int kBalOneLaunch = 128;  // tokens of one cluster, a row a warp (512 tokens, 512 experts: 9.9 us; two launches 7.4)

// V consecutive values of a row: 16 bytes, or one where rows are not 16-byte aligned.
template <class T, int V>
struct Raw;
template <>
struct Raw<float, 4> {
    float4 r;
    __device__ __forceinline__ void load(const float *p) { r = *reinterpret_cast<const float4 *>(p); }
    __device__ __forceinline__ void fill() { r = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY); }
    __device__ __forceinline__ void values(float *v) const { v[0] = r.x, v[1] = r.y, v[2] = r.z, v[3] = r.w; }
    static __device__ __forceinline__ void store(float *p, const float *v)
    {
        *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
    }
};
template <>
struct Raw<__nv_bfloat16, 8> {
    uint4 r;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { r = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void fill() { r = make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u); }
    __device__ __forceinline__ void values(float *v) const
    {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ void store(__nv_bfloat16 *p, const float *v)
    {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&b);
        }
        *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <>
struct Raw<float, 1> {
    float r;
    __device__ __forceinline__ void load(const float *p) { r = *p; }
    __device__ __forceinline__ void fill() { r = -INFINITY; }
    __device__ __forceinline__ void values(float *v) const { v[0] = r; }
    static __device__ __forceinline__ void store(float *p, const float *v) { *p = v[0]; }
};
template <>
struct Raw<__nv_bfloat16, 1> {
    __nv_bfloat16 r;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { r = *p; }
    __device__ __forceinline__ void fill() { r = __ushort_as_bfloat16(0xff80); }
    __device__ __forceinline__ void values(float *v) const { v[0] = __bfloat162float(r); }
    static __device__ __forceinline__ void store(__nv_bfloat16 *p, const float *v) { *p = __float2bfloat16_rn(v[0]); }
};

// A lane's NV values of a row as loaded (bf16 in half the registers): value (i, j) is column
// (i * 32 + lane) * V + j, -inf behind the row's end.
template <class T, int NV, int V>
struct Row {
    Raw<T, V> raw[NV / V];
    __device__ __forceinline__ void load(const T *row, int E, int lane)
    {
#pragma unroll
        for (int i = 0; i < NV / V; ++i) {
            const int c = (i * 32 + lane) * V;
            raw[i].fill();
            if (c < E) raw[i].load(row + c);  // V > 1 only where E is a multiple of V
        }
    }
    __device__ __forceinline__ void values(float (&v)[NV]) const
    {
#pragma unroll
        for (int i = 0; i < NV / V; ++i) raw[i].values(v + i * V);
    }
};

// v becomes the row's probabilities.  A row of only -inf has none (all zero); a
// NaN or +inf makes the whole row NaN, as the definition does.
template <int NV>
__device__ __forceinline__ void row_softmax(float (&v)[NV])
{
    float m = v[0];
#pragma unroll
    for (int i = 1; i < NV; ++i) m = fmaxf(m, v[i]);
#pragma unroll
    for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    // fmaxf passes over NaN: those come back through 2^NaN below; with m = -inf subtract
    // 0 so that an empty row gives 2^-inf = 0.  exp(l - m) = 2^(l log2(e) - m log2(e)) in one
    // FMA: the rounding of m log2(e) is a factor of the whole row, within 2^+-0.07 up to |m| = 2^20,
    // and cancels.  Beyond that it could overflow (as m log2(e) itself does for a row of the
    // type's lowest value): such rows, seldom enough, subtract first.
    constexpr float log2e = 1.44269504f;
    if (fabsf(m) > 1048576.f && m != -INFINITY) {
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i] -= m;
        m = 0.f;
    }
    const float shift = m == -INFINITY ? 0.f : -m * log2e;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(v[i]) : "f"(__fmaf_rn(v[i], log2e, shift)));
        s += v[i];
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    const float inv = s == 0.f ? 0.f : 1.f / s;
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] *= inv;
}

struct BalanceArgs {
    const void *logits;
    const int32_t *idx;
    const uint8_t *valid;
    int T, E, k, ctas;
    float *psum;      // [ctas][E] workspace
    int32_t *pcount;  // [ctas][E]
    int32_t *pvalid;  // [ctas]
    int32_t *counts;
    float *prob_mean, *loss;
};

// Column sums, counts and P, f, loss from the partial sums of `ctas` CTAs: the
// cluster's CTA r owns columns [r * cols, (r + 1) * cols), at most 128 of them
// where the cluster is full.  Partials lie in the workspace, or in the cluster's
// shared memory (DSMEM, ctas = the cluster's size).
template <bool DSMEM>
__device__ void balance_reduce(const BalanceArgs &a, const float *s_sum, const int32_t *s_cnt, const int32_t *s_valid)
{
    __shared__ float red_p[kBalThreads], warp_loss[4];
    __shared__ int32_t red_c[kBalThreads];
    __shared__ int n_valid;
    __shared__ float loss_part;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const unsigned rank = cluster_rank(), ranks = cluster_size();
    const int cols = (int)((a.E + ranks - 1) / ranks);
    const int c0 = (int)rank * cols, c1 = min(a.E, c0 + cols);
    // 32, 64 or 128 columns at a time, the CTAs' partials over the rest of the threads
    const int shift = cols <= 32 ? 5 : cols <= 64 ? 6 : 7, width = 1 << shift, parts = kBalThreads >> shift;
    const int part = threadIdx.x >> shift, col = threadIdx.x & (width - 1);
    const uint32_t sum_at = DSMEM ? static_cast<uint32_t>(__cvta_generic_to_shared(s_sum)) : 0;
    const uint32_t cnt_at = DSMEM ? static_cast<uint32_t>(__cvta_generic_to_shared(s_cnt)) : 0;
    const uint32_t valid_at = DSMEM ? static_cast<uint32_t>(__cvta_generic_to_shared(s_valid)) : 0;

    if (warp == 0) {
        int n = 0;
        for (int g = lane; g < a.ctas; g += 32) n += DSMEM ? (int)cluster_ld_u32(cluster_map(valid_at, g)) : a.pvalid[g];
#pragma unroll
        for (int d = 16; d; d >>= 1) n += __shfl_xor_sync(0xffffffffu, n, d);
        if (lane == 0) n_valid = n;
    }
    float loss = 0.f;
    for (int cb = c0; cb < c1; cb += width) {
        const int c = cb + col;
        float p = 0.f;
        int cnt = 0;
        if (c < c1) {
            for (int g0 = part; g0 < a.ctas; g0 += 8 * parts) {
                float x[8];
                int y[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int g = g0 + i * parts;
                    x[i] = 0.f;
                    y[i] = 0;
                    if (g < a.ctas) {
                        x[i] = DSMEM ? cluster_ld_f32(cluster_map(sum_at, g) + 4 * c) : a.psum[(size_t)g * a.E + c];
                        y[i] = DSMEM ? (int)cluster_ld_u32(cluster_map(cnt_at, g) + 4 * c) : a.pcount[(size_t)g * a.E + c];
                    }
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    p += x[i];
                    cnt += y[i];
                }
            }
        }
        red_p[threadIdx.x] = p;
        red_c[threadIdx.x] = cnt;
        __syncthreads();
        if (part == 0 && c < c1) {
            for (int w = 1; w < parts; ++w) {
                p += red_p[(w << shift) + col];
                cnt += red_c[(w << shift) + col];
            }
            const double n = (double)max(n_valid, 1);
            p *= (float)(1.0 / n);
            a.prob_mean[c] = p;
            a.counts[c] = cnt;
            loss += (float)cnt * (float)((double)a.E / ((double)a.k * n)) * p;
        }
        __syncthreads();
    }
    if (warp < 4) {
#pragma unroll
        for (int d = 16; d; d >>= 1) loss += __shfl_xor_sync(0xffffffffu, loss, d);
        if (lane == 0) warp_loss[warp] = loss;
    }
    __syncthreads();
    if (threadIdx.x == 0) loss_part = (warp_loss[0] + warp_loss[1]) + (warp_loss[2] + warp_loss[3]);
    if (ranks > 1) cluster_sync();
    else __syncthreads();
    if (rank == 0 && threadIdx.x == 0) {
        const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(&loss_part));
        float x[kBalCluster], l = 0.f;
#pragma unroll
        for (unsigned r = 0; r < kBalCluster; ++r) x[r] = r < ranks ? (ranks > 1 ? cluster_ld_f32(cluster_map(at, r)) : loss_part) : 0.f;
#pragma unroll
        for (unsigned r = 0; r < kBalCluster; ++r) l += x[r];
        *a.loss = l;
        a.counts[a.E] = n_valid;
    }
    if (ranks > 1) cluster_sync();  // the other CTAs' shared memory is read until here
}

// CLUSTER: the grid is one cluster and finishes the loss itself.
template <class T, int NV, int V, bool CLUSTER>
__global__ void __launch_bounds__(kBalThreads, 1) balance_forward_kernel(const BalanceArgs a)
{
    extern __shared__ __align__(16) float bal_smem[];  // stored to 16 bytes at a time
    float *warp_cols = bal_smem;                                   // [kBalWarps][E]
    float *cta_sum = warp_cols + kBalWarps * a.E;                  // [E]
    int32_t *hist = reinterpret_cast<int32_t *>(cta_sum + a.E);    // [E]
    __shared__ int32_t cta_valid;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const T *logits = static_cast<const T *>(a.logits);
    for (int e = threadIdx.x; e < a.E; e += kBalThreads) hist[e] = 0;
    if (threadIdx.x == 0) cta_valid = 0;
    __syncthreads();
    follow_previous();

    float acc[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) acc[i] = 0.f;
    int n_valid = 0;
    const int step = gridDim.x * kBalWarps;
    int t = blockIdx.x * kBalWarps + warp;
    // the next row's logits, mask and choices are in flight while this one is summed
    Row<T, NV, V> next;
    int next_choice = -1;
    bool next_valid = true;
    const auto fetch = [&](int row) {
        next.load(logits + (size_t)row * a.E, a.E, lane);
        next_valid = !a.valid || a.valid[row];
        next_choice = lane < a.k ? a.idx[(size_t)row * a.k + lane] : -1;
    };
    if (t < a.T) fetch(t);
    for (; t < a.T; t += step) {
        float v[NV];
        next.values(v);
        const int choice = next_choice;
        const bool counted = next_valid;
        if (t + step < a.T) fetch(t + step);
        if (!counted) continue;
        ++n_valid;
        if ((unsigned)choice < (unsigned)a.E) atomicAdd(&hist[choice], 1);
        for (int j = 32 + lane; j < a.k; j += 32) {
            const int e = a.idx[(size_t)t * a.k + j];
            if ((unsigned)e < (unsigned)a.E) atomicAdd(&hist[e], 1);
        }
        row_softmax<NV>(v);
#pragma unroll
        for (int i = 0; i < NV; ++i) acc[i] += v[i];
    }
#pragma unroll
    for (int i = 0; i < NV / V; ++i) {
        const int c = (i * 32 + lane) * V;
        if (c >= a.E) continue;
        float *col = warp_cols + warp * a.E + c;
        if constexpr (V == 1) {
            *col = acc[i];
        } else {  // (E is a multiple of V; one value at a time all lanes meet in 32 / V banks: 0.75 us more)
#pragma unroll
            for (int j = 0; j < V; j += 4)
                *reinterpret_cast<float4 *>(col + j) =
                    make_float4(acc[i * V + j], acc[i * V + j + 1], acc[i * V + j + 2], acc[i * V + j + 3]);
        }
    }
    if (lane == 0 && n_valid) atomicAdd(&cta_valid, n_valid);
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += kBalThreads) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < kBalWarps; ++w) s += warp_cols[w * a.E + e];
        if (CLUSTER) {
            cta_sum[e] = s;
        } else {
            a.psum[(size_t)blockIdx.x * a.E + e] = s;
            a.pcount[(size_t)blockIdx.x * a.E + e] = hist[e];
        }
    }
    if (CLUSTER) {
        if (cluster_size() > 1) cluster_sync();
        else __syncthreads();
        balance_reduce<true>(a, cta_sum, hist, &cta_valid);
    } else {
        if (threadIdx.x == 0) a.pvalid[blockIdx.x] = cta_valid;
    }
}

__global__ void __launch_bounds__(kBalThreads, 1) balance_reduce_kernel(const BalanceArgs a)
{
    follow_previous();
    balance_reduce<false>(a, nullptr, nullptr, nullptr);
}

constexpr int kBwdWarps = 8, kBwdThreads = 32 * kBwdWarps;

template <class T, int NV, int V>
__global__ void __launch_bounds__(kBwdThreads)
    balance_backward_kernel(const T *logits, const int32_t *counts,
                            const uint8_t *valid, const float *dloss, int tokens, int E, int k,
                            T *dlogits)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    follow_previous();
    const double n = (double)max(counts[E], 1);
    const float to_share = (float)((double)E / ((double)k * n));
    const float scale = *dloss / (float)n;
    float f[NV];
#pragma unroll
    for (int i = 0; i < NV / V; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int c = (i * 32 + lane) * V + j;
            f[i * V + j] = c < E ? (float)counts[c] * to_share : 0.f;
        }
    // (a row ahead in registers costs more warps than it hides: 30.6 against 46.4 us at 65,536 x 512)
    for (int t = blockIdx.x * kBwdWarps + warp; t < tokens; t += gridDim.x * kBwdWarps) {
        float v[NV];
        Row<T, NV, V> row;
        row.load(logits + (size_t)t * E, E, lane);  // not held up by the mask
        row.values(v);
        if (!valid || valid[t]) {
            row_softmax<NV>(v);
            float dot = 0.f;
#pragma unroll
            for (int i = 0; i < NV; ++i) dot += f[i] * v[i];
#pragma unroll
            for (int d = 16; d; d >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, d);
#pragma unroll
            for (int i = 0; i < NV; ++i) v[i] = scale * v[i] * (f[i] - dot);
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i) v[i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < NV / V; ++i) {
            const int c = (i * 32 + lane) * V;
            if (c < E) Raw<T, V>::store(dlogits + (size_t)t * E + c, v + i * V);
        }
    }
}

size_t balance_smem(int E) { return sizeof(float) * (size_t)E * (kBalWarps + 2); }

typedef void (*ForwardKernel)(const BalanceArgs);

template <class T, int NV, int V>
ForwardKernel forward_of(bool cluster)
{
    return cluster ? balance_forward_kernel<T, NV, V, true> : balance_forward_kernel<T, NV, V, false>;
}

// Rows are read 16 bytes at a time where every row starts on a 16-byte
// boundary, else value by value.
template <class T, int W>
ForwardKernel forward_pick(int E, bool wide, bool cluster)
{
    if (wide) {
        if (E <= 256) return forward_of<T, 8, W>(cluster);
        return E <= 512 ? forward_of<T, 16, W>(cluster) : forward_of<T, 32, W>(cluster);
    }
    if (E <= 256) return forward_of<T, 8, 1>(cluster);
    return E <= 512 ? forward_of<T, 16, 1>(cluster) : forward_of<T, 32, 1>(cluster);
}

template <class T, int W>
auto backward_pick(int E, bool wide) -> decltype(&balance_backward_kernel<T, 8, W>)
{
    if (wide) {
        if (E <= 256) return balance_backward_kernel<T, 8, W>;
        return E <= 512 ? balance_backward_kernel<T, 16, W> : balance_backward_kernel<T, 32, W>;
    }
    if (E <= 256) return balance_backward_kernel<T, 8, 1>;
    return E <= 512 ? balance_backward_kernel<T, 16, 1> : balance_backward_kernel<T, 32, 1>;
}

bool wide_rows(const void *p, const void *q, moe_dtype dt, int E)
{
    return aligned(p, 16) && aligned(q, 16) && E % (dt == MOE_DT_BF16 ? 8 : 4) == 0;
}

// One cluster (as many CTAs as have rows, or columns to add up), or partial sums of every SM.
int forward_ctas(int T, int E)
{
    if (T > kBalOneLaunch) return std::min(kBalMaxCtas, ceil_div(T, kBalWarps));
    const int rows = ceil_div(T, kBalWarps), cols = ceil_div(E, 64), n = std::max(rows, cols);
    return n > 4 ? 8 : n > 2 ? 4 : std::max(n, 1);
}

PerDevice g_balance;

cudaError_t balance_prepare()
{
    for (int E : {256, 512, 1024})
        for (int wide = 0; wide < 2; ++wide)
            for (int cluster = 0; cluster < 2; ++cluster)
                for (int bf = 0; bf < 2; ++bf) {
                    ForwardKernel f = bf ? forward_pick<__nv_bfloat16, 8>(E, wide, cluster)
                                         : forward_pick<float, 4>(E, wide, cluster);
                    const cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                               (int)balance_smem(kMaxExperts));
                    if (e != cudaSuccess) return e;
                }
    return cudaSuccess;
}

bool balance_sizes_ok(moe_dtype dt, int T, int E, int k)
{
    return (dt == MOE_DT_F32 || dt == MOE_DT_BF16) && T >= 0 && T <= (1 << 30) && E >= 1 && E <= kMaxExperts && k >= 1 &&
           k <= E;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" size_t moe_balance_loss_workspace_bytes(int n_tokens, int n_experts)
{
    if (n_tokens <= 0 || n_experts < 1 || n_experts > kMaxExperts) return 0;
    const int ctas = forward_ctas(n_tokens, n_experts);
    return ctas <= kBalCluster ? 0 : (size_t)ctas * n_experts * 8 + (size_t)ctas * 4;
}

extern "C" moe_status moe_balance_loss(const void *logits, moe_dtype dtype, const int32_t *idx, const uint8_t *valid,
                                       int n_tokens, int n_experts, int top_k, float *loss, int32_t *counts,
                                       float *prob_mean, void *workspace, size_t workspace_bytes, void *stream)
{
    if (!balance_sizes_ok(dtype, n_tokens, n_experts, top_k)) return MOE_ERR_INVALID_ARG;
    if ((int64_t)n_tokens * top_k > INT32_MAX) return MOE_ERR_INVALID_ARG;  // one expert may have them all
    if (!loss || !counts || !prob_mean) return MOE_ERR_INVALID_ARG;
    if (n_tokens && (!logits || !idx)) return MOE_ERR_INVALID_ARG;
    if (!aligned(logits, dtype == MOE_DT_BF16 ? 2 : 4) || !aligned(idx, 4) || !aligned(loss, 4) ||
        !aligned(counts, 4) || !aligned(prob_mean, 4))
        return MOE_ERR_INVALID_ARG;
    const size_t need = moe_balance_loss_workspace_bytes(n_tokens, n_experts);
    if (need && (!workspace || !aligned(workspace, 16) || workspace_bytes < need)) return MOE_ERR_INVALID_ARG;
    int sms = 0;
    const moe_status st = g_balance.get(&sms, balance_prepare);
    if (st != MOE_OK) return st;
    BalanceArgs a{};
    a.logits = logits;
    a.idx = idx;
    a.valid = valid;
    a.T = n_tokens;
    a.E = n_experts;
    a.k = top_k;
    a.ctas = forward_ctas(n_tokens, n_experts);
    a.counts = counts;
    a.prob_mean = prob_mean;
    a.loss = loss;
    const bool cluster = a.ctas <= kBalCluster;
    if (!cluster) {
        a.psum = static_cast<float *>(workspace);
        a.pcount = reinterpret_cast<int32_t *>(a.psum + (size_t)a.ctas * n_experts);
        a.pvalid = a.pcount + (size_t)a.ctas * n_experts;
    }
    const bool wide = wide_rows(logits, nullptr, dtype, n_experts);
    ForwardKernel f = dtype == MOE_DT_BF16 ? forward_pick<__nv_bfloat16, 8>(n_experts, wide, cluster)
                                           : forward_pick<float, 4>(n_experts, wide, cluster);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = launch(f, dim3(a.ctas), kBalThreads, balance_smem(n_experts), s, cluster ? a.ctas : 1, a);
    if (e == cudaSuccess && !cluster)
        e = launch(balance_reduce_kernel, dim3(kBalCluster), kBalThreads, 0, s, kBalCluster, a);
    return launched(e);
}

extern "C" moe_status moe_balance_loss_backward(const void *logits, moe_dtype dtype, const int32_t *counts,
                                                const uint8_t *valid, const float *dloss, int n_tokens, int n_experts,
                                                int top_k, void *dlogits, void *stream)
{
    if (!balance_sizes_ok(dtype, n_tokens, n_experts, top_k)) return MOE_ERR_INVALID_ARG;
    if (n_tokens == 0) return MOE_OK;
    if (!logits || !counts || !dloss || !dlogits) return MOE_ERR_INVALID_ARG;
    const unsigned size = dtype == MOE_DT_BF16 ? 2 : 4;
    if (!aligned(logits, size) || !aligned(dlogits, size) || !aligned(counts, 4) || !aligned(dloss, 4))
        return MOE_ERR_INVALID_ARG;
    int sms = 0;
    const moe_status st = g_balance.get(&sms, balance_prepare);
    if (st != MOE_OK) return st;
    const bool wide = wide_rows(logits, dlogits, dtype, n_experts);
    const int grid = std::min(ceil_div(n_tokens, kBwdWarps), sms * 4);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e =
        dtype == MOE_DT_BF16
            ? launch(backward_pick<__nv_bfloat16, 8>(n_experts, wide), dim3(grid), kBwdThreads, 0, s, 1,
                     static_cast<const __nv_bfloat16 *>(logits), counts, valid, dloss, n_tokens, n_experts, top_k,
                     static_cast<__nv_bfloat16 *>(dlogits))
            : launch(backward_pick<float, 4>(n_experts, wide), dim3(grid), kBwdThreads, 0, s, 1,
                     static_cast<const float *>(logits), counts, valid, dloss, n_tokens, n_experts, top_k,
                     static_cast<float *>(dlogits));
    return launched(e);
}
