// The expert plan: (token, choice) pairs sorted by expert, stable, with the
// experts' counts and row offsets.
//
//   counts[e]  = #{p : idx[p] = e}
//   offsets[e] = sum of counts[0..e)
//   slots[p]   = offsets[idx[p]] + #{q < p : idx[q] = idx[p]}
//   rows[slots[p]] = p / top_k
//
// A counting sort in one launch of one thread-block cluster.  Every warp owns a
// contiguous range of pairs and one row of a per-warp histogram in shared
// memory; 32 pairs at a time, __match_any_sync groups the lanes that chose the
// same expert, so a warp needs no atomics and the rank of a pair inside its
// group is the number of lower lanes in it.  The histograms are scanned over
// the CTA's warps, the CTAs' totals over the cluster (distributed shared
// memory), the experts' totals over the block; a second pass over the same
// pairs writes slots and rows.  No atomics anywhere: the order is that of the
// definition, and no workspace has to be kept or cleared.
//
// The work is latency: 12 bytes a pair (index read, slot and row written).
#include <algorithm>

#include "op_common.cuh"

namespace moe {
namespace {

using namespace op;

constexpr int kPlanThreads = 1024, kPlanWarps = kPlanThreads / 32;
constexpr int kPlanBatch = 4;  // index loads in flight per lane

__device__ __forceinline__ int load_choice(const int32_t *idx, int p, int end, int E)
{
    const int e = p < end ? __ldg(idx + p) : -1;
    return (unsigned)e < (unsigned)E ? e : -1;
}

__global__ void __launch_bounds__(kPlanThreads, 1)
    expert_plan_kernel(const int32_t *__restrict__ idx, int P, int k, int E, int warps, int32_t *__restrict__ counts,
                       int32_t *__restrict__ offsets, int32_t *__restrict__ rows, int32_t *__restrict__ slots)
{
    extern __shared__ int32_t smem[];
    int32_t *total = smem;           // [E] this CTA's pairs per expert (read by the cluster)
    int32_t *base = total + E;       // [E] first slot of this CTA's pairs of each expert
    int32_t *hist = base + E;        // [warps][E]
    __shared__ int32_t warp_sum[kPlanWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const unsigned rank = cluster_rank(), ctas = cluster_size();

    for (int i = threadIdx.x; i < warps * E; i += kPlanThreads) hist[i] = 0;
    __syncthreads();

    const int n_warps = warps * (int)ctas;
    const int chunk = (int)((((int64_t)P + n_warps - 1) / n_warps + 31) & ~31ll);
    const int64_t first = (int64_t)(rank * warps + warp) * chunk;
    const int begin = warp < warps && first < P ? (int)first : P;
    const int end = first + chunk < P ? (int)(first + chunk) : P;
    int32_t *own = hist + (warp < warps ? warp : 0) * E;
    for (int p0 = begin; p0 < end; p0 += 32 * kPlanBatch) {
        int e[kPlanBatch];
#pragma unroll
        for (int b = 0; b < kPlanBatch; ++b) e[b] = load_choice(idx, p0 + 32 * b + lane, end, E);
#pragma unroll
        for (int b = 0; b < kPlanBatch; ++b) {
            const unsigned same = __match_any_sync(0xffffffffu, e[b]);
            if (e[b] >= 0 && lane == __ffs(same) - 1) own[e[b]] += __popc(same);
            __syncwarp();
        }
    }
    __syncthreads();

    // over the CTA's warps: hist becomes the pairs of earlier warps
    for (int e = threadIdx.x; e < E; e += kPlanThreads) {
        int run = 0;
        for (int w = 0; w < warps; ++w) {
            const int n = hist[w * E + e];
            hist[w * E + e] = run;
            run += n;
        }
        total[e] = run;
    }
    if (ctas > 1) cluster_sync();
    else __syncthreads();

    // over the cluster, then over the experts (E <= the block's threads)
    int all = 0, before = 0;
    if (threadIdx.x < E) {
        if (ctas > 1) {
            const uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(total + threadIdx.x));
            for (unsigned c = 0; c < ctas; ++c) {
                const int n = (int)cluster_ld_u32(cluster_map(a, c));
                if (c < rank) before += n;
                all += n;
            }
        } else {
            all = total[threadIdx.x];
        }
    }
    int scan = all;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, scan, d);
        if (lane >= d) scan += v;
    }
    if (lane == 31) warp_sum[warp] = scan;
    __syncthreads();
    if (warp == 0) {
        int v = warp_sum[lane];
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, v, d);
            if (lane >= d) v += u;
        }
        warp_sum[lane] = v;
    }
    __syncthreads();
    const int upto = scan + (warp ? warp_sum[warp - 1] : 0);  // pairs of experts <= this thread's
    const int used = warp_sum[kPlanWarps - 1];
    if (threadIdx.x < E) {
        base[threadIdx.x] = upto - all + before;
        if (rank == 0) {
            counts[threadIdx.x] = all;
            offsets[threadIdx.x] = upto - all;
            if (threadIdx.x == E - 1) offsets[E] = upto;
        }
    }
    __syncthreads();

    for (int p0 = begin; p0 < end; p0 += 32 * kPlanBatch) {
        int e[kPlanBatch];
#pragma unroll
        for (int b = 0; b < kPlanBatch; ++b) e[b] = load_choice(idx, p0 + 32 * b + lane, end, E);
#pragma unroll
        for (int b = 0; b < kPlanBatch; ++b) {
            const int p = p0 + 32 * b + lane;
            const unsigned same = __match_any_sync(0xffffffffu, e[b]);
            int slot = -1;
            if (e[b] >= 0) {
                slot = base[e[b]] + own[e[b]] + __popc(same & ((1u << lane) - 1));
                rows[slot] = p / k;
            }
            __syncwarp();
            if (e[b] >= 0 && lane == __ffs(same) - 1) own[e[b]] += __popc(same);
            __syncwarp();
            if (p < end) slots[p] = slot;
        }
    }
    // rows behind the last group belong to no token
    for (int64_t s = used + (int64_t)rank * kPlanThreads + threadIdx.x; s < P; s += (int64_t)ctas * kPlanThreads)
        rows[s] = -1;
    if (ctas > 1) cluster_sync();  // `total` is read by the other CTAs until here
}

size_t plan_smem(int E, int warps) { return sizeof(int32_t) * (size_t)E * (2 + warps); }

PerDevice g_plan;

cudaError_t plan_prepare()
{
    return cudaFuncSetAttribute(expert_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)plan_smem(kMaxExperts, kPlanWarps));
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status moe_expert_plan(const int32_t *idx, int n_tokens, int top_k, int n_experts, int32_t *counts,
                                      int32_t *offsets, int32_t *rows, int32_t *slots, void *stream)
{
    if (n_tokens < 0 || n_experts < 1 || n_experts > kMaxExperts || top_k < 1 || top_k > n_experts)
        return MOE_ERR_INVALID_ARG;
    const int64_t pairs = (int64_t)n_tokens * top_k;
    if (pairs > (1ll << 30)) return MOE_ERR_INVALID_ARG;
    if (!counts || !offsets) return MOE_ERR_INVALID_ARG;
    if (pairs && (!idx || !rows || !slots)) return MOE_ERR_INVALID_ARG;
    if (!aligned(idx, 4) || !aligned(counts, 4) || !aligned(offsets, 4) || !aligned(rows, 4) || !aligned(slots, 4))
        return MOE_ERR_INVALID_ARG;
    int sms = 0;
    const moe_status st = g_plan.get(&sms, plan_prepare);
    if (st != MOE_OK) return st;
    const int warps = (int)std::min<int64_t>(kPlanWarps, std::max<int64_t>(1, (pairs + 31) / 32));
    const int ctas = pairs > 32 * kPlanWarps * kPlanBatch ? 8 : 1;
    return launched(launch(expert_plan_kernel, dim3(ctas), kPlanThreads, plan_smem(n_experts, warps),
                           static_cast<cudaStream_t>(stream), ctas, false, idx, (int)pairs, top_k, n_experts, warps,
                           counts, offsets, rows, slots));
}
