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
// memory; 32 pairs at a time, ballots group the lanes that chose the same
// expert, so a warp needs no atomics and the rank of a pair inside its
// group is the number of lower lanes in it plus what the warp has counted
// before.  The ranks wait in `slots` while the histograms are scanned over the
// CTA's warps, the CTAs' totals over the cluster (distributed shared memory)
// and the experts' totals over the block; a second pass adds each pair's base.
// No atomics anywhere: the order is that of the definition, and no workspace
// has to be kept or cleared.
//
// The work is latency: 12 bytes a pair (index read, slot and row written).  A
// cluster of 16 CTAs takes prefill chunks, one CTA the decode batches.  With 10
// choices among 512 experts: 8 tokens 3.1 us, 512 tokens 6.1, 8,192 tokens 12.1,
// 65,536 tokens 62 (there half of it ballots, half the second pass, of 16 SMs).
#include <algorithm>

#include "op_common.cuh"

namespace moe {
namespace {

using namespace op;

constexpr int kPlanThreads = 1024, kPlanWarps = kPlanThreads / 32;
constexpr int kPlanBatch = 8;  // index loads in flight per lane
constexpr int kPlanPairsOfOne = 2048;  // one CTA / a cluster: 1,280 pairs 4.9 / 6.0 us, 2,560 6.6 / 6.1
constexpr int kPlanCluster = 16;  // beyond the portable 8: checked when the kernel is prepared

__device__ __forceinline__ int load_choice(const int32_t *idx, int p, int end, int E)
{
    const int e = p < end ? idx[p] : -1;
    return (unsigned)e < (unsigned)E ? e : -1;
}

// The lanes that chose the same expert, from one ballot per bit of the expert's number.
// (__match_any_sync takes time with every distinct value: 78 against 62 us at 65,536
// tokens of 10 choices among 512.)
__device__ __forceinline__ unsigned same_choice(int e, int bits)
{
    unsigned same = __ballot_sync(0xffffffffu, e >= 0);
    for (int b = 0; b < bits; ++b) {
        const bool one = (e >> b) & 1;
        const unsigned ones = __ballot_sync(0xffffffffu, one);
        same &= one ? ones : ~ones;
    }
    return same;
}

__global__ void __launch_bounds__(kPlanThreads, 1)
    expert_plan_kernel(const int32_t *idx, int P, int k, int E, int bits, int warps, int32_t *counts,
                       int32_t *offsets, int32_t *rows, int32_t *slots)
{
    extern __shared__ __align__(16) int32_t smem[];  // cleared 16 bytes at a time
    int32_t *base = smem;                       // [E] first slot of this CTA's pairs of each expert
    int32_t *total = base + E;                  // [CTA of the cluster][E] pairs per expert, sent by each
    int32_t *hist = total + cluster_size() * E;  // [warps][E]
    __shared__ int32_t warp_sum[kPlanWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const unsigned rank = cluster_rank(), ctas = cluster_size();

    if (ctas > 1) cluster_started();

    const int words = warps * E;  // the histograms start on 16 bytes where E is a multiple of 4
    if ((E & 3) == 0) {
        int4 *h4 = reinterpret_cast<int4 *>(hist);
        for (int i = threadIdx.x; i < words / 4; i += kPlanThreads) h4[i] = make_int4(0, 0, 0, 0);
    } else {
        for (int i = threadIdx.x; i < words; i += kPlanThreads) hist[i] = 0;
    }
    __syncthreads();
    follow_previous();

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
            const int p = p0 + 32 * b + lane;
            if (p0 + 32 * b >= end) break;
            const unsigned same = same_choice(e[b], bits);
            const int before = e[b] >= 0 ? own[e[b]] : 0;
            __syncwarp();
            if (e[b] >= 0 && lane == __ffs(same) - 1) own[e[b]] = before + __popc(same);
            __syncwarp();
            if (p < end) slots[p] = before + __popc(same & ((1u << lane) - 1));
        }
    }
    __syncthreads();

    if (ctas > 1) cluster_wait_started();

    // over the CTA's warps: hist becomes the pairs of earlier warps
    for (int e = threadIdx.x; e < E; e += kPlanThreads) {
        int run = 0;
        for (int w0 = 0; w0 < warps; w0 += 8) {
            int n[8];
#pragma unroll
            for (int w = 0; w < 8; ++w) n[w] = w0 + w < warps ? hist[(w0 + w) * E + e] : 0;
#pragma unroll
            for (int w = 0; w < 8; ++w) {
                if (w0 + w < warps) hist[(w0 + w) * E + e] = run;
                run += n[w];
            }
        }
        if (ctas > 1) {  // every CTA gets every CTA's totals (reading them there costs 1.3 us more)
            const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(total + rank * E + e));
            for (unsigned c = 0; c < ctas; ++c) cluster_st_u32(cluster_map(at, c), run);
        } else {
            total[e] = run;
        }
    }
    if (ctas > 1) cluster_sync();
    else __syncthreads();

    // over the cluster, then over the experts (E <= the block's threads)
    int all = 0, before = 0;
    if (threadIdx.x < E) {
        for (unsigned c = 0; c < ctas; ++c) {
            const int n = total[c * E + threadIdx.x];
            if (c < rank) before += n;
            all += n;
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
        int e[kPlanBatch], r[kPlanBatch];
#pragma unroll
        for (int b = 0; b < kPlanBatch; ++b) {
            const int p = p0 + 32 * b + lane;
            e[b] = load_choice(idx, p, end, E);
            r[b] = p < end ? slots[p] : 0;  // written by this lane above
        }
#pragma unroll
        for (int b = 0; b < kPlanBatch; ++b) {
            const int p = p0 + 32 * b + lane;
            if (p >= end) continue;
            const int slot = e[b] >= 0 ? base[e[b]] + own[e[b]] + r[b] : -1;
            slots[p] = slot;
            if (slot >= 0) rows[slot] = p / k;
        }
    }
    // rows behind the last group belong to no token
    for (int64_t s = used + (int64_t)rank * kPlanThreads + threadIdx.x; s < P; s += (int64_t)ctas * kPlanThreads)
        rows[s] = -1;
}

size_t plan_smem(int E, int warps, int ctas) { return sizeof(int32_t) * (size_t)E * (1 + ctas + warps); }

PerDevice g_plan;
int g_plan_cluster[kMaxDevices];  // largest cluster of the device, 16 or 8

cudaError_t plan_prepare()
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(expert_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)plan_smem(kMaxExperts, kPlanWarps, kPlanCluster));
    if (e == cudaSuccess) e = cudaFuncSetAttribute(expert_plan_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = kPlanCluster;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(kPlanCluster);
    cfg.blockDim = dim3(kPlanThreads);
    cfg.dynamicSmemBytes = plan_smem(kMaxExperts, kPlanWarps, kPlanCluster);
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int fit = 0;
    if (cudaOccupancyMaxActiveClusters(&fit, expert_plan_kernel, &cfg) != cudaSuccess) {
        cudaGetLastError();
        fit = 0;
    }
    g_plan_cluster[dev] = fit > 0 ? kPlanCluster : 8;
    return cudaSuccess;
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
    int bits = 0, ctas = 1;
    while ((1 << bits) < n_experts) ++bits;
    if (pairs > kPlanPairsOfOne) {
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess) return MOE_ERR_CUDA;
        ctas = g_plan_cluster[dev];
    }
    return launched(launch(expert_plan_kernel, dim3(ctas), kPlanThreads, plan_smem(n_experts, warps, ctas),
                           static_cast<cudaStream_t>(stream), ctas, idx, (int)pairs, top_k, n_experts, bits, warps,
                           counts, offsets, rows, slots));
}
