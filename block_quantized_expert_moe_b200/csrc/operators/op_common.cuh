// Host and device helpers shared by the stand-alone operators (the expert
// plan, the balance loss, the E4M3 quantisers and the E4M3 product).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>

#include "../../../include/moe.h"

namespace moe {
namespace op {

constexpr int kMaxExperts = 1024;
constexpr int kScaleBlock = 128;  // columns that share a scale (weights: 128 x 128)
constexpr int kMaxDevices = 64;
constexpr int kMaxRows = 1 << 30;

inline bool aligned(const void *p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
inline int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

// The current device's SM count; `prepare` (kernel attributes) runs once per
// device, again by the next call if it failed.
struct PerDevice {
    std::mutex m;
    int sms[kMaxDevices] = {};
    template <class F>
    moe_status get(int *out, F prepare)
    {
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess) return MOE_ERR_CUDA;
        if (dev < 0 || dev >= kMaxDevices) return MOE_ERR_INVALID_ARG;
        std::lock_guard<std::mutex> lk(m);
        if (!sms[dev]) {
            int n = 0;
            if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || prepare() != cudaSuccess) {
                cudaGetLastError();  // reported here, not by a later call
                return MOE_ERR_CUDA;
            }
            sms[dev] = n;
        }
        *out = sms[dev];
        return MOE_OK;
    }
};

inline moe_status launched(cudaError_t e)
{
    if (e == cudaSuccess) return MOE_OK;
    cudaGetLastError();  // reported here, not by a later call
    return MOE_ERR_CUDA;
}

// Every operator is launched as a programmatic dependent of what precedes it on the stream:
// its blocks may be set up while that finishes, and each kernel begins with
// follow_previous(), before it touches global memory.
template <class K, class... A>
inline cudaError_t launch(K kernel, dim3 grid, int threads, size_t smem, cudaStream_t s, int cluster, A... args)
{
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    if (cluster > 1) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
        attr[cfg.numAttrs].val.clusterDim.x = cluster;
        attr[cfg.numAttrs].val.clusterDim.y = 1;
        attr[cfg.numAttrs].val.clusterDim.z = 1;
        ++cfg.numAttrs;
    }
    attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[cfg.numAttrs].val.programmaticStreamSerializationAllowed = 1;
    ++cfg.numAttrs;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// ---- device --------------------------------------------------------------------
__device__ __forceinline__ unsigned cluster_rank()
{
    unsigned r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ unsigned cluster_size()
{
    unsigned r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}

// (The .aligned forms take whole warps: lanes that come from a branch meet first.)
__device__ __forceinline__ void cluster_sync()
{
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// A CTA's shared memory may be written by the others once it has started: each arrives when
// it starts and waits before it sends.  (It waits for residents of one cluster, which are
// scheduled together.)
__device__ __forceinline__ void cluster_started()
{
    __syncwarp();
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}

__device__ __forceinline__ void cluster_wait_started()
{
    __syncwarp();
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}

// The shared::cluster address in CTA `rank` of a shared-memory address of this CTA.
__device__ __forceinline__ uint32_t cluster_map(uint32_t addr, unsigned rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}

__device__ __forceinline__ uint32_t cluster_ld_u32(uint32_t addr)
{
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ void cluster_st_u32(uint32_t addr, uint32_t v)
{
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

__device__ __forceinline__ void cluster_st_f32(uint32_t addr, float v)
{
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

__device__ __forceinline__ float cluster_ld_f32(uint32_t addr)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// Waits until everything before this kernel on the stream has finished and its memory is
// visible, then lets the next kernel's blocks be set up (in this order: a follower that
// reads weights before its own wait must not overtake what precedes this kernel).  One thread's
// call counts for its CTA: a CTA that allocates tensor memory has a barrier in between.  Global
// memory is read with plain loads and through pointers that are not __restrict__: a read-only
// load could be moved ahead of the wait, or hit a line cached before it.
__device__ __forceinline__ void follow_previous()
{
    asm volatile("griddepcontrol.wait;\n\tgriddepcontrol.launch_dependents;" ::: "memory");
}

}  // namespace op
}  // namespace moe
