// Shared parts of the E4M3 products: arguments, the table of groups, tiles and
// tensor maps.
#pragma once

#include <cuda.h>

#include <algorithm>

#include "op_common.cuh"
#include "../tc_common.cuh"
#include "../tma_maps.cuh"

namespace moe {
namespace fp8 {

using namespace op;
using namespace tc;

constexpr int kWeightRows = 128;            // weight rows of a CTA's tile (tensor-memory lanes)
constexpr int kABytes = kWeightRows * 128;  // weight rows of a stage (128 columns)

struct ProductArgs {
    const float *a_scale;
    int64_t ld_a_scale;
    const float *b_scale;
    const int32_t *offsets;  // null: one group of all rows
    int groups, rows, n, kblocks, n_tiles;
    void *out;
    int64_t ld_out;
    int32_t *status;
    int stall_after;  // K blocks a CTA loads before its producer stops, as if a copy never came (INT_MAX: never)
};

struct Operands {
    const uint8_t *a, *b;
    int64_t ld_a, ld_b, stride_b;
    int k;
};

// Sticky error of the products of a source file on a device (a word for each file: device code is not
// linked across them).
namespace {
__device__ int32_t device_error;

__device__ __forceinline__ void record_timeout(int32_t *status)
{
    atomicExch(&device_error, (int)MOE_ERR_TIMEOUT);
    if (status) atomicExch(status, (int)MOE_ERR_TIMEOUT);
}

// reads and clears the current device's word
inline cudaError_t take_error(int32_t *error)
{
    const int32_t none = 0;
    const cudaError_t e = cudaMemcpyFromSymbol(error, device_error, sizeof none);
    return e != cudaSuccess || *error == 0 ? e : cudaMemcpyToSymbol(device_error, &none, sizeof none);
}
}  // namespace

// kind::f8f6f4 instruction descriptor: E4M3 x E4M3 -> f32, both K-major.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N)
{
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// ---- shared memory by 32-bit addresses --------------------------------------------------
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity)
{
    if (bar_try(bar, parity)) return true;
    const long long t0 = clock64();
    while (!bar_try(bar, parity))
        if (clock64() - t0 > (1ll << 31)) return false;
    return true;
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one()
{
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one != 0;
}

// Position in a ring of N barriers: slot and the parity of its current use.
template <int N>
struct Ring {
    int slot = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next()
    {
        if (++slot == N) {
            slot = 0;
            phase ^= 1;
        }
    }
};

// One output tile: one weight tile of group g, token rows [row0, row0 + rows).
struct Tile {
    int group, n_tile, row0, rows;
};

// A warp's walk over its tiles (id, id + workers, ...): weight tile and token tile advance without
// a division, the group by a search of 32 at a time from the last one (up to 1900 clocks a tile
// less than dividing and bisecting).  A group's rows are cut into equal tiles: parts tiles of
// at most bn rows, (parts - 1) bn < rows, so each has at least one.
struct TileWalk {
    int token_tile, n_tile, group, step_token, step_n, n_tiles;
    __device__ __forceinline__ TileWalk(int id, int workers, int n_tiles_)
        : token_tile(id / n_tiles_), n_tile(id % n_tiles_), group(0), step_token(workers / n_tiles_),
          step_n(workers % n_tiles_), n_tiles(n_tiles_)
    {
    }
    __device__ __forceinline__ void next()
    {
        token_tile += step_token;
        n_tile += step_n;
        if (n_tile >= n_tiles) {
            n_tile -= n_tiles;
            ++token_tile;
        }
    }
    // the whole warp, converged
    __device__ __forceinline__ Tile tile(int groups, const int *first_tile, const int *offset)
    {
        const int lane = threadIdx.x & 31;
        for (;;) {  // groups whose successor starts at or before this token tile
            const int g = group + lane;
            const unsigned passed = __ballot_sync(0xffffffffu, g < groups - 1 && first_tile[min(g, groups - 1) + 1] <= token_tile);
            group += __popc(passed);
            if (passed != 0xffffffffu) break;
        }
        Tile t;
        t.group = group;
        t.n_tile = n_tile;
        const int first = first_tile[group], parts = first_tile[group + 1] - first;
        const int lo = offset[group], rows = offset[group + 1] - lo;
        if (parts == 1) {
            t.row0 = lo;
            t.rows = rows;
        } else {
            const int size = (((rows + parts - 1) / parts) + 15) & ~15;
            t.row0 = lo + (token_tile - first) * size;
            t.rows = min(size, lo + rows - t.row0);
        }
        return t;
    }
};

// Groups' row offsets, clamped to an ascending sequence inside [0, rows] (an offset below an
// earlier one counts as that one, so that no row has two groups), and each group's first token
// tile of at most bn rows, in shared memory.  Every thread of the CTA calls it; the caller
// synchronises afterwards.
template <int THREADS>
__device__ __forceinline__ void build_groups(const ProductArgs &a, int bn, int *offset, int *first_tile, int *warp_tiles)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (!a.offsets) {
        if (threadIdx.x == 0) {
            offset[0] = 0;
            offset[1] = a.rows;
            first_tile[0] = 0;
            first_tile[1] = (a.rows + bn - 1) / bn;
        }
        return;
    }
    // all offsets at once, then a thread's run of groups from shared memory
    constexpr int PER = (kMaxExperts + THREADS) / THREADS;
    int raw[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int g = i * THREADS + threadIdx.x;
        raw[i] = g <= a.groups ? a.offsets[g] : 0;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int g = i * THREADS + threadIdx.x;
        if (g <= a.groups) first_tile[g] = raw[i];
    }
    __syncthreads();
    const int per = (a.groups + THREADS - 1) / THREADS;
    const int g0 = min(a.groups, (int)threadIdx.x * per), g1 = min(a.groups, g0 + per);
    int tiles[PER], sum = 0;
    bool falls = false;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int g = g0 + i;
        tiles[i] = 0;
        if (g < g1) {
            const int lo = min(max(first_tile[g], 0), a.rows);
            const int next = min(max(first_tile[g + 1], 0), a.rows), hi = max(next, lo);
            falls = falls || next < lo;
            offset[g] = lo;
            if (g == a.groups - 1) offset[a.groups] = hi;
            tiles[i] = (hi - lo + bn - 1) / bn;
        }
        sum += tiles[i];
    }
    int scan = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, scan, d);
        if (lane >= d) scan += v;
    }
    if (lane == 31) warp_tiles[warp] = scan;
    if (__syncthreads_or(falls)) {
        // not a plan's offsets: one thread takes the running maximum
        if (threadIdx.x == 0) {
            int at = min(max(first_tile[0], 0), a.rows), count = 0;
            for (int g = 0; g < a.groups; ++g) {
                const int lo = at;
                at = max(lo, min(first_tile[g + 1], a.rows));
                offset[g] = lo;
                first_tile[g] = count;
                count += (at - lo + bn - 1) / bn;
            }
            offset[a.groups] = at;
            first_tile[a.groups] = count;
        }
        return;
    }
    int run = scan - sum;
    for (int w = 0; w < warp; ++w) run += warp_tiles[w];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int g = g0 + i;
        if (g < g1) {
            first_tile[g] = run;
            run += tiles[i];
            if (g == a.groups - 1) first_tile[a.groups] = run;
        }
    }
}

// uint8 rows of `cols` codes, row stride ld bytes; boxes of 128 columns in the 128-byte swizzle
inline bool code_map(CUtensorMap *m, const void *base, int cols, int64_t rows, int64_t ld, int64_t groups, int64_t stride,
              int box_rows)
{
    const tmaps::EncodeTiledFn f = tmaps::encode_fn();
    if (!f) return false;
    const int dim = groups > 0 ? 3 : 2;
    cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)groups};
    cuuint64_t strides[2] = {(cuuint64_t)ld, (cuuint64_t)stride};
    cuuint32_t box[3] = {128, (cuuint32_t)box_rows, 1}, es[3] = {1, 1, 1};
    return f(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, dim, const_cast<void *>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}


// The pair kernel (fp8_gemm_pair.cu): two CTAs share a 256-row weight tile.
constexpr int kPairTokens = 256;
cudaError_t pair_prepare();
cudaError_t pair_take_error(int32_t *error);
moe_status pair_product(const Operands &o, const ProductArgs &a, moe_dtype out_dtype, int pairs, cudaStream_t s);

}  // namespace fp8
}  // namespace moe
