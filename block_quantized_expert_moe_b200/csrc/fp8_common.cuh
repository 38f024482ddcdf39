// Shared parts of the E4M3 products: arguments, the table of groups, tiles and
// tensor maps.
#pragma once

#include <cuda.h>

#include <algorithm>

#include "op_common.cuh"
#include "tc_common.cuh"
#include "tma_maps.cuh"

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
};

struct Operands {
    const uint8_t *a, *b;
    int64_t ld_a, ld_b, stride_b;
    int k;
};

// kind::f8f6f4 instruction descriptor: E4M3 x E4M3 -> f32, both K-major.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N)
{
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// One output tile: one weight tile of group g, token rows [row0, row0 + rows).
struct Tile {
    int group, n_tile, row0, rows;
};

__device__ __forceinline__ Tile tile_at(int id, int n_tiles, int groups, const int *first_tile, const int *offset)
{
    const int tt = id / n_tiles;
    Tile t;
    t.n_tile = id - tt * n_tiles;
    int lo = 0, hi = groups;  // first_tile[lo] <= tt < first_tile[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first_tile[mid] <= tt) lo = mid;
        else hi = mid;
    }
    t.group = lo;
    const int i = tt - first_tile[lo], parts = first_tile[lo + 1] - first_tile[lo];
    const int r = offset[lo + 1] - offset[lo];
    const int size = (((r + parts - 1) / parts) + 15) & ~15;
    t.row0 = offset[lo] + i * size;
    t.rows = min(size, offset[lo] + r - t.row0);  // at least 1: (parts - 1) * bn < r and size <= bn
    return t;
}

// Groups' row offsets, clamped to an ascending sequence inside [0, rows], and each
// group's first token tile of at most bn rows, in shared memory.  Every thread
// of the CTA calls it; the caller synchronises afterwards.
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
    const int per = (a.groups + THREADS - 1) / THREADS;
    const int g0 = min(a.groups, (int)threadIdx.x * per), g1 = min(a.groups, g0 + per);
    int sum = 0;
    for (int g = g0; g < g1; ++g) {
        const int lo = min(max(__ldg(a.offsets + g), 0), a.rows);
        const int hi = min(max(__ldg(a.offsets + g + 1), lo), a.rows);
        offset[g] = lo;
        if (g == a.groups - 1) offset[a.groups] = hi;
        sum += (hi - lo + bn - 1) / bn;
    }
    int scan = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, scan, d);
        if (lane >= d) scan += v;
    }
    if (lane == 31) warp_tiles[warp] = scan;
    __syncthreads();
    int run = scan - sum;
    for (int w = 0; w < warp; ++w) run += warp_tiles[w];
    for (int g = g0; g < g1; ++g) {
        first_tile[g] = run;
        const int lo = offset[g];
        const int hi = min(max(__ldg(a.offsets + g + 1), lo), a.rows);
        run += (hi - lo + bn - 1) / bn;
        if (g == a.groups - 1) first_tile[a.groups] = run;
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
moe_status pair_product(const Operands &o, const ProductArgs &a, moe_dtype out_dtype, int pairs, cudaStream_t s);

}  // namespace fp8
}  // namespace moe
