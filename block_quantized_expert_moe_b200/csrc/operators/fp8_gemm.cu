// The E4M3 product with scales per block of 128, plain and per expert group:
//
//   out[r, n] = sum_b a_scale[b, r] * b_scale[g, n / 128, b]
//                     * sum_{c in block b} a[r, c] * b[g, n, c]
//
// for the rows r of group g, [offsets[g], offsets[g + 1]) (the plain product
// is one group of all rows).
//
// The weight rows are the M side of the tensor-core tile (128 of them, one
// weight scale per tile and block), the token rows its N side, so a group of
// any size fills the M side and pays for its own rows only (in steps of 16):
// a decode batch reads every weight once, and a prefill chunk's ragged groups
// waste at most 15 columns a tile.  A group with more rows than the widest
// tile is cut into equal tiles.
//
// Both scales change every 128 columns, so the tensor core's sum covers one
// block only (four 128 x N x 32 instructions into one of the tensor-memory
// buffers) and the epilogue warps add scale * partial to fp32 registers while
// the next block is multiplied: one FMA per 128 multiply-adds.  That split
// also keeps the tensor core's accumulation short.
//
//   warps 0-3  epilogue: a thread owns one weight row (tensor-memory lane) and the
//              tile's columns
//   warp 4     TMA producer of weight and token rows (128-byte swizzle)
//   warp 5     MMA issuer (one elected thread)
//   warp 6     scales: a_scale * b_scale of each block into a small ring
//
// Few tiles (decode): the K blocks of a tile are split over the CTAs of a
// cluster, whose partial sums meet through distributed shared memory in rank
// order: no workspace, no atomics, the same bits every run.
// Decode batches are bound by the weights' bytes: 64 tokens over 512 experts of 1024 x
// 2048 (352 read on average) 108.5 us, 6.8 TB/s.  Single tokens are bound by latency:
// one token's ten experts (20 MB) 9.3 us, one row x 1024 x 2048 4.2 us (group table
// 1.1 us when its offsets are cold, first tile 2 us, exchange 1 us).
// Every mbarrier wait is bounded.
#include <limits.h>

#include <atomic>

#include "fp8_common.cuh"

namespace moe {
namespace {

using namespace fp8;

constexpr int kEpiWarps = 4, kThreads = 32 * (kEpiWarps + 3);
constexpr int kBox = 16;   // token rows of one TMA box
constexpr int kBufs = 4;   // tensor-memory buffers
constexpr int kScales = 8;  // ring of scale rows

template <int BN_, int STAGES_>
struct Config {
    static constexpr int BN = BN_;          // widest token tile, columns of an epilogue thread
    static constexpr int STAGES = STAGES_;  // operand ring; two CTAs share an SM
    static constexpr int STAGE_BYTES = kABytes + BN * 128;
    static constexpr int TABLE = 2 * (kMaxExperts + 1) * 4;  // group offsets, first tiles
    static constexpr int SMEM = STAGES * STAGE_BYTES + kScales * BN * 4 + TABLE + 1024;
    static constexpr int PARTIAL = kWeightRows * BN * 4;  // partial sums of the cluster's ranks (K split)
    static_assert(2 * (SMEM + 2048) <= 228 * 1024, "two CTAs an SM");
};
typedef Config<64, 4> Narrow;
typedef Config<16, 5> Token;  // at most 16 rows: a deeper ring of smaller stages

__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                       uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// 16 columns of this thread's tensor-memory lane; the values are valid after tmem_wait16.
__device__ __forceinline__ void tmem_request16(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

__device__ __forceinline__ void tmem_wait16(uint32_t (&r)[16])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                   "+r"(r[15])::"memory");
}

// acc += v * s on a pair
__device__ __forceinline__ void fma_pair(float2 &acc, uint32_t v0, uint32_t v1, float s0, float s1)
{
    asm("{\n\t.reg .b64 rv, rs, ra;\n\t"
        "mov.b64 rv, {%2, %3};\n\tmov.b64 rs, {%4, %5};\n\tmov.b64 ra, {%0, %1};\n\t"
        "fma.rn.f32x2 ra, rv, rs, ra;\n\tmov.b64 {%0, %1}, ra;\n\t}"
        : "+f"(acc.x), "+f"(acc.y)
        : "r"(v0), "r"(v1), "f"(s0), "f"(s1));
}

// This thread's weight row of this rank's columns: the ranks' partial sums [rank][per][row] in
// rank order, 32 loads in flight.
template <int RANKS, class OUT>
__device__ __forceinline__ void add_partials(const float *p, int per, int cols, OUT *out, int64_t step)
{
    constexpr int N = 32 / RANKS;
#pragma unroll 1
    for (int c = 0; c < cols; c += N, p += N * kWeightRows, out += N * step) {
        float v[N][RANKS];
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int r = 0; r < RANKS; ++r) v[i][r] = c + i < cols ? p[(r * per + i) * kWeightRows] : 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
#pragma unroll
            for (int r = 1; r < RANKS; ++r) v[i][0] += v[i][r];
            if (c + i < cols) out[i * step] = OUT(v[i][0]);
        }
    }
}

template <class C, class OUT>
__global__ void __launch_bounds__(kThreads, 2)
    fp8_product_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
                       const ProductArgs a)
{
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t full[C::STAGES], empty[C::STAGES], acc_full[kBufs], acc_empty[kBufs],
        sc_full[kScales], sc_empty[kScales], drain_bar;
    __shared__ uint32_t tmem_base;
    __shared__ int warp_tiles[kThreads / 32];
    __shared__ volatile int abort_flag;
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float *scale_ring = reinterpret_cast<float *>(smem + C::STAGES * C::STAGE_BYTES);
    int *offset = reinterpret_cast<int *>(scale_ring + kScales * C::BN);
    int *first_tile = offset + kMaxExperts + 1;
    float *partial = reinterpret_cast<float *>(first_tile + kMaxExperts + 1);  // [rank][column][weight row], if ranks > 1
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const unsigned rank = cluster_rank(), ranks = cluster_size();

    if (warp == kEpiWarps + 1) {
        tmem_alloc(&tmem_base, kBufs * C::BN);
        tmem_relinquish();
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int s = 0; s < kBufs; ++s) {
            mbar_init(&acc_full[s], 1);
            mbar_init(&acc_empty[s], kEpiWarps);
        }
        for (int s = 0; s < kScales; ++s) {
            mbar_init(&sc_full[s], 1);
            mbar_init(&sc_empty[s], kEpiWarps);
        }
        mbar_init(&drain_bar, 1);
        abort_flag = 0;
        fence_mbar_init();
    }
    if (ranks > 1) cluster_started();
    // Tensor memory is this CTA's before any of its warps lets the next kernel be set up: that one
    // may allocate before its own wait, and would hold what this one still waits for.
    __syncthreads();
    follow_previous();
    build_groups<kThreads>(a, C::BN, offset, first_tile, warp_tiles);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (ranks > 1) cluster_wait_started();
    const uint32_t tmem = tmem_base;
    const int n_work = first_tile[a.groups] * a.n_tiles;
    const int shift = 31 - __clz(ranks);  // 1, 2, 4 or 8 ranks
    const int worker = blockIdx.x >> shift, workers = gridDim.x >> shift;
    const int kb0 = (int)((int64_t)a.kblocks * rank >> shift), kb1 = (int)((int64_t)a.kblocks * (rank + 1) >> shift);
    int issued = 0;

    // One tile of each role; after a wait that ran out a warp skips its work (and the others'
    // waits run out) but still meets the cluster's barriers.
    Ring<C::STAGES> ring;  // this warp's positions
    Ring<kBufs> buf;
    Ring<kScales> scale;
    bool go = true;
    TileWalk walk(worker, workers, a.n_tiles);
    for (int id = worker; id < n_work; id += workers, walk.next()) {
        const Tile t = walk.tile(a.groups, first_tile, offset);
        const int ncols = (max(t.rows, 1) + 15) & ~15;
        float2 acc[C::BN / 2];
        // (the issuing warps run converged and one lane issues: in a branch of one lane descriptors
        // do not count as uniform, and each instruction costs a sequence of moves)
        if (warp == kEpiWarps) {  // ---- TMA producer
            const int boxes = (ncols + kBox - 1) / kBox;
            for (int kb = kb0; kb < kb1 && go; ++kb) {
                go = issued < a.stall_after &&
                     __all_sync(0xffffffffu, bar_wait(smem_u32(empty) + 8 * ring.slot, ring.phase ^ 1));
                if (!go) break;
                if (elect_one()) {
                    uint8_t *w_s = smem + ring.slot * C::STAGE_BYTES, *x_s = w_s + kABytes;
                    uint64_t *bar = &full[ring.slot];
                    mbar_arrive_expect_tx(bar, kABytes + boxes * kBox * 128);
                    tma_load_3d(w_s, &map_w, bar, kb * 128, t.n_tile * kWeightRows, t.group);
                    for (int b = 0; b < boxes; ++b)
                        tma_load_2d(x_s + b * kBox * 128, &map_x, bar, kb * 128, t.row0 + b * kBox);
                }
                __syncwarp();
                ++issued;
                ring.next();
            }
        } else if (warp == kEpiWarps + 1) {  // ---- MMA issuer
            const uint32_t idesc = idesc_e4m3(kWeightRows, ncols);
            for (int kb = kb0; kb < kb1 && go; ++kb) {
                const bool ok = bar_wait(smem_u32(full) + 8 * ring.slot, ring.phase) &&
                                bar_wait(smem_u32(acc_empty) + 8 * buf.slot, buf.phase ^ 1);
                go = __all_sync(0xffffffffu, ok);
                if (!go) break;
                tc_fence_after_sync();
                if (elect_one()) {
                    const uint64_t step = (uint64_t)(ring.slot * (C::STAGE_BYTES >> 4));
                    const uint64_t wd = desc_kmajor_sw128(smem) + step, xd = desc_kmajor_sw128(smem + kABytes) + step;
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) mma_f8(tmem + buf.slot * C::BN, wd + 2 * kk, xd + 2 * kk, idesc, kk != 0);
                    mma_commit(&empty[ring.slot]);
                    mma_commit(&acc_full[buf.slot]);
                }
                __syncwarp();
                ring.next();
                buf.next();
            }
        } else if (warp == kEpiWarps + 2) {  // ---- scales
            constexpr int PER = (C::BN + 31) / 32;  // columns of a lane
            constexpr int AHEAD = PER == 1 ? 8 : 4;  // blocks of loads in flight
            const float *bs = a.b_scale + ((int64_t)t.group * a.n_tiles + t.n_tile) * a.kblocks;
            for (int k0 = kb0; k0 < kb1 && go; k0 += AHEAD) {
                // every load from a valid address, so that none waits behind a branch
                float v[AHEAD][PER], w[AHEAD];
#pragma unroll
                for (int i = 0; i < AHEAD; ++i) {
                    const int kb = min(k0 + i, kb1 - 1);
                    w[i] = bs[kb];
#pragma unroll
                    for (int j = 0; j < PER; ++j)
                        v[i][j] = *(a.a_scale + (int64_t)kb * a.ld_a_scale + t.row0 + min(j * 32 + lane, t.rows - 1));
                }
#pragma unroll
                for (int i = 0; i < AHEAD; ++i) {
                    if (k0 + i >= kb1) break;
                    const int s = scale.slot;
                    go = __all_sync(0xffffffffu, bar_wait(smem_u32(sc_empty) + 8 * s, scale.phase ^ 1));
                    if (!go) break;
                    scale.next();
#pragma unroll
                    for (int j = 0; j < PER; ++j)
                        if (j * 32 + lane < C::BN) scale_ring[s * C::BN + j * 32 + lane] = v[i][j] * w[i];
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sc_full[s]);
                }
            }
        } else {  // ---- epilogue warps
#pragma unroll
            for (int i = 0; i < C::BN / 2; ++i) acc[i] = make_float2(0.f, 0.f);
            for (int kb = kb0; kb < kb1 && go; ++kb) {
                const int d = buf.slot, s = scale.slot;
                const uint32_t sc_at = smem_u32(sc_full) + 8 * s, acc_at = smem_u32(acc_full) + 8 * d;
                const bool sc_ready = bar_try(sc_at, scale.phase), acc_ready = bar_try(acc_at, buf.phase);
                if (!__all_sync(0xffffffffu, sc_ready && acc_ready)) {
                    const bool ok = bar_wait(sc_at, scale.phase) && bar_wait(acc_at, buf.phase);
                    go = __all_sync(0xffffffffu, ok);
                    if (!go) break;
                }
                buf.next();
                scale.next();
                tc_fence_after_sync();
                const uint32_t td = tmem + d * C::BN + ((uint32_t)(warp * 32) << 16);
                const float *sc = scale_ring + s * C::BN;
#pragma unroll
                for (int c = 0; c < C::BN; c += 16) {
                    if (c < ncols) {
                        uint32_t v[16];
                        tmem_request16(td + c, v);
                        tmem_wait16(v);
#pragma unroll
                        for (int j = 0; j < 16; j += 4) {
                            const float4 f = *reinterpret_cast<const float4 *>(sc + c + j);
                            fma_pair(acc[(c + j) / 2], v[j], v[j + 1], f.x, f.y);
                            fma_pair(acc[(c + j) / 2 + 1], v[j + 2], v[j + 3], f.z, f.w);
                        }
                    }
                }
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&acc_empty[d]);
                    mbar_arrive(&sc_empty[s]);
                }
            }
        }
        __syncwarp();
        if (!go) abort_flag = 1;
        if (ranks > 1) {
            // Column c of the tile belongs to rank c % ranks: every rank sends its partial sums there,
            // and after one barrier the owner adds them in rank order from its own shared memory
            // (reading them from the others' instead costs 2 us more).
            const int per = (ncols + (int)ranks - 1) >> shift;  // columns of a rank
            if (warp < kEpiWarps) {
                const uint32_t own = smem_u32(partial + (rank * per * kWeightRows + threadIdx.x));
#pragma unroll
                for (int i = 0; i < C::BN / 2; ++i) {
                    if (2 * i < ncols) {
                        cluster_st_f32(cluster_map(own + (2 * i >> shift) * (kWeightRows * 4), 2 * i & (ranks - 1)), acc[i].x);
                        cluster_st_f32(cluster_map(own + ((2 * i + 1) >> shift) * (kWeightRows * 4), (2 * i + 1) & (ranks - 1)),
                                       acc[i].y);
                    }
                }
            }
            cluster_sync();
            const int n = t.n_tile * kWeightRows + (int)threadIdx.x;
            if (warp < kEpiWarps && !abort_flag && n < a.n) {
                OUT *out = static_cast<OUT *>(a.out) + (int64_t)(t.row0 + (int)rank) * a.ld_out + n;
                const float *p = partial + threadIdx.x;
                const int cols = (t.rows - (int)rank + (int)ranks - 1) >> shift;  // may be none
                const int64_t step = ranks * a.ld_out;
                if (ranks == 2) add_partials<2>(p, per, cols, out, step);
                else if (ranks == 4) add_partials<4>(p, per, cols, out, step);
                else add_partials<8>(p, per, cols, out, step);
            }
            if (id + workers < n_work) cluster_sync();  // the next tile's sums may come
        } else if (warp < kEpiWarps && !abort_flag) {
            const int n = t.n_tile * kWeightRows + (int)threadIdx.x;
            if (n < a.n) {
                OUT *out = static_cast<OUT *>(a.out) + (int64_t)t.row0 * a.ld_out + n;
#pragma unroll
                for (int i = 0; i < C::BN / 2; ++i) {
                    if (2 * i < t.rows) out[(int64_t)(2 * i) * a.ld_out] = OUT(acc[i].x);
                    if (2 * i + 1 < t.rows) out[(int64_t)(2 * i + 1) * a.ld_out] = OUT(acc[i].y);
                }
            }
        }
    }
    tc_fence_before_sync();
    __syncthreads();  // every warp is through: a wait that ran out in any of them is known here
    tc_fence_after_sync();
    // after one: let copies and MMAs in flight land before memory is released
    if (abort_flag) {
        if (warp == kEpiWarps && lane == 0) drain_ring(full, C::STAGES, issued);
        if (warp == kEpiWarps + 1 && elect_one()) drain_mma(&drain_bar);
        if (threadIdx.x == 0) record_timeout(a.status);
        __syncthreads();
    }
    __syncwarp();
    if (warp == kEpiWarps + 1) tmem_dealloc(tmem, kBufs * C::BN);
}

template <class C>
cudaError_t set_smem()
{
    cudaError_t e = cudaFuncSetAttribute(fp8_product_kernel<C, float>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM + C::PARTIAL);
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(fp8_product_kernel<C, __nv_bfloat16>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM + C::PARTIAL);
}

template <class C>
moe_status run_product(const Operands &o, const ProductArgs &a, moe_dtype out_dtype, int workers, int ranks,
                       cudaStream_t s)
{
    CUtensorMap mw, mx;
    if (!code_map(&mw, o.b, o.k, a.n, o.ld_b, a.groups, o.stride_b, kWeightRows)) return MOE_ERR_CUDA;
    if (!code_map(&mx, o.a, o.k, a.rows, o.ld_a, 0, 0, kBox)) return MOE_ERR_CUDA;
    const dim3 grid(workers * ranks);
    const int smem = C::SMEM + (ranks > 1 ? C::PARTIAL : 0);
    return launched(out_dtype == MOE_DT_BF16 ? launch(fp8_product_kernel<C, __nv_bfloat16>, grid, kThreads, smem, s,
                                                      ranks, mw, mx, a)
                                             : launch(fp8_product_kernel<C, float>, grid, kThreads, smem, s, ranks,
                                                      mw, mx, a));
}

PerDevice g_product;
std::atomic<int> g_stall_after{INT_MAX};  // tests only (moe_debug_fp8_stall_after)

cudaError_t product_prepare()
{
    if (!tmaps::encode_fn()) return cudaErrorUnknown;
    cudaError_t e = set_smem<Narrow>();
    if (e == cudaSuccess) e = set_smem<Token>();
    return e != cudaSuccess ? e : pair_prepare();
}

moe_status product(const uint8_t *a, int64_t ld_a, const float *a_scale, int64_t ld_a_scale, int rows, const uint8_t *b,
                   int64_t ld_b, int64_t stride_b, const float *b_scale, const int32_t *offsets, int groups, int n,
                   int k, void *out, moe_dtype out_dtype, int64_t ld_out, int32_t *status, void *stream)
{
    if (out_dtype != MOE_DT_F32 && out_dtype != MOE_DT_BF16) return MOE_ERR_INVALID_ARG;
    if (rows < 0 || rows > kMaxRows || n < 1 || n > (1 << 20) || k < 1 || k > (1 << 20) || groups < 1 || groups > kMaxExperts)
        return MOE_ERR_INVALID_ARG;
    if (ld_a < k || ld_a % 16 || ld_b < k || ld_b % 16 || stride_b % 16 || ld_out < n || ld_a_scale < rows)
        return MOE_ERR_INVALID_ARG;
    if (ld_a >= 1ll << 40 || ld_b >= 1ll << 40 || stride_b >= 1ll << 40) return MOE_ERR_INVALID_ARG;
    if (groups > 1 && stride_b < n * ld_b) return MOE_ERR_INVALID_ARG;
    if (rows == 0) return MOE_OK;
    if (!a || !a_scale || !b || !b_scale || !out) return MOE_ERR_INVALID_ARG;
    if (!aligned(a, 16) || !aligned(b, 16) || !aligned(a_scale, 4) || !aligned(b_scale, 4) || !aligned(offsets, 4) ||
        !aligned(out, out_dtype == MOE_DT_BF16 ? 2 : 4) || !aligned(status, 4))
        return MOE_ERR_INVALID_ARG;
    ProductArgs p{};
    p.a_scale = a_scale;
    p.ld_a_scale = ld_a_scale;
    p.b_scale = b_scale;
    p.offsets = offsets;
    p.groups = groups;
    p.rows = rows;
    p.n = n;
    p.kblocks = ceil_div(k, kScaleBlock);
    p.n_tiles = ceil_div(n, kWeightRows);
    p.out = out;
    p.ld_out = ld_out;
    p.status = status;
    p.stall_after = g_stall_after.load(std::memory_order_relaxed);
    int sms = 0;
    const moe_status st = g_product.get(&sms, product_prepare);
    if (st != MOE_OK) return st;
    const Operands o{a, b, ld_a, ld_b, stride_b ? stride_b : ld_b, k};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    // most tiles that any offsets could give: one per non-empty group and one per further full tile
    const auto most_tiles = [&](int bn) {
        const int64_t used = std::min<int64_t>(groups, rows);
        return std::min<int64_t>(rows, used + (rows - used) / bn) * p.n_tiles;
    };
    if (most_tiles(Narrow::BN) > INT32_MAX) return MOE_ERR_INVALID_ARG;
    const int64_t wide = most_tiles(kPairTokens) / p.n_tiles * ceil_div(n, 2 * kWeightRows);
    const int64_t narrow = most_tiles(Narrow::BN);
    const int slots = 2 * sms, pairs = sms / 2;
    const bool token = rows <= Token::BN;
    // few tiles: split each one's K blocks over a cluster
    int ranks = 1;
    while (ranks < 8 && narrow * ranks * 2 <= (token ? slots : sms) && ranks * 2 <= p.kblocks) ranks *= 2;
    // The pair kernel, or this one.  Many waves of tiles: by the rows a group has on average, since
    // both read every weight once (128 experts of 1024 x 2048, pair against narrow: 32 rows 67.0 /
    // 58.7 us, 48 rows 68.8 / 67.9, 64 rows 69.9 / 80.3, 128 rows 81.3 / 132.7; 512 experts of 2048 x
    // 512: 40 rows 162 / 170 to 181, 160 rows 224 / 458).  Few waves: by the blocks that the busiest CTA
    // takes one after another, 0.5 us each for a pair, 0.65 us for a narrow tile alone on its SM and
    // 0.9 us for two, and 1 us for a cluster's exchange (fitted when that read the others' sums; it
    // costs less since, which turns none of these; rows x n x k, pair / narrow: 64 x 4096 x 4096
    // 16.6 / 9.2 us, 128 x 4096 x 4096 17.1 / 13.2, 256 x 4096 x 4096 18.4 / 20.8, 512 x 4096 x 4096
    // 18.8 / 26.5, 1024 x 4096 x 4096 19.7 / 50.1, 256 x 1024 x 2048 11.5 / 7.4, 333 x 1000 x 1111
    // 8.8 / 7.5, 512 x 1024 x 1024 8.5 / 7.1, 1024 x 1024 x 1024 8.5 / 9.2, 4096 x 512 x 512 7.0 / 8.5;
    // 8 experts of 2048 x 2048, 64 rows 14.2 / 18.8).
    bool pair = !token;
    if (wide >= 4 * pairs) {
        pair = pair && (int64_t)rows > 56ll * groups;
    } else {
        const int64_t pair_cost = 10 * (int64_t)p.kblocks * ceil_div(wide, pairs) + 20;  // in 50 ns
        const int64_t each = (narrow * ranks > sms ? 18 : 13) * (int64_t)ceil_div(p.kblocks, ranks);
        pair = pair && pair_cost < each * ceil_div(narrow * ranks, slots) + (ranks > 1 ? 20 : 0);
    }
    if (pair) return pair_product(o, p, out_dtype, (int)std::min<int64_t>(wide, pairs), s);
    const int workers = (int)std::min<int64_t>(narrow, slots / ranks);
    return token ? run_product<Token>(o, p, out_dtype, workers, ranks, s)
                 : run_product<Narrow>(o, p, out_dtype, workers, ranks, s);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status moe_fp8_get_device_error(void)
{
    int32_t few = 0, pair = 0;
    if (cudaDeviceSynchronize() != cudaSuccess || take_error(&few) != cudaSuccess ||
        pair_take_error(&pair) != cudaSuccess) {
        cudaGetLastError();  // reported here, not by a later call
        return MOE_ERR_CUDA;
    }
    return (moe_status)(few ? few : pair);
}

extern "C" moe_status moe_debug_fp8_stall_after(int blocks)
{
    if (blocks < -1) return MOE_ERR_INVALID_ARG;
    g_stall_after.store(blocks < 0 ? INT_MAX : blocks, std::memory_order_relaxed);
    return MOE_OK;
}

extern "C" moe_status moe_fp8_matmul(const uint8_t *a, int64_t ld_a, const float *a_scale, int64_t ld_a_scale, int rows,
                                     const uint8_t *b, int64_t ld_b, const float *b_scale, int n, int k, void *out,
                                     moe_dtype out_dtype, int64_t ld_out, int32_t *status, void *stream)
{
    return product(a, ld_a, a_scale, ld_a_scale, rows, b, ld_b, 0, b_scale, nullptr, 1, n, k, out, out_dtype, ld_out,
                   status, stream);
}

extern "C" moe_status moe_fp8_grouped_matmul(const uint8_t *a, int64_t ld_a, const float *a_scale, int64_t ld_a_scale,
                                             int rows, const uint8_t *b, int64_t ld_b, int64_t group_stride_b,
                                             const float *b_scale, const int32_t *offsets, int n_groups, int n, int k,
                                             void *out, moe_dtype out_dtype, int64_t ld_out, int32_t *status,
                                             void *stream)
{
    if (!offsets) return MOE_ERR_INVALID_ARG;
    return product(a, ld_a, a_scale, ld_a_scale, rows, b, ld_b, group_stride_b, b_scale, offsets, n_groups, n, k, out,
                   out_dtype, ld_out, status, stream);
}
