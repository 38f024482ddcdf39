// The E4M3 product for many rows: a pair of CTAs (one cluster, two SMs of one
// TPC) multiplies up to 256 token rows by 256 weight rows, 128 columns at a time,
// with tcgen05.mma.cta_group::2.
//
// Each CTA brings up to 128 token rows and half of the weight rows, so a block of
// 128 columns costs an SM 32 KB of operands for 512 clocks of tensor work (a
// single CTA's 128 x 256 tile costs 48 KB, more than an SM gets from L2 in that
// time).  A CTA's accumulator holds its token rows (tensor-memory lanes) by all
// 256 weight rows, double buffered, one buffer per block: the epilogue adds scale *
// partial to fp32 registers while the next block is multiplied.  A group's last
// tile is cut in half between the two CTAs, so its empty lanes are whole warps of
// the epilogue, which skip.
//
// The epilogue is the other bound: 128 x 256 fused multiply-adds a block and CTA,
// 256 clocks of the FMA pipes.  Tokens on the lanes give a thread one row: its scale is
// one register, loaded two blocks ahead, and one product with the weights' block
// scale covers all its columns.  (With the weights on the lanes, as in the kernel
// for few rows, every column has a scale of its own, read from shared memory:
// 153.7 us at 8192 x 4096 x 4096.)  Sixteen warps, four per scheduler, hide the barrier
// and tensor-memory latencies of one another.
//
//   warps 0-15   epilogue: warpgroup q owns columns 64 q .. 64 q + 63
//   warp 16      TMA producer (both CTAs; all bytes count on the leader's barrier)
//   warp 17      MMA issuer (the leader's only)
//   warps 18-19  idle (a register split works on groups of four warps)
// Every mbarrier wait is bounded.
#include "fp8_common.cuh"

namespace moe {
namespace fp8 {
namespace {

constexpr int kEpiWarps = 16;
constexpr int kTmaWarp = kEpiWarps, kMmaWarp = kEpiWarps + 1;
constexpr int kPairThreads = 32 * (kEpiWarps + 4);
constexpr int kPairStages = 6, kPairBufs = 2;
constexpr int kPairWeights = 256;          // weight rows (accumulator columns) of a tile
constexpr int kPart = kPairWeights / 4;    // columns of a warpgroup
constexpr int kBox = 32;                   // token rows of one TMA box
constexpr int kPairStage = 2 * kABytes;    // 128 token rows, 128 weight rows
constexpr int kPairSmem = kPairStages * kPairStage + 2 * (kMaxExperts + 1) * 4 + 1024;
// registers: 640 threads at 96 are 512 at 112 and 128 at 32
constexpr int kEpilogueRegs = 112, kOtherRegs = 32;
static_assert(32 * kEpiWarps * kEpilogueRegs + 128 * kOtherRegs <= kPairThreads * 96, "register split exceeds the launch's");

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

// ---- cta_group::2 forms ------------------------------------------------------------
__device__ __forceinline__ void tmem_alloc2(uint32_t *dst, uint32_t ncols)
{
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(ncols)
                 : "memory");
}

__device__ __forceinline__ void tmem_relinquish2()
{
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_dealloc2(uint32_t taddr, uint32_t ncols)
{
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

__device__ __forceinline__ void mma2_f8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                        uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Arrive on `bar` of both CTAs once this thread's MMAs so far have completed.
__device__ __forceinline__ void mma2_commit(uint32_t bar)
{
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
}

// TMA loads into this CTA's shared memory whose bytes count on a barrier of either
// CTA of the pair (a shared::cluster address).
__device__ __forceinline__ void tma2_load_2d(void *dst, const void *tmap, uint32_t bar, int c0, int c1)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, "
        "%4}], [%2];" ::"r"(smem_u32(dst)),
        "l"(tmap), "r"(bar), "r"(c0), "r"(c1)
        : "memory");
}

__device__ __forceinline__ void tma2_load_3d(void *dst, const void *tmap, uint32_t bar, int c0, int c1, int c2)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, "
        "%4, %5}], [%2];" ::"r"(smem_u32(dst)),
        "l"(tmap), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}

// Arrive on a barrier of the pair (a shared::cluster address).  What it orders are
// tensor-memory reads, complete and fenced before it (tcgen05.wait::ld,
// fence::before_thread_sync): release and acquire at cluster scope, which order
// all memory, cost 344 instead of 219 us on a 8192 x 4096 x 4096 product.
__device__ __forceinline__ void pair_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// 16 columns of this thread's lane; valid after columns_wait.  They are no operands of the
// wait (they would be copied); the FMAs that use them are volatile and stay behind it.
// (32 at a time leave too few registers: spilled loop variables cost 1000 clocks a turn.)
constexpr int kStep = 16;
__device__ __forceinline__ void columns_request(uint32_t taddr, uint32_t (&v)[kStep])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(taddr));
}

__device__ __forceinline__ void columns_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// Volatile, so that the load stays where it is written, ahead of the blocks whose time hides it.
__device__ __forceinline__ float load_ahead(const float *p)
{
    float v;
    asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(v) : "l"(p));
    return v;
}

// Plain FMAs: the packed f32x2 form has the same rate, and its operand pairs cost moves
// (650 against 601 clocks a block of 256 columns, the loop alone).
__device__ __forceinline__ void fma_volatile(float &acc, uint32_t v, float s)
{
    asm volatile("fma.rn.f32 %0, %1, %2, %0;" : "+f"(acc) : "f"(__uint_as_float(v)), "f"(s));
}

// 32 bytes (a whole sector) of one output row
__device__ __forceinline__ void store_sector(void *p, const uint32_t (&w)[8])
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// `left` columns (of 64) of one row; WIDE: the row starts on 32 bytes.
template <bool WIDE>
__device__ __forceinline__ void store_row(float *out, const float (&acc)[kPart], int left)
{
#pragma unroll
    for (int c = 0; c < kPart; c += 8) {
        if (WIDE && c + 8 <= left) {
            uint32_t w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(acc[c + j]);
            store_sector(out + c, w);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (c + j < left) out[c + j] = acc[c + j];
        }
    }
}

template <bool WIDE>
__device__ __forceinline__ void store_row(__nv_bfloat16 *out, const float (&acc)[kPart], int left)
{
#pragma unroll
    for (int c = 0; c < kPart; c += 16) {
        if (WIDE && c + 16 <= left) {
            uint32_t w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const __nv_bfloat162 b = __floats2bfloat162_rn(acc[c + 2 * j], acc[c + 2 * j + 1]);
                w[j] = *reinterpret_cast<const uint32_t *>(&b);
            }
            store_sector(out + c, w);
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j)
                if (c + j < left) out[c + j] = __float2bfloat16_rn(acc[c + j]);
        }
    }
}

// The tile's token rows are split evenly between the CTAs; its columns (tcgen05 N) are a
// multiple of 16.
__device__ __forceinline__ int cta_rows(int rows) { return (rows + 1) / 2; }
__device__ __forceinline__ int tile_columns(int left) { return left >= kPairWeights ? kPairWeights : (left + 15) & ~15; }

// WIDE: output rows start on 32-byte boundaries.
template <class OUT, bool WIDE>
__global__ void __launch_bounds__(kPairThreads, 1)
    fp8_pair_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
                    const ProductArgs a)
{
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t full[kPairStages], empty[kPairStages], acc_full[kPairBufs], acc_empty[kPairBufs], drain_bar;
    __shared__ uint32_t tmem_base;
    __shared__ int warp_tiles[kPairThreads / 32];
    __shared__ volatile int abort_flag;
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    int *offset = reinterpret_cast<int *>(smem + kPairStages * kPairStage);
    int *first_tile = offset + kMaxExperts + 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const unsigned rank = cluster_rank();

    if (warp == kMmaWarp) {
        tmem_alloc2(&tmem_base, kPairBufs * kPairWeights);
        tmem_relinquish2();
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < kPairStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int s = 0; s < kPairBufs; ++s) {
            mbar_init(&acc_full[s], 1);
            mbar_init(&acc_empty[s], 2 * kEpiWarps);  // the epilogue warps of both CTAs (used by the leader)
        }
        mbar_init(&drain_bar, 1);
        abort_flag = 0;
        fence_mbar_init();
    }
    build_groups<kPairThreads>(a, kPairTokens, offset, first_tile, warp_tiles);
    tc_fence_before_sync();
    __syncthreads();
    cluster_sync();  // the other CTA's barriers and tensor memory exist from here on
    tc_fence_after_sync();
    const uint32_t tmem = tmem_base;
    const int n_pairs = (a.n + kPairWeights - 1) / kPairWeights;
    const int n_work = first_tile[a.groups] * n_pairs;
    const int worker = blockIdx.x >> 1, workers = gridDim.x >> 1;

    if (warp >= kTmaWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp == kTmaWarp) {  // ---- TMA producer
            if (lane == 0) {
                prefetch_tmap(&map_w);
                prefetch_tmap(&map_x);
            }
            const uint32_t full_at = smem_u32(full), empty_at = smem_u32(empty), leader_full = cluster_map(full_at, 0);
            Ring<kPairStages> r;
            int issued = 0;
            bool go = true;
            for (int id = worker; id < n_work && go; id += workers) {
                const Tile t = tile_at(id, n_pairs, a.groups, first_tile, offset);
                const int mine = cta_rows(t.rows), boxes = (mine + kBox - 1) / kBox;
                const uint32_t bytes = 2 * (kABytes + boxes * kBox * 128);
                const int n0 = t.n_tile * kPairWeights, w0 = n0 + (int)rank * tile_columns(a.n - n0) / 2;
                const int x0 = t.row0 + (int)rank * mine;
                for (int kb = 0; kb < a.kblocks; ++kb, ++issued, r.next()) {
                    // the slot's previous use has been multiplied (a fresh slot passes)
                    if (!__all_sync(0xffffffffu, bar_wait(empty_at + 8 * r.slot, r.phase ^ 1))) {
                        go = false;
                        break;
                    }
                    if (elect_one()) {
                        uint8_t *x_s = smem + r.slot * kPairStage, *w_s = x_s + kABytes;
                        if (rank == 0) mbar_arrive_expect_tx(&full[r.slot], bytes);
                        const uint32_t bar = leader_full + 8 * r.slot;
                        tma2_load_3d(w_s, &map_w, bar, kb * 128, w0, t.group);
                        for (int b = 0; b < boxes; ++b)
                            tma2_load_2d(x_s + b * kBox * 128, &map_x, bar, kb * 128, x0 + b * kBox);
                    }
                    __syncwarp();
                }
            }
            if (!go) {
                if (lane == 0) abort_flag = 1;
                if (rank == 0 && lane == 0) drain_ring(full, kPairStages, issued);
            }
        } else if (warp == kMmaWarp) {  // ---- MMA issuer
            // the whole warp runs the loop and one lane issues: in a branch of one lane the
            // descriptors do not count as uniform, and each instruction costs a sequence of moves
            if (rank == 0) {
                const uint32_t full_at = smem_u32(full), empty_at = smem_u32(empty), acc_full_at = smem_u32(acc_full),
                               acc_empty_at = smem_u32(acc_empty);
                const uint64_t x_desc = desc_kmajor_sw128(smem), w_desc = desc_kmajor_sw128(smem + kABytes);
                Ring<kPairStages> r;
                Ring<kPairBufs> d;
                bool go = true;
                for (int id = worker; id < n_work && go; id += workers) {
                    const Tile t = tile_at(id, n_pairs, a.groups, first_tile, offset);
                    const uint32_t idesc = idesc_e4m3(256, tile_columns(a.n - t.n_tile * kPairWeights));
                    for (int kb = 0; kb < a.kblocks; ++kb, r.next(), d.next()) {
                        const bool ok = bar_wait(full_at + 8 * r.slot, r.phase) &&
                                        bar_wait(acc_empty_at + 8 * d.slot, d.phase ^ 1);
                        if (!__all_sync(0xffffffffu, ok)) {
                            go = false;
                            break;
                        }
                        tc_fence_after_sync();
                        if (elect_one()) {
                            const uint64_t step = (uint64_t)(r.slot * (kPairStage >> 4));
                            const uint64_t wd = w_desc + step, xd = x_desc + step;
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                mma2_f8(tmem + d.slot * kPairWeights, xd + 2 * kk, wd + 2 * kk, idesc, kk != 0);
                            mma2_commit(empty_at + 8 * r.slot);
                            mma2_commit(acc_full_at + 8 * d.slot);
                        }
                        __syncwarp();
                    }
                }
                if (!go && elect_one()) {
                    abort_flag = 1;
                    mma2_commit(smem_u32(&drain_bar));
                    mbar_wait(&drain_bar, 0);
                }
            }
        }
    } else {  // ---- epilogue
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpilogueRegs));
        const int part = warp >> 2, quarter = warp & 3;
        const uint32_t acc_full_at = smem_u32(acc_full), leader_empty = cluster_map(smem_u32(acc_empty), 0);
        const uint32_t columns = tmem + ((uint32_t)(quarter * 32) << 16) + part * kPart;
        Ring<kPairBufs> d;
        bool go = true;
        for (int id = worker; id < n_work && go; id += workers) {
            const Tile t = tile_at(id, n_pairs, a.groups, first_tile, offset);
            const int mine = cta_rows(t.rows), n0 = t.n_tile * kPairWeights + part * kPart;
            const int lane_row = quarter * 32 + lane, row = (int)rank * mine + lane_row;
            const bool used = n0 < a.n && quarter * 32 < mine;  // this warp has outputs
            const float *as = a.a_scale + t.row0 + min(row, t.rows - 1);
            const float *bs = a.b_scale + ((int64_t)t.group * a.n_tiles + (used ? n0 / kWeightRows : 0)) * a.kblocks;
            float acc[kPart];
#pragma unroll
            for (int c = 0; c < kPart; ++c) acc[c] = 0.f;
            // one block: acc += scale * partial; false if the wait ran out
            const auto block = [&](float scale) {
                if (!__all_sync(0xffffffffu, bar_wait(acc_full_at + 8 * d.slot, d.phase))) return false;
                tc_fence_after_sync();
                if (used) {
#pragma unroll
                    for (int c = 0; c < kPart; c += kStep) {
                        uint32_t v[kStep];
                        columns_request(columns + d.slot * kPairWeights + c, v);
                        columns_wait();
                        if (c + kStep == kPart) {  // this warp has read its part of the buffer
                            tc_fence_before_sync();
                            __syncwarp();
                            if (lane == 0) pair_arrive(leader_empty + 8 * d.slot);
                        }
#pragma unroll
                        for (int j = 0; j < kStep; ++j) fma_volatile(acc[c + j], v[j], scale);
                    }
                } else if (lane == 0) {
                    pair_arrive(leader_empty + 8 * d.slot);
                }
                d.next();
                return true;
            };
            // two blocks a turn, with the next turn's scales loaded at its start
            float s0 = __ldg(as) * __ldg(bs), s1 = 0.f;
            if (a.kblocks > 1) s1 = __ldg(as + a.ld_a_scale) * __ldg(bs + 1);
            for (int left = a.kblocks; left > 0 && go; left -= 2) {
                float a2 = 0.f, b2 = 0.f, a3 = 0.f, b3 = 0.f;
                as += 2 * a.ld_a_scale;
                bs += 2;
                if (left > 2) {
                    a2 = load_ahead(as);
                    b2 = load_ahead(bs);
                }
                if (left > 3) {
                    a3 = load_ahead(as + a.ld_a_scale);
                    b3 = load_ahead(bs + 1);
                }
                go = block(s0);
                if (go && left > 1) go = block(s1);
                s0 = a2 * b2;
                s1 = a3 * b3;
            }
            if (!go) {
                abort_flag = 1;
                break;
            }
            if (used && lane_row < mine && row < t.rows)
                store_row<WIDE>(static_cast<OUT *>(a.out) + (int64_t)(t.row0 + row) * a.ld_out + n0, acc, a.n - n0);
        }
    }
    __syncwarp();
    if (abort_flag && threadIdx.x == 0 && a.status) atomicExch(a.status, (int)MOE_ERR_TIMEOUT);
    tc_fence_before_sync();
    __syncthreads();
    cluster_sync();  // neither CTA leaves while the other may still arrive here or read its operands
    tc_fence_after_sync();
    if (warp == kMmaWarp) tmem_dealloc2(tmem, kPairBufs * kPairWeights);
}

template <class OUT>
cudaError_t pair_launch(const CUtensorMap &mw, const CUtensorMap &mx, const ProductArgs &a, bool wide, int pairs,
                        cudaStream_t s)
{
    return wide ? launch(fp8_pair_kernel<OUT, true>, dim3(2 * pairs), kPairThreads, kPairSmem, s, 2, false, mw, mx, a)
                : launch(fp8_pair_kernel<OUT, false>, dim3(2 * pairs), kPairThreads, kPairSmem, s, 2, false, mw, mx, a);
}

}  // namespace

cudaError_t pair_prepare()
{
    const cudaFuncAttribute smem = cudaFuncAttributeMaxDynamicSharedMemorySize;
    cudaError_t e = cudaFuncSetAttribute(fp8_pair_kernel<float, true>, smem, kPairSmem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(fp8_pair_kernel<float, false>, smem, kPairSmem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(fp8_pair_kernel<__nv_bfloat16, true>, smem, kPairSmem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(fp8_pair_kernel<__nv_bfloat16, false>, smem, kPairSmem);
    return e;
}

moe_status pair_product(const Operands &o, const ProductArgs &a, moe_dtype out_dtype, int pairs, cudaStream_t s)
{
    const bool bf16 = out_dtype == MOE_DT_BF16;
    // 32-byte stores where every output row starts on a sector
    const bool wide = aligned(a.out, 32) && a.ld_out * (bf16 ? 2 : 4) % 32 == 0;
    CUtensorMap mw, mx;
    if (!code_map(&mw, o.b, o.k, a.n, o.ld_b, a.groups, o.stride_b, kPairWeights / 2)) return MOE_ERR_CUDA;
    if (!code_map(&mx, o.a, o.k, a.rows, o.ld_a, 0, 0, kBox)) return MOE_ERR_CUDA;
    return launched(bf16 ? pair_launch<__nv_bfloat16>(mw, mx, a, wide, pairs, s)
                         : pair_launch<float>(mw, mx, a, wide, pairs, s));
}

}  // namespace fp8
}  // namespace moe
