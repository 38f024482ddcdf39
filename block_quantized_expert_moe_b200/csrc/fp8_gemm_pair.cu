// The E4M3 product for many rows: a pair of CTAs (one cluster, two SMs of one
// TPC) multiplies 256 weight rows by up to 256 token rows, 128 columns at a
// time, with tcgen05.mma.cta_group::2.
//
// Each CTA brings 128 weight rows and half of the token rows, so a block of
// 128 columns costs an SM 32 KB of operands for 512 clocks of tensor work (a
// single CTA's 128 x 256 tile costs 48 KB, more than an SM gets from L2 in that
// time).  The accumulator of CTA r holds weight rows 128 r .. 128 r + 127 (its
// tensor-memory lanes) by all token columns, double buffered, one buffer per
// block: the epilogue adds scale * partial to fp32 registers while the next
// block is multiplied.
//
// The epilogue is the other bound: 128 x 256 fused multiply-adds a block and
// CTA (256 clocks of the FMA pipes), and a token scale per column.  With one
// weight row a thread would need all 128 scales of its half of the columns, and
// shared memory returns 128 bytes a clock: 1024 clocks a block.  The 16 x 256-bit
// tensor-memory load gives a thread 4 rows by a quarter of its columns instead,
// two neighbouring columns in neighbouring registers, so 8 16-byte loads bring
// its scales (256 clocks a block for the CTA) and a packed FMA serves two
// columns.
//
// A thread's 4 rows are tensor-memory lanes r, r + 8, r + 16, r + 24 of its
// warp's 32.  Where n is a multiple of 32 the weight rows are laid out by the
// TMA box (rows 4 r + g at lane 8 g + r) such that they are 4 consecutive weight
// rows: one 8-byte (bf16) or 16-byte (fp32) store a column, 8 lanes wide.
//
//   warps 0-15   epilogue: warpgroup q owns quarter q of the token columns
//   warp 16      TMA producer (both CTAs; all bytes count on the leader's barrier)
//   warp 17      MMA issuer (the leader's only)
//   warps 18-19  scales a_scale * b_scale of each block, one half of the columns
//                each, into a ring
// Every mbarrier wait is bounded.
#include "fp8_common.cuh"

namespace moe {
namespace fp8 {
namespace {

constexpr int kEpiWarps = 16;
constexpr int kTmaWarp = kEpiWarps, kMmaWarp = kEpiWarps + 1, kScaleWarp0 = kEpiWarps + 2;
constexpr int kPairThreads = 32 * (kEpiWarps + 4);
constexpr int kPairStages = 6, kPairBufs = 2, kPairScales = 4;
constexpr int kBox = 32;                                  // token rows of one TMA box
constexpr int kPairStage = kABytes + (kPairTokens / 2) * 128;
constexpr int kScaleStride = kPairTokens / 4 + 4;         // floats of a quarter of a block's scales, padded
constexpr int kScaleRow = 4 * kScaleStride;               // one block's scales
constexpr int kScaleAhead = 4;                            // blocks of scale loads in flight
constexpr int kPairSmem = kPairStages * kPairStage + kPairScales * kScaleRow * 4 + 2 * (kMaxExperts + 1) * 4 + 1024;
// registers: 640 threads at 96 are 512 at 104 and 128 at 64
constexpr int kEpilogueRegs = 104, kOtherRegs = 64;
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
    const long long t0 = clock64();
    while (!bar_try(bar, parity))
        if (clock64() - t0 > (1ll << 31)) return false;
    return true;
}

__device__ __forceinline__ void bar_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ float4 lds4(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
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

__device__ __forceinline__ void tma2_load_5d(void *dst, const void *tmap, uint32_t bar, int c0, int c1, int c2, int c3,
                                             int c4)
{
    asm volatile(
        "cp.async.bulk.tensor.5d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, "
        "%4, %5, %6, %7}], [%2];" ::"r"(smem_u32(dst)),
        "l"(tmap), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4)
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

// 16 columns of the warp's 32 lanes: v[4 i + 2 h + b] of group i (8 columns) are columns
// 8 i + 2 (lane % 4) + b, rows lane / 4 + 8 h of lanes 0-15 (v) and 16-31 (w).
struct Frag {
    uint32_t v[8], w[8];
};

__device__ __forceinline__ void frag_request(uint32_t taddr, Frag &f)
{
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(f.v[0]), "=r"(f.v[1]), "=r"(f.v[2]), "=r"(f.v[3]), "=r"(f.v[4]), "=r"(f.v[5]), "=r"(f.v[6]),
                   "=r"(f.v[7])
                 : "r"(taddr));
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(f.w[0]), "=r"(f.w[1]), "=r"(f.w[2]), "=r"(f.w[3]), "=r"(f.w[4]), "=r"(f.w[5]), "=r"(f.w[6]),
                   "=r"(f.w[7])
                 : "r"(taddr + (16u << 16)));
}

// Waits for every request of this warp.  The fragment is not an operand: it would be
// copied.  The FMAs that use it are volatile, so they stay behind the wait.
__device__ __forceinline__ void frag_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// Plain FMAs: the packed f32x2 form has the same rate (two a lane and two clocks), and
// its operand pairs cost two moves each here (196 against 133 us below, epilogue alone).
__device__ __forceinline__ void fma_volatile(float &acc, uint32_t v, float s)
{
    asm volatile("fma.rn.f32 %0, %1, %2, %0;" : "+f"(acc) : "f"(__uint_as_float(v)), "f"(s));
}

__device__ __forceinline__ void store4(float *p, float a, float b, float c, float d)
{
    *reinterpret_cast<float4 *>(p) = make_float4(a, b, c, d);
}

__device__ __forceinline__ void store4(__nv_bfloat16 *p, float a, float b, float c, float d)
{
    const __nv_bfloat162 lo = __floats2bfloat162_rn(a, b), hi = __floats2bfloat162_rn(c, d);
    *reinterpret_cast<uint2 *>(p) =
        make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
}

// Columns of a pair's tile (tcgen05 N: a multiple of 16), and of each quarter of the epilogue warps
__device__ __forceinline__ int tile_columns(int rows) { return (rows + 15) & ~15; }
__device__ __forceinline__ int quarter_columns(int cols) { return ((cols + 3) / 4 + 15) & ~15; }

// ---- the epilogue --------------------------------------------------------------------
// What one warp needs of its CTA: barrier arrays, the scales of this lane's columns, this
// warp's tensor-memory lanes.
struct Epilogue {
    uint32_t acc_full, sc_full, sc_empty;
    uint32_t acc_empty;  // the leader's (shared::cluster)
    uint32_t tmem, scales;
};

// All blocks of a tile for 16 * STEPS columns from c0, then the stores.  The step
// count is a template argument: with a branch per step the loads and FMAs of a
// step cannot overlap (844 against 602 clocks a block, the loop alone).  False: a
// wait ran out.
template <int STEPS, class OUT, bool PERM>
__device__ __forceinline__ bool epilogue_tile(const Epilogue &e, const ProductArgs &a, int c0, int rows, OUT *out,
                                              int n_left, int &it)
{
    const int lane = threadIdx.x & 31;
    float acc[2 * STEPS + 1][4][2];  // [column group][row group][column]
#pragma unroll
    for (int i = 0; i < 2 * STEPS; ++i)
#pragma unroll
        for (int g = 0; g < 4; ++g) acc[i][g][0] = acc[i][g][1] = 0.f;
    for (int kb = 0; kb < a.kblocks; ++kb, ++it) {
        const int d = it % kPairBufs, s = it % kPairScales;
        const uint32_t pa = (it / kPairBufs) & 1, ps = (it / kPairScales) & 1;
        const bool sc_ready = bar_try(e.sc_full + 8 * s, ps), acc_ready = bar_try(e.acc_full + 8 * d, pa);
        if (!__all_sync(0xffffffffu, sc_ready && acc_ready)) {
            const bool ok = bar_wait(e.sc_full + 8 * s, ps) && bar_wait(e.acc_full + 8 * d, pa);
            if (!__all_sync(0xffffffffu, ok)) return false;
        }
        tc_fence_after_sync();
        const uint32_t td = e.tmem + d * kPairTokens + c0;
        const uint32_t sc = e.scales + (s * kScaleRow + c0 / 4) * 4;
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
            Frag f;
            frag_request(td + 16 * i, f);
            const float4 w4 = lds4(sc + 16 * i);
            frag_wait();
            if (i == STEPS - 1) {  // every value of the buffer has been read
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) pair_arrive(e.acc_empty + 8 * d);
            }
            const float w[2][2] = {{w4.x, w4.y}, {w4.z, w4.w}};
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    fma_volatile(acc[2 * i + q][0][b], f.v[4 * q + b], w[q][b]);
                    fma_volatile(acc[2 * i + q][1][b], f.v[4 * q + 2 + b], w[q][b]);
                    fma_volatile(acc[2 * i + q][2][b], f.w[4 * q + b], w[q][b]);
                    fma_volatile(acc[2 * i + q][3][b], f.w[4 * q + 2 + b], w[q][b]);
                }
        }
        __syncwarp();
        if (lane == 0) {
            if (STEPS == 0) pair_arrive(e.acc_empty + 8 * d);
            bar_arrive(e.sc_empty + 8 * s);
        }
    }
    // out: column c0 + 2 (lane % 4), this lane's first weight row, of which n_left are left
    const int64_t group = 8 * a.ld_out;
    int left = rows - c0 - 2 * (lane & 3);
    if (n_left <= 0) return true;
#pragma unroll
    for (int i = 0; i < 2 * STEPS; ++i, out += group, left -= 8) {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            OUT *o = b ? out + a.ld_out : out;
            if (left <= b) continue;
            if (PERM) {
                store4(o, acc[i][0][b], acc[i][1][b], acc[i][2][b], acc[i][3][b]);
            } else {
#pragma unroll
                for (int g = 0; g < 4; ++g)
                    if (8 * g < n_left) o[8 * g] = OUT(acc[i][g][b]);
            }
        }
    }
    return true;
}

// PERM: weight rows permuted by the tensor map (n a multiple of 32), 4-wide stores.
template <class OUT, bool PERM>
__global__ void __launch_bounds__(kPairThreads, 1)
    fp8_pair_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
                    const ProductArgs a)
{
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t full[kPairStages], empty[kPairStages], acc_full[kPairBufs], acc_empty[kPairBufs],
        sc_full[kPairScales], sc_empty[kPairScales], drain_bar;
    __shared__ uint32_t tmem_base;
    __shared__ int warp_tiles[kPairThreads / 32];
    __shared__ volatile int abort_flag;
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float *scale_ring = reinterpret_cast<float *>(smem + kPairStages * kPairStage);  // [slot][kScaleRow]
    int *offset = reinterpret_cast<int *>(scale_ring + kPairScales * kScaleRow);
    int *first_tile = offset + kMaxExperts + 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const unsigned rank = cluster_rank();

    if (warp == kMmaWarp) {
        tmem_alloc2(&tmem_base, kPairBufs * kPairTokens);
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
        for (int s = 0; s < kPairScales; ++s) {
            mbar_init(&sc_full[s], 2);
            mbar_init(&sc_empty[s], kEpiWarps);
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
    const int n_pairs = (a.n + 2 * kWeightRows - 1) / (2 * kWeightRows);
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
                const int mine = tile_columns(t.rows) / 2;  // token rows of each CTA
                const int boxes = (mine + kBox - 1) / kBox;
                const uint32_t bytes = 2 * (kABytes + boxes * kBox * 128);
                const int w0 = (t.n_tile * 2 + (int)rank) * kWeightRows, x0 = t.row0 + (int)rank * mine;
                for (int kb = 0; kb < a.kblocks; ++kb, ++issued, r.next()) {
                    // the slot's previous use has been multiplied (a fresh slot passes)
                    if (!__all_sync(0xffffffffu, bar_wait(empty_at + 8 * r.slot, r.phase ^ 1))) {
                        go = false;
                        break;
                    }
                    if (elect_one()) {
                        uint8_t *w_s = smem + r.slot * kPairStage, *x_s = w_s + kABytes;
                        if (rank == 0) mbar_arrive_expect_tx(&full[r.slot], bytes);
                        const uint32_t bar = leader_full + 8 * r.slot;
                        if (PERM) tma2_load_5d(w_s, &map_w, bar, kb * 128, 0, 0, w0 / 32, t.group);
                        else tma2_load_3d(w_s, &map_w, bar, kb * 128, w0, t.group);
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
                const uint64_t w_desc = desc_kmajor_sw128(smem), x_desc = desc_kmajor_sw128(smem + kABytes);
                Ring<kPairStages> r;
                Ring<kPairBufs> d;
                bool go = true;
                for (int id = worker; id < n_work && go; id += workers) {
                    const Tile t = tile_at(id, n_pairs, a.groups, first_tile, offset);
                    const uint32_t idesc = idesc_e4m3(2 * kWeightRows, tile_columns(t.rows));
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
                                mma2_f8(tmem + d.slot * kPairTokens, wd + 2 * kk, xd + 2 * kk, idesc, kk != 0);
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
        } else {  // ---- scales of half of the columns
            const int c0 = (warp - kScaleWarp0) * (kPairTokens / 2);
            int it = 0;
            bool go = true;
            for (int id = worker; id < n_work && go; id += workers) {
                const Tile t = tile_at(id, n_pairs, a.groups, first_tile, offset);
                const int nb = t.n_tile * 2 + (int)rank;
                const bool has_w = nb < a.n_tiles;
                const float *bs = a.b_scale + ((int64_t)t.group * a.n_tiles + (has_w ? nb : 0)) * a.kblocks;
                const float *as = a.a_scale + t.row0;
                int at[4];  // this lane's columns, inside the tile
#pragma unroll
                for (int j = 0; j < 4; ++j) at[j] = min(c0 + j * 32 + lane, t.rows - 1);
                for (int k0 = 0; k0 < a.kblocks && go; k0 += kScaleAhead) {
                    // every load from a valid address, so that none waits behind a branch
                    float v[kScaleAhead][4], w[kScaleAhead];
#pragma unroll
                    for (int i = 0; i < kScaleAhead; ++i) {
                        const int kb = min(k0 + i, a.kblocks - 1);
                        w[i] = __ldg(bs + kb);
#pragma unroll
                        for (int j = 0; j < 4; ++j) v[i][j] = __ldg(as + (int64_t)kb * a.ld_a_scale + at[j]);
                    }
#pragma unroll
                    for (int i = 0; i < kScaleAhead; ++i) {
                        if (k0 + i >= a.kblocks) break;
                        const int s = it % kPairScales, u = it / kPairScales;
                        ++it;
                        if (lane == 0) {
                            go = u == 0 || mbar_wait(&sc_empty[s], (u - 1) & 1);
                            if (!go) abort_flag = 1;
                        }
                        go = __shfl_sync(0xffffffffu, go, 0);
                        if (!go) break;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int c = c0 + j * 32 + lane;
                            scale_ring[s * kScaleRow + ((c & 7) >> 1) * kScaleStride + (c >> 3) * 2 + (c & 1)] = has_w ? v[i][j] * w[i] : 0.f;
                        }
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&sc_full[s]);
                    }
                }
            }
        }
    } else {  // ---- epilogue
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpilogueRegs));
        const int part = warp >> 2, quarter = warp & 3;
        const Epilogue e{smem_u32(acc_full),
                         smem_u32(sc_full),
                         smem_u32(sc_empty),
                         cluster_map(smem_u32(acc_empty), 0),
                         tmem + ((uint32_t)(quarter * 32) << 16),
                         smem_u32(scale_ring + (lane & 3) * kScaleStride)};
        int it = 0;
        bool go = true;
        for (int id = worker; id < n_work && go; id += workers) {
            const Tile t = tile_at(id, n_pairs, a.groups, first_tile, offset);
            const int all = tile_columns(t.rows), most = quarter_columns(all);
            const int c0 = min(part * most, all), cols = min(most, all - c0);
            const int n = (t.n_tile * 2 + (int)rank) * kWeightRows + quarter * 32 + (PERM ? 4 : 1) * (lane >> 2);
            OUT *out = static_cast<OUT *>(a.out) + (int64_t)(t.row0 + c0 + 2 * (lane & 3)) * a.ld_out + n;
            switch (cols / 16) {
            case 0: go = epilogue_tile<0, OUT, PERM>(e, a, c0, t.rows, out, a.n - n, it); break;
            case 1: go = epilogue_tile<1, OUT, PERM>(e, a, c0, t.rows, out, a.n - n, it); break;
            case 2: go = epilogue_tile<2, OUT, PERM>(e, a, c0, t.rows, out, a.n - n, it); break;
            case 3: go = epilogue_tile<3, OUT, PERM>(e, a, c0, t.rows, out, a.n - n, it); break;
            default: go = epilogue_tile<4, OUT, PERM>(e, a, c0, t.rows, out, a.n - n, it); break;
            }
            if (!go) abort_flag = 1;
        }
    }
    __syncwarp();
    if (abort_flag && threadIdx.x == 0 && a.status) atomicExch(a.status, (int)MOE_ERR_TIMEOUT);
    tc_fence_before_sync();
    __syncthreads();
    cluster_sync();  // neither CTA leaves while the other may still arrive here or read its operands
    tc_fence_after_sync();
    if (warp == kMmaWarp) tmem_dealloc2(tmem, kPairBufs * kPairTokens);
}

// Weight rows as [group][q][g][r][k] with row = 32 q + 4 r + g: a box of 128 rows puts
// row 4 r + g of each 32 at shared-memory row 8 g + r.
bool permuted_map(CUtensorMap *m, const Operands &o, const ProductArgs &a)
{
    const tmaps::EncodeTiledFn f = tmaps::encode_fn();
    if (!f) return false;
    cuuint64_t dims[5] = {(cuuint64_t)o.k, 8, 4, (cuuint64_t)(a.n / 32), (cuuint64_t)a.groups};
    cuuint64_t strides[4] = {(cuuint64_t)o.ld_b * 4, (cuuint64_t)o.ld_b, (cuuint64_t)o.ld_b * 32, (cuuint64_t)o.stride_b};
    cuuint32_t box[5] = {128, 8, 4, kWeightRows / 32, 1}, es[5] = {1, 1, 1, 1, 1};
    return f(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, const_cast<uint8_t *>(o.b), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class OUT>
cudaError_t pair_launch(const CUtensorMap &mw, const CUtensorMap &mx, const ProductArgs &a, bool perm, int pairs,
                        cudaStream_t s)
{
    return perm ? launch(fp8_pair_kernel<OUT, true>, dim3(2 * pairs), kPairThreads, kPairSmem, s, 2, false, mw, mx, a)
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
    const bool perm = a.n % 32 == 0 && a.ld_out % 4 == 0 && aligned(a.out, bf16 ? 8 : 16);
    CUtensorMap mw, mx;
    if (perm ? !permuted_map(&mw, o, a) : !code_map(&mw, o.b, o.k, a.n, o.ld_b, a.groups, o.stride_b, kWeightRows))
        return MOE_ERR_CUDA;
    if (!code_map(&mx, o.a, o.k, a.rows, o.ld_a, 0, 0, kBox)) return MOE_ERR_CUDA;
    return launched(bf16 ? pair_launch<__nv_bfloat16>(mw, mx, a, perm, pairs, s)
                         : pair_launch<float>(mw, mx, a, perm, pairs, s));
}

}  // namespace fp8
}  // namespace moe
