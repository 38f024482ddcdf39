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
// 256 clocks of the FMA pipes, and a chain of latencies (MMA, commit, wait, read, release)
// over the two buffers: 784 clocks a block measured.  Tokens on the lanes give a thread
// one row: its scale is one register, loaded two blocks ahead, and one product with the
// weights' block scale covers all its columns.  (With the weights on the lanes, as in
// the kernel for few rows, every column has a scale of its own, read from shared memory:
// 153.7 us at 8192 x 4096 x 4096.)
//
// 8192 x 4096 x 4096 takes 122 us, 2.26 PFLOP/s, and 143 us (1.92) in a loop of a second:
// the power cap holds the SMs at 1.5 to 1.7 GHz, without the epilogue's work the same
// loop runs 105 us, with one of the four instructions a block 108.  81,920 rows over 512
// experts of 1024 x 2048 take 330 us (weights alone 163 us of HBM): each expert's 160
// rows fill 62 % of its tile.
//
//   warps 0-7    epilogue: warpgroup h owns columns 128 h .. 128 h + 127
//   warp 8       TMA producer (both CTAs; all bytes count on the leader's barrier)
//   warp 9       MMA issuer (the leader's only)
//   warps 10-11  idle (a register split works on groups of four warps)
// Every mbarrier wait is bounded.
#include "fp8_common.cuh"

namespace moe {
namespace fp8 {
namespace {

constexpr int kEpiWarps = 8;
constexpr int kTmaWarp = kEpiWarps, kMmaWarp = kEpiWarps + 1;
constexpr int kPairThreads = 32 * (kEpiWarps + 4);
constexpr int kPairStages = 5, kPairBufs = 2;
constexpr int kPairWeights = 256;          // weight rows (accumulator columns) of a tile
constexpr int kPart = kPairWeights * 4 / kEpiWarps;    // columns of a warpgroup
constexpr int kBox = 32;                   // token rows of one TMA box
constexpr int kPairStage = 2 * kABytes;    // 128 token rows, 128 weight rows
constexpr int kOutBytes = 32 * 128;        // a warp's output box: 32 rows of 128 bytes
constexpr int kPairSmem =
    kPairStages * kPairStage + kEpiWarps * kOutBytes + 2 * (kMaxExperts + 1) * 4 + 1024;
// registers: 384 threads at 168 are 256 at 216 and 128 at 72
constexpr int kEpilogueRegs = 216, kOtherRegs = 72;
static_assert(32 * kEpiWarps * kEpilogueRegs + 128 * kOtherRegs <= kPairThreads * 168, "register split exceeds the launch's");

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
// wait (they would be copied); the FMAs that use them are volatile and stay behind it.  (32 at
// a time spill registers: 361 against 344 us for 81,920 rows over 512 experts of 1024 x 2048.)
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
    asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(p));
    return v;
}

// Plain FMAs: the packed f32x2 form has the same rate, and its operand pairs cost moves
// (650 against 601 clocks a block of 256 columns, the loop alone).
__device__ __forceinline__ void fma_volatile(float &acc, uint32_t v, float s)
{
    asm volatile("fma.rn.f32 %0, %1, %2, %0;" : "+f"(acc) : "f"(__uint_as_float(v)), "f"(s));
}

// ---- stores -----------------------------------------------------------------------------
// A warp's 32 rows go through shared memory (128-byte rows in the 128-byte swizzle) and
// leave as TMA boxes: a thread's own row would be 32 lines an instruction, and the epilogue
// would wait for them before the next tile (131.3 us at 8192 x 4096 x 4096).
__device__ __forceinline__ void tma_store_2d(const void *tmap, uint32_t src, int c0, int c1)
{
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(tmap), "r"(src),
                 "r"(c0), "r"(c1)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

// this thread's stores have left shared memory / have been written
__device__ __forceinline__ void stores_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void stores_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

__device__ __forceinline__ uint4 pack16(const float *v, float)
{
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
}

__device__ __forceinline__ uint4 pack16(const float *v, __nv_bfloat16)
{
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
        w[j] = *reinterpret_cast<const uint32_t *>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void copy_from_shared(float *out, uint32_t at)
{
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
    *out = v;
}

__device__ __forceinline__ void copy_from_shared(__nv_bfloat16 *out, uint32_t at)
{
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at) : "memory");
    *out = __ushort_as_bfloat16(v);
}

// The warp's columns of its 32 rows, all of them inside the tile, a box at a time.  A TMA store ends
// on 16 bytes, beyond the map's last column if that does not (513 columns of fp32 in a wider buffer:
// three more of each row were written): such a box leaves value by value.
template <class OUT>
__device__ __forceinline__ void store_rows(const CUtensorMap *map, uint32_t stage, const float (&acc)[kPart], int row0,
                                           int n0, int n, OUT *out, int64_t ld)
{
    constexpr int per = 16 / sizeof(OUT), cols = 128 / sizeof(OUT);  // columns of 16 bytes, of a box
    int lane;  // volatile: addresses computed from it are not kept in registers over the block loop
    asm volatile("mov.u32 %0, %%laneid;" : "=r"(lane));
#pragma unroll
    for (int c = 0; c < kPart; c += cols) {
        if (lane == 0) stores_read();
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint4 w = pack16(acc + c + j * per, OUT());
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(stage + lane * 128 + ((j ^ (lane & 7)) << 4)),
                         "r"(w.x), "r"(w.y), "r"(w.z), "r"(w.w)
                         : "memory");
        }
        fence_proxy_async_smem();
        __syncwarp();
        const int left = n - n0 - c;
        if (left > 0 && left < cols && left % per) {
            for (int r = 0; r < 32; ++r)
                for (int j = lane; j < left; j += 32)
                    copy_from_shared(out + r * ld + c + j,
                                     stage + r * 128 + ((j / per ^ (r & 7)) << 4) + j % per * (int)sizeof(OUT));
        } else if (lane == 0 && left > 0) {
            tma_store_2d(map, stage, n0 + c, row0);
        }
    }
}

// `left` columns (of the warp's part) of one row that starts on 16 bytes.
template <class OUT>
__device__ __forceinline__ void store_row(OUT *out, const float (&acc)[kPart], int left)
{
    constexpr int per = 16 / sizeof(OUT);
#pragma unroll
    for (int c = 0; c < kPart; c += per) {
        if (c + per <= left) {
            *reinterpret_cast<uint4 *>(out + c) = pack16(acc + c, OUT());
        } else {
#pragma unroll
            for (int j = 0; j < per; ++j)
                if (c + j < left) out[c + j] = OUT(acc[c + j]);
        }
    }
}

// The warp's first `rows` rows anywhere: 32 columns at a time through shared memory, so that a
// store is 32 columns of one row (a thread writing its own row is 32 lines a store: 95 against
// 26 us for 4001 x 2047 x 2049 in bf16).
template <class OUT>
__device__ __forceinline__ void store_rows_anywhere(OUT *out, int64_t ld, uint32_t stage, const float (&acc)[kPart],
                                                    int rows, int left)
{
    int lane;  // volatile: addresses computed from it are not kept in registers over the block loop
    asm volatile("mov.u32 %0, %%laneid;" : "=r"(lane));
#pragma unroll
    for (int c = 0; c < kPart; c += 32) {
        if (c >= left) break;
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 32; ++j)
            asm volatile("st.shared.f32 [%0], %1;" ::"r"(stage + (lane * 32 + (j ^ lane)) * 4), "f"(acc[c + j]) : "memory");
        __syncwarp();
        OUT *o = out + c + lane;
        for (int r = 0; r < rows; ++r, o += ld) {
            float v;
            asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(stage + (r * 32 + (lane ^ r)) * 4) : "memory");
            if (c + lane < left) *o = OUT(v);
        }
    }
}

// The tile's token rows are split evenly between the CTAs, and so are its columns (tcgen05 N): a
// multiple of 32, so that each CTA brings whole steps of 16 as a single one's instruction takes them.
__device__ __forceinline__ int cta_rows(int rows) { return (rows + 1) / 2; }
__device__ __forceinline__ int tile_columns(int left) { return left >= kPairWeights ? kPairWeights : (left + 31) & ~31; }

// WIDE: output rows start on 16-byte boundaries (map_y is then a map of the output).
template <class OUT, bool WIDE>
__global__ void __launch_bounds__(kPairThreads, 1)
    fp8_pair_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
                    const __grid_constant__ CUtensorMap map_y, const ProductArgs a)
{
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t full[kPairStages], empty[kPairStages], acc_full[kPairBufs], acc_empty[kPairBufs], drain_bar;
    __shared__ uint32_t tmem_base;
    __shared__ int warp_tiles[kPairThreads / 32];
    __shared__ volatile int abort_flag;
    __shared__ int blocks_issued;
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *out_stage = smem + kPairStages * kPairStage;  // [warp][32][128]
    int *offset = reinterpret_cast<int *>(out_stage + kEpiWarps * kOutBytes);
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
    __syncthreads();  // tensor memory is this CTA's before the next kernel may be set up and take it
    follow_previous();
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
            TileWalk walk(worker, workers, n_pairs);
            for (int id = worker; id < n_work && go; id += workers, walk.next()) {
                const Tile t = walk.tile(a.groups, first_tile, offset);
                const int mine = cta_rows(t.rows), boxes = (mine + kBox - 1) / kBox;
                const uint32_t bytes = 2 * (kABytes + boxes * kBox * 128);
                const int n0 = t.n_tile * kPairWeights, w0 = n0 + (int)rank * tile_columns(a.n - n0) / 2;
                const int x0 = t.row0 + (int)rank * mine;
                for (int kb = 0; kb < a.kblocks; ++kb, ++issued, r.next()) {
                    // the slot's previous use has been multiplied (a fresh slot passes)
                    if (issued >= a.stall_after ||
                        !__all_sync(0xffffffffu, bar_wait(empty_at + 8 * r.slot, r.phase ^ 1))) {
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
            if (lane == 0) {
                blocks_issued = issued;
                if (!go) abort_flag = 1;
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
                TileWalk walk(worker, workers, n_pairs);
                for (int id = worker; id < n_work && go; id += workers, walk.next()) {
                    const uint32_t idesc = idesc_e4m3(256, tile_columns(a.n - walk.n_tile * kPairWeights));
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
                if (!go && elect_one()) abort_flag = 1;
            }
        }
    } else {  // ---- epilogue
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpilogueRegs));
        const int part = warp >> 2, quarter = warp & 3;
        const uint32_t acc_full_at = smem_u32(acc_full), leader_empty = cluster_map(smem_u32(acc_empty), 0);
        const uint32_t columns = tmem + ((uint32_t)(quarter * 32) << 16) + part * kPart;
        int it = 0;  // block of the CTA: buffer it % 2
        bool go = true;
        TileWalk walk(worker, workers, n_pairs);
        int n0, row0, rows;  // this warp's first column and row, and its rows that have outputs
        const float *as, *bs;
        float a0, b0, a1 = 0.f, b1 = 0.f;
        const auto begin = [&]() {
            const Tile t = walk.tile(a.groups, first_tile, offset);
            const int mine = cta_rows(t.rows);
            n0 = t.n_tile * kPairWeights + part * kPart;
            row0 = t.row0 + (int)rank * mine + quarter * 32;
            rows = n0 < a.n ? min(mine, t.rows - (int)rank * mine) - quarter * 32 : 0;
            as = a.a_scale + min(row0 + lane, t.row0 + t.rows - 1);
            bs = a.b_scale + ((int64_t)t.group * a.n_tiles + min(n0, a.n - 1) / kWeightRows) * a.kblocks;
            a0 = load_ahead(as);
            b0 = load_ahead(bs);
            if (a.kblocks > 1) {
                a1 = load_ahead(as + a.ld_a_scale);
                b1 = load_ahead(bs + 1);
            }
            walk.next();
        };
        if (worker < n_work) begin();
        for (int id = worker; id < n_work; id += workers) {
            float acc[kPart];
#pragma unroll
            for (int c = 0; c < kPart; ++c) acc[c] = 0.f;
            // one block: acc += scale * partial; false if the wait ran out
            const auto block = [&](float scale) {
                const uint32_t d = it & 1;
                if (!__all_sync(0xffffffffu, bar_wait(acc_full_at + 8 * d, (it >> 1) & 1))) return false;
                ++it;
                tc_fence_after_sync();
                if (rows > 0) {
#pragma unroll
                    for (int c = 0; c < kPart; c += kStep) {
                        uint32_t v[kStep];
                        columns_request(columns + d * kPairWeights + c, v);
                        columns_wait();
                        if (c + kStep == kPart) {  // this warp has read its part of the buffer
                            tc_fence_before_sync();
                            __syncwarp();
                            if (lane == 0) pair_arrive(leader_empty + 8 * d);
                        }
#pragma unroll
                        for (int j = 0; j < kStep; ++j) fma_volatile(acc[c + j], v[j], scale);
                    }
                } else if (lane == 0) {
                    pair_arrive(leader_empty + 8 * d);
                }
                return true;
            };
            // two blocks a turn, with the next turn's scales loaded at its start
            for (int left = a.kblocks; left > 0 && go; left -= 2) {
                const float s0 = a0 * b0;
                as += 2 * a.ld_a_scale;
                bs += 2;
                if (left > 2) {
                    a0 = load_ahead(as);
                    b0 = load_ahead(bs);
                }
                go = block(s0);
                const float s1 = a1 * b1;
                if (left > 3) {
                    a1 = load_ahead(as + a.ld_a_scale);
                    b1 = load_ahead(bs + 1);
                }
                if (go && left > 1) go = block(s1);
            }
            if (!go) {
                abort_flag = 1;
                break;
            }
            const int out_row = row0, out_col = n0, out_rows = rows;
            if (id + workers < n_work) begin();
            const uint32_t stage = smem_u32(out_stage) + warp * kOutBytes;
            OUT *out = static_cast<OUT *>(a.out) + (int64_t)out_row * a.ld_out + out_col;
            if (!WIDE) {
                if (out_rows > 0) store_rows_anywhere<OUT>(out, a.ld_out, stage, acc, min(out_rows, 32), a.n - out_col);
            } else if (out_rows >= 32) {
                store_rows<OUT>(&map_y, stage, acc, out_row, out_col, a.n, out, a.ld_out);
            } else if (lane < out_rows) {
                store_row<OUT>(out + lane * a.ld_out, acc, a.n - out_col);
            }
        }
        if (WIDE && lane == 0) stores_done();
    }
    __syncwarp();
    tc_fence_before_sync();
    __syncthreads();  // every warp is through: a wait that ran out in any of them is known here
    // after one: let copies (of both CTAs, on the leader's barriers) and MMAs in flight land
    if (abort_flag) {
        if (rank == 0 && warp == kTmaWarp && lane == 0) drain_ring(full, kPairStages, blocks_issued);
        if (rank == 0 && warp == kMmaWarp && elect_one()) {
            mma2_commit(smem_u32(&drain_bar));
            mbar_wait(&drain_bar, 0);
        }
        if (threadIdx.x == 0) record_timeout(a.status);
    }
    cluster_sync();  // neither CTA leaves while the other may still arrive here or read its operands
    tc_fence_after_sync();
    if (warp == kMmaWarp) tmem_dealloc2(tmem, kPairBufs * kPairWeights);
}

// The output as boxes of 32 rows x 128 bytes.
bool out_map(CUtensorMap *m, const ProductArgs &a, bool bf16)
{
    const tmaps::EncodeTiledFn f = tmaps::encode_fn();
    if (!f) return false;
    const int size = bf16 ? 2 : 4;
    cuuint64_t dims[2] = {(cuuint64_t)a.n, (cuuint64_t)a.rows};
    cuuint64_t strides[1] = {(cuuint64_t)a.ld_out * size};
    cuuint32_t box[2] = {(cuuint32_t)(128 / size), 32}, es[2] = {1, 1};
    return f(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, a.out, dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class OUT>
cudaError_t pair_launch(const CUtensorMap &mw, const CUtensorMap &mx, const CUtensorMap &my, const ProductArgs &a,
                        bool wide, int pairs, cudaStream_t s)
{
    return wide ? launch(fp8_pair_kernel<OUT, true>, dim3(2 * pairs), kPairThreads, kPairSmem, s, 2, mw, mx, my, a)
                : launch(fp8_pair_kernel<OUT, false>, dim3(2 * pairs), kPairThreads, kPairSmem, s, 2, mw, mx, my, a);
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

cudaError_t pair_take_error(int32_t *error) { return take_error(error); }

moe_status pair_product(const Operands &o, const ProductArgs &a, moe_dtype out_dtype, int pairs, cudaStream_t s)
{
    const bool bf16 = out_dtype == MOE_DT_BF16;
    const bool wide = aligned(a.out, 16) && a.ld_out * (bf16 ? 2 : 4) % 16 == 0 && a.ld_out < 1ll << 37;
    CUtensorMap mw, mx, my{};
    if (!code_map(&mw, o.b, o.k, a.n, o.ld_b, a.groups, o.stride_b, kPairWeights / 2)) return MOE_ERR_CUDA;
    if (!code_map(&mx, o.a, o.k, a.rows, o.ld_a, 0, 0, kBox)) return MOE_ERR_CUDA;
    if (wide && !out_map(&my, a, bf16)) return MOE_ERR_CUDA;
    return launched(bf16 ? pair_launch<__nv_bfloat16>(mw, mx, my, a, wide, pairs, s)
                         : pair_launch<float>(mw, mx, my, a, wide, pairs, s));
}

}  // namespace fp8
}  // namespace moe
