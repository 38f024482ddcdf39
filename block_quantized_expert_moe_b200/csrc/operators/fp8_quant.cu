// Quantisers to E4M3 codes with an fp32 scale per block of 128.
//
//   a     = max(max |x| over the block, 448 * 2^-126)
//   scale = a / 448,   code = E4M3(x * (448 / a))     (nearest even)
//
// in fp32, so scale * code is x within half an E4M3 step of the block's largest
// magnitude's scale, and 448 / a and the product never overflow.  The floor
// keeps an all-zero block at codes 0 (its scale is 2^-126).  A NaN or infinity
// makes its whole block NaN.  Blocks are 128 columns of one row (activations)
// or 128 rows x 128 columns (weights); the last ones may be shorter.
//
// Activations may be gathered (output row r is source row rows[r]) or be the
// SwiGLU of a gate/up row, silu(x[:cols]) * x[cols:], so that neither the
// gathered rows nor h is ever written: bytes are one read of the source and one
// write of codes and scales.  Half a warp owns a block: eight values a lane,
// four shuffles for the maximum (of two blocks at once).  A CTA takes 8 rows by all their blocks, so
// the scales of a block (stored block by block over the rows, the layout the
// product reads) leave as whole 32-byte sectors.  SwiGLU over 81,920 rows of 512 in
// bf16: 34.1 us, 6.2 TB/s of the 211 MB it must move (94 % of a plain copy's
// rate); 81,920 gathered rows of 2048: 69 to 71 us, bound by instruction issue; 81,920 contiguous ones
// 84 us of a floor of 77.  Where a half-warp's second block is not whole, the turn is read value by
// value: SwiGLU of 81,920 rows of 128, 256 and 768 columns 23, 41 and 66 us (floors 8, 16 and 48).
#include <algorithm>

#include "op_common.cuh"

namespace moe {
namespace {

using namespace op;

constexpr float kE4m3Max = 448.f;
constexpr float kAmaxFloor = 448.f * 1.17549435e-38f;  // 448 * 2^-126
constexpr int kQuantThreads = 256, kQuantRows = 8;

// scale = a / 448 and inv = 448 / a, both correctly rounded.  The division by a constant is
// Markstein's (IBM J. Res. Dev. 34, 1990): with c the rounded 1 / 448 and q = a c, one
// exact residual corrects q to the rounded quotient; an infinite a is left as it is.
// (x times the rounded 448 / a leaves a tie between two codes one fp32 step off in one of ten cases,
// so that the odd code is taken, equally near; a second term of 448 / a mends that and costs 69.5 ->
// 80.6 us for 81,920 gathered rows of 2048.)
__device__ __forceinline__ void block_scale(float amax, float &scale, float &inv)
{
    const float a = amax < kAmaxFloor ? kAmaxFloor : amax;  // NaN stays
    constexpr float c = 1.f / kE4m3Max;
    const float q = a * c;
    scale = a == INFINITY ? a : __fmaf_rn(__fmaf_rn(-q, kE4m3Max, a), c, q);
    inv = __fdiv_rn(kE4m3Max, a);
}

// two E4M3 codes (lo in the low byte), round to nearest even, |x| <= 448
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// largest magnitude of three values; NaN if one is
__device__ __forceinline__ float amax3(float a, float b, float c)
{
    float m;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(a), "f"(b), "f"(c));
    return m;
}

__device__ __forceinline__ float amax8(const float (&v)[8])
{
    return amax3(amax3(v[0], v[1], v[2]), amax3(v[3], v[4], v[5]), amax3(v[6], v[7], 0.f));
}

__device__ __forceinline__ float amax2(float a, float b) { return amax3(a, b, 0.f); }

// g / (1 + exp(-g)) from the hardware's 2^t and reciprocal (2^-22 relative each); t = -g log2(e)
// is rounded, which adds |g| 2^-24 for negative g.  Down to kSiluFar the sigmoid is a normal number
// (the reciprocal gives 0 for smaller ones).
constexpr float kSiluFar = -87.f;
__device__ __forceinline__ float silu(float g)
{
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.44269504f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return g * r;
}

// Below kSiluFar, where 1 + exp(-g) rounds to exp(-g) and silu(g) is an fp32 number down to -104:
// g exp(g) as (g h) h with h = exp(g / 2), which leaves the normal numbers in the last product only.
__device__ __forceinline__ float silu_far(float g)
{
    const float h = expf(0.5f * g);
    return (g * h) * h;
}

__device__ __forceinline__ float min3(float a, float b, float c)
{
    float m;
    asm("min.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(a), "f"(b), "f"(c));
    return m;
}

__device__ __forceinline__ float min8(const float (&v)[8], float m)
{
    return min3(min3(v[0], v[1], v[2]), min3(v[3], v[4], v[5]), min3(v[6], v[7], m));
}

// Eight values as loaded, and as fp32.
template <class T>
struct Raw8;
template <>
struct Raw8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p)
    {
        a = *reinterpret_cast<const float4 *>(p);
        b = reinterpret_cast<const float4 *>(p)[1];
    }
    __device__ __forceinline__ void pack(const float (&v)[8])
    {
        a = make_float4(v[0], v[1], v[2], v[3]);
        b = make_float4(v[4], v[5], v[6], v[7]);
    }
    __device__ __forceinline__ void values(float (&v)[8]) const
    {
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
};
template <>
struct Raw8<__nv_bfloat16> {
    uint4 r;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { r = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void pack(const __nv_bfloat16 (&v)[8])
    {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = __bfloat16_as_ushort(v[2 * i]) | (uint32_t)__bfloat16_as_ushort(v[2 * i + 1]) << 16;
        r = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ __forceinline__ void values(float (&v)[8]) const
    {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
};

__device__ __forceinline__ float as_float(float v) { return v; }
__device__ __forceinline__ float as_float(__nv_bfloat16 v) { return __bfloat162float(v); }

struct QuantArgs {
    const void *x;
    int64_t ld_x;
    const int32_t *index;  // output row -> source row, or null
    int src_rows, rows, cols, blocks;
    uint8_t *codes;
    int64_t ld_codes;
    float *scales;
    int64_t ld_scales;
};

// Eight consecutive values of a row from column c0 (zero from `cols` on, and where there is no row),
// kept as loaded: bf16 in half the registers.
template <class T, bool WIDE>
struct Kept {
    Raw8<T> r = {};
    __device__ __forceinline__ void load(const T *row, int c0, int cols)
    {
        if (!row) return;
        if (WIDE && c0 + 8 <= cols) {
            r.load(row + c0);
        } else {
            T v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = c0 + j < cols ? row[c0 + j] : T(0.f);
            r.pack(v);
        }
    }
    __device__ __forceinline__ void values(float (&v)[8]) const { r.values(v); }
};

// The lane's eight columns of a block: 8 in a row, or for fp32 rows off 16-byte boundaries every
// 16th, so that a load is consecutive.  (28,968 gathered rows of 1309: 36.1 us, 41.8 with 8 in a
// row; for bf16 the codes' byte stores cost more: 60,000 SwiGLU rows of 513 46.4 us then, 56.6 with
// every 16th.)
template <class T, bool WIDE>
struct Columns {
    static constexpr bool SPREAD = !WIDE && sizeof(T) == 4;
    static constexpr int STEP = SPREAD ? 16 : 1;
    static __device__ __forceinline__ int first(int b, int lane) { return b * kScaleBlock + lane * (SPREAD ? 1 : 8); }
};

// The lane's values of a block of a source row, or of its SwiGLU (WIDE: then `far` is set where a gate
// is below kSiluFar, whose value is not right yet); zeros for no row.
template <class T, bool SWIGLU, bool WIDE>
__device__ __forceinline__ void row_values(const T *x, int b, int lane, int cols, float (&v)[8], bool &far)
{
    const int c0 = Columns<T, WIDE>::first(b, lane);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int c = c0 + j * Columns<T, WIDE>::STEP;
        v[j] = x && c < cols ? as_float(x[c]) : 0.f;
    }
    if (SWIGLU) {
        float w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = c0 + j * Columns<T, WIDE>::STEP;
            w[j] = x && c < cols ? as_float(x[cols + c]) : 0.f;
        }
        const bool some_far = min8(v, 0.f) < kSiluFar;
        if (!WIDE && some_far) {  // (out of line 60,000 rows of 513 in bf16 take 51.7 us, so 47.3)
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = (v[j] < kSiluFar ? silu_far(v[j]) : silu(v[j])) * w[j];
        } else {
            far = far || some_far;
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = silu(v[j]) * w[j];
        }
    }
}

// Whether a lane's sixteen gates may hold one below kSiluFar.  bf16: such a gate's bits are, as an
// unsigned number, at or above those of -87.5 (NaNs with a sign are too), two gates an instruction on
// the words as loaded.
__device__ __forceinline__ bool has_far(const Raw8<__nv_bfloat16> &a, const Raw8<__nv_bfloat16> &b)
{
    const uint32_t m = __vmaxu2(__vmaxu2(__vmaxu2(a.r.x, a.r.y), __vmaxu2(a.r.z, a.r.w)),
                                __vmaxu2(__vmaxu2(b.r.x, b.r.y), __vmaxu2(b.r.z, b.r.w)));
    return m >= 0xc2af0000u || (m << 16) >= 0xc2af0000u;
}
__device__ __forceinline__ bool has_far(const Raw8<float> &a, const Raw8<float> &b)
{
    float v[8], w[8];
    a.values(v);
    b.values(w);
    return min8(v, min8(w, 0.f)) < kSiluFar;
}

// The lane's values of a block, read once more, where some gate is far: seldom, so out of line (in line,
// or with fp32 minima for the test, the usual path gets 48 registers or another order of its loads:
// 36.5 to 43.4 us for 81,920 x 512 in bf16, 34.1 so).
struct Eight {
    float v[8];
};

template <class T>
__device__ __noinline__ Eight far_values(const T *x, int b, int lane, int cols)
{
    Eight r;
#pragma unroll 1
    for (int j = 0; j < 8; ++j) {
        const int c = Columns<T, true>::first(b, lane) + j * Columns<T, true>::STEP;
        const float g = x && c < cols ? as_float(x[c]) : 0.f, u = x && c < cols ? as_float(x[cols + c]) : 0.f;
        r.v[j] = (g < kSiluFar ? silu_far(g) : silu(g)) * u;
    }
    return r;
}

template <class T, bool WIDE>
__device__ __forceinline__ void store_codes(const QuantArgs &a, const float (&v)[8], float inv, int row, int b, int lane)
{
    uint2 q;
    q.x = e4m3x2(v[0] * inv, v[1] * inv) | e4m3x2(v[2] * inv, v[3] * inv) << 16;
    q.y = e4m3x2(v[4] * inv, v[5] * inv) | e4m3x2(v[6] * inv, v[7] * inv) << 16;
    const int c0 = Columns<T, WIDE>::first(b, lane);
    uint8_t *dst = a.codes + (int64_t)row * a.ld_codes;
    if (!Columns<T, WIDE>::SPREAD && c0 + 8 <= a.cols) {
        *reinterpret_cast<uint2 *>(dst + c0) = q;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = c0 + j * Columns<T, WIDE>::STEP;
            if (c < a.cols) dst[c] = (uint8_t)((j < 4 ? q.x : q.y) >> (8 * (j & 3)));
        }
    }
}

// Two blocks of a row at a time: all their loads first, and one sequence of shuffles and
// divisions for both (lanes 0-7 of the half-warp end up with the first block's maximum,
// lanes 8-15 with the second's).  The kernel is bound by instruction issue on bf16.
constexpr int kQuantPer = kQuantThreads / 16 / kQuantRows;  // half-warps on a row
constexpr int kQuantTurn = 2 * kQuantPer;                   // blocks of a row a CTA takes at a time

template <class T, bool SWIGLU, bool WIDE>
__global__ void __launch_bounds__(kQuantThreads, SWIGLU && WIDE && sizeof(T) == 2 ? 6 : 0)
    quantize_rows_kernel(const QuantArgs a)
{
    const int half = threadIdx.x >> 4, lane = threadIdx.x & 15;
    const int row = blockIdx.x * kQuantRows + (half & (kQuantRows - 1));
    follow_previous();
    const T *x = nullptr;
    if (row < a.rows) {
        const int src = a.index ? a.index[row] : row;
        if ((unsigned)src < (unsigned)a.src_rows) x = static_cast<const T *>(a.x) + (int64_t)src * a.ld_x;
    }
    for (int b0 = half / kQuantRows + blockIdx.y * kQuantTurn; b0 < a.blocks; b0 += kQuantTurn * gridDim.y) {
        const int b1 = b0 + kQuantPer;
        float v0[8], v1[8];
        bool far = false;
        if (WIDE && (b1 + 1) * kScaleBlock <= a.cols) {
            Raw8<T> g0 = {}, g1 = {}, u0 = {}, u1 = {};
            if (x) {
                const T *p0 = x + b0 * kScaleBlock + lane * 8, *p1 = p0 + kQuantPer * kScaleBlock;
                g0.load(p0);
                g1.load(p1);
                if (SWIGLU) {
                    u0.load(p0 + a.cols);
                    u1.load(p1 + a.cols);
                }
            }
            g0.values(v0);
            g1.values(v1);
            if (SWIGLU) {
                far = has_far(g0, g1);
                float w0[8], w1[8];
                u0.values(w0);
                u1.values(w1);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    v0[j] = silu(v0[j]) * w0[j];
                    v1[j] = silu(v1[j]) * w1[j];
                }
            }
        } else {
            row_values<T, SWIGLU, WIDE>(x, b0, lane, a.cols, v0, far);
            row_values<T, SWIGLU, WIDE>(x, b1, lane, a.cols, v1, far);
        }
        if (SWIGLU && WIDE && far) {
            const Eight f0 = far_values<T>(x, b0, lane, a.cols), f1 = far_values<T>(x, b1, lane, a.cols);
#pragma unroll
            for (int j = 0; j < 8; ++j) v0[j] = f0.v[j], v1[j] = f1.v[j];
        }
        const bool second = lane & 8;
        const float m0 = amax8(v0), m1 = amax8(v1);
        float m = amax2(second ? m1 : m0, __shfl_xor_sync(0xffffffffu, second ? m0 : m1, 8));
#pragma unroll
        for (int d = 4; d; d >>= 1) m = amax2(m, __shfl_xor_sync(0xffffffffu, m, d));
        float scale, inv;
        block_scale(m, scale, inv);
        const float inv0 = __shfl_sync(0xffffffffu, inv, 0, 16), inv1 = __shfl_sync(0xffffffffu, inv, 8, 16);
        if (row >= a.rows) continue;
        store_codes<T, WIDE>(a, v0, inv0, row, b0, lane);
        if (b1 < a.blocks) store_codes<T, WIDE>(a, v1, inv1, row, b1, lane);
        const int b = second ? b1 : b0;
        if ((lane & 7) == 0 && b < a.blocks) a.scales[(int64_t)b * a.ld_scales + row] = scale;
    }
}

// One CTA per 128 x 128 block: thread t holds 8 columns of rows t / 16 + 16 i.
// The loads come before everything else and the values stay as loaded, so that four CTAs of
// bf16 fit an SM (three of fp32): 64 matrices of 1024 x 2048 bf16 67 us of a floor of 61, with the
// values as fp32 136; fp32 97 against 149.
template <class T, bool WIDE>
__global__ void __launch_bounds__(kQuantThreads, sizeof(T) == 2 ? 4 : 3)
    quantize_weight_kernel(const T *w, int64_t ld_w, int64_t group_stride, int n, int cols,
                           uint8_t *codes, int64_t ld_codes, int64_t codes_stride,
                           float *scales)
{
    __shared__ float red[kQuantThreads / 32];
    const int kb = blockIdx.x, nb = blockIdx.y, g = blockIdx.z;
    const int c0 = kb * kScaleBlock + (threadIdx.x & 15) * 8;
    const int r0 = nb * kScaleBlock + (threadIdx.x >> 4);
    const T *src = w + (int64_t)g * group_stride;
    follow_previous();
    Kept<T, WIDE> v[8];
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i].load(r0 + 16 * i < n ? src + (int64_t)(r0 + 16 * i) * ld_w : nullptr, c0, cols);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float x[8];
        v[i].values(x);
        m = amax2(m, amax8(x));
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) m = amax2(m, __shfl_xor_sync(0xffffffffu, m, d));
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kQuantThreads / 32; ++i) m = amax2(m, red[i]);
    float scale, inv;
    block_scale(m, scale, inv);
    if (threadIdx.x == 0) scales[((int64_t)g * gridDim.y + nb) * gridDim.x + kb] = scale;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = r0 + 16 * i;
        if (r >= n) continue;
        float x[8];
        v[i].values(x);
        uint2 q;
        q.x = e4m3x2(x[0] * inv, x[1] * inv) | e4m3x2(x[2] * inv, x[3] * inv) << 16;
        q.y = e4m3x2(x[4] * inv, x[5] * inv) | e4m3x2(x[6] * inv, x[7] * inv) << 16;
        uint8_t *dst = codes + (int64_t)g * codes_stride + (int64_t)r * ld_codes + c0;
        if (c0 + 8 <= cols) {
            *reinterpret_cast<uint2 *>(dst) = q;
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (c0 + j < cols) dst[j] = (uint8_t)((j < 4 ? q.x : q.y) >> (8 * (j & 3)));
        }
    }
}

typedef void (*QuantKernel)(const QuantArgs);

template <class T>
QuantKernel quant_pick(bool swiglu, bool wide)
{
    if (swiglu) return wide ? quantize_rows_kernel<T, true, true> : quantize_rows_kernel<T, true, false>;
    return wide ? quantize_rows_kernel<T, false, true> : quantize_rows_kernel<T, false, false>;
}

unsigned dtype_size(moe_dtype dt) { return dt == MOE_DT_BF16 ? 2 : 4; }

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status moe_fp8_quantize(const void *x, moe_dtype x_dtype, int64_t ld_x, const int32_t *rows,
                                       int n_src_rows, int n_rows, int cols, int swiglu, uint8_t *codes,
                                       int64_t ld_codes, float *scales, int64_t ld_scales, void *stream)
{
    if ((x_dtype != MOE_DT_F32 && x_dtype != MOE_DT_BF16) || (swiglu != 0 && swiglu != 1)) return MOE_ERR_INVALID_ARG;
    if (n_rows < 0 || n_rows > kMaxRows || n_src_rows < 0 || cols < 1 || cols > (1 << 20)) return MOE_ERR_INVALID_ARG;
    if (!rows && n_src_rows != n_rows) return MOE_ERR_INVALID_ARG;
    if (ld_x < (swiglu ? 2 : 1) * (int64_t)cols || ld_codes < cols || ld_codes % 16 || ld_scales < n_rows)
        return MOE_ERR_INVALID_ARG;
    if (n_rows == 0) return MOE_OK;
    if (!codes || !scales || (!x && n_src_rows)) return MOE_ERR_INVALID_ARG;
    const unsigned size = dtype_size(x_dtype);
    if (!aligned(x, size) || !aligned(rows, 4) || !aligned(codes, 16) || !aligned(scales, 4)) return MOE_ERR_INVALID_ARG;
    QuantArgs a{};
    a.x = x;
    a.ld_x = ld_x;
    a.index = rows;
    a.src_rows = n_src_rows;
    a.rows = n_rows;
    a.cols = cols;
    a.blocks = ceil_div(cols, kScaleBlock);
    a.codes = codes;
    a.ld_codes = ld_codes;
    a.scales = scales;
    a.ld_scales = ld_scales;
    // 16-byte loads where every block of every row (and of its up half) starts on one
    const bool wide = aligned(x, 16) && ld_x * size % 16 == 0 && (!swiglu || (int64_t)cols * size % 16 == 0);
    QuantKernel f = x_dtype == MOE_DT_BF16 ? quant_pick<__nv_bfloat16>(swiglu, wide) : quant_pick<float>(swiglu, wide);
    const int row_ctas = ceil_div(n_rows, kQuantRows);
    // few rows: a CTA per turn of blocks; many: a CTA walks its rows' blocks
    const int by = std::max(1, std::min(ceil_div(a.blocks, kQuantTurn), 1184 / row_ctas));
    return launched(launch(f, dim3(row_ctas, by), kQuantThreads, 0, static_cast<cudaStream_t>(stream), 1, a));
}

extern "C" moe_status moe_fp8_quantize_weight(const void *w, moe_dtype w_dtype, int64_t ld_w, int64_t group_stride_w,
                                              int n_groups, int n, int cols, uint8_t *codes, int64_t ld_codes,
                                              int64_t group_stride_codes, float *scales, void *stream)
{
    if (w_dtype != MOE_DT_F32 && w_dtype != MOE_DT_BF16) return MOE_ERR_INVALID_ARG;
    if (n_groups < 0 || n_groups > 65535 || n < 0 || n > (1 << 20) || cols < 1 || cols > (1 << 20))
        return MOE_ERR_INVALID_ARG;
    if (ld_w < cols || ld_codes < cols || ld_codes % 16 || group_stride_codes % 16) return MOE_ERR_INVALID_ARG;
    if (n_groups > 1 && (group_stride_w < n * ld_w || group_stride_codes < n * ld_codes)) return MOE_ERR_INVALID_ARG;
    if (n_groups == 0 || n == 0) return MOE_OK;
    if (!w || !codes || !scales) return MOE_ERR_INVALID_ARG;
    const unsigned size = dtype_size(w_dtype);
    if (!aligned(w, size) || !aligned(codes, 16) || !aligned(scales, 4)) return MOE_ERR_INVALID_ARG;
    const bool wide = aligned(w, 16) && ld_w * size % 16 == 0 && group_stride_w * size % 16 == 0;
    const dim3 grid(ceil_div(cols, kScaleBlock), ceil_div(n, kScaleBlock), n_groups);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (w_dtype == MOE_DT_BF16) {
        auto f = wide ? quantize_weight_kernel<__nv_bfloat16, true> : quantize_weight_kernel<__nv_bfloat16, false>;
        return launched(launch(f, grid, kQuantThreads, 0, s, 1, static_cast<const __nv_bfloat16 *>(w), ld_w,
                               group_stride_w, n, cols, codes, ld_codes, group_stride_codes, scales));
    }
    auto f = wide ? quantize_weight_kernel<float, true> : quantize_weight_kernel<float, false>;
    return launched(launch(f, grid, kQuantThreads, 0, s, 1, static_cast<const float *>(w), ld_w, group_stride_w, n, cols,
                           codes, ld_codes, group_stride_codes, scales));
}
