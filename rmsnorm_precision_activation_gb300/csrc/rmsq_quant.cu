// rmsq_quant.cu -- quantisation to NVFP4 and MXFP4 without a norm, and NVFP4's global scale (declared in
// include/rmsq.h).
//
//   NVFP4  per 16 elements: s_b = E4M3(min(gs amax_b / 6, 448));  q = E2M1(x gs / s_b);  gs = 2688 / max |x|
//   MXFP4  per 32 elements: e_b = clamp(ceil(log2(amax_b / 6)) + 127, 0, 255);  q = E2M1(x 2^(127 - e_b)), 0 where e_b = 0
//
// Bound by HBM: an element of 16 bits is read once and leaves as 4 bits and its part of a scale. A thread takes 16
// neighbours, so a block's maximum needs no more than one exchange, and codes leave as 8 bytes a thread.
#include <cstdint>

#include "rmsq_norm.cuh"
#include "rmsq_ops.h"

namespace rmsq {

struct QuantParams {
    const void* x;
    const float* gs;                 // or null (1)
    unsigned char* out;
    unsigned char* scale;
    long long rows, units;           // rows, and units of 16 elements in all
    long long row_units;             // per row
    int chunks;                      // swizzled: of kQuantChunk units per row
    int k_tiles;                     // swizzled: tiles of 4 scales per row
};

constexpr int kQuantThreads = 256;

// 16 elements, as they are in memory and as fp32 pairs.
template <int DT> struct Unit {
    static constexpr int N = DT == DT_F32 ? 4 : 2;
    uint4 v[N];

    __device__ __forceinline__ void load(const void* x, long long unit, bool in)
    {
        const uint4* const p = static_cast<const uint4*>(x) + unit * N;
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = in ? ld_stream_v4(p + i) : make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void pairs(float2 (&f)[8]) const
    {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float2 t[8 / N];
            Elem<DT>::pairs(v[i], t);
#pragma unroll
            for (int j = 0; j < 8 / N; ++j) f[i * (8 / N) + j] = t[j];
        }
    }
};

// max |f|, NaN where one of them is.
__device__ __forceinline__ float amax16(const float2 (&f)[8])
{
    float a = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) a = max3_nan(a, fabsf(f[j].x), fabsf(f[j].y));
    return a;
}

// E4M3 code of gs a / 6: the quotient is formed as the nearest fp32 to the exact one (a near one and the remainders of both
// steps), because with 16-bit elements it lies on a boundary of E4M3, or a rounding of gs away from one, far more
// often than chance would have it.
__device__ __forceinline__ uint32_t nvfp4_scale(float gs, float a)
{
    if (!(a < __int_as_float(0x7F800000))) return 0x7Fu;               // a NaN or an infinity: scale NaN
    const float p = __fmul_rn(gs, a), q = __fmul_rn(p, 1.0f / 6.0f);
    const float rest = __fadd_rn(__fmaf_rn(-6.0f, q, p), __fmaf_rn(gs, a, -p));
    const float sum = __fmaf_rn(rest, 1.0f / 6.0f, q);
    return cvt_e4m3x2(p > 3000.0f ? 448.0f : sum, 0.f) & 0xFFu;        // (above 2688 it saturates; p may be an infinity, or NaN)
}

// The nearest E2M1 value to T = x gs / s, exactly, ties to even. T is first formed with a rounded factor and brought to a
// multiple of 2^-19 by adding 24 (which is in [16, 32); |T| is at most 6.4 unless it saturates): t, off by less than 2^-19, so
// on T's side of every boundary (a multiple of 1/4) that it is not on. Where it is on one, the sign of x gs - t s tells T's
// side. With 16-bit elements that is frequent: boundaries are hit, or missed by a rounding of gs, whenever gs is
// near a ratio of small numbers.
constexpr float kNudge = 2.384185791015625e-7f;                        // 2^-22

// bf16 elements: one sign for all of a tensor's. An element whose t is on a boundary m has gs within 2^-17 of m s / x, a
// quotient of N, the odd parts of m (1, 3, 5, 7) times the significand of s (8 to 15), and one of x (128 to 255), times a
// power of two. Different ones are at least 1 / (105 255) = 2^-14.7 apart, so there is one such quotient at most, and gs is
// above or below it for all. Each lane tries one N with the bf16 that comes nearest. Returns what t is multiplied by: 1,
// or 1 +- 2^-22, which moves t off the boundary to its side and, by 1.5e-6 at most, over no other (2^-19 = 1.9e-6 away).
__device__ __forceinline__ float bf16_side(float gs)
{
    const int lane = threadIdx.x & 31;
    const float n = static_cast<float>((2 * (lane & 3) + 1) * (8 + (lane >> 2)));
    const float normal = gs < 1e-37f ? gs * 1.8446744073709552e19f : gs;               // (2^64)
    const float g = __uint_as_float((__float_as_uint(normal) & 0x7FFFFFu) | 0x3F800000u);
    const float x = Scalar<DT_BF16>::get(Scalar<DT_BF16>::put(__fdividef(n, g)));      // (near enough: 2^-8 apart)
    const float r = __fmaf_rn(x, g, -n);                               // its sign is exact
    const uint32_t near = __ballot_sync(0xFFFFFFFFu, fabsf(r) <= n * 7.62939453125e-6f);          // 2^-17
    if (near == 0) return 1.0f;
    const float side = __shfl_sync(0xFFFFFFFFu, r, __ffs(near) - 1);
    return side > 0.f ? 1.0f + kNudge : side < 0.f ? 1.0f - kNudge : 1.0f;
}

// Other elements: each its own sign, from a fused product and difference (t s is exact where t is on a boundary).
__device__ __forceinline__ float2 beside(float2 t, float2 x, float gs, float s)
{
    const float2 r = fma2(x, splat(gs), mul2(t, splat(-s)));
    const float step = 9.5367431640625e-7f;                            // 2^-20
    return add2(t, make_float2(r.x == 0.f ? 0.f : copysignf(step, r.x), r.y == 0.f ? 0.f : copysignf(step, r.y)));
}

// Scale code and E2M1 codes of a thread's unit (MXFP4: of half a block, the other half being the neighbour's).
template <int DT, bool NV> __device__ __forceinline__ uint32_t quantise16(const Unit<DT>& unit, float gs, float c, uint2& codes)
{
    float2 f[8];
    unit.pairs(f);
    float a = amax16(f);
    uint32_t code;
    float2 t[8];
    if (NV) {
        code = nvfp4_scale(gs, a);
        const float s = e4m3_value(code);
        // (a block below the normal floats, under the gs of a tensor as small: gs / s would leave their range at the top)
        if (a < 1e-30f && s > 0.f) {
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = mul2(f[j], splat(1.099511627776e12f));            // 2^40
            gs *= 9.094947017729282379e-13f;
        }
        const float inv = s > 0.f ? __fmul_rn(gs, __frcp_rn(s)) : 0.f;
        if (DT == DT_BF16) {
#pragma unroll
            for (int j = 0; j < 8; ++j) t[j] = fma2(fma2(f[j], splat(inv), splat(24.f)), splat(c), splat(-24.f * c));     // (24 c is exact)
        } else {
            uint32_t low = 0xFFFFFFFFu;                                // 0: some t is a multiple of 1/4
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float2 u = fma2(f[j], splat(inv), splat(24.f));
                low = min(min(low, __float_as_uint(u.x) & 0x1FFFFu), __float_as_uint(u.y) & 0x1FFFFu);
                t[j] = add2(u, splat(-24.f));
            }
            if (low == 0) {
#pragma unroll
                for (int j = 0; j < 8; ++j) t[j] = beside(t[j], f[j], gs, s);
            }
        }
    } else {
        a = max3_nan(a, __shfl_xor_sync(0xFFFFFFFFu, a, 1), 0.f);
        code = a < __int_as_float(0x7F800000) ? ue8m0_code(a) : 255u;
        const float inv = code < 255u ? ue8m0_inv_factor(code) : 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) t[j] = mul2(f[j], splat(inv));
    }
    const float lo[8] = {t[0].x, t[0].y, t[1].x, t[1].y, t[2].x, t[2].y, t[3].x, t[3].y};
    const float hi[8] = {t[4].x, t[4].y, t[5].x, t[5].y, t[6].x, t[6].y, t[7].x, t[7].y};
    codes = make_uint2(cvt_e2m1x8(lo), cvt_e2m1x8(hi));
    return code;
}

// CTAs go through the tensor from its end: what was written or read last before, by the kernel that made it or by
// nvfp4_global_scale, is still in L2.
//
// A thread's units are all on their way before the first is used. Row-major scales: two units, in their order. Swizzled ones:
// four units (fp32: two); a CTA takes kQuantChunk units of 8 (4) neighbouring rows of each of the four groups of 32 rows that a
// tile of scales has, so that its scales leave as 128 (64) neighbouring bytes of each of its tiles. Measured, 16384 x 8192 bf16
// to NVFP4: row-major 50 us (one unit a thread: 52, four: 50); swizzled 52 us, MXFP4 49 (two units a thread: 55 / 49, one:
// 71 / 54; chunks of 8 units instead of 16: 51 / 49, of 32: 55 / 49); fp32 to NVFP4 88 us with two units, 89 with four.
constexpr int kQuantChunk = 16, kSwizzledThreads = 8 * kQuantChunk, kRowMajorUnits = 2;
template <int DT> constexpr int kSwizzledUnits = DT == DT_F32 ? 2 : 4;

template <int DT, bool NV> __global__ void __launch_bounds__(kQuantThreads) rmsq_quant_kernel(const QuantParams p)
{
    constexpr int PER = NV ? 1 : 2, U = kRowMajorUnits;                 // units per scale, per thread
    const long long first = static_cast<long long>(gridDim.x - 1 - blockIdx.x) * (U * kQuantThreads) + threadIdx.x;
    pdl_wait();
    Unit<DT> x[U];
#pragma unroll
    for (int i = 0; i < U; ++i) x[i].load(p.x, first + i * kQuantThreads, first + i * kQuantThreads < p.units);
    const float gs = NV && p.gs != nullptr ? __ldg(p.gs) : 1.0f, c = NV && DT == DT_BF16 ? bf16_side(gs) : 1.0f;
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const long long unit = first + i * kQuantThreads;
        uint2 codes;
        const uint32_t code = quantise16<DT, NV>(x[i], gs, c, codes);
        if (unit >= p.units) continue;
        st_v2(p.out + unit * 8, codes.x, codes.y);
        if (threadIdx.x % PER == 0) p.scale[unit / PER] = static_cast<unsigned char>(code);
    }
}

template <int DT, bool NV> __global__ void __launch_bounds__(kSwizzledThreads) rmsq_quant_swizzled_kernel(const QuantParams p)
{
    constexpr int PER = NV ? 1 : 2, SPAN = 4 * PER;                     // units per scale, per four scales
    constexpr int TILES = kQuantChunk / SPAN, U = kSwizzledUnits<DT>, NEXT = 2 * U;       // neighbouring rows of a group
    __shared__ uint32_t words[TILES * 8 * U];                           // [tile][row of a group][group]: a row's four scales
    const unsigned block = gridDim.x - 1 - blockIdx.x;
    const unsigned strip = block / static_cast<unsigned>(p.chunks), chunk = block - strip * static_cast<unsigned>(p.chunks);
    const int u = threadIdx.x % kQuantChunk, which = threadIdx.x / kQuantChunk;      // unit of the chunk; of 8 rows
    const long long row0 = static_cast<long long>(strip / (32 / NEXT)) * 128 + strip % (32 / NEXT) * NEXT;
    const long long row = row0 + (which >> 1) * 32 + (which & 1);
    const int in_row = static_cast<int>(chunk) * kQuantChunk + u;
    const long long unit = row * p.row_units + in_row;
    pdl_wait();
    Unit<DT> x[U];
#pragma unroll
    for (int i = 0; i < U; ++i) x[i].load(p.x, unit + 2 * i * p.row_units, row + 2 * i < p.rows && in_row < p.row_units);
    const float gs = NV && p.gs != nullptr ? __ldg(p.gs) : 1.0f, c = NV && DT == DT_BF16 ? bf16_side(gs) : 1.0f;
#pragma unroll
    for (int i = 0; i < U; ++i) {
        uint2 codes;
        uint32_t w = quantise16<DT, NV>(x[i], gs, c, codes) << (8 * (u / PER & 3));
        if (row + 2 * i < p.rows && in_row < p.row_units) st_v2(p.out + (unit + 2 * i * p.row_units) * 8, codes.x, codes.y);
        // the four scales of a tile's row come from neighbouring lanes
        w |= __shfl_xor_sync(0xFFFFFFFFu, w, PER);
        w |= __shfl_xor_sync(0xFFFFFFFFu, w, 2 * PER);
        if (u % SPAN == 0) words[(u / SPAN * NEXT + 2 * i + (which & 1)) * 4 + (which >> 1)] = w;
    }
    __syncthreads();
    if (threadIdx.x >= TILES * 8 * U) return;
    const int tile = threadIdx.x / (4 * NEXT), of = threadIdx.x / 4 % NEXT, group = threadIdx.x & 3;
    const long long r = row0 + group * 32 + of;
    const int scale = static_cast<int>(chunk) * (kQuantChunk / PER) + tile * 4, left = static_cast<int>(p.row_units) / PER - scale;
    if (r >= p.rows || left <= 0) return;
    unsigned char* const at = p.scale + (r / 128 * p.k_tiles + scale / 4) * 512 + r % 32 * 16 + group * 4;
    const uint32_t w = words[threadIdx.x];
    if (left >= 4) st_u32(at, w);
    else
        for (int i = 0; i < left; ++i) at[i] = static_cast<unsigned char>(w >> (8 * i));     // the padding stays
}

// The global scale, in two steps: the maxima of parts of the tensor, one per CTA, then their maximum. A tensor that one
// CTA reads in about the time of a launch takes one step.
struct AmaxParams {
    const void* x;
    long long vectors, count;        // whole vectors of 16 bytes, elements
    float* part;                     // or null: out is written
    float* out;
};

constexpr int kAmaxThreads = 512;

// The reciprocal's product, both rounded: the value that a number over a tensor has in PyTorch, and so in programs that form it
// there. (A step of the quotient's last place would decide other ties: 0.4 % of the codes where the maximum is 52.) It is off by 1.16
// units of the last place at most: half a unit, and the reciprocal's half times the ratio of their significands, 1.3125.
// Past 2^126 the reciprocal is a subnormal float and would cost up to 3.1; the quotient itself is taken there.
__device__ __forceinline__ float gs_of(float a)
{
    if (a > 8.507059173e37f) return __fdiv_rn(448.0f * 6.0f, a);
    return a == 0.f ? 1.0f : a != a ? a : fminf(__fmul_rn(448.0f * 6.0f, __frcp_rn(a)), 3.402823466e38f);
}

// Maximum over the CTA, in thread 0; NaN where one is.
__device__ __forceinline__ float cta_max_nan(float a)
{
    __shared__ float w[kAmaxThreads / 32];
    a = warp_max_nan(a);
    if ((threadIdx.x & 31) == 0) w[threadIdx.x >> 5] = a;
    __syncthreads();
    if (threadIdx.x < 32) a = warp_max_nan(threadIdx.x < kAmaxThreads / 32 ? w[threadIdx.x] : 0.f);
    return a;
}

template <int DT> __global__ void __launch_bounds__(kAmaxThreads) rmsq_amax_kernel(const AmaxParams p)
{
    constexpr int VW = Elem<DT>::EPV, U = 4;
    pdl_wait();
    float a = 0.f;
    const long long stride = static_cast<long long>(gridDim.x) * kAmaxThreads;
    const uint4* const x = static_cast<const uint4*>(p.x);
    for (long long i = static_cast<long long>(blockIdx.x) * kAmaxThreads + threadIdx.x; i < p.vectors; i += U * stride) {
        uint4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] = i + u * stride < p.vectors ? ld_v4(x + i + u * stride) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float2 f[VW / 2];
            Elem<DT>::pairs(v[u], f);
#pragma unroll
            for (int j = 0; j < VW / 2; ++j) a = max3_nan(a, fabsf(f[j].x), fabsf(f[j].y));
        }
    }
    if (blockIdx.x == 0 && threadIdx.x < p.count - p.vectors * VW) {
        const typename Scalar<DT>::T e = static_cast<const typename Scalar<DT>::T*>(p.x)[p.vectors * VW + threadIdx.x];
        a = max3_nan(a, fabsf(Scalar<DT>::get(e)), 0.f);
    }
    a = cta_max_nan(a);
    if (threadIdx.x == 0) {
        if (p.part != nullptr) p.part[blockIdx.x] = a;
        else *p.out = gs_of(a);
    }
}

static __global__ void __launch_bounds__(kAmaxThreads) rmsq_amax_join_kernel(const float* part, int parts, float* out)
{
    pdl_wait();
    float a = 0.f;
    for (int i = threadIdx.x; i < parts; i += kAmaxThreads) a = max3_nan(a, part[i], 0.f);
    a = cta_max_nan(a);
    if (threadIdx.x == 0) *out = gs_of(a);
}

static bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

static bool known_dtype(int dtype) { return dtype == RMSQ_BF16 || dtype == RMSQ_FP16 || dtype == RMSQ_F32; }

static rmsq_status status_of(cudaError_t e)
{
    if (e == cudaSuccess) return RMSQ_OK;
    cudaGetLastError();
    return RMSQ_ERR_LAUNCH;
}

template <int DT, bool NV> static const void* quant_fn(bool swizzled)
{
    return swizzled ? reinterpret_cast<const void*>(&rmsq_quant_swizzled_kernel<DT, NV>)
                    : reinterpret_cast<const void*>(&rmsq_quant_kernel<DT, NV>);
}
template <bool NV> static const void* quant_fn(int dtype, bool swizzled)
{
    return dtype == RMSQ_BF16   ? quant_fn<DT_BF16, NV>(swizzled)
           : dtype == RMSQ_FP16 ? quant_fn<DT_FP16, NV>(swizzled)
                                : quant_fn<DT_F32, NV>(swizzled);
}

static rmsq_status quantise(bool nv, const void* input, int64_t rows, int64_t hidden, int dtype, const float* global_scale,
                            void* output, void* block_scale, int scale_layout, void* stream)
{
    const int block = nv ? 16 : 32;
    if (!known_dtype(dtype)) return RMSQ_ERR_DTYPE;
    if (scale_layout != RMSQ_SCALE_ROW_MAJOR && scale_layout != RMSQ_SCALE_SWIZZLED_128x4) return RMSQ_ERR_DTYPE;
    if (rows < 0 || hidden < block || hidden % block != 0 || hidden > RMSQ_QUANT_MAX_HIDDEN || rows > RMSQ_QUANT_MAX_ROWS)
        return RMSQ_ERR_SHAPE;
    if (rows == 0) return RMSQ_OK;
    if (!input || !output || !block_scale) return RMSQ_ERR_NULL;
    if (!aligned16(input) || !aligned16(output) || !aligned16(block_scale) || reinterpret_cast<uintptr_t>(global_scale) % 4 != 0)
        return RMSQ_ERR_ALIGN;
    QuantParams p = {};
    p.x = input;
    p.gs = global_scale;
    p.out = static_cast<unsigned char*>(output);
    p.scale = static_cast<unsigned char*>(block_scale);
    const bool swizzled = scale_layout == RMSQ_SCALE_SWIZZLED_128x4;
    p.rows = rows;
    p.row_units = hidden / 16;
    p.units = rows * p.row_units;
    p.chunks = static_cast<int>((p.row_units + kQuantChunk - 1) / kQuantChunk);
    p.k_tiles = static_cast<int>((hidden / block + 3) / 4);
    const long long grid = swizzled ? (rows + 127) / 128 * (16 / (dtype == RMSQ_F32 ? kSwizzledUnits<DT_F32> : kSwizzledUnits<DT_BF16>)) * p.chunks
                                    : (p.units + kRowMajorUnits * kQuantThreads - 1) / (kRowMajorUnits * kQuantThreads);
    if (grid > INT32_MAX) return RMSQ_ERR_SHAPE;
    DeviceView dv;
    if (!device_view(&dv)) return RMSQ_ERR_DEVICE;
    void* args[] = {&p};
    return status_of(launch_kernel(nv ? quant_fn<true>(dtype, swizzled) : quant_fn<false>(dtype, swizzled), dim3(static_cast<unsigned>(grid)),
                                   swizzled ? kSwizzledThreads : kQuantThreads, 0, 1, static_cast<cudaStream_t>(stream), args));
}

}  // namespace rmsq

using namespace rmsq;

extern "C" rmsq_status quant_nvfp4(const void* input, int64_t rows, int64_t hidden, int dtype, const float* global_scale,
                                   void* output, void* block_scale, int scale_layout, void* stream)
{
    return quantise(true, input, rows, hidden, dtype, global_scale, output, block_scale, scale_layout, stream);
}

extern "C" rmsq_status quant_mxfp4(const void* input, int64_t rows, int64_t hidden, int dtype, void* output,
                                   void* block_scale, int scale_layout, void* stream)
{
    return quantise(false, input, rows, hidden, dtype, nullptr, output, block_scale, scale_layout, stream);
}

// Elements that one CTA takes alone.
constexpr int64_t kAmaxAlone = 65536;

extern "C" int64_t nvfp4_global_scale_workspace(int64_t count)
{
    return count > kAmaxAlone ? RMSQ_GLOBAL_SCALE_PARTS * static_cast<int64_t>(sizeof(float)) : 0;
}

extern "C" rmsq_status nvfp4_global_scale(const void* input, int64_t count, int dtype, float* gs_out, void* workspace,
                                          int64_t workspace_bytes, void* stream)
{
    if (!known_dtype(dtype)) return RMSQ_ERR_DTYPE;
    if (count < 0) return RMSQ_ERR_SHAPE;
    if (!gs_out) return RMSQ_ERR_NULL;
    if (reinterpret_cast<uintptr_t>(gs_out) % 4 != 0) return RMSQ_ERR_ALIGN;
    if (count > 0) {
        const int64_t need = nvfp4_global_scale_workspace(count);
        if (!input || (need > 0 && !workspace)) return RMSQ_ERR_NULL;
        if (!aligned16(input) || !aligned16(workspace)) return RMSQ_ERR_ALIGN;
        if (workspace_bytes < need) return RMSQ_ERR_SHAPE;
    }
    DeviceView dv;
    if (!device_view(&dv)) return RMSQ_ERR_DEVICE;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    AmaxParams p = {};
    p.x = input;
    p.count = count;
    p.out = gs_out;
    const int es = dtype == RMSQ_F32 ? 4 : 2;
    p.vectors = count / (16 / es);
    long long grid = 1;
    if (count > kAmaxAlone) {
        grid = (p.vectors + 4 * kAmaxThreads - 1) / (4 * kAmaxThreads);
        if (grid > 4LL * dv.sms) grid = 4LL * dv.sms;
        if (grid > RMSQ_GLOBAL_SCALE_PARTS) grid = RMSQ_GLOBAL_SCALE_PARTS;
        p.part = static_cast<float*>(workspace);
    }
    const void* fn = dtype == RMSQ_BF16   ? reinterpret_cast<const void*>(&rmsq_amax_kernel<DT_BF16>)
                     : dtype == RMSQ_FP16 ? reinterpret_cast<const void*>(&rmsq_amax_kernel<DT_FP16>)
                                          : reinterpret_cast<const void*>(&rmsq_amax_kernel<DT_F32>);
    void* args[] = {&p};
    const rmsq_status s = status_of(launch_kernel(fn, dim3(static_cast<unsigned>(grid)), kAmaxThreads, 0, 1, st, args));
    if (s != RMSQ_OK || p.part == nullptr) return s;
    const float* part = p.part;
    int parts = static_cast<int>(grid);
    void* join[] = {&part, &parts, &gs_out};
    return status_of(launch_kernel(reinterpret_cast<const void*>(&rmsq_amax_join_kernel), dim3(1), kAmaxThreads, 0, 1, st, join));
}
