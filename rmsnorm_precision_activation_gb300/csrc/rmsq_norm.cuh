// rmsq_norm.cuh -- forward norms whose row stays in registers: layer norm in the input's type, and
// layer norm or RMS norm to int8 codes with one scale per row.
//
//   s    = RN_dtype(x + r)                          (s = x without a residual)
//   mean = sum s / H,  var = sum (s - mean)^2 / H   (RMS: mean = 0)
//   y    = (s - mean) / sqrt(var + eps) * (gamma + offset) + beta
//   int8: scale = max |y| / 127,  q = RN_even(y / scale)
//
// The row is read once into registers, so the variance is formed in a second pass over registers
// about the mean: no cancellation for rows far off centre. Warps do that about their own mean and
// the row's totals follow from (sum, squares about the own mean, count) of each warp,
//   M2 = sum_w M2_w + n_w (mean_w - mean)^2,
// which costs one block barrier instead of two.
//
// Bound by HBM. Two kernels:
//  - rmsq_norm_direct_kernel, rows of up to 16384 columns: straight into registers, each row by a warp or
//    CTA of its own.
//  - rmsq_norm_ring_kernel, wider rows: split over a cluster, whose CTAs would read gamma and beta anew with
//    every row. They take several rows, which come through a ring of shared-memory slots filled by bulk
//    copies, and keep gamma and beta in shared memory.
#pragma once

#include "rmsq_device.cuh"

namespace rmsq {

enum { SCOPE_WARP = 0, SCOPE_CTA = 1, SCOPE_CLUSTER = 2 };    // threads of a row group, or that a wait acquires from
enum { NORM_LAYER = 0, NORM_LAYER_INT8 = 1, NORM_RMS_INT8 = 2 };

// The rows a kernel reads through its rings.
struct RowTensors {
    const void* in[3];     // tensors [rows x hidden]
    long long total;       // bytes of one
    int ntens;
    int rows;
    int hidden;
    int slice;             // elements of a row per CTA
    int stages;            // ring slots per row group
    int slot;              // bytes of one tensor's row in a slot (multiple of 16)
};

struct NormParams {
    RowTensors r;          // x, and the residual where there is one
    void* res_out;         // or null
    const void* gamma;
    const void* beta;      // or null
    void* out;             // input's type, or int8 codes
    float* scale;          // int8: one per row
    float* mean;           // or null
    float* rstd;           // or null
    int T;                 // threads per row group
    float eps;
    float offset;
    unsigned int* err;
    unsigned long long timeout_ns;
};

// One element of a 16-bit or 32-bit type, by type code.
template <int DT> struct Scalar;
template <> struct Scalar<DT_BF16> {
    using T = uint16_t;
    static __device__ __forceinline__ float get(T v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }
    static __device__ __forceinline__ T put(float f)
    {
        T h;
        asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(h) : "f"(f));
        return h;
    }
    static __device__ __forceinline__ uint32_t put2(float lo, float hi)
    {
        uint32_t r;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
        return r;
    }
    static __device__ __forceinline__ T add(T a, T b)
    {
        T r;
        asm("add.rn.bf16 %0, %1, %2;" : "=h"(r) : "h"(a), "h"(b));
        return r;
    }
};
template <> struct Scalar<DT_FP16> {
    using T = uint16_t;
    static __device__ __forceinline__ float get(T v)
    {
        float f;
        asm("cvt.f32.f16 %0, %1;" : "=f"(f) : "h"(v));
        return f;
    }
    static __device__ __forceinline__ T put(float f)
    {
        T h;
        asm("cvt.rn.f16.f32 %0, %1;" : "=h"(h) : "f"(f));
        return h;
    }
    static __device__ __forceinline__ uint32_t put2(float lo, float hi)
    {
        uint32_t r;
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
        return r;
    }
    static __device__ __forceinline__ T add(T a, T b)
    {
        T r;
        asm("add.rn.f16 %0, %1, %2;" : "=h"(r) : "h"(a), "h"(b));
        return r;
    }
};
template <> struct Scalar<DT_F32> {
    using T = float;
    static __device__ __forceinline__ float get(T v) { return v; }
    static __device__ __forceinline__ T put(float f) { return f; }
    static __device__ __forceinline__ T add(T a, T b) { return __fadd_rn(a, b); }
};

// fp32 pairs -> one 16-byte vector of the type.
template <int DT> __device__ __forceinline__ uint4 pack_pairs(const float2* f)
{
    if constexpr (DT == DT_F32)
        return make_uint4(__float_as_uint(f[0].x), __float_as_uint(f[0].y), __float_as_uint(f[1].x), __float_as_uint(f[1].y));
    else
        return make_uint4(Scalar<DT>::put2(f[0].x, f[0].y), Scalar<DT>::put2(f[1].x, f[1].y),
                          Scalar<DT>::put2(f[2].x, f[2].y), Scalar<DT>::put2(f[3].x, f[3].y));
}

__device__ __forceinline__ uint4 ld_v4(const void* p)
{
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

// Maxima that are NaN where one of their operands is.
__device__ __forceinline__ float max3_nan(float a, float b, float c)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float warp_max_nan(float v)
{
    float r;
    asm volatile("redux.sync.max.abs.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

__device__ __forceinline__ void pdl_wait()
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
}

// mbar_wait_bounded for kernels whose warps wait much of the time. The thread is suspended for up to
// 10 us at a time, so waiting warps do not crowd the shared-memory pipe that the working ones need
// (measured in the tensor-core product: polling made every ready wait take 350 cycles), and the
// timer, which takes about a microsecond to read, is only read by waits that last. SCOPE_CLUSTER
// also acquires what the cluster's other CTAs wrote before they arrived.
template <int SCOPE> __device__ __forceinline__ bool mbar_try_wait_long(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    if constexpr (SCOPE == SCOPE_CLUSTER)
        asm volatile(
            "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok) : "r"(bar), "r"(parity), "r"(10000u) : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok) : "r"(bar), "r"(parity), "r"(10000u) : "memory");
    return ok != 0;
}

// Whether the phase is over, without waiting: asked one step ahead, its latency (about 150 cycles,
// which a wait for a finished phase costs too) passes behind other work.
template <int SCOPE> __device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    if constexpr (SCOPE == SCOPE_CLUSTER)
        asm volatile(
            "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0;
}

// A timeout as mbar_wait takes it: 32 bits of nanoseconds (registers are scarce where it waits).
__device__ __forceinline__ uint32_t wait_limit(unsigned long long timeout_ns)
{
    return timeout_ns < 4000000000ull ? static_cast<uint32_t>(timeout_ns) : 4000000000u;
}

__device__ __forceinline__ uint32_t globaltimer_lo()
{
    uint32_t t;
    asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
    return t;
}

template <int SCOPE> __device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, uint32_t limit_ns)
{
    if (mbar_test<SCOPE>(bar, parity)) return true;
    if (mbar_try_wait_long<SCOPE>(bar, parity)) return true;
    const uint32_t t0 = globaltimer_lo();
#pragma unroll 1
    do {
        if (mbar_try_wait_long<SCOPE>(bar, parity)) return true;
    } while (globaltimer_lo() - t0 <= limit_ns);
    return false;
}

// A row in vectors of 16 bytes, dealt to T threads: vector c of a thread is vector c * T + t, so that a
// warp's accesses are contiguous. Rows whose width is no whole number of vectors start `shift` elements
// behind a 16-byte boundary; such a row is taken from that boundary on ("columns"), and its elements are
// columns shift to shift + hidden. All accesses but those of its first and last vector are then whole
// vectors, as in other rows.
template <int DT, int E> struct Deal {
    static constexpr int VW = Elem<DT>::EPV, NC = E / VW, PV = VW / 2;
    static __device__ __forceinline__ int col(int c, int t, int T) { return (c * T + t) * VW; }
    // how many of the columns lo to hi the 32 threads from t0 on hold
    static __device__ __forceinline__ int count(int t0, int T, int lo, int hi)
    {
        int n = 0;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int first = (c * T + t0) * VW;
            n += max(0, min(hi, first + 32 * VW) - max(lo, first));
        }
        return n;
    }
};

// Which of a thread's vectors have columns lo to hi at all, and which of those also have others. EDGE: bits,
// the same for all rows of one shift, so that testing one is all a row costs.
template <int DT, int E, bool FULL, bool EDGE> struct Part {
    uint32_t some = 0, cut = 0;
    int hi;
    __device__ __forceinline__ Part(int t, int T, int lo, int hi_) : hi(hi_)
    {
        using D = Deal<DT, E>;
        if (EDGE) {
#pragma unroll
            for (int c = 0; c < D::NC; ++c) {
                const int k = D::col(c, t, T);
                if (k < hi) some |= 1u << c;
                if (k < hi && (k < lo || k + D::VW > hi)) cut |= 1u << c;
            }
        }
    }
    __device__ __forceinline__ bool in(int c, int k) const { return FULL || (EDGE ? (some >> c & 1u) != 0 : k < hi); }
    __device__ __forceinline__ bool whole(int c) const { return !EDGE || !(cut >> c & 1u); }
};

// Zeros in place of a vector's columns outside lo to hi.
template <int PV> __device__ __forceinline__ void clear_outside(float2 (&f)[PV], int k, int lo, int hi)
{
#pragma unroll
    for (int j = 0; j < PV; ++j) {
        if (k + 2 * j < lo || k + 2 * j >= hi) f[j].x = 0.f;
        if (k + 2 * j + 1 < lo || k + 2 * j + 1 >= hi) f[j].y = 0.f;
    }
}

// A vector's columns lo to hi to p + k, element by element.
template <int DT> __device__ __forceinline__ void store_inside(typename Scalar<DT>::T* p, const uint4& v, int k, int lo, int hi)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < Elem<DT>::EPV; ++j)
        if (k + j >= lo && k + j < hi) {
            if constexpr (DT == DT_F32) p[k + j] = __uint_as_float(w[j]);
            else p[k + j] = static_cast<uint16_t>(j & 1 ? w[j / 2] >> 16 : w[j / 2] & 0xFFFFu);
        }
}

// Two 16-bit elements of a word, exact.
template <int DT> __device__ __forceinline__ float2 unpack2(uint32_t w)
{
    if constexpr (DT == DT_BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    else return make_float2(Scalar<DT>::get(static_cast<uint16_t>(w & 0xFFFFu)), Scalar<DT>::get(static_cast<uint16_t>(w >> 16)));
}

// A thread's share of gamma over all rows, as raw 32-bit words (two 16-bit elements each).
template <int DT, int E, bool EDGE> struct Held {
    using D = Deal<DT, E>;
    using T = typename Scalar<DT>::T;
    static constexpr int PER = 4 / sizeof(T), N = E / PER;
    uint32_t w[N];

    // Column k is p[k - lo] in columns lo to hi, 0 elsewhere.
    __device__ __forceinline__ void load(const T* p, int t, int threads, int lo, int hi)
    {
#pragma unroll
        for (int c = 0; c < D::NC; ++c) {
            const int k = D::col(c, t, threads);
            if constexpr (!EDGE) {
                const uint4 v = k < hi ? ld_v4(p + k) : make_uint4(0, 0, 0, 0);
                w[4 * c] = v.x;
                w[4 * c + 1] = v.y;
                w[4 * c + 2] = v.z;
                w[4 * c + 3] = v.w;
            } else {
#pragma unroll
                for (int j = 0; j < D::VW; j += PER) {
                    uint32_t v = 0;
#pragma unroll
                    for (int q = 0; q < PER; ++q)
                        if (k + j + q >= lo && k + j + q < hi) {
                            if constexpr (PER == 1) v = __float_as_uint(p[k + j - lo]);
                            else v |= static_cast<uint32_t>(p[k + j + q - lo]) << (16 * q);
                        }
                    w[(c * D::VW + j) / PER] = v;
                }
            }
        }
    }
    // Keeps the compiler from holding the words unpacked across rows, which the registers do not allow.
    __device__ __forceinline__ void pin()
    {
#pragma unroll
        for (int i = 0; i < N; ++i) asm volatile("" : "+r"(w[i]));
    }
    __device__ __forceinline__ float2 pair(int i) const          // elements 2 i and 2 i + 1
    {
        if constexpr (PER == 1) return make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
        else return unpack2<DT>(w[i]);
    }
};

// A thread's share of a row, columns lo to hi, as int8 codes of y * 127 / amax. 127 / amax overflows for
// rows of tiny y: those are scaled up by 2^100 first (exact). amax is NaN for a row with a NaN, and so is
// the scale; the codes are then any.
template <int DT, int E, bool FULL, bool EDGE>
__device__ __forceinline__ void store_codes(float2 (&v)[E / 2], float amax, signed char* o, int t, int T, int lo, int hi)
{
    using D = Deal<DT, E>;
    constexpr int PV = D::PV, VW = D::VW;
    const float pre = amax < 1e-30f ? 0x1p100f : 1.0f;
    const float2 inv = splat(amax > 0.f ? __fdiv_rn(127.0f, amax * pre) : 0.f);
    if (pre != 1.0f) {
#pragma unroll
        for (int j = 0; j < E / 2; ++j) v[j] = mul2(v[j], splat(pre));
    }
    // adding 1.5 * 2^23 rounds to nearest even and leaves the code in the low byte
    const float2 magic = splat(12582912.0f);
#pragma unroll
    for (int c = 0; c < D::NC; ++c) {
        const int k = D::col(c, t, T);
        if (FULL || k < hi) {
            uint32_t h[PV];
#pragma unroll
            for (int j = 0; j < PV; ++j) {
                const float2 q = add2(mul2(v[c * PV + j], inv), magic);
                h[j] = __byte_perm(__float_as_uint(q.x), __float_as_uint(q.y), 0x0040);
            }
            if (!EDGE || (k >= lo && k + VW <= hi)) {
                if constexpr (PV == 4) st_v2(o + k, __byte_perm(h[0], h[1], 0x5410), __byte_perm(h[2], h[3], 0x5410));
                else st_u32(o + k, __byte_perm(h[0], h[1], 0x5410));
            } else {
#pragma unroll
                for (int j = 0; j < VW; ++j)
                    if (k + j >= lo && k + j < hi) o[k + j] = static_cast<signed char>(h[j / 2] >> (8 * (j & 1)) & 0xFFu);
            }
        }
    }
}

// ------------------------------------------------------------------------------------------
// Rows straight into registers
// ------------------------------------------------------------------------------------------

// The vector at column k of a tensor's row, which starts at element at (the row's columns lo to hi);
// what is not the row's is not cleared. The last vector can reach past the tensor's `total` elements.
template <int DT, bool EDGE>
__device__ __forceinline__ uint4 load_columns(const typename Scalar<DT>::T* p, long long at, long long total, int k, int hi)
{
    if (!EDGE || at + k + Elem<DT>::EPV <= total) return ld_stream_v4(reinterpret_cast<const uint4*>(p + at + k));
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < Elem<DT>::EPV; ++j)
        if (k + j < hi) {
            if constexpr (DT == DT_F32) w[j] = __float_as_uint(p[at + k + j]);
            else w[j / 2] |= static_cast<uint32_t>(p[at + k + j]) << (16 * (j & 1));
        }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// gamma's or beta's elements for the vector at column k of a row with the given shift: elements k - shift
// on, taken out of the two aligned vectors they lie in (shift is the same for the whole row, so its
// branches are uniform). Elements outside 0 to hidden are any value.
template <int DT, bool EDGE>
__device__ __forceinline__ uint4 load_param(const typename Scalar<DT>::T* p, int k, int shift, int hidden)
{
    constexpr int VW = Elem<DT>::EPV;
    if constexpr (!EDGE) {
        return ld_v4(p + k);
    } else {
        uint32_t w[9];
        w[8] = 0;
        const uint4 lower = shift > 0 && k >= VW ? ld_v4(p + k - VW) : make_uint4(0, 0, 0, 0);
        w[0] = lower.x;
        w[1] = lower.y;
        w[2] = lower.z;
        w[3] = lower.w;
        if (k + VW <= hidden) {
            const uint4 upper = ld_v4(p + k);
            w[4] = upper.x;
            w[5] = upper.y;
            w[6] = upper.z;
            w[7] = upper.w;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) w[4 + j] = 0;
#pragma unroll
            for (int j = 0; j < VW; ++j)
                if (k + j < hidden) {
                    if constexpr (DT == DT_F32) w[4 + j] = __float_as_uint(p[k + j]);
                    else w[4 + j / 2] |= static_cast<uint32_t>(p[k + j]) << (16 * (j & 1));
                }
        }
        // the vector starts (VW - shift) elements into lower, upper: words first, then half a word
        const int words = DT == DT_F32 ? 4 - shift : 4 - (shift + 1) / 2;
        uint32_t v[5];
        switch (words) {
        case 0:
#pragma unroll
            for (int j = 0; j < 5; ++j) v[j] = w[j];
            break;
        case 1:
#pragma unroll
            for (int j = 0; j < 5; ++j) v[j] = w[j + 1];
            break;
        case 2:
#pragma unroll
            for (int j = 0; j < 5; ++j) v[j] = w[j + 2];
            break;
        case 3:
#pragma unroll
            for (int j = 0; j < 5; ++j) v[j] = w[j + 3];
            break;
        default:
#pragma unroll
            for (int j = 0; j < 5; ++j) v[j] = w[j + 4];
        }
        if (DT != DT_F32 && (shift & 1)) {
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = __funnelshift_r(v[j], v[j + 1], 16);
        }
        return make_uint4(v[0], v[1], v[2], v[3]);
    }
}

// A warp (SCOPE_WARP, rows of up to 1024 columns) or a CTA (up to 16384, 32 elements a thread) per row.
// FULL: the threads' shares cover the row exactly, so nothing is checked. EDGE: rows whose width is no
// whole number of vectors.
// Every row has its own thread group and no loop: the hardware's CTA scheduler overlaps rows and evens
// out SMs of unequal bandwidth. Bound by HBM with a residual and by instructions without one: 32
// elements a thread halve what a row costs in reductions against 16.
template <int DT, int E, bool FULL, bool EDGE, int SCOPE, int KIND>
__global__ void __launch_bounds__(SCOPE == SCOPE_WARP ? 256 : 512, SCOPE == SCOPE_WARP ? 4 : 2) rmsq_norm_direct_kernel(const __grid_constant__ NormParams p)
{
    using D = Deal<DT, E>;
    using S = Scalar<DT>;
    using TT = typename S::T;
    constexpr bool RMS = KIND == NORM_RMS_INT8;
    constexpr bool INT8 = KIND != NORM_LAYER;
    constexpr int NC = D::NC, PV = D::PV, VW = D::VW;
    __shared__ float2 part[16];
    __shared__ float part_max[16];

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int T = SCOPE == SCOPE_WARP ? 32 : blockDim.x;
    const int t = SCOPE == SCOPE_WARP ? lane : threadIdx.x;
    const int nwarps = SCOPE == SCOPE_WARP ? 1 : blockDim.x >> 5;
    const int row = SCOPE == SCOPE_WARP ? static_cast<int>(blockIdx.x) * (blockDim.x >> 5) + warp : blockIdx.x;
    pdl_wait();
    if (SCOPE == SCOPE_WARP && row >= p.r.rows) return;

    const int shift = EDGE ? static_cast<int>(static_cast<long long>(row) * p.r.hidden % VW) : 0;
    const int lo = shift, hi = shift + p.r.hidden;
    const long long at = static_cast<long long>(row) * p.r.hidden - shift;      // of column 0
    const long long total = static_cast<long long>(p.r.rows) * p.r.hidden;
    const auto in = [&](int c) { return FULL || D::col(c, t, T) < hi; };
    const auto whole = [&](int k) { return !EDGE || (k >= lo && k + VW <= hi); };

    // ---- s into registers, fp32 (exact), 0 outside the row ----
    float2 v[E / 2];
    {
        const uint4 zero = make_uint4(0, 0, 0, 0);
        uint4 raw[NC];
#pragma unroll
        for (int c = 0; c < NC; ++c)
            raw[c] = in(c) ? load_columns<DT, EDGE>(static_cast<const TT*>(p.r.in[0]), at, total, D::col(c, t, T), hi) : zero;
        if (p.r.ntens == 2) {
            TT* const ro = static_cast<TT*>(p.res_out) + at;
            uint4 add[NC];
#pragma unroll
            for (int c = 0; c < NC; ++c)
                add[c] = in(c) ? load_columns<DT, EDGE>(static_cast<const TT*>(p.r.in[1]), at, total, D::col(c, t, T), hi) : zero;
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const int k = D::col(c, t, T);
                raw[c] = Elem<DT>::add(raw[c], add[c]);
                if (in(c)) {
                    if (whole(k)) st_v4(ro + k, raw[c]);
                    else store_inside<DT>(ro, raw[c], k, lo, hi);
                }
            }
        }
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            float2 f[PV];
            Elem<DT>::pairs(raw[c], f);
            if (!whole(D::col(c, t, T))) clear_outside(f, D::col(c, t, T), lo, hi);
#pragma unroll
            for (int j = 0; j < PV; ++j) v[c * PV + j] = f[j];
        }
    }

    // ---- mean and squares about it ----
    const int n_w = FULL ? 32 * E : D::count(SCOPE == SCOPE_WARP ? 0 : warp * 32, T, lo, hi);
    float sum = 0.f, m2, mean = 0.f;
    if constexpr (!RMS) {
        float2 a = v[0];
#pragma unroll
        for (int j = 1; j < E / 2; ++j) a = add2(a, v[j]);
        sum = warp_sum(a.x + a.y);
        mean = FULL ? sum * (1.0f / (32 * E)) : n_w > 0 ? __fdividef(sum, static_cast<float>(n_w)) : 0.f;
    }
    {
        const float2 m = splat(-mean);
        float2 a = make_float2(0.f, 0.f);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            if (in(c)) {
                float2 d[PV];
#pragma unroll
                for (int j = 0; j < PV; ++j) d[j] = add2(v[c * PV + j], m);
                if (!whole(D::col(c, t, T))) clear_outside(d, D::col(c, t, T), lo, hi);
#pragma unroll
                for (int j = 0; j < PV; ++j) a = fma2(d[j], d[j], a);
            }
        }
        m2 = warp_sum(a.x + a.y);
    }
    const float inv_h = __frcp_rn(static_cast<float>(p.r.hidden));
    if constexpr (SCOPE != SCOPE_WARP) {
        if (lane == 0) part[warp] = make_float2(sum, m2);
        __syncthreads();
        const float2 q = lane < nwarps ? part[lane] : make_float2(0.f, 0.f);
        float d = 0.f, n_l = 0.f;
        if constexpr (!RMS) {
            mean = warp_sum(q.x) * inv_h;
            if (lane < nwarps) {
                n_l = FULL ? static_cast<float>(32 * E) : static_cast<float>(D::count(lane * 32, T, lo, hi));
                d = FULL ? q.x * (1.0f / (32 * E)) - mean : n_l > 0.f ? __fdividef(q.x, n_l) - mean : 0.f;
            }
        }
        m2 = warp_sum(fmaf(n_l * d, d, q.y));
    }
    const float rstd = __frsqrt_rn(fmaf(m2, inv_h, p.eps));

    // ---- y ----
    const float2 m = splat(-mean), r2 = splat(rstd), offset = splat(p.offset);
    const TT* const gamma = static_cast<const TT*>(p.gamma);
    const TT* const beta = static_cast<const TT*>(p.beta);
    float amax = 0.f;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        if (in(c)) {
            const int k = D::col(c, t, T);
            float2 w[PV], b[PV];
            Elem<DT>::pairs(load_param<DT, EDGE>(gamma, k, shift, p.r.hidden), w);
            if (p.offset != 0.f) {
#pragma unroll
                for (int j = 0; j < PV; ++j) w[j] = add2(w[j], offset);
            }
            if (!RMS && beta != nullptr) {
                Elem<DT>::pairs(load_param<DT, EDGE>(beta, k, shift, p.r.hidden), b);
            } else {
#pragma unroll
                for (int j = 0; j < PV; ++j) b[j] = make_float2(0.f, 0.f);
            }
            float2 y[PV];
#pragma unroll
            for (int j = 0; j < PV; ++j) {
                if constexpr (RMS) y[j] = mul2(mul2(v[c * PV + j], r2), w[j]);
                else y[j] = fma2(mul2(add2(v[c * PV + j], m), r2), w[j], b[j]);
            }
            if constexpr (INT8) {
                if (!whole(k)) clear_outside(y, k, lo, hi);
#pragma unroll
                for (int j = 0; j < PV; ++j) {
                    amax = max3_nan(amax, fabsf(y[j].x), fabsf(y[j].y));
                    v[c * PV + j] = y[j];
                }
            } else {
                TT* const o = static_cast<TT*>(p.out) + at;
                const uint4 raw = pack_pairs<DT>(y);
                if (whole(k)) st_v4(o + k, raw);
                else store_inside<DT>(o, raw, k, lo, hi);
            }
        }
    }
    const bool leader = t == 0;
    if constexpr (INT8) {
        amax = warp_max_nan(amax);
        if constexpr (SCOPE != SCOPE_WARP) {
            if (lane == 0) part_max[warp] = amax;
            __syncthreads();
            amax = warp_max_nan(lane < nwarps ? part_max[lane] : 0.f);
        }
        store_codes<DT, E, FULL, EDGE>(v, amax, static_cast<signed char*>(p.out) + at, t, T, lo, hi);
        if (leader) p.scale[row] = amax / 127.0f;
    } else if (leader) {
        if (p.mean) p.mean[row] = mean;
        if (p.rstd) p.rstd[row] = rstd;
    }
}

// ------------------------------------------------------------------------------------------
// Rows through shared memory
// ------------------------------------------------------------------------------------------

constexpr int kRingStages = 8;      // slots per group at most
constexpr int kRingGroups = 16;     // row groups per CTA at most
// The rows a group works on: `first`, and every `stride`-th from there. Group g of cluster c starts at
// row g * clusters + c; the host makes the number of clusters a multiple of the rows after which the shift
// repeats (or gives every group one row at most), so a CTA's rows have one shift.
struct Rows {
    int first, stride, n;
    __device__ __forceinline__ Rows(int group, int groups, int rows)
    {
        const int clusters = static_cast<int>(cluster_count());
        first = group * clusters + static_cast<int>(cluster_id());
        stride = clusters * groups;
        n = first < rows ? (rows - first + stride - 1) / stride : 0;
    }
};

constexpr int kRingBars = 2 * kRingStages * kRingGroups * 8;      // bytes of barriers

// A row group's ring of slots: its next rows, brought by bulk copies while the group works. EDGE: rows of
// a width that is no whole number of vectors, taken from the 16-byte boundary below. The group's rows all
// have the same shift (Rows).
template <int DT, bool EDGE> struct RowRing {
    using T = typename Scalar<DT>::T;
    static constexpr int ES = sizeof(T), VW = Elem<DT>::EPV;
    const RowTensors& r;
    int c0;                        // the CTA's first column
    int lo, hi;                    // its columns that are the row's, from c0 on
    int shift;                     // of the rows
    uint32_t bars, base;           // shared addresses of the group's barriers (kRingStages full, as many
                                   // empty) and slots
    __device__ __forceinline__ uint32_t full(int stage) const { return bars + 8 * stage; }
    __device__ __forceinline__ uint32_t empty(int stage) const { return bars + 8 * (kRingStages + stage); }

    __device__ __forceinline__ uint32_t at(uint32_t stage, int i) const { return base + (stage * r.ntens + i) * r.slot; }
    // Where the CTA's first column of a row is in a tensor, in elements (whole vectors).
    __device__ __forceinline__ long long origin(int row) const { return static_cast<long long>(row) * r.hidden - shift + c0; }

    // One row's pieces of every tensor into a slot (one thread).
    __device__ __forceinline__ void fetch(int row, uint32_t stage, uint64_t policy) const
    {
        const long long a0 = origin(row) * ES;
        long long a1 = a0 + (hi + VW - 1) / VW * 16;
        if (EDGE && a1 > (r.total & ~15LL)) a1 = r.total & ~15LL;
        const uint32_t bytes = hi > lo && a1 > a0 ? static_cast<uint32_t>(a1 - a0) : 0u;
        if (EDGE && hi > lo) {
            // the tensors' last bytes, which no whole piece covers, by hand (before the arrival below)
            const long long end = origin(row) + hi;
            for (long long e = a1 / ES; e < end; ++e)
                for (int i = 0; i < r.ntens; ++i) {
                    const uint32_t to = at(stage, i) + static_cast<uint32_t>(e * ES - a0);
                    const T v = static_cast<const T*>(r.in[i])[e];
                    if constexpr (ES == 2) asm volatile("st.shared.u16 [%0], %1;" ::"r"(to), "h"(v) : "memory");
                    else asm volatile("st.shared.f32 [%0], %1;" ::"r"(to), "f"(v) : "memory");
                }
        }
        mbar_arrive_expect_tx(full(stage), bytes * r.ntens);
        if (bytes > 0)
            for (int i = 0; i < r.ntens; ++i)
                bulk_load(at(stage, i), static_cast<const unsigned char*>(r.in[i]) + a0, bytes, full(stage), policy);
    }

    // The vector at column k of tensor i, as raw bits; what is not the row's is not cleared.
    __device__ __forceinline__ uint4 vec(uint32_t stage, int i, int k) const { return ld_shared_v4(at(stage, i) + k * ES); }

    // One thread sets the barriers up: a slot is empty when `warps` warps have left it.
    __device__ __forceinline__ void init(int warps) const
    {
        for (int i = 0; i < r.stages; ++i) {
            mbar_init(full(i), 1);
            mbar_init(empty(i), warps);
        }
    }

    // Brings the group's rows (one thread of the CTA's copying warp: issuing a row's copies takes about
    // 1000 cycles, which a working warp would keep its group waiting for). After a wait that ran out,
    // waits (bounded) for the copies in flight, so that they end before the CTA does.
    __device__ __forceinline__ void feed(const Rows& rows, unsigned long long timeout_ns, unsigned int* err) const
    {
        const uint64_t policy = l2_evict_normal_policy();
        const uint32_t limit = wait_limit(timeout_ns);
        int stage = 0, phase = 1, i = 0;
        for (; i < rows.n; ++i) {
            if (!mbar_wait<SCOPE_CTA>(empty(stage), phase, limit)) break;
            fence_proxy_async_smem();
            fetch(rows.first + i * rows.stride, stage, policy);
            if (++stage == r.stages) {
                stage = 0;
                phase ^= 1;
            }
        }
        if (i < rows.n) {
            bool drained = true;
            for (int j = i > r.stages ? i - r.stages : 0; j < i; ++j)
                drained &= mbar_wait<SCOPE_CTA>(full(j % r.stages), (j / r.stages) & 1, wait_limit(4 * timeout_ns));
            atomicOr(err, drained ? ERRF_WAIT_TIMEOUT : ERRF_WAIT_TIMEOUT | ERRF_DRAIN_TIMEOUT);
        }
    }
};

// The threads of a row group (T a multiple of 32).
__device__ __forceinline__ void group_sync(int group, int T)
{
    if (T == 32) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(T) : "memory");
}

// A row's sums among the CTAs of a cluster: each writes its own into a slot of every CTA, which counts
// the bytes on its own barrier. Two sets in turn: a CTA sends a row's sums after it has read those of
// the row before, so nobody writes a set that is still read. No cluster barrier, which the copying
// warp would have to join; every wait is bounded.
struct ClusterSums {
    uint32_t bars, slots;          // shared addresses: 2 barriers, [2][16] float4
    int nc, rank;
    static constexpr int BYTES = 16 + 2 * 16 * 16;

    __device__ __forceinline__ void init() const
    {
        mbar_init(bars, 1);
        mbar_init(bars + 8, 1);
    }
    // By the lanes of one warp.
    __device__ __forceinline__ void send(int lane, int flip, float4 v) const
    {
        const uint32_t bar = bars + 8 * flip, slot = slots + (flip * 16 + rank) * 16;
        if (lane == 0) mbar_arrive_expect_tx(bar, nc * 16);
        if (lane < nc)
            asm volatile(
                "{\n\t.reg .b32 a, b;\n\tmapa.shared::cluster.u32 a, %0, %2;\n\tmapa.shared::cluster.u32 b, %1, %2;\n\t"
                "st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [a], {%3, %4, %5, %6}, [b];\n\t}"
                ::"r"(slot), "r"(bar), "r"(lane), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w) : "memory");
    }
    // Lane r of every warp gets rank r's (zeros past the cluster); false: the wait ran out.
    __device__ __forceinline__ bool receive(int lane, int flip, int phase, uint32_t limit_ns, float4& v) const
    {
        const bool ok = mbar_wait<SCOPE_CLUSTER>(bars + 8 * flip, phase, limit_ns);
        v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (lane < nc) {
            const uint4 w = ld_shared_v4(slots + (flip * 16 + lane) * 16);
            v = make_float4(__uint_as_float(w.x), __uint_as_float(w.y), __uint_as_float(w.z), __uint_as_float(w.w));
        }
        return ok;
    }
};

constexpr int kRingSlice = 16384;             // bytes of a tensor's row per CTA at most
constexpr int kRingWorkers = 256;             // threads that work on rows; a warp more copies

// Shared memory before gamma, beta and the ring: barriers, the groups' warp sums and maxima (each for
// two rows in turn: one barrier a row then keeps a row's from the next but one's), the cluster's sums.
constexpr int kNormHead = (kRingBars + 2 * 8 * 8 + 2 * 8 * 4 + 2 * ClusterSums::BYTES + 127) / 128 * 128;

template <int DT, int E, bool EDGE, bool FULL, int KIND>
__global__ void __launch_bounds__(kRingWorkers + 32, 3) rmsq_norm_ring_kernel(const __grid_constant__ NormParams p)
{
    using D = Deal<DT, E>;
    using S = Scalar<DT>;
    using TT = typename S::T;
    constexpr bool RMS = KIND == NORM_RMS_INT8;
    constexpr bool INT8 = KIND != NORM_LAYER;
    constexpr int VW = D::VW, NC = D::NC, PV = D::PV;
    extern __shared__ __align__(128) unsigned char smem[];

    float2* const part = reinterpret_cast<float2*>(smem + kRingBars);
    float* const part_max = reinterpret_cast<float*>(part + 16);
    unsigned char* const cluster_part = reinterpret_cast<unsigned char*>(part_max + 16);

    const int T = p.T, thread = threadIdx.x;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = T >> 5;
    const int nc = static_cast<int>(cluster_size()), rank = static_cast<int>(cluster_rank());

    const bool copies = threadIdx.x >= T;
    const Rows rows(0, 1, p.r.rows);
    const int c0 = rank * p.r.slice;
    const int shift = EDGE ? static_cast<int>(static_cast<long long>(rows.first) * p.r.hidden % VW) : 0;
    const int lo = max(shift - c0, 0), hi = FULL ? p.r.slice : max(min(shift + p.r.hidden - c0, p.r.slice), 0);
    const RowRing<DT, EDGE> ring{p.r, c0, lo, hi, shift, smem_u32(smem),
                                 smem_u32(smem + kNormHead) + 2 * p.r.slot};
    const ClusterSums sums{smem_u32(cluster_part), smem_u32(cluster_part + 16), nc, rank};
    const ClusterSums maxima{sums.bars + ClusterSums::BYTES, sums.slots + ClusterSums::BYTES, nc, rank};

    const bool has_res = p.r.ntens == 2;
    if (copies && lane == 0) {
        ring.init(warps);
        sums.init();
        maxima.init();
        fence_mbar_init();
        fence_proxy_async_smem();
    }
    __syncthreads();
    cluster_sync();                               // the other CTAs' barriers are set up
    pdl_wait();
    if (copies) {
        if (lane == 0) ring.feed(rows, p.timeout_ns, p.err);
        return;
    }

    // gamma and beta of the slice stay in shared memory, in their own type
    TT* const ws = reinterpret_cast<TT*>(smem + kNormHead);
    TT* const bs = reinterpret_cast<TT*>(smem + kNormHead + p.r.slot);
    const TT* const gamma = static_cast<const TT*>(p.gamma) + (c0 - shift);
    const TT* const beta = p.beta != nullptr ? static_cast<const TT*>(p.beta) + (c0 - shift) : nullptr;
    if constexpr (!EDGE) {
        const uint4 zero = make_uint4(0, 0, 0, 0);
        for (int k = threadIdx.x * VW; k < hi; k += T * VW) {
            st_shared_v4(smem_u32(ws + k), ld_v4(gamma + k));
            st_shared_v4(smem_u32(bs + k), beta != nullptr ? ld_v4(beta + k) : zero);
        }
    } else {
#pragma unroll 4
        for (int k = lo + threadIdx.x; k < hi; k += T) {
            const TT w = gamma[k], b = beta != nullptr ? beta[k] : TT(0);
            ws[k] = w;
            bs[k] = b;
        }
    }
    asm volatile("bar.sync 15, %0;" ::"r"(T) : "memory");

    // Counts of elements and their reciprocals: this warp's, lane's warp's of the group, the CTA's, lane's
    // CTA's of the cluster. A count that is not a power of two makes a mean off by half a step more.
    const uint32_t limit = wait_limit(p.timeout_ns);
    const auto inverse = [](int k) { return k > 0 ? 1.0f / static_cast<float>(k) : 0.f; };
    const Part<DT, E, FULL, EDGE> mine(thread, T, lo, hi);
    const int n_w = FULL ? 32 * E : D::count(warp * 32, T, lo, hi);
    const int n_l = lane >= warps ? 0 : FULL ? 32 * E : D::count(lane * 32, T, lo, hi);
    const int n_r = lane < nc
                        ? max(min(shift + p.r.hidden - lane * p.r.slice, p.r.slice), 0) - (lane == 0 ? shift : 0) : 0;
    const float inv_w = inverse(n_w), inv_l = inverse(n_l), inv_c = inverse(hi - lo), inv_r = inverse(n_r);
    const float inv_h = 1.0f / static_cast<float>(p.r.hidden), f_l = static_cast<float>(n_l), f_r = static_cast<float>(n_r);
    bool dead = false;                            // a wait ran out: finish without waiting again
    int stage = 0, phase = 0;
    int flip = 0;
    for (int i = 0; i < rows.n; ++i) {
        // made opaque to the compiler again and again, which would keep every element's address and test
        // in registers from row to row and from phase to phase
        int t = thread;
        asm volatile("" : "+r"(t));
        const int row = rows.first + i * rows.stride;
        if (!dead && !mbar_wait<SCOPE_CTA>(ring.full(stage), phase, limit)) dead = true;
        const long long at = ring.origin(row);

        // ---- s into registers, fp32 (exact), 0 outside the slice ----
        float2 v[E / 2];
        {
            TT* const ro = static_cast<TT*>(p.res_out) + at;
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const int k = D::col(c, t, T);
                uint4 raw = make_uint4(0, 0, 0, 0);
                if (mine.in(c, k)) {
                    raw = ring.vec(stage, 0, k);
                    if (has_res) {
                        raw = Elem<DT>::add(raw, ring.vec(stage, 1, k));
                        if (mine.whole(c)) st_v4(ro + k, raw);
                        else store_inside<DT>(ro, raw, k, lo, hi);
                    }
                }
                float2 f[PV];
                Elem<DT>::pairs(raw, f);
                if (!mine.whole(c)) clear_outside(f, k, lo, hi);
#pragma unroll
                for (int j = 0; j < PV; ++j) v[c * PV + j] = f[j];
            }
        }

        // ---- mean and squares about it ----
        asm volatile("" : "+r"(t));
        float sum = 0.f, m2, mean = 0.f;
        if constexpr (!RMS) {
            float2 a = v[0];
#pragma unroll
            for (int j = 1; j < E / 2; ++j) a = add2(a, v[j]);
            sum = warp_sum(a.x + a.y);
            mean = sum * inv_w;
        }
        {
            const float2 m = splat(-mean);
            float2 a = make_float2(0.f, 0.f);
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const int k = D::col(c, t, T);
                if (mine.in(c, k)) {
                    float2 d[PV];
#pragma unroll
                    for (int j = 0; j < PV; ++j) d[j] = add2(v[c * PV + j], m);
                    if (!mine.whole(c)) clear_outside(d, k, lo, hi);
#pragma unroll
                    for (int j = 0; j < PV; ++j) a = fma2(d[j], d[j], a);
                }
            }
            m2 = warp_sum(a.x + a.y);
        }
        if (lane == 0) mbar_arrive(ring.empty(stage));       // the warp has read the slot
        if (lane == 0) part[flip * 8 + warp] = make_float2(sum, m2);
        group_sync(0, T);
        {
            const float2 q = lane < warps ? part[flip * 8 + lane] : make_float2(0.f, 0.f);
            float d = 0.f;
            if constexpr (!RMS) {
                sum = warp_sum(q.x);
                mean = sum * inv_c;
                d = f_l > 0.f ? q.x * inv_l - mean : 0.f;
            }
            m2 = warp_sum(fmaf(f_l * d, d, q.y));
        }
        {
            float4 q;
            if (warp == 0) sums.send(lane, flip, make_float4(sum, m2, 0.f, 0.f));
            if (!sums.receive(lane, flip, (i >> 1) & 1, dead ? 0 : limit, q)) dead = true;
            float d = 0.f;
            if constexpr (!RMS) {
                mean = warp_sum(q.x) * inv_h;
                d = f_r > 0.f ? q.x * inv_r - mean : 0.f;
            }
            m2 = warp_sum(fmaf(f_r * d, d, q.y));
        }
        const float rstd = __frsqrt_rn(m2 * inv_h + p.eps);

        // ---- y ----
        asm volatile("" : "+r"(t));
        const float2 m = splat(-mean), r2 = splat(rstd);
        float amax = 0.f;
        TT* const o = static_cast<TT*>(p.out) + at;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int k = D::col(c, t, T);
            if (mine.in(c, k)) {
                float2 w[PV], b[PV];
                Elem<DT>::pairs(ld_shared_v4(smem_u32(ws + k)), w);
                Elem<DT>::pairs(ld_shared_v4(smem_u32(bs + k)), b);
                if (p.offset != 0.f) {
#pragma unroll
                    for (int j = 0; j < PV; ++j) w[j] = add2(w[j], splat(p.offset));
                }
                float2 y[PV];
#pragma unroll
                for (int j = 0; j < PV; ++j) {
                    if constexpr (RMS) y[j] = mul2(mul2(v[c * PV + j], r2), w[j]);
                    else y[j] = fma2(mul2(add2(v[c * PV + j], m), r2), w[j], b[j]);
                }
                if constexpr (INT8) {
                    if (!mine.whole(c)) clear_outside(y, k, lo, hi);
#pragma unroll
                    for (int j = 0; j < PV; ++j) {
                        amax = max3_nan(amax, fabsf(y[j].x), fabsf(y[j].y));
                        v[c * PV + j] = y[j];
                    }
                } else {
                    const uint4 raw = pack_pairs<DT>(y);
                    if (mine.whole(c)) st_v4(o + k, raw);
                    else store_inside<DT>(o, raw, k, lo, hi);
                }
            }
        }
        const bool leader = t == 0 && rank == 0;
        if constexpr (INT8) {
            amax = warp_max_nan(amax);
            if (lane == 0) part_max[flip * 8 + warp] = amax;
            group_sync(0, T);
            amax = warp_max_nan(lane < warps ? part_max[flip * 8 + lane] : 0.f);
            float4 q;
            if (warp == 0) maxima.send(lane, flip, make_float4(amax, 0.f, 0.f, 0.f));
            if (!maxima.receive(lane, flip, (i >> 1) & 1, dead ? 0 : limit, q)) dead = true;
            amax = warp_max_nan(q.x);
            asm volatile("" : "+r"(t));
            signed char* const codes = static_cast<signed char*>(p.out) + at;
            store_codes<DT, E, FULL, EDGE>(v, amax, codes, t, T, lo, hi);
            if (leader) p.scale[row] = amax / 127.0f;
        } else if (leader) {
            if (p.mean) p.mean[row] = mean;
            if (p.rstd) p.rstd[row] = rstd;
        }
        flip ^= 1;
        if (++stage == p.r.stages) {
            stage = 0;
            phase ^= 1u;
        }
    }
    if (dead && lane == 0) atomicOr(p.err, ERRF_WAIT_TIMEOUT);
    cluster_sync();                               // nobody sends to a CTA that has left
}

}  // namespace rmsq
