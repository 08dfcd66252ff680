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
// The kernel is rmsq_norm_kernel; this header also has what the other kernels of these operators share.
#pragma once

#include "rmsq_device.cuh"
#include "rmsq_param.h"

namespace rmsq {

enum { SCOPE_WARP = 0, SCOPE_CTA = 1, SCOPE_CLUSTER = 2 };    // threads of a row group, or that a wait acquires from
enum { NORM_LAYER = 0, NORM_LAYER_INT8 = 1, NORM_RMS_INT8 = 2 };

struct NormParams {
    const void* x;
    const void* residual;  // or null
    void* res_out;         // or null
    const void* gamma;
    const void* beta;      // or null
    void* out;             // input's type, or int8 codes
    float* scale;          // int8: one per row
    float* mean;           // or null
    float* rstd;           // or null
    int rows;
    int hidden;
    int slice;             // columns of a row per CTA of a cluster
    float eps;
    float offset;
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
};
template <> struct Scalar<DT_F32> {
    using T = float;
    static __device__ __forceinline__ float get(T v) { return v; }
    static __device__ __forceinline__ T put(float f) { return f; }
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

// The kernels before this one on the stream are done and their writes visible.
__device__ __forceinline__ void pdl_wait_alone() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// The same, and the next kernel's CTAs may come as soon as every CTA has got here. A CTA that allocates
// TMEM does so first: a CTA of the next kernel could take the columns and then wait for this kernel.
__device__ __forceinline__ void pdl_wait()
{
    pdl_wait_alone();
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

// Time in units of 1024 ns, as bounds are given (rmsq_ops_plan.h).
__device__ __forceinline__ uint32_t time_units()
{
    unsigned long long t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return static_cast<uint32_t>(t >> 10);
}

template <int SCOPE> __device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, uint32_t limit)
{
    if (mbar_test<SCOPE>(bar, parity)) return true;
    if (mbar_try_wait_long<SCOPE>(bar, parity)) return true;
    const uint32_t t0 = time_units();
#pragma unroll 1
    do {
        if (mbar_try_wait_long<SCOPE>(bar, parity)) return true;
    } while (time_units() - t0 <= limit);
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

// int8 codes of a row: y * 127 / amax to the nearest, even at ties. 127 / amax overflows for rows of tiny
// y: those are scaled up by 2^100 first (exact). amax is NaN for a row with a NaN, and so is the scale;
// the codes are then any.
struct Coder {
    float pre, inv;
    __device__ __forceinline__ explicit Coder(float amax)
    {
        pre = amax < 1e-30f ? 0x1p100f : 1.0f;
        inv = amax > 0.f ? __fdiv_rn(127.0f, amax * pre) : 0.f;
    }
    // A vector of y at column k, of which the row has columns lo to hi. EDGE: perhaps not the whole of it.
    template <bool EDGE, int PV>
    __device__ __forceinline__ void store(float2 (&y)[PV], signed char* o, int k, int lo, int hi) const
    {
        constexpr int VW = 2 * PV;
        if (pre != 1.0f) {
#pragma unroll
            for (int j = 0; j < PV; ++j) y[j] = mul2(y[j], splat(pre));
        }
        // adding 1.5 * 2^23 rounds to nearest even and leaves the code in the low byte
        uint32_t h[PV];
#pragma unroll
        for (int j = 0; j < PV; ++j) {
            const float2 q = add2(mul2(y[j], splat(inv)), splat(12582912.0f));
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
};

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

// A parameter in device memory, as param_words reads it.
template <int DT> struct ParamReader {
    const typename Scalar<DT>::T* p;
    __device__ __forceinline__ void vector(int k, uint32_t* w) const
    {
        const uint4 v = ld_v4(p + k);
        w[0] = v.x;
        w[1] = v.y;
        w[2] = v.z;
        w[3] = v.w;
    }
    __device__ __forceinline__ uint32_t element(int k) const
    {
        if constexpr (DT == DT_F32) return __float_as_uint(p[k]);
        else return p[k];
    }
};

// gamma's or beta's elements for the vector at column k of a row with the given shift (param_words).
template <int DT, bool EDGE>
__device__ __forceinline__ uint4 load_param(const typename Scalar<DT>::T* p, int k, int shift, int hidden)
{
    if constexpr (!EDGE) {
        return ld_v4(p + k);
    } else {
        uint32_t v[4];
        param_words<Elem<DT>::EPV>(ParamReader<DT>{p}, k, shift, hidden, v);
        return make_uint4(v[0], v[1], v[2], v[3]);
    }
}

// One CTA's v to slot `rank` of every CTA of the cluster (lanes of warp 0), and everybody's read back:
// lane r of every warp gets rank r's, 0 past the cluster.
__device__ __forceinline__ float2 cluster_exchange(float2* slots, int warp, int lane, int nc, int rank, float2 v)
{
    if (warp == 0 && lane < nc)
        asm volatile(
            "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, %1;\n\tst.shared::cluster.v2.f32 [a], {%2, %3};\n\t}"
            ::"r"(smem_u32(slots + rank)), "r"(lane), "f"(v.x), "f"(v.y) : "memory");
    cluster_arrive_as(warp == 0);
    cluster_wait();
    return lane < nc ? slots[lane] : make_float2(0.f, 0.f);
}

// A warp, a CTA or a cluster per row, with E elements a thread: as fp32, or, 64 of 16 bits, packed as they
// were read and unpacked for each use. FULL: the threads' shares cover the row (a CTA's slice of it)
// exactly, so nothing is checked. EDGE: rows whose width is no whole number of vectors.
// Every row has its own thread group and no loop: the hardware's CTA scheduler overlaps rows and evens
// out SMs of unequal bandwidth (CTAs that walk rows through rings in shared memory: 2048 x 65536 fp16 128
// us against 107, 4096 x 20000 bf16 89 against 58, 512 x 20000 with residual 26 against 21). Bound by HBM
// with a residual (16384 x 8192 bf16 155 us, 1.02 of the copy rate of 6787 GB/s), by instructions without
// one (85.6 us, 0.92; to int8 87.6, 0.68); rows off 16-byte boundaries by instructions (8192 x 5121 bf16
// 54.6 us, 0.45: their parameters are shifted into place and their accesses checked, twice the instructions;
// staging the shifted parameters in shared memory for several rows took 58).
// The launch bounds leave 64 registers, which not every form fits. What each thread stores and reloads,
// in bytes: fp32 to 44 (fp32 rows of no whole vectors 100 to 164); to int8 fp32 16 to 96 (96 to 228, a warp
// per row the most), packed 72 to 140, 16-bit rows of no whole vectors up to 100; other forms under 40 or
// none. Wide rows to int8 lose most by it (2048 x 65536 158 us, 0.38).
template <int DT, int E, bool FULL, bool EDGE, int SCOPE, int KIND>
__global__ void __launch_bounds__(SCOPE == SCOPE_WARP ? 256 : 512, SCOPE == SCOPE_WARP ? 4 : 2) rmsq_norm_kernel(const __grid_constant__ NormParams p)
{
    using D = Deal<DT, E>;
    using S = Scalar<DT>;
    using TT = typename S::T;
    constexpr bool RMS = KIND == NORM_RMS_INT8;
    constexpr bool INT8 = KIND != NORM_LAYER;
    constexpr int NC = D::NC, PV = D::PV, VW = D::VW;
    __shared__ float4 part[16];                     // sum, squares, elements
    __shared__ float part_max[16];
    __shared__ float2 cluster_part[2][16];          // sums, maxima

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int T = SCOPE == SCOPE_WARP ? 32 : blockDim.x;
    const int t = SCOPE == SCOPE_WARP ? lane : threadIdx.x;
    const int nwarps = SCOPE == SCOPE_WARP ? 1 : blockDim.x >> 5;
    const int nc = SCOPE == SCOPE_CLUSTER ? static_cast<int>(cluster_size()) : 1;
    const int rank = SCOPE == SCOPE_CLUSTER ? static_cast<int>(cluster_rank()) : 0;
    const int row = SCOPE == SCOPE_WARP ? static_cast<int>(blockIdx.x) * (blockDim.x >> 5) + warp
                  : SCOPE == SCOPE_CTA  ? blockIdx.x : static_cast<int>(cluster_id());
    if (SCOPE == SCOPE_CLUSTER) cluster_arrive_as(false);
    pdl_wait();
    if (SCOPE == SCOPE_WARP && row >= p.rows) return;

    const int shift = EDGE ? static_cast<int>(static_cast<long long>(row) * p.hidden % VW) : 0;
    const int c0 = SCOPE == SCOPE_CLUSTER ? rank * p.slice : 0;               // the CTA's first column
    const int lo = SCOPE == SCOPE_CLUSTER ? max(shift - c0, 0) : shift;
    const int hi = SCOPE == SCOPE_CLUSTER ? max(min(shift + p.hidden - c0, p.slice), 0) : shift + p.hidden;
    const long long at = static_cast<long long>(row) * p.hidden - shift + c0; // of the CTA's first column
    const long long total = static_cast<long long>(p.rows) * p.hidden;
    const auto in = [&](int c) { return FULL || D::col(c, t, T) < hi; };
    const auto whole = [&](int k) { return !EDGE || (k >= lo && k + VW <= hi); };

    // ---- s into registers, exact, 0 outside the row: as fp32, or packed ----
    constexpr bool PACKED = E > 32;
    constexpr int BATCH = NC < 4 || DT == DT_F32 ? NC : 4;          // vectors in flight with a residual's
    float2 v[PACKED ? 1 : E / 2];
    uint4 raw[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c)
        raw[c] = in(c) ? load_columns<DT, EDGE>(static_cast<const TT*>(p.x), at, total, D::col(c, t, T), hi)
                       : make_uint4(0, 0, 0, 0);
    if (p.residual != nullptr) {
        TT* const ro = static_cast<TT*>(p.res_out) + at;
#pragma unroll
        for (int c0 = 0; c0 < NC; c0 += BATCH) {
            uint4 add[BATCH];
#pragma unroll
            for (int c = 0; c < BATCH; ++c)
                add[c] = in(c0 + c) ? load_columns<DT, EDGE>(static_cast<const TT*>(p.residual), at, total,
                                                             D::col(c0 + c, t, T), hi)
                                    : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int c = c0; c < c0 + BATCH; ++c) {
                const int k = D::col(c, t, T);
                raw[c] = Elem<DT>::add(raw[c], add[c - c0]);
                if (in(c)) {
                    if (whole(k)) st_v4(ro + k, raw[c]);
                    else store_inside<DT>(ro, raw[c], k, lo, hi);
                }
            }
        }
    }
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        float2 f[PV];
        Elem<DT>::pairs(raw[c], f);
        if (!whole(D::col(c, t, T))) {
            clear_outside(f, D::col(c, t, T), lo, hi);
            if constexpr (PACKED) raw[c] = pack_pairs<DT>(f);
        }
        if constexpr (!PACKED) {
#pragma unroll
            for (int j = 0; j < PV; ++j) v[c * PV + j] = f[j];
        }
    }
    // Keeps the compiler from holding packed vectors unpacked from one use to the next, which the registers
    // do not allow: 200 bytes of spills without it, none to 28 with it (to int8 up to 140: the comment at the
    // kernel). It takes a zero that the compiler does not know.
    const uint32_t zero = static_cast<uint32_t>(p.hidden >> 31);
    auto pin = [&]() {
        if constexpr (PACKED) {
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                raw[c].x ^= zero;
                raw[c].y ^= zero;
                raw[c].z ^= zero;
                raw[c].w ^= zero;
                asm volatile("" : "+r"(raw[c].x), "+r"(raw[c].y), "+r"(raw[c].z), "+r"(raw[c].w));
            }
        }
    };
    // vector c
    auto held = [&](int c, float2 (&f)[PV]) {
        if constexpr (PACKED) {
            Elem<DT>::pairs(raw[c], f);
        } else {
#pragma unroll
            for (int j = 0; j < PV; ++j) f[j] = v[c * PV + j];
        }
    };

    // ---- mean and squares about it ----
    const int n_w = FULL ? 32 * E : D::count(SCOPE == SCOPE_WARP ? 0 : warp * 32, T, lo, hi);
    float sum = 0.f, m2, mean = 0.f;
    if constexpr (!RMS) {
        float2 a = make_float2(0.f, 0.f);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            float2 f[PV];
            held(c, f);
#pragma unroll
            for (int j = 0; j < PV; ++j) a = add2(a, f[j]);
        }
        sum = warp_sum(a.x + a.y);
        mean = FULL ? sum * (1.0f / (32 * E)) : n_w > 0 ? __fdividef(sum, static_cast<float>(n_w)) : 0.f;
    }
    pin();
    {
        const float2 m = splat(-mean);
        float2 a = make_float2(0.f, 0.f);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            if (in(c)) {
                float2 d[PV];
                held(c, d);
#pragma unroll
                for (int j = 0; j < PV; ++j) d[j] = add2(d[j], m);
                if (!whole(D::col(c, t, T))) clear_outside(d, D::col(c, t, T), lo, hi);
#pragma unroll
                for (int j = 0; j < PV; ++j) a = fma2(d[j], d[j], a);
            }
        }
        m2 = warp_sum(a.x + a.y);
    }
    const float inv_h = __frcp_rn(static_cast<float>(p.hidden));
    if constexpr (SCOPE != SCOPE_WARP) {
        if (lane == 0) part[warp] = make_float4(sum, m2, static_cast<float>(n_w), 0.f);
        __syncthreads();
        const float4 q = lane < nwarps ? part[lane] : make_float4(0.f, 0.f, 0.f, 0.f);
        const float n_l = FULL ? (lane < nwarps ? static_cast<float>(32 * E) : 0.f) : q.z;
        float d = 0.f;
        if constexpr (!RMS) {
            sum = warp_sum(q.x);
            mean = sum * (SCOPE == SCOPE_CTA ? inv_h : hi > lo ? 1.0f / static_cast<float>(hi - lo) : 0.f);
            if (lane < nwarps) d = FULL ? q.x * (1.0f / (32 * E)) - mean : n_l > 0.f ? __fdividef(q.x, n_l) - mean : 0.f;
        }
        m2 = warp_sum(fmaf(n_l * d, d, q.y));
    }
    if constexpr (SCOPE == SCOPE_CLUSTER) {
        cluster_wait();                               // the other CTAs have started
        const float2 q = cluster_exchange(cluster_part[0], warp, lane, nc, rank, make_float2(sum, m2));
        float d = 0.f, n_r = 0.f;
        if constexpr (!RMS) {
            mean = warp_sum(q.x) * inv_h;
            if (lane < nc) {
                n_r = static_cast<float>(max(min(shift + p.hidden - lane * p.slice, p.slice), 0) - (lane == 0 ? shift : 0));
                d = n_r > 0.f ? __fdividef(q.x, n_r) - mean : 0.f;
            }
        }
        m2 = warp_sum(fmaf(n_r * d, d, q.y));
    }
    const float rstd = __frsqrt_rn(fmaf(m2, inv_h, p.eps));

    // ---- y ----
    pin();
    const float2 m = splat(-mean), r2 = splat(rstd), offset = splat(p.offset);
    const TT* const gamma = static_cast<const TT*>(p.gamma);
    const TT* const beta = static_cast<const TT*>(p.beta);
    auto norm = [&](int c, int k, float2 (&y)[PV]) {
        float2 w[PV], b[PV];
        Elem<DT>::pairs(load_param<DT, EDGE>(gamma, c0 + k, shift, p.hidden), w);
        if (p.offset != 0.f) {
#pragma unroll
            for (int j = 0; j < PV; ++j) w[j] = add2(w[j], offset);
        }
        if (!RMS && beta != nullptr) {
            Elem<DT>::pairs(load_param<DT, EDGE>(beta, c0 + k, shift, p.hidden), b);
        } else {
#pragma unroll
            for (int j = 0; j < PV; ++j) b[j] = make_float2(0.f, 0.f);
        }
        held(c, y);
#pragma unroll
        for (int j = 0; j < PV; ++j) {
            if constexpr (RMS) y[j] = mul2(mul2(y[j], r2), w[j]);
            else y[j] = fma2(mul2(add2(y[j], m), r2), w[j], b[j]);
        }
    };
    const bool leader = t == 0 && rank == 0;
    if constexpr (!INT8) {
        TT* const o = static_cast<TT*>(p.out) + at;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int k = D::col(c, t, T);
            if (in(c)) {
                float2 y[PV];
                norm(c, k, y);
                const uint4 v4 = pack_pairs<DT>(y);
                if (whole(k)) st_v4(o + k, v4);
                else store_inside<DT>(o, v4, k, lo, hi);
            }
        }
        if (leader) {
            if (p.mean) p.mean[row] = mean;
            if (p.rstd) p.rstd[row] = rstd;
        }
    } else {
        // packed rows form y twice, for want of registers
        float amax = 0.f;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int k = D::col(c, t, T);
            if (in(c)) {
                float2 y[PV];
                norm(c, k, y);
                if (!whole(k)) clear_outside(y, k, lo, hi);
#pragma unroll
                for (int j = 0; j < PV; ++j) {
                    amax = max3_nan(amax, fabsf(y[j].x), fabsf(y[j].y));
                    if constexpr (!PACKED) v[c * PV + j] = y[j];
                }
                if constexpr (PACKED) asm volatile("" : "+f"(amax));      // before the next vectors' loads
            }
        }
        amax = warp_max_nan(amax);
        if constexpr (SCOPE != SCOPE_WARP) {
            if (lane == 0) part_max[warp] = amax;
            __syncthreads();
            amax = warp_max_nan(lane < nwarps ? part_max[lane] : 0.f);
        }
        if constexpr (SCOPE == SCOPE_CLUSTER)
            amax = warp_max_nan(cluster_exchange(cluster_part[1], warp, lane, nc, rank, make_float2(amax, 0.f)).x);
        const Coder coder(amax);
        pin();
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int k = D::col(c, t, T);
            if (in(c)) {
                float2 y[PV];
                if constexpr (PACKED) norm(c, k, y);
                else held(c, y);
                coder.store<EDGE>(y, static_cast<signed char*>(p.out) + at, k, lo, hi);
            }
        }
        if (leader) p.scale[row] = amax / 127.0f;
    }
}

}  // namespace rmsq
