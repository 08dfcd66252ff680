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
// Bound by HBM. A warp, a CTA or a cluster of CTAs owns a row (SCOPE_*); every row has its own
// thread group and no loop, so the hardware's CTA scheduler evens out SMs of unequal bandwidth.
// gamma and beta stay in L1.
#pragma once

#include "rmsq_device.cuh"

namespace rmsq {

enum { SCOPE_WARP = 0, SCOPE_CTA = 1, SCOPE_CLUSTER = 2 };
enum { NORM_LAYER = 0, NORM_LAYER_INT8 = 1, NORM_RMS_INT8 = 2 };

struct NormParams {
    const void* x;
    const void* res;       // or null
    void* res_out;         // or null
    const void* gamma;
    const void* beta;      // or null
    void* out;             // input's type, or int8 codes
    float* scale;          // int8: one per row
    float* mean;           // or null
    float* rstd;           // or null
    long long rows;
    int hidden;
    int slice;             // elements of a row per CTA (SCOPE_CLUSTER), else hidden
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

// fp32 values -> one 16-byte vector of the type.
template <int DT> __device__ __forceinline__ uint4 pack_vec(const float* f)
{
    if constexpr (DT == DT_F32) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                          __float_as_uint(f[3]));
    } else {
        return make_uint4(Scalar<DT>::put2(f[0], f[1]), Scalar<DT>::put2(f[2], f[3]),
                          Scalar<DT>::put2(f[4], f[5]), Scalar<DT>::put2(f[6], f[7]));
    }
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

// The thread's share of a slice of len elements, dealt to T threads. VEC: vector c of a thread is
// vector c * T + t of the slice (rows start on 16-byte boundaries); otherwise element j is element
// j * T + t, so that a warp's accesses are contiguous either way.
template <int DT, int E, bool VEC> struct Deal {
    static constexpr int VW = VEC ? Elem<DT>::EPV : 1;
    static constexpr int NC = E / VW;
    static __device__ __forceinline__ int col(int c, int t, int T) { return (c * T + t) * VW; }
    // how many of the slice's elements the 32 threads from t0 on hold
    static __device__ __forceinline__ int count(int t0, int T, int len)
    {
        int n = 0;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int left = len - (c * T + t0) * VW;
            n += left < 0 ? 0 : left < 32 * VW ? left : 32 * VW;
        }
        return n;
    }
};

// int8 codes of values already scaled to [-127, 127]: adding 1.5 * 2^23 rounds to nearest even
// and leaves the code in the low byte.
__device__ __forceinline__ uint32_t code_bits(float v) { return __float_as_uint(__fadd_rn(v, 12582912.0f)); }

__device__ __forceinline__ uint32_t pack_codes(float a, float b, float c, float d)
{
    const uint32_t lo = __byte_perm(code_bits(a), code_bits(b), 0x0040);
    const uint32_t hi = __byte_perm(code_bits(c), code_bits(d), 0x0040);
    return __byte_perm(lo, hi, 0x5410);
}

template <int DT, int E, bool VEC, int SCOPE, int KIND>
__global__ void __launch_bounds__(SCOPE == SCOPE_WARP ? 256 : 512)
rmsq_norm_kernel(const NormParams p)
{
    using D = Deal<DT, E, VEC>;
    using S = Scalar<DT>;
    constexpr bool RMS = KIND == NORM_RMS_INT8;
    constexpr bool INT8 = KIND != NORM_LAYER;
    constexpr int VW = D::VW, NC = D::NC;

    __shared__ float2 part[16];
    __shared__ float part_max[16];
    __shared__ float4 xch[2];

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int T = SCOPE == SCOPE_WARP ? 32 : blockDim.x;
    const int t = SCOPE == SCOPE_WARP ? lane : threadIdx.x;
    const int nwarps = blockDim.x >> 5;
    long long row;
    int c0 = 0, len = p.hidden;
    if constexpr (SCOPE == SCOPE_WARP) {
        row = static_cast<long long>(blockIdx.x) * nwarps + warp;
    } else if constexpr (SCOPE == SCOPE_CTA) {
        row = blockIdx.x;
    } else {
        row = cluster_id();
        c0 = static_cast<int>(cluster_rank()) * p.slice;
        len = p.hidden - c0;
        len = len < 0 ? 0 : len < p.slice ? len : p.slice;
    }
    pdl_wait();
    if (SCOPE == SCOPE_WARP && row >= p.rows) return;

    const long long base = row * p.hidden + c0;
    const typename S::T* const x = static_cast<const typename S::T*>(p.x) + base;
    float v[E];

    // ---- s into registers, fp32 (exact) ----
    if constexpr (VEC) {
        uint4 raw[NC];
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int k = D::col(c, t, T);
            raw[c] = k < len ? ld_stream_v4(reinterpret_cast<const uint4*>(x + k)) : make_uint4(0, 0, 0, 0);
        }
        if (p.res != nullptr) {
            const typename S::T* const r = static_cast<const typename S::T*>(p.res) + base;
            typename S::T* const ro = static_cast<typename S::T*>(p.res_out) + base;
            uint4 add[NC];
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const int k = D::col(c, t, T);
                add[c] = k < len ? ld_stream_v4(reinterpret_cast<const uint4*>(r + k)) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const int k = D::col(c, t, T);
                raw[c] = Elem<DT>::add(raw[c], add[c]);
                if (k < len) st_v4(ro + k, raw[c]);
            }
        }
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            float f[VW];
            Elem<DT>::unpack(raw[c], f);
#pragma unroll
            for (int j = 0; j < VW; ++j) v[c * VW + j] = f[j];
        }
    } else {
        typename S::T raw[E];
#pragma unroll
        for (int c = 0; c < E; ++c) {
            const int k = D::col(c, t, T);
            raw[c] = k < len ? x[k] : typename S::T(0);
        }
        if (p.res != nullptr) {
            const typename S::T* const r = static_cast<const typename S::T*>(p.res) + base;
            typename S::T* const ro = static_cast<typename S::T*>(p.res_out) + base;
            typename S::T add[E];
#pragma unroll
            for (int c = 0; c < E; ++c) {
                const int k = D::col(c, t, T);
                add[c] = k < len ? r[k] : typename S::T(0);
            }
#pragma unroll
            for (int c = 0; c < E; ++c) {
                const int k = D::col(c, t, T);
                raw[c] = S::add(raw[c], add[c]);
                if (k < len) ro[k] = raw[c];
            }
        }
#pragma unroll
        for (int c = 0; c < E; ++c) v[c] = S::get(raw[c]);
    }

    // ---- mean and squares about it ----
    float sum = 0.f, m2 = 0.f;
    const int n_w = D::count(SCOPE == SCOPE_WARP ? 0 : warp * 32, T, len);
    float mean = 0.f;
    if constexpr (!RMS) {
#pragma unroll
        for (int j = 0; j < E; ++j) sum += v[j];
        sum = warp_sum(sum);
        mean = n_w > 0 ? sum / static_cast<float>(n_w) : 0.f;
    }
    if (n_w == 32 * E) {
#pragma unroll
        for (int j = 0; j < E; ++j) {
            const float d = v[j] - mean;
            m2 = fmaf(d, d, m2);
        }
    } else {
#pragma unroll
        for (int c = 0; c < NC; ++c)
            if (D::col(c, t, T) < len) {
#pragma unroll
                for (int j = 0; j < VW; ++j) {
                    const float d = v[c * VW + j] - mean;
                    m2 = fmaf(d, d, m2);
                }
            }
    }
    m2 = warp_sum(m2);
    if constexpr (SCOPE != SCOPE_WARP) {
        if (lane == 0) part[warp] = make_float2(sum, m2);
        __syncthreads();
        const float2 q = lane < nwarps ? part[lane] : make_float2(0.f, 0.f);
        if constexpr (RMS) {
            m2 = warp_sum(q.y);
        } else {
            const float n_l = lane < nwarps ? static_cast<float>(D::count(lane * 32, T, len)) : 0.f;
            sum = warp_sum(q.x);
            mean = len > 0 ? sum / static_cast<float>(len) : 0.f;
            const float d = n_l > 0.f ? q.x / n_l - mean : 0.f;
            m2 = warp_sum(fmaf(n_l * d, d, q.y));
        }
    }
    if constexpr (SCOPE == SCOPE_CLUSTER) {
        if (threadIdx.x == 0) xch[0] = make_float4(sum, m2, static_cast<float>(len), 0.f);
        cluster_sync();
        const uint32_t nc = cluster_size();
        const float4 q = lane < static_cast<int>(nc) ? ld_cluster_f4(smem_u32(&xch[0]), lane)
                                                     : make_float4(0.f, 0.f, 0.f, 0.f);
        if constexpr (RMS) {
            m2 = warp_sum(q.y);
        } else {
            sum = warp_sum(q.x);
            mean = sum / static_cast<float>(p.hidden);
            const float d = q.z > 0.f ? q.x / q.z - mean : 0.f;
            m2 = warp_sum(fmaf(q.z * d, d, q.y));
        }
    }
    const float rstd = 1.0f / sqrtf(m2 / static_cast<float>(p.hidden) + p.eps);

    // ---- y ----
    const typename S::T* const gamma = static_cast<const typename S::T*>(p.gamma) + c0;
    const typename S::T* const beta = p.beta ? static_cast<const typename S::T*>(p.beta) + c0 : nullptr;
    float amax = 0.f;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int k = D::col(c, t, T);
        if (k < len) {
            float w[VW], b[VW];
            if constexpr (VEC) {
                Elem<DT>::unpack(ld_v4(gamma + k), w);
                if (beta) {
                    Elem<DT>::unpack(ld_v4(beta + k), b);
                } else {
#pragma unroll
                    for (int j = 0; j < VW; ++j) b[j] = 0.f;
                }
            } else {
                w[0] = S::get(gamma[k]);
                b[0] = beta ? S::get(beta[k]) : 0.f;
            }
#pragma unroll
            for (int j = 0; j < VW; ++j) {
                float& y = v[c * VW + j];
                y = fmaf((y - mean) * rstd, w[j] + p.offset, b[j]);
                if constexpr (INT8) amax = fmaxf(amax, fabsf(y));
            }
            if constexpr (!INT8) {
                typename S::T* const o = static_cast<typename S::T*>(p.out) + base;
                if constexpr (VEC) st_v4(o + k, pack_vec<DT>(&v[c * VW]));
                else o[k] = S::put(v[c]);
            }
        }
    }
    const bool leader = SCOPE == SCOPE_WARP ? lane == 0
                                            : threadIdx.x == 0 && (SCOPE == SCOPE_CTA || cluster_rank() == 0);
    if constexpr (INT8) {
        amax = warp_max(amax);
        if constexpr (SCOPE != SCOPE_WARP) {
            if (lane == 0) part_max[warp] = amax;
            __syncthreads();
            amax = warp_max(lane < nwarps ? part_max[lane] : 0.f);
        }
        if constexpr (SCOPE == SCOPE_CLUSTER) {
            if (threadIdx.x == 0) xch[1] = make_float4(amax, 0.f, 0.f, 0.f);
            cluster_sync();
            amax = warp_max(lane < static_cast<int>(cluster_size())
                                ? ld_cluster_f4(smem_u32(&xch[1]), lane).x : 0.f);
        }
        // 127 / amax overflows for rows of tiny y: those are scaled up by 2^100 first (exact).
        const float pre = amax < 1e-30f ? 0x1p100f : 1.0f;
        const float inv = amax > 0.f ? 127.0f / (amax * pre) : 0.f;
        signed char* const o = static_cast<signed char*>(p.out) + base;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int k = D::col(c, t, T);
            if (k < len) {
                float f[VW];
#pragma unroll
                for (int j = 0; j < VW; ++j) f[j] = v[c * VW + j] * pre * inv;
                if constexpr (VW == 8)
                    st_v2(o + k, pack_codes(f[0], f[1], f[2], f[3]), pack_codes(f[4], f[5], f[6], f[7]));
                else if constexpr (VW == 4)
                    st_u32(o + k, pack_codes(f[0], f[1], f[2], f[3]));
                else
                    o[k] = static_cast<signed char>(code_bits(f[0]) & 0xFFu);
            }
        }
        if (leader) p.scale[row] = amax / 127.0f;
    } else if (leader) {
        if (p.mean) p.mean[row] = mean;
        if (p.rstd) p.rstd[row] = rstd;
    }
    // a CTA's exchange slots are read by the others of its cluster: none leaves before all have
    if constexpr (SCOPE == SCOPE_CLUSTER) cluster_sync();
}

}  // namespace rmsq
