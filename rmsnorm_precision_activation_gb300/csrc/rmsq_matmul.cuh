// rmsq_matmul.cuh -- product of int8 codes with a scale per token and per output channel.
//
//   out[m][n] = RN((sum_k a[m][k] w[n][k]) * a_scale[m] * w_scale[n] + bias[n])
//
// The integer sums are exact in every kernel.
#pragma once

#include "rmsq_norm.cuh"

namespace rmsq {

struct MatmulParams {
    const signed char* a;      // [m x k] codes of the tokens
    const float* a_scale;      // [m]
    const signed char* w;      // [n x k] codes of the weight, a row per output channel
    const float* w_scale;      // [n]
    const void* bias;          // [n] of the output's type, or null
    void* out;                 // [m x n]
    unsigned int* err;
    long long m, n;
    int k;
    int dt;                    // output's type
    int ksplit;                // few-token kernel: warps that share a channel's sum
    unsigned long long timeout_ns;
};

__device__ __forceinline__ float load_as(const void* p, long long i, int dt)
{
    if (dt == DT_F32) return static_cast<const float*>(p)[i];
    const uint16_t v = static_cast<const uint16_t*>(p)[i];
    return dt == DT_BF16 ? Scalar<DT_BF16>::get(v) : Scalar<DT_FP16>::get(v);
}

__device__ __forceinline__ void store_as(void* p, long long i, int dt, float v)
{
    if (dt == DT_F32) static_cast<float*>(p)[i] = v;
    else static_cast<uint16_t*>(p)[i] = dt == DT_BF16 ? Scalar<DT_BF16>::put(v) : Scalar<DT_FP16>::put(v);
}

// A sum to the output's fp32 value: one rounding each, in the same order in every kernel.
__device__ __forceinline__ float scaled(int sum, float a_scale, float w_scale, float bias, bool has_bias)
{
    const float v = __fmul_rn(__fmul_rn(__int2float_rn(sum), a_scale), w_scale);
    return has_bias ? __fadd_rn(v, bias) : v;
}

__device__ __forceinline__ int dot16(const uint4& a, const uint4& b, int acc)
{
    acc = __dp4a(static_cast<int>(a.x), static_cast<int>(b.x), acc);
    acc = __dp4a(static_cast<int>(a.y), static_cast<int>(b.y), acc);
    acc = __dp4a(static_cast<int>(a.z), static_cast<int>(b.z), acc);
    return __dp4a(static_cast<int>(a.w), static_cast<int>(b.w), acc);
}

// Few tokens: bound by the weight's bytes. A warp takes kFewRows channels and MT tokens and walks
// k in 512-byte pieces, 16 bytes per lane; ksplit warps of the CTA share a channel's k where there
// are too few channels to fill the SMs. Sums by dp4a (four products per instruction, exact).
constexpr int kFewRows = 4;
constexpr int kFewWarps = 8;

template <int MT>
__global__ void __launch_bounds__(kFewWarps * 32) rmsq_matmul_few_kernel(const MatmulParams p)
{
    __shared__ int part[kFewWarps][kFewRows * MT];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int piece = warp % p.ksplit;
    const long long n0 = (static_cast<long long>(blockIdx.x) * (kFewWarps / p.ksplit) + warp / p.ksplit) * kFewRows;
    const long long m0 = static_cast<long long>(blockIdx.y) * MT;
    pdl_wait();

    int acc[kFewRows][MT];
#pragma unroll
    for (int r = 0; r < kFewRows; ++r)
#pragma unroll
        for (int i = 0; i < MT; ++i) acc[r][i] = 0;

    if (n0 < p.n) {
#pragma unroll 2
        for (int c = (piece * 32 + lane) * 16; c < p.k; c += p.ksplit * 512) {
            uint4 w[kFewRows];
#pragma unroll
            for (int r = 0; r < kFewRows; ++r) {
                const long long n = n0 + r < p.n ? n0 + r : p.n - 1;
                w[r] = ld_stream_v4(reinterpret_cast<const uint4*>(p.w + n * p.k + c));
            }
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const long long m = m0 + i < p.m ? m0 + i : p.m - 1;
                const uint4 a = ld_v4(p.a + m * p.k + c);
#pragma unroll
                for (int r = 0; r < kFewRows; ++r) acc[r][i] = dot16(w[r], a, acc[r][i]);
            }
        }
    }
#pragma unroll
    for (int r = 0; r < kFewRows; ++r)
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const int s = __reduce_add_sync(0xFFFFFFFFu, acc[r][i]);
            if (lane == 0) part[warp][r * MT + i] = s;
        }
    __syncthreads();
    for (int e = threadIdx.x; e < kFewWarps / p.ksplit * kFewRows * MT; e += kFewWarps * 32) {
        const int row = e / MT, i = e % MT;
        const long long n = static_cast<long long>(blockIdx.x) * (kFewWarps / p.ksplit) * kFewRows + row, m = m0 + i;
        if (n < p.n && m < p.m) {
            int s = 0;
            for (int q = 0; q < p.ksplit; ++q) s += part[row / kFewRows * p.ksplit + q][row % kFewRows * MT + i];
            store_as(p.out, m * p.n + n, p.dt,
                     scaled(s, p.a_scale[m], p.w_scale[n], p.bias ? load_as(p.bias, n, p.dt) : 0.f, p.bias));
        }
    }
}

}  // namespace rmsq
