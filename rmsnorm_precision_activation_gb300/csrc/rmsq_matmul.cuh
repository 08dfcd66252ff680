// rmsq_matmul.cuh -- product of int8 codes with a scale per token and per output channel.
//
//   out[m][n] = RN((sum_k a[m][k] w[n][k]) * a_scale[m] * w_scale[n] + bias[n])
//
// The integer sums are exact in every kernel.
#pragma once

#include "rmsq_norm.cuh"
#include "rmsq_ops_plan.h"

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
    uint32_t wait, drain;      // bounds of waits, and of what a stopping CTA has in flight (rmsq_ops_plan.h)
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

// Four codes to four fp16: with the sign bit flipped a code is b = code + 128; the fp16 with high
// byte 0x64 and low byte b is 1024 + b, from which 1152 is subtracted exactly.
__device__ __forceinline__ void codes_to_half(uint32_t w, uint32_t& lo, uint32_t& hi)
{
    const uint32_t u = w ^ 0x80808080u;
    lo = __byte_perm(u, 0x64646464u, 0x4140);
    hi = __byte_perm(u, 0x64646464u, 0x4342);
    asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(lo) : "r"(0x64806480u));
    asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(hi) : "r"(0x64806480u));
}

// Single tokens and decode batches (NB x 8 tokens): bound by the weight's bytes. A CTA takes 16 or 32
// channels; its 8 warps take k in turn, 64 bytes of every row at a time, load the codes straight into
// registers, turn them into fp16 there and multiply with mma.sync (fp32 sums of up to 1024 products
// are exact, then they go to integers). No shared memory or barrier stands between a load and its
// use, so a short call costs little more than its bytes, where the tcgen05 kernels' hand-overs cost
// about 8 us. Measured (GB300, weights from HBM, calls in a captured graph): 1 to 8 tokens x 7168 x 8192
// 12.1 us, 4.9 TB/s (tcgen05: 20.2; a dp4a kernel took 18.7 us a call for 1 token, 28 for 8); x 28672 x 8192
// 39.0 us, 6.0 TB/s; 16 x 8192 x 8192 16.8 us (tcgen05: 20.4); 32 tokens 23.9 us (tcgen05: 20.7, so those go
// there).
// A fragment's k order is free as long as both operands share it: lane (g, t) loads 16 bytes of row
// g at 16 t, and the j-th four of them are its elements in the j-th of four MMAs.
constexpr int kStreamWarps = 8;
constexpr int kStreamHalves = 3;         // CTAs of 16 channels on an SM

template <int NB, int ROWS>
__global__ void __launch_bounds__(kStreamWarps * 32, ROWS == 16 ? kStreamHalves : 2) rmsq_matmul_stream_kernel(const MatmulParams p)
{
    // steps of 64 elements held in registers: one is multiplied while the loads of the others run
    constexpr int U = NB == 1 ? 4 : 3;
    __shared__ int part[kStreamWarps][NB * 8][ROWS + 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const long long n0 = static_cast<long long>(blockIdx.x) * ROWS;
    constexpr int I = ROWS / 16, R = ROWS / 8;      // MMAs of 16 rows, loads of 8
    const signed char* wp[R];
    const signed char* ap[NB];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const long long n = n0 + 8 * i + g;
        wp[i] = p.w + (n < p.n ? n : p.n - 1) * p.k + 16 * t;
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        const long long m = 8 * b + g;
        ap[b] = p.a + (m < p.m ? m : p.m - 1) * p.k + 16 * t;
    }
    pdl_wait();

    float c[I][NB][4];
#pragma unroll
    for (int i = 0; i < I; ++i)
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int e = 0; e < 4; ++e) c[i][b][e] = 0.f;
    bool fresh = true;                                     // nothing in part yet
    auto flush = [&]() {
#pragma unroll
        for (int i = 0; i < I; ++i)
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    int& sum = part[warp][8 * b + 2 * t + (e & 1)][16 * i + g + 8 * (e >> 1)];
                    sum = (fresh ? 0 : sum) + __float2int_rn(c[i][b][e]);
                    c[i][b][e] = 0.f;
                }
        fresh = false;
    };

    uint4 wv[U][R], av[U][NB];
    auto load = [&](int u, int step) {                     // past the end: zeros, nothing is read
        const int k = step * 64;
        const bool in = k + 16 * t < p.k;
#pragma unroll
        for (int i = 0; i < R; ++i)
            wv[u][i] = in ? ld_stream_v4(reinterpret_cast<const uint4*>(wp[i] + k)) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int b = 0; b < NB; ++b) av[u][b] = in ? ld_v4(ap[b] + k) : make_uint4(0, 0, 0, 0);
    };
    const int steps = (p.k + 63) / 64;
#pragma unroll
    for (int u = 0; u < U; ++u) load(u, warp + u * kStreamWarps);
    int held = 0;                                          // steps in c: at most 16, 1024 products
    for (int s = warp; s < steps; s += U * kStreamWarps) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            uint32_t w[R][4];
#pragma unroll
            for (int i = 0; i < R; ++i) {
                w[i][0] = wv[u][i].x;
                w[i][1] = wv[u][i].y;
                w[i][2] = wv[u][i].z;
                w[i][3] = wv[u][i].w;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t lo[R], hi[R];
#pragma unroll
                for (int i = 0; i < R; ++i) codes_to_half(w[i][j], lo[i], hi[i]);
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const uint32_t a[4] = {av[u][b].x, av[u][b].y, av[u][b].z, av[u][b].w};
                    uint32_t b0, b1;
                    codes_to_half(a[j], b0, b1);
#pragma unroll
                    for (int i = 0; i < I; ++i)
                        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
                            "{%8, %9}, {%0, %1, %2, %3};"
                            : "+f"(c[i][b][0]), "+f"(c[i][b][1]), "+f"(c[i][b][2]), "+f"(c[i][b][3])
                            : "r"(lo[2 * i]), "r"(lo[2 * i + 1]), "r"(hi[2 * i]), "r"(hi[2 * i + 1]), "r"(b0), "r"(b1));
                }
            }
            load(u, s + (u + U) * kStreamWarps);
            if (++held == 16) {
                flush();
                held = 0;
            }
        }
    }
    flush();
    __syncthreads();
    for (int e = threadIdx.x; e < NB * 8 * ROWS; e += kStreamWarps * 32) {
        const int row = e % ROWS, m = e / ROWS;
        const long long n = n0 + row;
        if (n < p.n && m < p.m) {
            int v = 0;
#pragma unroll
            for (int q = 0; q < kStreamWarps; ++q) v += part[q][m][row];
            store_as(p.out, m * p.n + n, p.dt,
                     scaled(v, p.a_scale[m], p.w_scale[n], p.bias ? load_as(p.bias, n, p.dt) : 0.f, p.bias));
        }
    }
}

}  // namespace rmsq
