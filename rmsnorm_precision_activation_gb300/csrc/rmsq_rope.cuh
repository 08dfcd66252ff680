// rmsq_rope.cuh -- RMS norm of every head's query and key with the rotation by its position, and the
// gradients of both.
//
//   xhat = x / sqrt(sum x^2 / D + eps);  z = xhat (gamma + offset)                       (fp32)
//   rotation of the first R of D elements: pairs (a, b) -> (a cos - b sin, b cos + a sin), the pair i being
//   elements (i, i + R/2), or (2i, 2i + 1) when neighbours are rotated together
//   backward: g = the rotation by the opposite angle of dy;  u = g (gamma + offset)
//             dx = rstd (u - xhat <u xhat>),  dgamma = sum over tokens and heads of g xhat    (<.>: mean over D)
//
// A head is a short row (64 to 256 elements), so a few lanes take one: every lane holds 8 pairs (16 elements)
// as both of their halves, and the rotation needs no exchange between lanes. A warp has 32 / lanes rows at
// a time and keeps its token's cosines and sines, and gamma, in registers over the heads it goes through.
// Bound by HBM: each element is read and written once.
#pragma once

#include "rmsq_norm.cuh"

namespace rmsq {

constexpr int kRopeAxes = 4;

struct RopeSide {                    // queries or keys: [tokens][heads][D], strides in elements
    const void* x;
    void* out;                       // y, or dx
    const void* dy;                  // backward
    const void* gamma;
    long long xt, xh, ot, oh, dt, dh;
    int heads;
    int items;                       // per token: runs of `run` turns of rows
};

struct RopeParams {
    RopeSide side[2];
    const float* cos;                // [places][half]
    const float* sin;
    const void* positions;           // [axes][tokens]
    float* part;                     // backward: [CTAs][2][D]
    long long tokens;
    long long places;
    int dim, half, wide;             // wide: positions are 64-bit
    int lanes;                       // per row, a power of two
    int run;                         // turns of rows per item
    int axes;
    int until[kRopeAxes];            // frequencies below until[a] go by axis a (or one before it)
    int vec_table;                   // table rows are whole vectors of 16 bytes
    float eps, offset, inv_dim;
};

// What a lane holds: 16 elements as 16 / V vectors of V neighbours; element f[8 s + j] belongs to the pair's
// half s (INTER: f[2 i] and f[2 i + 1] are pair i).
template <int V, bool INTER> struct RopeLane {
    static constexpr int C = 8 / V, NV = 2 * C;      // vectors per half, in all
    int at[NV];                                       // element a vector starts at; -1: none
    int pair[NV];                                     // its first pair, -1: not rotated

    __device__ __forceinline__ void init(int l, int lanes, int dim, int half)
    {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int s = i / C, c = i % C;
            if (INTER) {
                constexpr int VV = V < 2 ? 2 : V;             // a pair stays with one lane
                const int e = (i * V / VV * lanes + l) * VV + i * V % VV;
                at[i] = e < dim ? e : -1;
                pair[i] = e < 2 * half ? e / 2 : -1;
            } else {
                const int q = (c * lanes + l) * V, rest = dim / 2 - half;
                pair[i] = q < half ? q : -1;
                at[i] = q < half ? q + s * half : q < dim / 2 ? half + q + s * rest : -1;
            }
        }
    }
    static __device__ __forceinline__ int a(int i) { return INTER ? 2 * i : i; }
    static __device__ __forceinline__ int b(int i) { return INTER ? 2 * i + 1 : 8 + i; }
    // the vector that pair i of the lane is in (half-split: of its first half)
    static __device__ __forceinline__ int of(int i) { return INTER ? 2 * i / V : i / V; }
};

// V elements of a type, as raw words (a 16-bit element alone: in the low half).
template <int DT, int V> struct RopeVec {
    static constexpr int BYTES = V * (DT == DT_F32 ? 4 : 2), W = BYTES < 4 ? 1 : BYTES / 4;
    static __device__ __forceinline__ void load(const void* p, uint32_t* w)
    {
        if constexpr (BYTES == 16) {
            const uint4 v = ld_v4(p);
            w[0] = v.x;
            w[1] = v.y;
            w[2] = v.z;
            w[3] = v.w;
        } else if constexpr (BYTES == 8) {
            asm volatile("ld.global.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(p) : "memory");
        } else if constexpr (BYTES == 4) {
            asm volatile("ld.global.u32 %0, [%1];" : "=r"(w[0]) : "l"(p) : "memory");
        } else {
            uint16_t h;
            asm volatile("ld.global.u16 %0, [%1];" : "=h"(h) : "l"(p) : "memory");
            w[0] = h;
        }
    }
    static __device__ __forceinline__ void unpack(const uint32_t* w, float* f)
    {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if constexpr (DT == DT_F32) f[i] = __uint_as_float(w[i]);
            else f[i] = Scalar<DT>::get(static_cast<uint16_t>(w[i / 2] >> (16 * (i & 1))));
        }
    }
    static __device__ __forceinline__ void store(void* p, const float* f)
    {
        uint32_t w[W];
        if constexpr (DT == DT_F32) {
#pragma unroll
            for (int i = 0; i < V; ++i) w[i] = __float_as_uint(f[i]);
        } else if constexpr (V == 1) {
            st_u16(p, Scalar<DT>::put(f[0]));
            return;
        } else {
#pragma unroll
            for (int i = 0; i < V / 2; ++i) w[i] = Scalar<DT>::put2(f[2 * i], f[2 * i + 1]);
        }
        if constexpr (BYTES == 16) st_v4(p, make_uint4(w[0], w[1], w[2], w[3]));
        else if constexpr (BYTES == 8) st_v2(p, w[0], w[1]);
        else if constexpr (BYTES == 4) st_u32(p, w[0]);
    }
};

// A lane's 16 elements of a row, as raw words; zeros where it has none.
template <int DT, int V, bool INTER> struct RopeRow {
    using Vec = RopeVec<DT, V>;
    using Lane = RopeLane<V, INTER>;
    static constexpr int ES = DT == DT_F32 ? 4 : 2;
    uint32_t w[Lane::NV][Vec::W];

    __device__ __forceinline__ void load(const char* row, const Lane& lane, bool in)
    {
#pragma unroll
        for (int i = 0; i < Lane::NV; ++i) {
#pragma unroll
            for (int j = 0; j < Vec::W; ++j) w[i][j] = 0;
            if (in && lane.at[i] >= 0) Vec::load(row + static_cast<long long>(lane.at[i]) * ES, w[i]);
        }
    }
    __device__ __forceinline__ void unpack(float (&f)[16]) const
    {
#pragma unroll
        for (int i = 0; i < Lane::NV; ++i) Vec::unpack(w[i], f + i * V);
    }
    static __device__ __forceinline__ void store(char* row, const Lane& lane, const float (&f)[16])
    {
#pragma unroll
        for (int i = 0; i < Lane::NV; ++i)
            if (lane.at[i] >= 0) Vec::store(row + static_cast<long long>(lane.at[i]) * ES, f + i * V);
    }
};

__device__ __forceinline__ long long rope_place(const RopeParams& p, int axis, long long t)
{
    const long long i = axis * p.tokens + t;
    return p.wide ? static_cast<const long long*>(p.positions)[i] : static_cast<const int*>(p.positions)[i];
}

// Cosines and sines of the lane's 8 pairs for token t. A place outside the table reads nothing and gives NaN.
template <int V, bool INTER>
__device__ __forceinline__ void rope_angles(const RopeParams& p, const RopeLane<V, INTER>& lane, long long t,
                                            float (&c)[8], float (&s)[8])
{
    using Lane = RopeLane<V, INTER>;
    constexpr int PV = !INTER ? V : V > 2 ? V / 2 : 1, N = 8 / PV;     // pairs read together
    const float nan = __int_as_float(0x7FFFFFFF);
    const long long place0 = rope_place(p, 0, t);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int q = lane.pair[Lane::of(i * PV)];
#pragma unroll
        for (int j = 0; j < PV; ++j) {
            c[i * PV + j] = nan;
            s[i * PV + j] = nan;
        }
        if (q < 0) continue;
        if (p.axes == 1) {
            if (place0 < 0 || place0 >= p.places) continue;
            const float* const cr = p.cos + place0 * p.half + q;
            const float* const sr = p.sin + place0 * p.half + q;
            if (PV % 4 == 0 && p.vec_table) {
#pragma unroll
                for (int j = 0; j < PV; j += 4) {
                    const float4 a = __ldg(reinterpret_cast<const float4*>(cr + j));
                    const float4 b = __ldg(reinterpret_cast<const float4*>(sr + j));
                    c[i * PV + j] = a.x, c[i * PV + j + 1] = a.y, c[i * PV + j + 2] = a.z, c[i * PV + j + 3] = a.w;
                    s[i * PV + j] = b.x, s[i * PV + j + 1] = b.y, s[i * PV + j + 2] = b.z, s[i * PV + j + 3] = b.w;
                }
            } else {
#pragma unroll
                for (int j = 0; j < PV; ++j) {
                    c[i * PV + j] = __ldg(cr + j);
                    s[i * PV + j] = __ldg(sr + j);
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < PV; ++j) {
                int axis = 0;
#pragma unroll
                for (int a = 0; a < kRopeAxes - 1; ++a) axis += q + j >= p.until[a];
                const long long place = axis == 0 ? place0 : rope_place(p, axis, t);
                if (place < 0 || place >= p.places) continue;
                c[i * PV + j] = __ldg(p.cos + place * p.half + q + j);
                s[i * PV + j] = __ldg(p.sin + place * p.half + q + j);
            }
        }
    }
}

__device__ __forceinline__ float rope_row_sum(float v, int lanes)
{
    for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

constexpr int kRopeWarps = 8;

// Where item i of a side's tokens * items lies: its token and its first head.
__device__ __forceinline__ void rope_item(const RopeParams& p, const RopeSide& sd, long long i, int rows, long long& t, int& h)
{
    t = i / sd.items;
    h = static_cast<int>(i - t * sd.items) * p.run * rows;
}

template <int DT, int V, bool INTER>
__global__ void __launch_bounds__(kRopeWarps * 32) rmsq_rope_kernel(const __grid_constant__ RopeParams p)
{
    using Lane = RopeLane<V, INTER>;
    using Row = RopeRow<DT, V, INTER>;
    constexpr int U = DT == DT_F32 ? 2 : 4;                  // rows whose loads are in flight together
    constexpr int ES = Row::ES;
    const int l = threadIdx.x & (p.lanes - 1), rows = 32 / p.lanes, mine = (threadIdx.x & 31) / p.lanes;
    Lane lane;
    lane.init(l, p.lanes, p.dim, p.half);
    pdl_wait();
    const long long nq = p.tokens * p.side[0].items;
    long long i = static_cast<long long>(blockIdx.x) * kRopeWarps + (threadIdx.x >> 5);
    const bool key = i >= nq;
    if (key) i -= nq;
    const RopeSide& sd = p.side[key];
    if (i >= p.tokens * sd.items) return;
    long long t;
    int h0;
    rope_item(p, sd, i, rows, t, h0);
    const char* const x = static_cast<const char*>(sd.x) + t * sd.xt * ES;
    char* const out = static_cast<char*>(sd.out) + t * sd.ot * ES;
    float cs[8], sn[8], g[16];
    Row graw;
    graw.load(static_cast<const char*>(sd.gamma), lane, true);
    rope_angles<V, INTER>(p, lane, t, cs, sn);
    graw.unpack(g);
#pragma unroll
    for (int j = 0; j < 16; ++j) g[j] += p.offset;
    for (int r = 0; r < p.run; r += U) {
        Row raw[U];
        int h[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            h[u] = h0 + (r + u) * rows + mine;
            raw[u].load(x + h[u] * sd.xh * ES, lane, r + u < p.run && h[u] < sd.heads);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float f[16], ss = 0.f;
            raw[u].unpack(f);
#pragma unroll
            for (int j = 0; j < 16; ++j) ss = fmaf(f[j], f[j], ss);
            ss = rope_row_sum(ss, p.lanes);
            const float rstd = __frcp_rn(__fsqrt_rn(fmaf(ss, p.inv_dim, p.eps)));
#pragma unroll
            for (int j = 0; j < 16; ++j) f[j] = f[j] * rstd * g[j];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float a = f[Lane::a(j)], b = f[Lane::b(j)];
                if (lane.pair[Lane::of(j)] >= 0) {
                    f[Lane::a(j)] = a * cs[j] - b * sn[j];
                    f[Lane::b(j)] = b * cs[j] + a * sn[j];
                }
            }
            if (r + u < p.run && h[u] < sd.heads) Row::store(out + h[u] * sd.oh * ES, lane, f);
        }
    }
}

// Persistent: a warp goes through its queries' items, then through its keys', and adds each side's gamma
// gradient in registers (a lane has the same elements in every row). The row groups of a CTA are joined through
// shared memory, the CTAs by the column reduction of the layer norm, all in a fixed order.
template <int DT, int V, bool INTER>
__global__ void __launch_bounds__(kRopeWarps * 32) rmsq_rope_bwd_kernel(const __grid_constant__ RopeParams p)
{
    using Lane = RopeLane<V, INTER>;
    using Row = RopeRow<DT, V, INTER>;
    constexpr int ES = Row::ES;
    __shared__ float sums[kRopeWarps][512];
    const int l = threadIdx.x & (p.lanes - 1), rows = 32 / p.lanes, mine = (threadIdx.x & 31) / p.lanes;
    const int warp = threadIdx.x >> 5;
    Lane lane;
    lane.init(l, p.lanes, p.dim, p.half);
    pdl_wait();
#pragma unroll 1
    for (int k = 0; k < 2; ++k) {
        const RopeSide& sd = p.side[k];
        float g[16], acc[16];
        {
            Row graw;
            graw.load(static_cast<const char*>(sd.gamma), lane, true);
            graw.unpack(g);
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            g[j] += p.offset;
            acc[j] = 0.f;
        }
        const long long items = p.tokens * sd.items;
        for (long long i = static_cast<long long>(blockIdx.x) * kRopeWarps + warp; i < items;
             i += static_cast<long long>(gridDim.x) * kRopeWarps) {
            long long t;
            int h0;
            rope_item(p, sd, i, rows, t, h0);
            const char* const x = static_cast<const char*>(sd.x) + t * sd.xt * ES;
            const char* const dy = static_cast<const char*>(sd.dy) + t * sd.dt * ES;
            char* const out = static_cast<char*>(sd.out) + t * sd.ot * ES;
            float cs[8], sn[8];
            rope_angles<V, INTER>(p, lane, t, cs, sn);
            for (int r = 0; r < p.run; ++r) {
                const int h = h0 + r * rows + mine;
                const bool in = h < sd.heads;
                Row rx, rd;
                rx.load(x + h * sd.xh * ES, lane, in);
                rd.load(dy + h * sd.dh * ES, lane, in);
                float f[16], d[16], ss = 0.f, dot = 0.f;
                rx.unpack(f);
                rd.unpack(d);
#pragma unroll
                for (int j = 0; j < 16; ++j) ss = fmaf(f[j], f[j], ss);
                ss = rope_row_sum(ss, p.lanes);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float a = d[Lane::a(j)], b = d[Lane::b(j)];
                    if (in && lane.pair[Lane::of(j)] >= 0) {
                        d[Lane::a(j)] = a * cs[j] + b * sn[j];
                        d[Lane::b(j)] = b * cs[j] - a * sn[j];
                    }
                }
                const float rstd = __frcp_rn(__fsqrt_rn(fmaf(ss, p.inv_dim, p.eps)));
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    f[j] *= rstd;
                    if (in) acc[j] = fmaf(d[j], f[j], acc[j]);
                    d[j] *= g[j];
                    dot = fmaf(d[j], f[j], dot);
                }
                dot = rope_row_sum(dot, p.lanes) * p.inv_dim;
#pragma unroll
                for (int j = 0; j < 16; ++j) d[j] = rstd * (d[j] - f[j] * dot);
                if (in) Row::store(out + h * sd.oh * ES, lane, d);
            }
        }
        // the warp's row groups, then the CTA's warps
#pragma unroll
        for (int j = 0; j < 16; ++j)
            for (int o = p.lanes; o < 32; o <<= 1) acc[j] += __shfl_xor_sync(0xFFFFFFFFu, acc[j], o);
        if (mine == 0) {
#pragma unroll
            for (int i = 0; i < Lane::NV; ++i)
#pragma unroll
                for (int j = 0; j < V; ++j)
                    if (lane.at[i] >= 0) sums[warp][lane.at[i] + j] = acc[i * V + j];
        }
        __syncthreads();
        for (int e = threadIdx.x; e < p.dim; e += kRopeWarps * 32) {
            float a = 0.f;
#pragma unroll
            for (int w = 0; w < kRopeWarps; ++w) a += sums[w][e];
            p.part[(static_cast<long long>(blockIdx.x) * 2 + k) * p.dim + e] = a;
        }
        __syncthreads();
    }
}

}  // namespace rmsq
