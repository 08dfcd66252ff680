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
// a time (a turn) and keeps its token's cosines and sines, and gamma, in registers over the heads it goes through.
// Bound by HBM: each element is read and written once. Registers hold too few rows for that, so a lane's vectors come
// through a ring of its own in shared memory by asynchronous copies, several turns ahead; nobody else reads them, so
// nothing waits but the lane.
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
    int turns, items;                // per token: of heads, and runs of `run` of them
};

struct RopeParams {
    RopeSide side[2];
    const float* cos;                // [places][half]
    const float* sin;
    const void* positions;           // [axes][tokens]
    float* part;                     // backward: [CTAs][D]
    int split;                       // CTAs that take queries; the others take keys
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
    // The same by way of shared memory. (Two bytes cannot be copied asynchronously.)
    static __device__ __forceinline__ void copy(uint32_t to, const void* p)
    {
        if constexpr (BYTES == 16)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + threadIdx.x * BYTES), "l"(p) : "memory");
        else if constexpr (BYTES >= 4)
            asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to + threadIdx.x * BYTES), "l"(p), "n"(BYTES) : "memory");
        else {
            uint16_t h;
            asm volatile("ld.global.u16 %0, [%1];" : "=h"(h) : "l"(p) : "memory");
            asm volatile("st.shared.u16 [%0], %1;" ::"r"(to + threadIdx.x * BYTES), "h"(h) : "memory");
        }
    }
    static __device__ __forceinline__ void get(uint32_t from, uint32_t* w)
    {
        from += threadIdx.x * BYTES;
        if constexpr (BYTES == 16) {
            const uint4 v = ld_shared_v4(from);
            w[0] = v.x;
            w[1] = v.y;
            w[2] = v.z;
            w[3] = v.w;
        } else if constexpr (BYTES == 8) {
            asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(from) : "memory");
        } else if constexpr (BYTES == 4) {
            asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(from) : "memory");
        } else {
            uint16_t h;
            asm volatile("ld.shared.u16 %0, [%1];" : "=h"(h) : "r"(from) : "memory");
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

constexpr int kRopeWarps = 8, kRopeThreads = 32 * kRopeWarps;

// A lane's rings: TENSORS rows of 16 elements in each of STAGES slots, vector i of thread t at (i * threads + t) vectors.
template <int DT, int V, bool INTER, int TENSORS, int STAGES> struct RopeRing {
    using Vec = RopeVec<DT, V>;
    using Lane = RopeLane<V, INTER>;
    static constexpr int ES = DT == DT_F32 ? 4 : 2, ROW = 16 * ES * kRopeThreads, BYTES = TENSORS * STAGES * ROW;
    uint32_t base;

    __device__ __forceinline__ uint32_t at(int stage, int tensor, int i) const
    {
        return base + static_cast<uint32_t>((stage * TENSORS + tensor) * ROW + (i * kRopeThreads) * Vec::BYTES);
    }
    // Starts the copies of a row (in: the lane has one).
    __device__ __forceinline__ void fetch(int stage, int tensor, const char* row, const Lane& lane, bool in) const
    {
#pragma unroll
        for (int i = 0; i < Lane::NV; ++i)
            if (in && lane.at[i] >= 0) Vec::copy(at(stage, tensor, i), row + static_cast<long long>(lane.at[i]) * ES);
    }
    // Zeros where the lane has nothing.
    __device__ __forceinline__ void get(int stage, int tensor, const Lane& lane, bool in, float (&f)[16]) const
    {
#pragma unroll
        for (int i = 0; i < Lane::NV; ++i) {
            uint32_t w[Vec::W];
#pragma unroll
            for (int j = 0; j < Vec::W; ++j) w[j] = 0;
            if (in && lane.at[i] >= 0) Vec::get(at(stage, tensor, i), w);
            Vec::unpack(w, f + i * V);
        }
    }
};

// A row to memory, and gamma from it.
template <int DT, int V, bool INTER>
__device__ __forceinline__ void rope_store(char* row, const RopeLane<V, INTER>& lane, const float (&f)[16])
{
#pragma unroll
    for (int i = 0; i < RopeLane<V, INTER>::NV; ++i)
        if (lane.at[i] >= 0) RopeVec<DT, V>::store(row + static_cast<long long>(lane.at[i]) * (DT == DT_F32 ? 4 : 2), f + i * V);
}

template <int DT, int V, bool INTER>
__device__ __forceinline__ void rope_gamma(const void* gamma, const RopeLane<V, INTER>& lane, float offset, float (&g)[16])
{
#pragma unroll
    for (int i = 0; i < RopeLane<V, INTER>::NV; ++i) {
        uint32_t w[RopeVec<DT, V>::W];
#pragma unroll
        for (int j = 0; j < RopeVec<DT, V>::W; ++j) w[j] = 0;
        if (lane.at[i] >= 0)
            RopeVec<DT, V>::load(static_cast<const char*>(gamma) + static_cast<long long>(lane.at[i]) * (DT == DT_F32 ? 4 : 2), w);
        RopeVec<DT, V>::unpack(w, g + i * V);
    }
#pragma unroll
    for (int j = 0; j < 16; ++j) g[j] += offset;
}

// The turns of a warp, one after another: items w, w + W, ... of a side's tokens * items, each of up to `run` turns of
// `rows` heads of one token.
struct RopeCursor {
    long long t;
    int item, left, head;            // within the token; turns left of the item; this lane's head
    __device__ __forceinline__ void enter(const RopeParams& p, const RopeSide& sd, int rows, int mine)
    {
        left = min(p.run, sd.turns - item * p.run);
        head = item * p.run * rows + mine;
    }
    __device__ __forceinline__ void start(const RopeParams& p, const RopeSide& sd, int rows, int mine, int w)
    {
        t = w / sd.items;
        item = static_cast<int>(w - t * sd.items);
        enter(p, sd, rows, mine);
    }
    // dt, di: the warps' stride in items, as tokens and items. True where an item begins.
    __device__ __forceinline__ bool next(const RopeParams& p, const RopeSide& sd, int rows, int mine, int dt, int di)
    {
        head += rows;
        if (--left > 0) return false;
        t += dt;
        item += di;
        if (item >= sd.items) {
            item -= sd.items;
            ++t;
        }
        enter(p, sd, rows, mine);
        return true;
    }
};

// Where a lane's row of a tensor lies: found at the start of an item, and a turn's heads on from there.
struct RopeAt {
    const char* p;
    __device__ __forceinline__ void enter(const void* base, long long t, long long st, int head, long long sh, int es)
    {
        p = static_cast<const char*>(base) + (t * st + head * sh) * es;
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

__device__ __forceinline__ float rope_rstd(float squares, const RopeParams& p) { return rsqrtf(fmaf(squares, p.inv_dim, p.eps)); }

// Pairs of neighbouring registers, for the packed instructions.
__device__ __forceinline__ float2 rope_two(const float (&f)[16], int j) { return make_float2(f[2 * j], f[2 * j + 1]); }
__device__ __forceinline__ void rope_put(float (&f)[16], int j, float2 v)
{
    f[2 * j] = v.x;
    f[2 * j + 1] = v.y;
}

__device__ __forceinline__ float rope_dot(const float (&a)[16], const float (&b)[16])
{
    float2 s = mul2(rope_two(a, 0), rope_two(b, 0));
#pragma unroll
    for (int j = 1; j < 8; ++j) s = fma2(rope_two(a, j), rope_two(b, j), s);
    return s.x + s.y;
}

// f with its pairs rotated by the angles, or by the opposite ones.
template <bool BACK, int V, bool INTER>
__device__ __forceinline__ void rope_turn(float (&f)[16], const RopeLane<V, INTER>& lane, const float (&cs)[8], const float (&sn)[8])
{
    using Lane = RopeLane<V, INTER>;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float a = f[Lane::a(j)], b = f[Lane::b(j)];
        if (lane.pair[Lane::of(j)] >= 0) {
            f[Lane::a(j)] = BACK ? fmaf(a, cs[j], b * sn[j]) : fmaf(a, cs[j], -b * sn[j]);
            f[Lane::b(j)] = BACK ? fmaf(b, cs[j], -a * sn[j]) : fmaf(b, cs[j], a * sn[j]);
        }
    }
}

// Slots of the rings: 64 KB a CTA, of which two or three run on an SM (32-bit gradients: 128 KB, one).
template <int DT, bool BACKWARD> struct RopeStages {
    static constexpr int N = DT != DT_F32 && !BACKWARD ? 8 : 4;
};

// What the kernels do with a side's turns: fetch several ahead, then body(stage, cursor, an item begins, the lane has a row).
// fetch(stage, cursor, an item begins, the lane has a row) starts the copies.
template <int STAGES, class Fetch, class Body>
__device__ __forceinline__ void rope_turns(const RopeParams& p, const RopeSide& sd, int rows, int mine, int w, int W, Fetch fetch, Body body)
{
    const int dt = W / sd.items, di = W - dt * sd.items;
    RopeCursor ahead, now;
    ahead.start(p, sd, rows, mine, w);
    now = ahead;
    bool begins = true, begins_ahead = true;
    const auto bring = [&](int stage) {
        if (ahead.t < p.tokens) {
            fetch(stage, ahead, begins_ahead, ahead.head < sd.heads);
            begins_ahead = ahead.next(p, sd, rows, mine, dt, di);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll 1
    for (int s = 0; s < STAGES - 1; ++s) bring(s);
    int stage = 0;
#pragma unroll 1
    while (now.t < p.tokens) {
        bring((stage + STAGES - 1) & (STAGES - 1));
        asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 1) : "memory");
        body(stage, now, begins, now.head < sd.heads);
        begins = now.next(p, sd, rows, mine, dt, di);
        stage = (stage + 1) & (STAGES - 1);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

template <int DT, int V, bool INTER>
__global__ void __launch_bounds__(kRopeThreads, DT == DT_F32 || V < 8 ? 2 : 3) rmsq_rope_kernel(const __grid_constant__ RopeParams p)
{
    using Lane = RopeLane<V, INTER>;
    constexpr int STAGES = RopeStages<DT, false>::N;
    using Ring = RopeRing<DT, V, INTER, 1, STAGES>;
    extern __shared__ __align__(16) unsigned char smem[];
    const int l = threadIdx.x & (p.lanes - 1), rows = 32 / p.lanes, mine = (threadIdx.x & 31) / p.lanes;
    const bool key = static_cast<int>(blockIdx.x) >= p.split;
    const RopeSide& sd = p.side[key];
    const int cta = static_cast<int>(blockIdx.x) - (key ? p.split : 0), ctas = key ? static_cast<int>(gridDim.x) - p.split : p.split;
    Lane lane;
    lane.init(l, p.lanes, p.dim, p.half);
    const Ring ring = {smem_u32(smem)};
    pdl_wait();
    float cs[8], sn[8], g[16];
    rope_gamma<DT, V, INTER>(sd.gamma, lane, p.offset, g);
    RopeAt x, y;
    const long long xs = rows * sd.xh * Ring::ES, ys = rows * sd.oh * Ring::ES;          // a turn's heads on
    rope_turns<STAGES>(
        p, sd, rows, mine, cta * kRopeWarps + (threadIdx.x >> 5), ctas * kRopeWarps,
        [&](int stage, const RopeCursor& c, bool begins, bool in) {
            if (begins) x.enter(sd.x, c.t, sd.xt, c.head, sd.xh, Ring::ES);
            ring.fetch(stage, 0, x.p, lane, in);
            x.p += xs;
        },
        [&](int stage, const RopeCursor& c, bool begins, bool in) {
            if (begins) {
                rope_angles<V, INTER>(p, lane, c.t, cs, sn);
                y.enter(sd.out, c.t, sd.ot, c.head, sd.oh, Ring::ES);
            }
            float f[16];
            ring.get(stage, 0, lane, in, f);
            const float2 rstd = splat(rope_rstd(rope_row_sum(rope_dot(f, f), p.lanes), p));
#pragma unroll
            for (int j = 0; j < 8; ++j) rope_put(f, j, mul2(mul2(rope_two(f, j), rstd), rope_two(g, j)));
            rope_turn<false>(f, lane, cs, sn);
            if (in) rope_store<DT, V, INTER>(const_cast<char*>(y.p), lane, f);
            y.p += ys;
        });
}

// A lane has the same elements in every row and adds their part of gamma's gradient in registers. The row groups of a warp
// are joined by exchanges, the warps of a CTA through shared memory, the CTAs by rmsq_rope_reduce_kernel, all in a
// fixed order.
template <int DT, int V, bool INTER>
__global__ void __launch_bounds__(kRopeThreads, DT == DT_F32 ? 1 : 2) rmsq_rope_bwd_kernel(const __grid_constant__ RopeParams p)
{
    using Lane = RopeLane<V, INTER>;
    constexpr int STAGES = RopeStages<DT, true>::N;
    using Ring = RopeRing<DT, V, INTER, 2, STAGES>;
    extern __shared__ __align__(16) unsigned char smem[];
    const int l = threadIdx.x & (p.lanes - 1), rows = 32 / p.lanes, mine = (threadIdx.x & 31) / p.lanes, warp = threadIdx.x >> 5;
    const bool key = static_cast<int>(blockIdx.x) >= p.split;
    const RopeSide& sd = p.side[key];
    const int cta = static_cast<int>(blockIdx.x) - (key ? p.split : 0), ctas = key ? static_cast<int>(gridDim.x) - p.split : p.split;
    Lane lane;
    lane.init(l, p.lanes, p.dim, p.half);
    const Ring ring = {smem_u32(smem)};
    pdl_wait();
    float cs[8], sn[8], g[16], acc[16];
    rope_gamma<DT, V, INTER>(sd.gamma, lane, p.offset, g);
#pragma unroll
    for (int j = 0; j < 16; ++j) acc[j] = 0.f;
    RopeAt x, dy, dx;
    const long long xs = rows * sd.xh * Ring::ES, ds = rows * sd.dh * Ring::ES, os = rows * sd.oh * Ring::ES;   // a turn's heads on
    rope_turns<STAGES>(
        p, sd, rows, mine, cta * kRopeWarps + warp, ctas * kRopeWarps,
        [&](int stage, const RopeCursor& c, bool begins, bool in) {
            if (begins) {
                x.enter(sd.x, c.t, sd.xt, c.head, sd.xh, Ring::ES);
                dy.enter(sd.dy, c.t, sd.dt, c.head, sd.dh, Ring::ES);
            }
            ring.fetch(stage, 0, x.p, lane, in);
            ring.fetch(stage, 1, dy.p, lane, in);
            x.p += xs;
            dy.p += ds;
        },
        [&](int stage, const RopeCursor& c, bool begins, bool in) {
            if (begins) {
                rope_angles<V, INTER>(p, lane, c.t, cs, sn);
                dx.enter(sd.out, c.t, sd.ot, c.head, sd.oh, Ring::ES);
            }
            float f[16], d[16];
            ring.get(stage, 0, lane, in, f);
            ring.get(stage, 1, lane, in, d);
            const float rstd = rope_rstd(rope_row_sum(rope_dot(f, f), p.lanes), p);
            rope_turn<true>(d, lane, cs, sn);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float2 xhat = mul2(rope_two(f, j), splat(rstd));
                // (a lane without a row has NaN here where its group has no place in the table)
                if (in) rope_put(acc, j, fma2(rope_two(d, j), xhat, rope_two(acc, j)));
                rope_put(f, j, xhat);
                rope_put(d, j, mul2(rope_two(d, j), rope_two(g, j)));
            }
            const float2 dot = splat(-rope_row_sum(rope_dot(f, d), p.lanes) * p.inv_dim);
#pragma unroll
            for (int j = 0; j < 8; ++j) rope_put(d, j, mul2(fma2(rope_two(f, j), dot, rope_two(d, j)), splat(rstd)));
            if (in) rope_store<DT, V, INTER>(const_cast<char*>(dx.p), lane, d);
            dx.p += os;
        });
    __syncthreads();                                       // the rings are free: they take the warps' sums
    float* const sums = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int j = 0; j < 16; ++j)
        for (int o = p.lanes; o < 32; o <<= 1) acc[j] += __shfl_xor_sync(0xFFFFFFFFu, acc[j], o);
    if (mine == 0) {
#pragma unroll
        for (int i = 0; i < Lane::NV; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (lane.at[i] >= 0) sums[warp * p.dim + lane.at[i] + j] = acc[i * V + j];
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.dim; e += kRopeThreads) {
        float a = 0.f;
#pragma unroll
        for (int w = 0; w < kRopeWarps; ++w) a += sums[w * p.dim + e];
        p.part[static_cast<long long>(blockIdx.x) * p.dim + e] = a;
    }
}

// The gammas' gradients from the CTAs' rows: 32 elements of one side per CTA; 32 warps share an element's rows and their sums
// are added in warp order.
struct RopeReduceParams {
    const float* part;
    void* out[2];
    int rows[2];                     // the queries' first, then the keys'
    int dim, dt;
};

static __global__ void __launch_bounds__(1024) rmsq_rope_reduce_kernel(const RopeReduceParams p)
{
    __shared__ float sum[32][33];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5, side = blockIdx.y, e = blockIdx.x * 32 + tx;
    pdl_wait();
    const float* const part = p.part + (side == 0 ? 0 : static_cast<long long>(p.rows[0]) * p.dim);
    float a = 0.f;
    if (e < p.dim) {
#pragma unroll 4
        for (int i = ty; i < p.rows[side]; i += 32) a += part[static_cast<long long>(i) * p.dim + e];
    }
    sum[ty][tx] = a;
    __syncthreads();
    if (ty != 0 || e >= p.dim) return;
    a = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) a += sum[i][tx];
    if (p.dt == DT_F32) static_cast<float*>(p.out[side])[e] = a;
    else static_cast<uint16_t*>(p.out[side])[e] = p.dt == DT_BF16 ? Scalar<DT_BF16>::put(a) : Scalar<DT_FP16>::put(a);
}

}  // namespace rmsq
