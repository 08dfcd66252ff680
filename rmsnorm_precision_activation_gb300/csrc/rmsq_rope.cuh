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
// as both of their halves, and the rotation needs no exchange between lanes. A warp has two groups of 32 / lanes rows at
// a time (a turn); gamma and the token's cosines and sines come to the lanes by way of shared memory.
// Bound by HBM: each element is read and written once. Registers hold too few rows for that, so a lane's vectors come
// through a ring of its own in shared memory by asynchronous copies, a turn ahead; nobody else reads them, so
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
    unsigned xt, xh, ot, oh, dt, dh; // (below 2^31)
    int heads;
    int groups;                      // of heads that a warp takes at a time, per token
};

struct RopeParams {
    RopeSide side[2];
    const float* cos;                // [places][half]
    const float* sin;
    const void* positions;           // [axes][tokens]
    float* part;                     // backward: [CTAs][D]
    int split;                       // CTAs that take queries; the others take keys
    int tokens;
    long long places;
    int dim, half, wide;             // wide: positions are 64-bit
    int lanes;                       // per row, a power of two
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

// Threads of a CTA and CTAs on an SM: 16 warps of 128 registers a thread, backward 12 of 168 (16 of 128 spill: 146 us,
// 16384 tokens of 40 heads of 128 in bf16, against 81). Two slots in a ring, one turn ahead: with three, forward takes 53 us there
// instead of 54, 4099 tokens of 14 heads of 80 in fp32 10.7 instead of 10.2 (two groups of one token a turn). Forward with 20 warps of 96
// registers: heads of 96 47 us instead of 49.5, but 32 + 32 heads of 128 93 instead of 85 and of 256 112 instead of 108.
template <bool BACKWARD> struct RopeShape {
    static constexpr int THREADS = BACKWARD ? 192 : 128, CTAS = BACKWARD ? 2 : 4, STAGES = 2;
};

// A lane's ring: ROWS rows of 16 elements in each of STAGES slots, vector i of thread t at (i * threads + t) vectors. Where
// a lane has no elements its slots stay zero; where it has no row they keep what an earlier row left.
template <int DT, int V, bool INTER, int ROWS, int STAGES, int THREADS> struct RopeRing {
    using Vec = RopeVec<DT, V>;
    using Lane = RopeLane<V, INTER>;
    static constexpr int ES = DT == DT_F32 ? 4 : 2, ROW = 16 * ES * THREADS, BYTES = ROWS * STAGES * ROW;
    uint32_t base;

    __device__ __forceinline__ uint32_t at(int stage, int row, int i) const
    {
        return base + static_cast<uint32_t>((stage * ROWS + row) * ROW + (i * THREADS) * Vec::BYTES);
    }
    __device__ __forceinline__ void clear() const
    {
        for (uint32_t i = threadIdx.x * 16; i < BYTES; i += THREADS * 16) st_shared_v4(base + i, make_uint4(0, 0, 0, 0));
    }
    // Starts the copies of a row.
    __device__ __forceinline__ void fetch(int stage, int row, const char* from, const Lane& lane) const
    {
#pragma unroll
        for (int i = 0; i < Lane::NV; ++i)
            if (lane.at[i] >= 0) Vec::copy(at(stage, row, i), from + static_cast<long long>(lane.at[i]) * ES);
    }
    __device__ __forceinline__ void get(int stage, int row, float (&f)[16]) const
    {
#pragma unroll
        for (int i = 0; i < Lane::NV; ++i) {
            uint32_t w[Vec::W];
            Vec::get(at(stage, row, i), w);
            Vec::unpack(w, f + i * V);
        }
    }
};

// A row to memory.
template <int DT, int V, bool INTER>
__device__ __forceinline__ void rope_store(char* row, const RopeLane<V, INTER>& lane, const float (&f)[16])
{
#pragma unroll
    for (int i = 0; i < RopeLane<V, INTER>::NV; ++i)
        if (lane.at[i] >= 0) RopeVec<DT, V>::store(row + static_cast<long long>(lane.at[i]) * (DT == DT_F32 ? 4 : 2), f + i * V);
}

// L floats from shared memory.
template <int L> __device__ __forceinline__ void rope_read(uint32_t from, float* f)
{
    if constexpr (L == 4)
        asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3]) : "r"(from) : "memory");
    else if constexpr (L == 2)
        asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(f[0]), "=f"(f[1]) : "r"(from) : "memory");
    else
        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(f[0]) : "r"(from) : "memory");
}

// gamma + offset in fp32, a CTA's together: registers go to the rows instead.
template <int DT> struct RopeGamma {
    uint32_t base;
    __device__ __forceinline__ void load(const void* gamma, int dim, float offset) const
    {
        for (int i = threadIdx.x; i < dim; i += blockDim.x) {
            const float v = Scalar<DT>::get(static_cast<const typename Scalar<DT>::T*>(gamma)[i]) + offset;
            asm volatile("st.shared.f32 [%0], %1;" ::"r"(base + i * 4), "f"(v) : "memory");
        }
    }
    template <int V, bool INTER> __device__ __forceinline__ void get(const RopeLane<V, INTER>& lane, float (&g)[16]) const
    {
        constexpr int L = V < 4 ? V : 4;
#pragma unroll
        for (int i = 0; i < RopeLane<V, INTER>::NV; ++i)
#pragma unroll
            for (int j = 0; j < V; j += L) rope_read<L>(base + (max(lane.at[i], 0) + j) * 4, g + i * V + j);
    }
};

// The turns of a warp, one after another: w, w + W, ... of a side's, each two of its tokens * groups groups of heads, which follow one
// another: the second is the next token's first where the first is its token's last, so that few heads, or an odd
// number of groups, leave no half of a turn empty (4099 tokens of 12 + 2 heads of 80 in fp32: 9.0 us, with two groups of one
// token a turn 10.1). Kernels of their own do that (BOTH): where both sides' groups are even no turn has two tokens, and
// allowing for it takes 56.5 us instead of 54.5 below. Neighbouring warps have neighbouring turns, so what an SM reads and writes at a time
// lies together: forward takes 59 us where a warp takes four turns in a row, 56.5 with two and 54.5 so, though angles are
// copied for every turn (16384 tokens of 40 heads of 128 in bf16, 6.3 TB/s; backward 84, 83 and 80 us, 6.4 TB/s). Heads of 192,
// where a quarter of the lanes has nothing, lose by it: 95 and 98 us, backward 146 and 156.
constexpr int kRopeRows = 2;

struct RopeCursor {
    int t, group;                    // of the first group
    __device__ __forceinline__ void start(const RopeSide& sd, int w)
    {
        t = 2 * w / sd.groups;
        group = 2 * w - t * sd.groups;
    }
    // dt, di: the warps' stride, as tokens and groups.
    __device__ __forceinline__ void next(const RopeSide& sd, int dt, int di)
    {
        t += dt;
        group += di;
        if (group >= sd.groups) {
            group -= sd.groups;
            ++t;
        }
    }
    // Whether the second group is the next token's.
    __device__ __forceinline__ bool splits(const RopeSide& sd) const { return group + 1 == sd.groups; }
};

// A lane's rows of a turn. Where a tensor's lie: first() and, `rows` heads on or in the next token, second().
template <bool BOTH> struct RopeRows {
    int t, head, mine;
    bool split, in[2];
    __device__ __forceinline__ RopeRows(const RopeParams& p, const RopeSide& sd, const RopeCursor& c, int rows, int mine_)
    {
        t = c.t;
        mine = mine_;
        head = c.group * rows + mine;
        split = BOTH && c.splits(sd);
        in[0] = head < sd.heads;
        in[1] = split ? mine < sd.heads && t + 1 < p.tokens : head + rows < sd.heads;
    }
    static __device__ __forceinline__ char* at(const void* base, int t, int head, unsigned st, unsigned sh, int es)
    {
        const unsigned long long e = static_cast<unsigned long long>(static_cast<unsigned>(t)) * st +
                                     static_cast<unsigned long long>(static_cast<unsigned>(head)) * sh;
        return const_cast<char*>(static_cast<const char*>(base)) + e * static_cast<unsigned>(es);
    }
    __device__ __forceinline__ char* first(const void* base, unsigned st, unsigned sh, int es) const { return at(base, t, head, st, sh, es); }
    __device__ __forceinline__ char* second(char* first, unsigned long long step, const void* base, unsigned st, unsigned sh, int es) const
    {
        return split ? at(base, t + 1, mine, st, sh, es) : first + step;
    }
};

// A warp's cosines and sines, [slot][token of a turn][cosines, then sines][half], a slot for each turn whose rows are in the ring. The
// warp copies its tokens' rows of both tables together. Lane a holds the first token's place on axis a, lane 16 + a
// the second's, read a turn before it is needed.
template <int STAGES, bool BOTH> struct RopeAngles {
    uint32_t base;                       // this warp's
    long long place;

    static __host__ __device__ constexpr int bytes(int half) { return STAGES * (1 + BOTH) * 2 * ((half + 3) / 4 * 4) * 4; }
    __device__ __forceinline__ uint32_t at(const RopeParams& p, int slot, int second, int sine) const
    {
        return base + static_cast<uint32_t>(((slot * (1 + BOTH) + second) * 2 + sine) * ((p.half + 3) / 4 * 4) * 4);
    }
    __device__ __forceinline__ void look(const RopeParams& p, int t)
    {
        const int lane = threadIdx.x & 31, axis = lane & 15;
        if (BOTH) t += lane >> 4;
        if (axis >= p.axes || t >= p.tokens) return;
        const long long i = static_cast<long long>(axis) * p.tokens + t;
        place = p.wide ? static_cast<const long long*>(p.positions)[i] : static_cast<const int*>(p.positions)[i];
    }
    // Starts the copies for a token of the turn whose first token look() was given. A place outside the table reads nothing and gives NaN.
    __device__ __forceinline__ void fetch(const RopeParams& p, int slot, int second)
    {
        const int lane = threadIdx.x & 31;
        const uint32_t c = at(p, slot, second, 0), s = at(p, slot, second, 1);
        if (p.axes == 1 && p.vec_table) {
            const long long row = __shfl_sync(0xFFFFFFFFu, place, 16 * second);
            const bool in = row >= 0 && row < p.places;
            for (int i = lane; i < p.half / 2; i += 32) {                 // the cosines' vectors, then the sines'
                const int sine = i >= p.half / 4, v = 4 * (i - sine * (p.half / 4));
                const uint32_t to = (sine ? s : c) + v * 4;
                if (in)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"((sine ? p.sin : p.cos) + row * p.half + v) : "memory");
                else
                    st_shared_v4(to, make_uint4(0x7FFFFFFFu, 0x7FFFFFFFu, 0x7FFFFFFFu, 0x7FFFFFFFu));
            }
        } else {
            for (int i0 = 0; i0 < p.half; i0 += 32) {
                const int i = i0 + lane;
                int axis = 0;
#pragma unroll
                for (int a = 0; a < kRopeAxes - 1; ++a) axis += i >= p.until[a];
                const long long row = __shfl_sync(0xFFFFFFFFu, place, 16 * second + axis);
                if (i >= p.half) continue;
                if (row >= 0 && row < p.places) {
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(c + i * 4), "l"(p.cos + row * p.half + i) : "memory");
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(s + i * 4), "l"(p.sin + row * p.half + i) : "memory");
                } else {
                    asm volatile("st.shared.u32 [%0], %1;" ::"r"(c + i * 4), "r"(0x7FFFFFFFu) : "memory");
                    asm volatile("st.shared.u32 [%0], %1;" ::"r"(s + i * 4), "r"(0x7FFFFFFFu) : "memory");
                }
            }
        }
    }
    // Cosines and sines of the lane's 8 pairs (any where it has none).
    template <int V, bool INTER>
    __device__ __forceinline__ void get(const RopeParams& p, int slot, int second, const RopeLane<V, INTER>& lane, float (&c)[8], float (&s)[8]) const
    {
        using Lane = RopeLane<V, INTER>;
        constexpr int PV = !INTER ? V : V > 2 ? V / 2 : 1, N = 8 / PV, L = PV < 4 ? PV : 4;     // pairs together; floats of a read
        const uint32_t ca = at(p, slot, second, 0), sa = at(p, slot, second, 1);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int q = max(lane.pair[Lane::of(i * PV)], 0);
#pragma unroll
            for (int j = 0; j < PV; j += L) {
                rope_read<L>(ca + (q + j) * 4, c + i * PV + j);
                rope_read<L>(sa + (q + j) * 4, s + i * PV + j);
            }
        }
    }
};

// Sums over the lanes of a row, of every row of a lane.
__device__ __forceinline__ void rope_row_sums(float (&v)[2], int lanes)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        if (o >= lanes) continue;
        v[0] += __shfl_xor_sync(0xFFFFFFFFu, v[0], o);
        v[1] += __shfl_xor_sync(0xFFFFFFFFu, v[1], o);
    }
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

// What the kernels do with a side's turns: fetch(stage, cursor) starts the copies of a turn ahead of body(stage, cursor), when
// they and the angles are there.
template <int STAGES, bool BOTH, class Fetch, class Body>
__device__ __forceinline__ void rope_turns(const RopeParams& p, const RopeSide& sd, int w, int W, RopeAngles<STAGES, BOTH>& angles, Fetch fetch, Body body)
{
    const int dt = 2 * W / sd.groups, di = 2 * W - dt * sd.groups;
    RopeCursor ahead, now;
    ahead.start(sd, w);
    now = ahead;
    angles.look(p, ahead.t);
    const auto bring = [&](int stage) {
        if (ahead.t < p.tokens) {
            angles.fetch(p, stage, 0);
            if (BOTH && ahead.splits(sd) && ahead.t + 1 < p.tokens) angles.fetch(p, stage, 1);
            fetch(stage, ahead);
            ahead.next(sd, dt, di);
            angles.look(p, ahead.t);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll 1
    for (int s = 0; s < STAGES - 1; ++s) bring(s);
    int stage = 0;
#pragma unroll 1
    while (now.t < p.tokens) {
        bring(stage == 0 ? STAGES - 1 : stage - 1);
        asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 1) : "memory");
        __syncwarp();                                     // the angles are the warp's together
        body(stage, now);
        now.next(sd, dt, di);
        __syncwarp();
        if (++stage == STAGES) stage = 0;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

// Two rows of a lane at a time: two chains of dependent instructions in flight, and half the bookkeeping.
template <int DT, int V, bool INTER, bool BOTH>
__global__ void __launch_bounds__(RopeShape<false>::THREADS, RopeShape<false>::CTAS) rmsq_rope_kernel(const __grid_constant__ RopeParams p)
{
    using Lane = RopeLane<V, INTER>;
    using Shape = RopeShape<false>;
    constexpr int STAGES = Shape::STAGES, WARPS = Shape::THREADS / 32, R = kRopeRows;
    using Ring = RopeRing<DT, V, INTER, R, STAGES, Shape::THREADS>;
    extern __shared__ __align__(16) unsigned char smem[];
    const int l = threadIdx.x & (p.lanes - 1), rows = 32 / p.lanes, mine = (threadIdx.x & 31) / p.lanes, warp = threadIdx.x >> 5;
    const bool key = static_cast<int>(blockIdx.x) >= p.split;
    const RopeSide& sd = p.side[key];
    const int cta = static_cast<int>(blockIdx.x) - (key ? p.split : 0), ctas = key ? static_cast<int>(gridDim.x) - p.split : p.split;
    Lane lane;
    lane.init(l, p.lanes, p.dim, p.half);
    const Ring ring = {smem_u32(smem)};
    RopeAngles<STAGES, BOTH> angles;
    angles.base = smem_u32(smem) + Ring::BYTES + warp * RopeAngles<STAGES, BOTH>::bytes(p.half);
    const RopeGamma<DT> gamma = {smem_u32(smem) + Ring::BYTES + WARPS * RopeAngles<STAGES, BOTH>::bytes(p.half)};
    ring.clear();
    pdl_wait();
    gamma.load(sd.gamma, p.dim, p.offset);
    __syncthreads();
    const unsigned long long xs = 1ull * rows * sd.xh * Ring::ES, ys = 1ull * rows * sd.oh * Ring::ES;      // `rows` heads on
    rope_turns<STAGES, BOTH>(
        p, sd, cta * WARPS + warp, ctas * WARPS, angles,
        [&](int stage, const RopeCursor& c) {
            const RopeRows<BOTH> row(p, sd, c, rows, mine);
            char* x = row.first(sd.x, sd.xt, sd.xh, Ring::ES);
            if (row.in[0]) ring.fetch(stage, 0, x, lane);
            x = row.second(x, xs, sd.x, sd.xt, sd.xh, Ring::ES);
            if (row.in[1]) ring.fetch(stage, 1, x, lane);
        },
        [&](int stage, const RopeCursor& c) {
            float f[R][16], ss[R];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                ring.get(stage, r, f[r]);
                ss[r] = rope_dot(f[r], f[r]);
            }
            rope_row_sums(ss, p.lanes);
            {
                float g[16];
                gamma.get(lane, g);
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float2 rstd = splat(rope_rstd(ss[r], p));
#pragma unroll
                    for (int j = 0; j < 8; ++j) rope_put(f[r], j, mul2(mul2(rope_two(f[r], j), rstd), rope_two(g, j)));
                }
            }
            float cs[8], sn[8];
            const RopeRows<BOTH> row(p, sd, c, rows, mine);
            char* y = row.first(sd.out, sd.ot, sd.oh, Ring::ES);
            angles.get(p, stage, 0, lane, cs, sn);
            rope_turn<false>(f[0], lane, cs, sn);
            if (row.in[0]) rope_store<DT, V, INTER>(y, lane, f[0]);
            if (row.split) angles.get(p, stage, 1, lane, cs, sn);
            y = row.second(y, ys, sd.out, sd.ot, sd.oh, Ring::ES);
            rope_turn<false>(f[1], lane, cs, sn);
            if (row.in[1]) rope_store<DT, V, INTER>(y, lane, f[1]);
        });
}

// A lane has the same elements in every row and adds their part of gamma's gradient in registers. The row groups of a warp
// are joined by exchanges, the warps of a CTA through shared memory, the CTAs by rmsq_rope_reduce_kernel, all in a
// fixed order.
template <int DT, int V, bool INTER, bool BOTH>
__global__ void __launch_bounds__(RopeShape<true>::THREADS, RopeShape<true>::CTAS) rmsq_rope_bwd_kernel(const __grid_constant__ RopeParams p)
{
    using Lane = RopeLane<V, INTER>;
    using Shape = RopeShape<true>;
    constexpr int STAGES = Shape::STAGES, WARPS = Shape::THREADS / 32, R = kRopeRows;
    using Ring = RopeRing<DT, V, INTER, 2 * R, STAGES, Shape::THREADS>;                  // rows of x, then of dy
    extern __shared__ __align__(16) unsigned char smem[];
    const int l = threadIdx.x & (p.lanes - 1), rows = 32 / p.lanes, mine = (threadIdx.x & 31) / p.lanes, warp = threadIdx.x >> 5;
    const bool key = static_cast<int>(blockIdx.x) >= p.split;
    const RopeSide& sd = p.side[key];
    const int cta = static_cast<int>(blockIdx.x) - (key ? p.split : 0), ctas = key ? static_cast<int>(gridDim.x) - p.split : p.split;
    Lane lane;
    lane.init(l, p.lanes, p.dim, p.half);
    const Ring ring = {smem_u32(smem)};
    RopeAngles<STAGES, BOTH> angles;
    angles.base = smem_u32(smem) + Ring::BYTES + warp * RopeAngles<STAGES, BOTH>::bytes(p.half);
    const RopeGamma<DT> gamma = {smem_u32(smem) + Ring::BYTES + WARPS * RopeAngles<STAGES, BOTH>::bytes(p.half)};
    ring.clear();
    pdl_wait();
    gamma.load(sd.gamma, p.dim, p.offset);
    __syncthreads();
    float acc[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) acc[j] = 0.f;
    const unsigned long long xs = 1ull * rows * sd.xh * Ring::ES, ds = 1ull * rows * sd.dh * Ring::ES, os = 1ull * rows * sd.oh * Ring::ES;
    rope_turns<STAGES, BOTH>(
        p, sd, cta * WARPS + warp, ctas * WARPS, angles,
        [&](int stage, const RopeCursor& c) {
            const RopeRows<BOTH> row(p, sd, c, rows, mine);
            char *x = row.first(sd.x, sd.xt, sd.xh, Ring::ES), *dy = row.first(sd.dy, sd.dt, sd.dh, Ring::ES);
            if (row.in[0]) {
                ring.fetch(stage, 0, x, lane);
                ring.fetch(stage, R, dy, lane);
            }
            x = row.second(x, xs, sd.x, sd.xt, sd.xh, Ring::ES);
            dy = row.second(dy, ds, sd.dy, sd.dt, sd.dh, Ring::ES);
            if (row.in[1]) {
                ring.fetch(stage, 1, x, lane);
                ring.fetch(stage, R + 1, dy, lane);
            }
        },
        [&](int stage, const RopeCursor& c) {
            const RopeRows<BOTH> row(p, sd, c, rows, mine);
            float f[R][16], d[R][16], ss[R], dot[R];
            {
                float cs[8], sn[8];
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    if (r == 0 || row.split) angles.get(p, stage, r, lane, cs, sn);
                    ring.get(stage, r, f[r]);
                    ring.get(stage, R + r, d[r]);
                    ss[r] = rope_dot(f[r], f[r]);
                    rope_turn<true>(d[r], lane, cs, sn);
                }
            }
            rope_row_sums(ss, p.lanes);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                ss[r] = rope_rstd(ss[r], p);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    rope_put(f[r], j, mul2(rope_two(f[r], j), splat(ss[r])));
                    // (a lane without a row has anything here)
                    if (row.in[r]) rope_put(acc, j, fma2(rope_two(d[r], j), rope_two(f[r], j), rope_two(acc, j)));
                }
            }
            {
                float g[16];
                gamma.get(lane, g);
#pragma unroll
                for (int r = 0; r < R; ++r) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) rope_put(d[r], j, mul2(rope_two(d[r], j), rope_two(g, j)));
                    dot[r] = rope_dot(f[r], d[r]);
                }
            }
            rope_row_sums(dot, p.lanes);
            char* dx = nullptr;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float2 back = splat(-dot[r] * p.inv_dim);
#pragma unroll
                for (int j = 0; j < 8; ++j) rope_put(d[r], j, mul2(fma2(rope_two(f[r], j), back, rope_two(d[r], j)), splat(ss[r])));
                dx = r == 0 ? row.first(sd.out, sd.ot, sd.oh, Ring::ES) : row.second(dx, os, sd.out, sd.ot, sd.oh, Ring::ES);
                if (row.in[r]) rope_store<DT, V, INTER>(dx, lane, d[r]);
            }
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
    for (int e = threadIdx.x; e < p.dim; e += Shape::THREADS) {
        float a = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) a += sums[w * p.dim + e];
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
