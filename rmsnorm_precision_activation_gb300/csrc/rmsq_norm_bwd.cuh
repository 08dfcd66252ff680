// rmsq_norm_bwd.cuh -- layer norm's backward pass.
//
//   xhat = (s - mean) * rstd,  w = gamma + offset,  g = dy * w
//   ds     = rstd * (g - <g> - xhat * <g * xhat>) + dres        <.>: mean over the row
//   dgamma = sum over rows of dy * xhat,  dbeta = sum over rows of dy
//
// Bound by HBM: dy, s (and dres) are read once and ds written once. Persistent CTAs walk the rows;
// a thread owns the same columns in every row, so its shares of dgamma and dbeta stay in fp32
// registers until the end, when each CTA (cluster) writes one partial row of both. A second kernel
// adds the partials in a fixed order: no atomics, the same bits every time.
//
// The rows come through a ring of shared-memory slots (RowRing), so loads of the next rows run while a
// row is reduced. A row is read from its slot twice (sums, then ds) rather than held in registers,
// which the column sums need.
//
// A CTA holds several row groups of T threads when rows are short; rows wider than 16 KB are split
// over a cluster whose CTAs exchange the two row sums.
//
// Measured (GB300, of the copy rate of 6787 GB/s; with dres where it says so): 16384 x 8192 fp16 with dres
// 175 us (0.90), 16384 x 4096 bf16 with dres 92.4 (0.86), 32768 x 2048 72.5 (0.82), 8192 x 16384 164 (0.72),
// 2048 x 65536 209 (0.57), fp32 4096 x 16384 124 (0.95). Wide rows are bound by the SMs that clusters of 8
// leave idle (120 of 152 work) and by the latency of a pair of rows in 11 warps: sums formed a pair ahead of
// the exchange gave 3 % at 65536 and cost 4 % at 8192. Rows off 16-byte boundaries are bound by checked and
// unaligned accesses (5003 x 2051 fp32 32, 0.57). Row groups add their column sums side by side: one after
// another, 4000 x 512 took 26 us, not 10.
#pragma once

#include "rmsq_norm.cuh"
#include "rmsq_ops_plan.h"

namespace rmsq {

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

struct NormBwdParams {
    RowTensors r;            // dy, s, and dres where there is one
    const void* gamma;
    const float* mean;
    const float* rstd;
    void* ds;
    float* part;             // [parts][2][hidden]
    unsigned int* err;
    float offset;
    int T;                   // threads per row group
    int groups;              // row groups per CTA
    uint32_t wait, drain;    // bounds of waits, and of what a stopping CTA has in flight (rmsq_ops_plan.h)
};

struct NormBwdReduceParams {
    const float* part;
    void* dgamma;
    void* dbeta;
    int parts;
    int hidden;
    int dt;                  // type of dgamma and dbeta
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
    // 1000 cycles, which a working warp would keep its group waiting for). At its end it waits (bounded)
    // for the copies in flight, so that they end before the CTA does, whichever thread's wait ran out.
    __device__ __forceinline__ void feed(const Rows& rows, uint32_t limit, uint32_t drain, unsigned int* err) const
    {
        const uint64_t policy = l2_evict_normal_policy();
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
        bool drained = true;
        for (int j = i > r.stages ? i - r.stages : 0; j < i; ++j)
            drained &= mbar_wait<SCOPE_CTA>(full(j % r.stages), (j / r.stages) & 1, drain);
        if (i < rows.n || !drained) atomicOr(err, drained ? ERRF_WAIT_TIMEOUT : ERRF_WAIT_TIMEOUT | ERRF_DRAIN_TIMEOUT);
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
// warp would have to join; every wait is bounded. A CTA whose wait ran out sends no more, so the others'
// waits run out too, and it stays (linger) until what they had sent it has landed.
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
    __device__ __forceinline__ bool receive(int lane, int flip, int phase, uint32_t limit, float4& v) const
    {
        const bool ok = mbar_wait<SCOPE_CLUSTER>(bars + 8 * flip, phase, limit);
        v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (lane < nc) {
            const uint4 w = ld_shared_v4(slots + (flip * 16 + lane) * 16);
            v = make_float4(__uint_as_float(w.x), __uint_as_float(w.y), __uint_as_float(w.z), __uint_as_float(w.w));
        }
        return ok;
    }
    // After the cluster's last barrier, when nobody sends any more: time for what was sent to land, which
    // takes about a microsecond. A CTA that received every row's sums has nothing under way to it.
    static __device__ __forceinline__ void linger()
    {
        const uint32_t t0 = time_units();
        while (time_units() - t0 < 1000) __nanosleep(100000);
    }
};

constexpr int kRingSlice = 16384;             // bytes of a tensor's row per CTA at most

// Elements of a row per thread: 8, 16 or 24, and the warps of a CTA that work on rows then (one more
// copies). Registers are dealt to a quarter of the SM's warps each: 16 warps get 128, 12 get 168.
constexpr int row_warps(int elems) { return elems <= 16 ? 15 : 11; }

// Shared memory before the ring: barriers, the groups' warp sums (of two iterations in turn), the
// cluster's sums.
constexpr int kBwdHead = (kRingBars + 2 * 16 * 16 + ClusterSums::BYTES + 127) / 128 * 128;

// CLUSTER: the row may be split over a cluster. (Leaving its code out where it cannot be gives 3 % with 16
// elements a thread: 16384 x 4096 bf16 with dres 92 us against 95. With 24 the registers are dealt out worse
// without it, 16384 x 8192 fp16 with dres 193 us against 176, so those have it always.)
template <int DT, int E, bool FULL, bool EDGE, bool CLUSTER>
__global__ void __launch_bounds__(32 * row_warps(E) + 32) rmsq_norm_bwd_kernel(const __grid_constant__ NormBwdParams p)
{
    using D = Deal<DT, E>;
    using S = Scalar<DT>;
    using TT = typename S::T;
    constexpr int VW = D::VW, NC = D::NC, PV = D::PV;
    extern __shared__ __align__(128) unsigned char smem[];

    float4* const red = reinterpret_cast<float4*>(smem + kRingBars);
    unsigned char* const cluster_part = reinterpret_cast<unsigned char*>(red + 32);

    const int T = p.T, group = threadIdx.x / T, thread = threadIdx.x % T;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int group_warps = T >> 5, warp0 = group * group_warps;
    const int nc = CLUSTER ? static_cast<int>(cluster_size()) : 1, rank = CLUSTER ? static_cast<int>(cluster_rank()) : 0;

    // a lane of the copying warp stands for the group it feeds
    const bool copies = threadIdx.x >= T * p.groups;
    const int mine = copies ? (lane < p.groups ? lane : 0) : group;
    const Rows rows(mine, p.groups, p.r.rows);
    const int c0 = rank * p.r.slice;
    const int shift = EDGE ? static_cast<int>(static_cast<long long>(rows.first) * p.r.hidden % VW) : 0;
    const int lo = max(shift - c0, 0), hi = FULL ? p.r.slice : max(min(shift + p.r.hidden - c0, p.r.slice), 0);
    const RowRing<DT, EDGE> ring{p.r, c0, lo, hi, shift, smem_u32(smem) + mine * 2 * kRingStages * 8,
                                 smem_u32(smem + kBwdHead) + mine * p.r.stages * p.r.ntens * p.r.slot};
    const ClusterSums sums{smem_u32(cluster_part), smem_u32(cluster_part + 16), nc, rank};
    const bool has_res = p.r.ntens == 3;

    if (copies && lane < p.groups) {
        ring.init(group_warps);
        if (CLUSTER) sums.init();
        fence_mbar_init();
        fence_proxy_async_smem();
    }
    __syncthreads();
    if (CLUSTER && nc > 1) cluster_sync();                   // the other CTAs' barriers are set up
    pdl_wait();
    if (copies) {
        if (lane < p.groups) ring.feed(rows, p.wait, p.drain, p.err);
        return;
    }
    const int workers = T * p.groups;

    float2 acc_g[E / 2], acc_b[E / 2];
    Held<DT, E, EDGE> w;                          // gamma, in its own type
    w.load(static_cast<const TT*>(p.gamma) + (c0 + lo - shift), thread, T, lo, hi);
#pragma unroll
    for (int e = 0; e < E / 2; ++e) acc_g[e] = acc_b[e] = make_float2(0.f, 0.f);

    // (the minimum changes nothing but keeps the limit in a register: read from the parameters where it is
    // used, 16384 x 4096 bf16 with dres takes 94.2 us, so 92.5)
    const uint32_t limit = min(p.wait, kWaitMost);
    const float inv_h = 1.0f / static_cast<float>(p.r.hidden);
    bool dead = false;                            // a wait ran out: finish without waiting again
    int stage = 0, phase = 0;
    int flip = 0;
    const Part<DT, E, FULL, EDGE> share(thread, T, lo, hi);
    // The thread's vector c, at column k, of tensor i, 0 outside the row.
    auto load = [&](int c, int slot, int i, int k, float2 (&f)[PV]) {
        Elem<DT>::pairs(share.in(c, k) ? ring.vec(slot, i, k) : make_uint4(0, 0, 0, 0), f);
        if (!share.whole(c)) clear_outside(f, k, lo, hi);
    };
    const float2 offset = splat(p.offset);
    // the statistics of the next two rows, loaded an iteration ahead
    float next_mean[2], next_rstd[2];
    auto ahead = [&](int i) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int row = rows.first + min(i + r, rows.n - 1) * rows.stride;
            next_mean[r] = rows.n > 0 ? p.mean[row] : 0.f;
            next_rstd[r] = rows.n > 0 ? p.rstd[row] : 0.f;
        }
    };
    ahead(0);
    // Two rows at a time, so that one barrier and one round of shuffles serve both. Every CTA of a
    // cluster, and every thread of a group, runs the same iterations.
    for (int i = 0; i < rows.n; i += 2) {
        // opaque to the compiler, which would keep every element's address in registers across rows
        int t = thread;
        asm volatile("" : "+r"(t));
        const int pair = rows.n - i < 2 ? 1 : 2;
        const float mean[2] = {next_mean[0], next_mean[1]}, rstd[2] = {next_rstd[0], next_rstd[1]};
        float s1[2] = {0.f, 0.f}, s2[2] = {0.f, 0.f};
        ahead(i + 2);
        // (one row's code, not unrolled: both rows' operands at once take more registers than there are)
#pragma unroll 1
        for (int r = 0; r < pair; ++r) {
            if (!dead && !mbar_wait<SCOPE_CTA>(ring.full(stage + r), phase, limit)) dead = true;
            w.pin();
            const float2 m = splat(r ? -mean[1] : -mean[0]), rs = splat(r ? rstd[1] : rstd[0]);
            float2 a1 = make_float2(0.f, 0.f), a2 = a1;
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const int k = D::col(c, t, T);
                float2 dy[PV], s[PV];
                load(c, stage + r, 0, k, dy);
                load(c, stage + r, 1, k, s);
#pragma unroll
                for (int j = 0; j < PV; ++j) {
                    const int e = c * PV + j;
                    const float2 xh = mul2(add2(s[j], m), rs), g = mul2(dy[j], add2(w.pair(e), offset));
                    a1 = add2(a1, g);
                    a2 = fma2(g, xh, a2);
                    acc_g[e] = fma2(dy[j], xh, acc_g[e]);
                    acc_b[e] = add2(acc_b[e], dy[j]);
                }
            }
            if (r) {
                s1[1] = a1.x + a1.y;
                s2[1] = a2.x + a2.y;
            } else {
                s1[0] = a1.x + a1.y;
                s2[0] = a2.x + a2.y;
            }
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            s1[r] = warp_sum(s1[r]);
            s2[r] = warp_sum(s2[r]);
        }
        if (T > 32) {
            if (lane == 0) red[flip * 16 + warp] = make_float4(s1[0], s2[0], s1[1], s2[1]);
            group_sync(group, T);
            const float4 q = lane < group_warps ? red[flip * 16 + warp0 + lane] : make_float4(0.f, 0.f, 0.f, 0.f);
            s1[0] = warp_sum(q.x);
            s2[0] = warp_sum(q.y);
            s1[1] = warp_sum(q.z);
            s2[1] = warp_sum(q.w);
        }
        if (CLUSTER && nc > 1) {
            float4 q;
            // (a lane whose wait ran out sends no more: its arrival could fall into the phase it did not see end)
            if (warp == 0 && !dead) sums.send(lane, flip, make_float4(s1[0], s2[0], s1[1], s2[1]));
            if (!sums.receive(lane, flip, (i >> 2) & 1, dead ? 0 : limit, q)) dead = true;
            s1[0] = warp_sum(q.x);
            s2[0] = warp_sum(q.y);
            s1[1] = warp_sum(q.z);
            s2[1] = warp_sum(q.w);
        }
#pragma unroll 1
        for (int r = 0; r < pair; ++r) {
            const int row = rows.first + (i + r) * rows.stride;
            w.pin();
            TT* const out = static_cast<TT*>(p.ds) + ring.origin(row);
            const float2 m = splat(r ? -mean[1] : -mean[0]), rs = splat(r ? rstd[1] : rstd[0]);
            const float2 n1 = splat((r ? s1[1] : s1[0]) * -inv_h), n2 = splat((r ? s2[1] : s2[0]) * -inv_h);
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const int k = D::col(c, t, T);
                if (share.in(c, k)) {
                    float2 dy[PV], s[PV], d[PV];
                    load(c, stage + r, 0, k, dy);
                    load(c, stage + r, 1, k, s);
                    if (has_res) {
                        load(c, stage + r, 2, k, d);
                    } else {
#pragma unroll
                        for (int j = 0; j < PV; ++j) d[j] = make_float2(0.f, 0.f);
                    }
#pragma unroll
                    for (int j = 0; j < PV; ++j) {
                        const float2 xh = mul2(add2(s[j], m), rs), g = mul2(dy[j], add2(w.pair(c * PV + j), offset));
                        d[j] = fma2(rs, fma2(xh, n2, add2(g, n1)), d[j]);
                    }
                    const uint4 raw = pack_pairs<DT>(d);
                    if (share.whole(c)) st_v4(out + k, raw);
                    else store_inside<DT>(out, raw, k, lo, hi);
                }
            }
        }
        __syncwarp();
        if (lane == 0) {                          // the warp has read the slots
            mbar_arrive(ring.empty(stage));
            if (pair == 2) mbar_arrive(ring.empty(stage + 1));
        }
        flip ^= 1;
        stage += 2;
        if (stage == p.r.stages) {
            stage = 0;
            phase ^= 1u;
        }
    }

    if (dead && lane == 0) atomicOr(p.err, ERRF_WAIT_TIMEOUT);

    const auto workers_sync = [&]() { asm volatile("bar.sync 15, %0;" ::"r"(workers) : "memory"); };
    const auto acc = [](const float2* a, int e) { return e & 1 ? a[e / 2].y : a[e / 2].x; };
    // ---- partial rows: the groups' sums side by side in the ring's memory, then added in group order ----
    workers_sync();
    float* const part = p.part + static_cast<long long>(cluster_id()) * 2 * p.r.hidden + (c0 + lo - shift);
    float* const sums_all = reinterpret_cast<float*>(smem + kBwdHead);
    float* const own = p.groups == 1 ? part : sums_all + group * 2 * p.r.slice;
    const int other = p.groups == 1 ? p.r.hidden : p.r.slice;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int k = D::col(c, thread, T);
#pragma unroll
        for (int j = 0; j < VW; ++j)
            if (k + j >= lo && k + j < hi) {
                own[k + j - lo] = acc(acc_g, c * VW + j);
                own[other + k + j - lo] = acc(acc_b, c * VW + j);
            }
    }
    if (p.groups > 1) {
        workers_sync();
        for (int k = threadIdx.x; k < 2 * (hi - lo); k += workers) {
            const bool beta = k >= hi - lo;
            const int e = beta ? k - (hi - lo) : k, at = beta ? p.r.slice + e : e;
            float a = 0.f;
            for (int g = 0; g < p.groups; ++g) a += sums_all[g * 2 * p.r.slice + at];
            part[beta ? p.r.hidden + e : e] = a;
        }
    }
    if (CLUSTER && nc > 1) {
        cluster_sync();                                      // nobody sends to a CTA that has left
        if (dead) ClusterSums::linger();
    }
}

// dgamma and dbeta from the partial rows: 32 columns per CTA, 16 threads share a column's partials
// and their sums are added in thread order.
static __global__ void __launch_bounds__(512) rmsq_norm_bwd_reduce_kernel(const NormBwdReduceParams p)
{
    __shared__ float sum[16][33];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + tx;          // of 2 * hidden
    pdl_wait();
    float a = 0.f;
    if (col < 2 * p.hidden)
        for (int i = ty; i < p.parts; i += 16) a += p.part[static_cast<long long>(i) * 2 * p.hidden + col];
    sum[ty][tx] = a;
    __syncthreads();
    if (ty == 0 && col < 2 * p.hidden) {
        a = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) a += sum[i][tx];
        void* const out = col < p.hidden ? p.dgamma : p.dbeta;
        const int k = col < p.hidden ? col : col - p.hidden;
        if (out != nullptr) {
            if (p.dt == DT_F32) static_cast<float*>(out)[k] = a;
            else static_cast<uint16_t*>(out)[k] = p.dt == DT_BF16 ? Scalar<DT_BF16>::put(a)
                                                                 : Scalar<DT_FP16>::put(a);
        }
    }
}

}  // namespace rmsq
