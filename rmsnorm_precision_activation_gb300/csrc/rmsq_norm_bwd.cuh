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
#pragma once

#include "rmsq_norm.cuh"

namespace rmsq {

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
    unsigned long long timeout_ns;
};

struct NormBwdReduceParams {
    const float* part;
    void* dgamma;
    void* dbeta;
    int parts;
    int hidden;
    int dt;                  // type of dgamma and dbeta
};

// Elements of a row per thread: 8, 16 or 24, and the warps of a CTA that work on rows then (one more
// copies). Registers are dealt to a quarter of the SM's warps each: 16 warps get 128, 12 get 168.
constexpr int row_warps(int elems) { return elems <= 16 ? 15 : 11; }

// Shared memory before the ring: barriers, the groups' warp sums (of two iterations in turn), the
// cluster's sums.
constexpr int kBwdHead = (kRingBars + 2 * 16 * 16 + ClusterSums::BYTES + 127) / 128 * 128;

template <int DT, int E, bool FULL, bool EDGE>
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
    const int nc = static_cast<int>(cluster_size()), rank = static_cast<int>(cluster_rank());

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
        sums.init();
        fence_mbar_init();
        fence_proxy_async_smem();
    }
    __syncthreads();
    if (nc > 1) cluster_sync();                   // the other CTAs' barriers are set up
    pdl_wait();
    if (copies) {
        if (lane < p.groups) ring.feed(rows, p.timeout_ns, p.err);
        return;
    }
    const int workers = T * p.groups;

    float2 acc_g[E / 2], acc_b[E / 2];
    Held<DT, E, EDGE> w;                          // gamma, in its own type
    w.load(static_cast<const TT*>(p.gamma) + (c0 + lo - shift), thread, T, lo, hi);
#pragma unroll
    for (int e = 0; e < E / 2; ++e) acc_g[e] = acc_b[e] = make_float2(0.f, 0.f);

    const uint32_t limit = wait_limit(p.timeout_ns);
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
            const int row = rows.first + (i + r) * rows.stride;
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
        if (nc > 1) {
            float4 q;
            if (warp == 0) sums.send(lane, flip, make_float4(s1[0], s2[0], s1[1], s2[1]));
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
    // ---- partial rows: the groups' sums in group order, through the ring's memory ----
    workers_sync();
    float* const part = p.part + static_cast<long long>(cluster_id()) * 2 * p.r.hidden + (c0 + lo - shift);
    float* const sum = reinterpret_cast<float*>(smem + kBwdHead);
    for (int g = 0; g < p.groups; ++g) {
        if (g == group) {
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const int k = D::col(c, thread, T);
#pragma unroll
                for (int j = 0; j < VW; ++j)
                    if (k + j >= lo && k + j < hi) {
                        const int e = k + j - lo;
                        const float a = acc(acc_g, c * VW + j), b = acc(acc_b, c * VW + j);
                        if (p.groups == 1) {
                            part[e] = a;
                            part[p.r.hidden + e] = b;
                        } else {
                            sum[e] = (g == 0 ? 0.f : sum[e]) + a;
                            sum[p.r.slice + e] = (g == 0 ? 0.f : sum[p.r.slice + e]) + b;
                        }
                    }
            }
        }
        if (p.groups > 1) workers_sync();
    }
    if (p.groups > 1)
        for (int k = threadIdx.x; k < hi - lo; k += workers) {
            part[k] = sum[k];
            part[p.r.hidden + k] = sum[p.r.slice + k];
        }
    if (nc > 1) cluster_sync();                   // nobody sends to a CTA that has left
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
