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
// The rows come through a ring of shared-memory slots filled by bulk copies (cp.async.bulk +
// mbarrier), so loads of the next rows run while a row is reduced. A row is read from its slot
// twice (sums, then ds) rather than held in registers, which the column sums need. Rows that do
// not start on 16-byte boundaries are copied from the boundary below; the last bytes of the
// tensors, which no whole 16-byte piece covers, are read directly.
//
// A CTA holds several row groups of T threads when rows are short; rows too wide for 512 threads
// of 16 elements are split over a cluster whose CTAs exchange the two row sums.
#pragma once

#include "rmsq_norm.cuh"

namespace rmsq {

constexpr int kBwdThreads = 512;
constexpr int kBwdMaxStages = 8;

struct NormBwdParams {
    const void* in[3];       // dy, s, dres (or null)
    const void* gamma;
    const float* mean;
    const float* rstd;
    void* ds;
    float* part;             // [parts][2][hidden]
    unsigned int* err;
    long long rows;
    int hidden;
    int slice;               // elements per CTA of a row
    float offset;
    int T;                   // threads per row group
    int groups;              // row groups per CTA
    int stages;              // ring slots per group
    int slot;                // bytes of one tensor's row in a slot (multiple of 16)
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

// Shared memory before the ring: mbarriers of every slot, the groups' warp sums (two rows in
// turn), the cluster's exchange slots (two rows in turn).
constexpr int kBwdHead = kBwdMaxStages * 16 * 8 + 2 * 16 * 8 + 2 * 16;

__device__ __forceinline__ void group_sync(int group, int T)
{
    if (T == 32) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(T) : "memory");
}

template <int DT, int E, bool VEC>
__global__ void __launch_bounds__(kBwdThreads) rmsq_norm_bwd_kernel(const NormBwdParams p)
{
    using D = Deal<DT, E, VEC>;
    using S = Scalar<DT>;
    using TT = typename S::T;
    constexpr int VW = D::VW, NC = D::NC, ES = sizeof(TT);
    extern __shared__ __align__(128) unsigned char smem[];

    uint64_t* const bars = reinterpret_cast<uint64_t*>(smem);
    float2* const red = reinterpret_cast<float2*>(smem + kBwdMaxStages * 16 * 8);
    float4* const xch = reinterpret_cast<float4*>(smem + kBwdMaxStages * 16 * 8 + 2 * 16 * 8);
    unsigned char* const ring = smem + kBwdHead;

    const int T = p.T, group = threadIdx.x / T, t = threadIdx.x % T;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int group_warps = T >> 5, warp0 = group * group_warps;
    const uint32_t nc = cluster_size(), rank = cluster_rank();
    const int c0 = static_cast<int>(rank) * p.slice;
    int len = p.hidden - c0;
    len = len < 0 ? 0 : len < p.slice ? len : p.slice;
    const int ntens = p.in[2] != nullptr ? 3 : 2;
    const uint32_t slot_bytes = static_cast<uint32_t>(p.slot) * ntens;
    unsigned char* const my_ring = ring + static_cast<size_t>(group) * p.stages * slot_bytes;
    const long long first = static_cast<long long>(cluster_id()) * p.groups + group;
    const long long stride = static_cast<long long>(cluster_count()) * p.groups;
    const long long total = p.rows * p.hidden * ES;      // bytes of a tensor

    if (t == 0)
        for (int i = 0; i < p.stages; ++i) mbar_init(smem_u32(&bars[group * kBwdMaxStages + i]), 1);
    fence_mbar_init();
    __syncthreads();
    pdl_wait();

    // One row's pieces of every tensor into a slot (one thread per group).
    const uint64_t policy = l2_evict_normal_policy();
    auto fetch = [&](long long row, int slot) {
        const long long b0 = (row * p.hidden + c0) * ES;
        const long long a0 = b0 & ~15LL;
        long long a1 = (b0 + static_cast<long long>(len) * ES + 15) & ~15LL;
        if (a1 > (total & ~15LL)) a1 = total & ~15LL;
        const uint32_t bytes = len > 0 && a1 > a0 ? static_cast<uint32_t>(a1 - a0) : 0u;
        const uint32_t bar = smem_u32(&bars[group * kBwdMaxStages + slot]);
        mbar_arrive_expect_tx(bar, bytes * ntens);
        if (bytes > 0)
            for (int i = 0; i < ntens; ++i)
                bulk_load(smem_u32(my_ring + slot * slot_bytes + i * p.slot),
                          static_cast<const unsigned char*>(p.in[i]) + a0, bytes, bar, policy);
    };

    float acc_g[E], acc_b[E], w[E];
    const TT* const gamma = static_cast<const TT*>(p.gamma) + c0;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int k = D::col(c, t, T);
#pragma unroll
        for (int j = 0; j < VW; ++j) {
            acc_g[c * VW + j] = acc_b[c * VW + j] = 0.f;
            w[c * VW + j] = k < len ? S::get(gamma[k + j]) + p.offset : 0.f;
        }
    }

    long long issued = first;                     // next row to fetch (thread t == 0)
    if (t == 0)
        for (int i = 0; i < p.stages && issued < p.rows; ++i, issued += stride) fetch(issued, i);

    const float inv_h = 1.0f / static_cast<float>(p.hidden);
    bool dead = false;                            // a wait ran out: finish without waiting again
    int slot = 0, phase = 0, flip = 0;
    long long done = 0;                           // rows finished by this group
    // every CTA of a cluster, and every thread of a group, runs the same iterations
    for (long long row = first; row < p.rows; row += stride) {
        const uint32_t bar = smem_u32(&bars[group * kBwdMaxStages + slot]);
        const float mean = p.mean[row], rstd = p.rstd[row];
        if (!dead && !mbar_wait<SCOPE_CTA>(bar, phase, wait_limit(p.timeout_ns))) dead = true;

        const unsigned char* const sl = my_ring + slot * slot_bytes;
        const long long b0 = (row * p.hidden + c0) * ES;
        const int shift = VEC ? 0 : static_cast<int>(b0 & 15);
        // elements of the slice that the copies brought (all but the tensor's last few)
        const int have = VEC ? len : static_cast<int>(((total & ~15LL) - b0) / ES);
        // vector / element k of tensor i
        auto get = [&](int i, int k, float* f) {
            const unsigned char* const a = sl + i * p.slot + shift + k * ES;
            if constexpr (VEC) {
                Elem<DT>::unpack(ld_shared_v4(smem_u32(a)), *reinterpret_cast<float(*)[VW]>(f));
            } else {
                f[0] = S::get(k < have ? *reinterpret_cast<const TT*>(a)
                                       : static_cast<const TT*>(p.in[i])[row * p.hidden + c0 + k]);
            }
        };

        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int k = D::col(c, t, T);
            if (k < len) {
                float dy[VW], s[VW];
                get(0, k, dy);
                get(1, k, s);
#pragma unroll
                for (int j = 0; j < VW; ++j) {
                    const int e = c * VW + j;
                    const float xh = (s[j] - mean) * rstd, g = dy[j] * w[e];
                    s1 += g;
                    s2 = fmaf(g, xh, s2);
                    acc_g[e] = fmaf(dy[j], xh, acc_g[e]);
                    acc_b[e] += dy[j];
                }
            }
        }
        s1 = warp_sum(s1);
        s2 = warp_sum(s2);
        if (T > 32) {
            if (lane == 0) red[flip * 16 + warp] = make_float2(s1, s2);
            group_sync(group, T);
            const float2 q = lane < group_warps ? red[flip * 16 + warp0 + lane] : make_float2(0.f, 0.f);
            s1 = warp_sum(q.x);
            s2 = warp_sum(q.y);
        } else {
            __syncwarp();
        }
        // the group has left the previous row's slot: refill it
        if (t == 0 && done > 0 && issued < p.rows && !dead) {
            fence_proxy_async_smem();
            fetch(issued, slot == 0 ? p.stages - 1 : slot - 1);
            issued += stride;
        }
        if (nc > 1) {
            if (threadIdx.x == 0) xch[flip] = make_float4(s1, s2, 0.f, 0.f);
            cluster_sync();
            const float4 q = lane < static_cast<int>(nc) ? ld_cluster_f4(smem_u32(&xch[flip]), lane)
                                                         : make_float4(0.f, 0.f, 0.f, 0.f);
            s1 = warp_sum(q.x);
            s2 = warp_sum(q.y);
        }
        s1 *= inv_h;
        s2 *= inv_h;

        TT* const out = static_cast<TT*>(p.ds) + row * p.hidden + c0;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int k = D::col(c, t, T);
            if (k < len) {
                float dy[VW], s[VW], d[VW];
                get(0, k, dy);
                get(1, k, s);
                if (ntens == 3) {
                    get(2, k, d);
                } else {
#pragma unroll
                    for (int j = 0; j < VW; ++j) d[j] = 0.f;
                }
#pragma unroll
                for (int j = 0; j < VW; ++j) {
                    const float xh = (s[j] - mean) * rstd, g = dy[j] * w[c * VW + j];
                    d[j] = fmaf(rstd, fmaf(-xh, s2, g - s1), d[j]);
                }
                if constexpr (VEC) st_v4(out + k, pack_vec<DT>(d));
                else out[k] = S::put(d[0]);
            }
        }
        flip ^= 1;
        ++done;
        if (++slot == p.stages) {
            slot = 0;
            phase ^= 1;
        }
    }

    if (dead) {
        if (lane == 0) atomicOr(p.err, ERRF_WAIT_TIMEOUT);
        // the copies in flight end before the CTA does
        if (t == 0) {
            bool drained = true;
            long long k = 0;
            for (long long r = first; r < issued; r += stride, ++k)
                if (issued - r <= stride * p.stages)
                    drained &= mbar_wait<SCOPE_CTA>(
                        smem_u32(&bars[group * kBwdMaxStages + static_cast<int>(k % p.stages)]),
                        static_cast<uint32_t>(k / p.stages) & 1u, wait_limit(4 * p.timeout_ns));
            if (!drained) atomicOr(p.err, ERRF_DRAIN_TIMEOUT);
        }
    }

    // ---- partial rows: the groups' sums in group order, through the ring's memory ----
    __syncthreads();
    float* const part = p.part + static_cast<long long>(cluster_id()) * 2 * p.hidden + c0;
    if (p.groups == 1) {
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int k = D::col(c, t, T);
#pragma unroll
            for (int j = 0; j < VW; ++j)
                if (k < len) {
                    part[k + j] = acc_g[c * VW + j];
                    part[p.hidden + k + j] = acc_b[c * VW + j];
                }
        }
    } else {
        float* const sum = reinterpret_cast<float*>(ring);
        for (int g = 0; g < p.groups; ++g) {
            if (g == group) {
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    const int k = D::col(c, t, T);
#pragma unroll
                    for (int j = 0; j < VW; ++j)
                        if (k < len) {
                            float& a = sum[k + j];
                            float& b = sum[len + k + j];
                            a = (g == 0 ? 0.f : a) + acc_g[c * VW + j];
                            b = (g == 0 ? 0.f : b) + acc_b[c * VW + j];
                        }
                }
            }
            __syncthreads();
        }
        for (int k = threadIdx.x; k < len; k += blockDim.x) {
            part[k] = sum[k];
            part[p.hidden + k] = sum[len + k];
        }
    }
    if (nc > 1) cluster_sync();   // exchange slots are read by the other CTAs until here
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
