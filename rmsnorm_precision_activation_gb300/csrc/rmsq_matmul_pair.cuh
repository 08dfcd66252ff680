// rmsq_matmul_pair.cuh -- the int8 product on the tensor cores for many tokens: a CTA pair per tile.
//
// As rmsq_matmul_tc_kernel, but two CTAs (a cluster of 2) share one MMA (cta_group::2) of 256 output
// channels by TOKENS tokens: each converts its own 128 channels into its TMEM and half of the tokens
// into its shared memory, and holds the sums of its channels for all of the tokens. Per product that
// halves the codes a CTA turns into fp16 and the shared memory the MMA reads, which bound the one-CTA
// kernel (shared memory moves 8-bit and 16-bit copies of both operands through one port).
//
// Tiles have 192 tokens, or 128 where those fill the SMs better, rather than 256: two accumulators then
// fit TMEM beside the operand stages, and reading one out (bound by the float-to-integer conversions, at
// 256 tokens 2500 cycles per 8192 of MMA) overlaps the next one's products. Measured (GB300, boost clock):
// 8192^3 in 622 to 634 us, 1770 to 1735 TFLOP/s, 0.93 to 0.91 of the measured burst rate of a library product
// in bf16 (665 us, 1650, under the power cap: 0.97 of its sustained rate); pairs of 128 tokens 720 us, of 160
// 679; 256 tokens with one accumulator 863.
//
// The leader (rank 0) issues the MMAs. Its op_full and acc_empty barriers count arrivals of both
// CTAs; its commits arrive in both. Copy rings are each CTA's own. The reading warps hold TOKENS / 2
// sums per thread, so registers move to them from the other warps (setmaxnreg).
#pragma once

#include "rmsq_matmul_tc.cuh"

namespace rmsq {

// Per tile width in tokens.
template <int TOKENS> struct PairShape {
    static constexpr int HALF = TOKENS / 2;                       // tokens whose codes a CTA brings and converts
    static constexpr int RAWS = 6;                                // code stages
    static constexpr int OPS = 4;                                 // operand stages
    static constexpr int RAW_A = kTcRows * kTcCodes;              // codes of 128 channels
    static constexpr int RAW = RAW_A + HALF * kTcCodes;           // and of half the tokens
    static constexpr int OP = HALF * kTcStep * 2;                 // half the tokens in fp16
    static constexpr int SMEM = 2048 + RAWS * RAW + OPS * OP;     // 1024 to align the ring, 1024 for barriers
    static_assert(RAW % 1024 == 0 && OP % 1024 == 0 && RAW_A % 1024 == 0, "swizzle atoms");
    static_assert(2 * TOKENS + OPS * 32 <= 512, "two accumulators and the operand stages fit TMEM");
    static_assert(SMEM > 116 * 1024 && SMEM <= 232448, "one CTA per SM");
};
// registers: 12 warps give up what 8 take; the launch has kPairRegs for every thread
constexpr int kPairRegs = 96, kPairRegsIssue = 32, kPairRegsConvert = 80, kPairRegsRead = 144;
static_assert(128 * kPairRegsIssue + 256 * (kPairRegsConvert + kPairRegsRead) <= kTcThreads * kPairRegs, "within the launch's registers");

// Arrive on the leader's barrier at this CTA's address bar. What the arrival publishes stays in this
// CTA's own shared memory and TMEM, where the MMA reads it: fence.proxy.async and tcgen05.fence before
// the arrival make it visible there, so the arrival need not release at cluster scope (which took about
// 1000 cycles behind the converting warps' stores: 863 us against 768 at 8192^3 when it was tried, in
// tiles of 256 tokens).
__device__ __forceinline__ void mbar_arrive_leader(uint32_t bar)
{
    asm volatile(
        "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, 0;\n\t"
        "mbarrier.arrive.shared::cluster.b64 _, [a];\n\t}" ::"r"(bar) : "memory");
}

// The same after tcgen05 operations alone, which tcgen05.fence orders: nothing else to release.
__device__ __forceinline__ void mbar_arrive_leader_relaxed(uint32_t bar)
{
    asm volatile(
        "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, 0;\n\t"
        "mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [a];\n\t}" ::"r"(bar) : "memory");
}

// Arrives on bar in both CTAs when every MMA this thread has issued is done.
__device__ __forceinline__ void tc_commit_pair(uint32_t bar)
{
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
        ::"r"(bar), "h"(static_cast<uint16_t>(3)) : "memory");
}

template <int TOKENS>
__global__ void __launch_bounds__(kTcThreads, 1) __cluster_dims__(2, 1, 1)
rmsq_matmul_pair_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_a,
                        const MatmulParams p, const TcTiles tiles)
{
    using S = PairShape<TOKENS>;
    constexpr int RAWS = S::RAWS, OPS = S::OPS, HALF = S::HALF;
    extern __shared__ unsigned char smem_raw[];
    __shared__ uint32_t tmem_slot;

    unsigned char* const smem = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    unsigned char* const raw = smem;
    unsigned char* const ops = smem + RAWS * S::RAW;
    const uint32_t bars = smem_u32(ops + OPS * S::OP);
    const uint32_t raw_full = bars, raw_empty = raw_full + 8 * RAWS;
    const uint32_t op_full = raw_empty + 8 * RAWS, op_empty = op_full + 8 * OPS;
    const uint32_t acc_full = op_empty + 8 * OPS, acc_empty = acc_full + 16, drain = acc_empty + 16;

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int rank = static_cast<int>(cluster_rank());

    const int steps = (p.k + kTcCodes - 1) / kTcCodes;      // code stages
    const long long ntiles = static_cast<long long>(tiles.n_tiles) * tiles.m_tiles;
    const long long first = cluster_id(), stride = cluster_count();

    // Code stage s of a tile into this CTA's ring (one thread).
    auto fetch = [&](uint32_t slot, int s, int tn, int tm) {
        const uint32_t full = raw_full + 8 * slot, dst = smem_u32(raw) + slot * S::RAW;
        mbar_arrive_expect_tx(full, S::RAW);
        tma_load_2d(dst, &map_w, s * kTcCodes, (tn * 2 + rank) * kTcRows, full);
        tma_load_2d(dst + S::RAW_A, &map_a, s * kTcCodes, tm * TOKENS + rank * HALF, full);
    };
    int started = 0;                          // stages of the first tile fetched ahead

    if (threadIdx.x == 0) {
        prefetch_map(&map_w);
        prefetch_map(&map_a);
        for (int i = 0; i < RAWS; ++i) {
            mbar_init(raw_full + 8 * i, 1);
            mbar_init(raw_empty + 8 * i, 8);
        }
        for (int i = 0; i < OPS; ++i) {
            mbar_init(op_full + 8 * i, 8);
            mbar_init(op_empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(acc_full + 8 * i, 1);
            mbar_init(acc_empty + 8 * i, 16);
        }
        mbar_init(drain, 1);
        fence_mbar_init();
        fence_proxy_async_smem();
        // the first loads run while the pair sets itself up
        pdl_wait_alone();
        int tn, tm;
        tc_tile(first, tiles, tn, tm);
        for (; started < RAWS && started < steps; ++started) fetch(started, started, tn, tm);
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&tmem_slot))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
        tc_fence_before();
    }
    __syncthreads();
    cluster_sync();                          // the other CTA's barriers are set up
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    const uint32_t tmem_a = tmem + 2 * TOKENS;      // operand stages of 32 columns behind the accumulators
    pdl_wait();

    // (the minima change nothing but keep the limits in registers: read from the parameters where they are
    // used, 512 x 8192 x 8192 takes 63.9 us, so 60.5)
    const uint32_t limit = min(p.wait, kWaitMost), drain_limit = min(p.drain, 2 * kWaitMost);
    bool ok = true;

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPairRegsIssue));
        if (warp == 0 && lane == 0) {
            long long it = 0;
            for (long long tile = first; tile < ntiles && ok; tile += stride) {
                int tn, tm;
                tc_tile(tile, tiles, tn, tm);
                for (int s = 0; s < steps; ++s, ++it) {
                    if (it < started) continue;
                    const uint32_t slot = static_cast<uint32_t>(it % RAWS);
                    ok = mbar_wait<SCOPE_CTA>(raw_empty + 8 * slot, (static_cast<uint32_t>(it / RAWS) & 1u) ^ 1u, limit);
                    if (!ok) break;
                    fetch(slot, s, tn, tm);
                }
            }
            // the copies in flight end before the CTA does, whichever role stopped waiting
            bool drained = true;
            for (long long i = it > RAWS ? it - RAWS : 0; i < it; ++i)
                drained &= mbar_wait<SCOPE_CTA>(raw_full + 8 * static_cast<int>(i % RAWS),
                                             static_cast<uint32_t>(i / RAWS) & 1u, drain_limit);
            if (!ok || !drained) atomicOr(p.err, drained ? ERRF_WAIT_TIMEOUT : ERRF_WAIT_TIMEOUT | ERRF_DRAIN_TIMEOUT);
        } else if (warp == 1 && rank == 0) {
            constexpr uint32_t idesc = (1u << 4) | ((TOKENS / 8u) << 17) | ((2u * kTcRows / 16u) << 24);
            const bool one = elect_one();
            const uint32_t desc0 = tc_desc_lo(smem_u32(ops));
            uint32_t slot = 0, phase = 0, chunks = 0;    // a code stage fills operand stages slot and slot + 1
            bool ready0 = false, ready1 = false;         // asked a stage ahead
            for (long long tile = first; tile < ntiles && ok; tile += stride) {
                int left = 0;                            // code stages until the read-out
                for (int s = 0; s < steps; ++s) {
                    const bool fresh = left == 0;
                    if (fresh) {
                        left = kTcChunk;
                        ok = mbar_wait<SCOPE_CTA>(acc_empty + 8 * (chunks & 1u), ((chunks >> 1) & 1u) ^ 1u, limit);
                        ++chunks;
                    }
                    const uint32_t buf = (chunks - 1) & 1u, acc = tmem + buf * TOKENS;
                    const bool tail = --left == 0 || s == steps - 1;
                    const uint32_t next = slot + 2 == OPS ? 0 : slot + 2, next_phase = slot + 2 == OPS ? phase ^ 1u : phase;
                    if (!ready0) ok = ok && mbar_wait<SCOPE_CTA>(op_full + 8 * slot, phase, limit);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) break;
                    tc_fence_after();
                    if (one) {
                        tc_mma_step<true>(acc, tmem_a + slot * 32, desc0 + slot * (S::OP / 16), idesc, fresh);
                        tc_commit_pair(op_empty + 8 * slot);
                    }
                    __syncwarp();
                    if (!ready1) ok = mbar_wait<SCOPE_CTA>(op_full + 8 * slot + 8, phase, limit);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) break;
                    tc_fence_after();
                    const bool peek0 = mbar_test<SCOPE_CTA>(op_full + 8 * next, next_phase);
                    const bool peek1 = mbar_test<SCOPE_CTA>(op_full + 8 * next + 8, next_phase);
                    if (one) {
                        tc_mma_step<true>(acc, tmem_a + slot * 32 + 32, desc0 + (slot + 1) * (S::OP / 16), idesc, false);
                        tc_commit_pair(op_empty + 8 * slot + 8);
                        if (tail) tc_commit_pair(acc_full + 8 * buf);
                    }
                    __syncwarp();
                    ready0 = __all_sync(0xFFFFFFFFu, peek0);
                    ready1 = __all_sync(0xFFFFFFFFu, peek1);
                    slot = next;
                    phase = next_phase;
                }
            }
            if (one) {
                tc_commit_pair(drain);
                if (!ok) atomicOr(p.err, ERRF_WAIT_TIMEOUT);
            }
        }
        __syncwarp();
    } else if (warp < 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPairRegsConvert));
        constexpr int PB = (HALF * 4 + 127) / 128;    // a thread's pieces of the tokens' HALF x 4
        const int wg = (warp - 4) >> 2, t = threadIdx.x & 127;
        const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;     // this warp's TMEM lanes, in bits 16+
        uint32_t rs = 0, rphase = 0, os = wg, ophase = 0;
        bool ready = false;                  // the next code stage, asked ahead
        for (long long tile = first; tile < ntiles && ok; tile += stride) {
            for (int s = 0; s < steps; ++s) {
                if (!ready) ok = mbar_wait<SCOPE_CTA>(raw_full + 8 * rs, rphase, limit);
                const uint32_t rnext = rs + 1 == RAWS ? 0 : rs + 1, rnext_phase = rs + 1 == RAWS ? rphase ^ 1u : rphase;
                const uint32_t ra = smem_u32(raw) + rs * S::RAW, rb = ra + S::RAW_A;
                const uint32_t ob = smem_u32(ops) + os * S::OP;
                // thread t: channel t, and its pieces of the tokens; all loads first, to overlap
                uint4 va[4], vb[PB];
#pragma unroll
                for (int c = 0; c < 4; ++c) va[c] = ld_shared_v4(ra + t * 128 + (((4 * wg + c) ^ (t & 7)) << 4));
#pragma unroll
                for (int j = 0; j < PB; ++j) {
                    const int i = j * 128 + t, r = i % HALF, c = i / HALF;
                    if (c < 4) vb[j] = ld_shared_v4(rb + r * 128 + (((4 * wg + c) ^ (r & 7)) << 4));
                }
                ok = ok && mbar_wait<SCOPE_CTA>(op_empty + 8 * os, ophase ^ 1u, limit);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                const bool peek = mbar_test<SCOPE_CTA>(raw_full + 8 * rnext, rnext_phase);
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < 4; c += 2) {
                    uint32_t h[16];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        codes_to_half(va[c + i].x, h[8 * i], h[8 * i + 1]);
                        codes_to_half(va[c + i].y, h[8 * i + 2], h[8 * i + 3]);
                        codes_to_half(va[c + i].z, h[8 * i + 4], h[8 * i + 5]);
                        codes_to_half(va[c + i].w, h[8 * i + 6], h[8 * i + 7]);
                    }
                    tmem_st_x16(tmem_a + lanes + os * 32 + c * 8, h);
                }
#pragma unroll
                for (int j = 0; j < PB; ++j) {
                    const int i = j * 128 + t, r = i % HALF, c = i / HALF;
                    if (c >= 4) continue;
                    uint4 lo, hi;
                    codes_to_half(vb[j].x, lo.x, lo.y);
                    codes_to_half(vb[j].y, lo.z, lo.w);
                    codes_to_half(vb[j].z, hi.x, hi.y);
                    codes_to_half(vb[j].w, hi.z, hi.w);
                    st_shared_v4(ob + r * 128 + (((2 * c) ^ (r & 7)) << 4), lo);
                    st_shared_v4(ob + r * 128 + (((2 * c + 1) ^ (r & 7)) << 4), hi);
                }
                fence_proxy_async_smem();
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(raw_empty + 8 * rs);
                    mbar_arrive_leader(op_full + 8 * os);
                }
                ready = __all_sync(0xFFFFFFFFu, peek);
                rs = rnext;
                rphase = rnext_phase;
                os += 2;
                if (os >= OPS) {
                    os -= OPS;
                    ophase ^= 1u;
                }
            }
        }
        if (!ok && lane == 0) atomicOr(p.err, ERRF_WAIT_TIMEOUT);
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kPairRegsRead));
        const int wg = (warp - 12) >> 2, row = threadIdx.x & 127;
        const uint32_t base = tmem + (static_cast<uint32_t>(warp & 3) << 21) + wg * HALF;
        uint32_t chunks = 0;
        for (long long tile = first; tile < ntiles && ok; tile += stride) {
            int acc[HALF];
#pragma unroll
            for (int i = 0; i < HALF; ++i) acc[i] = 0;
            for (int s = 0; s < steps; s += kTcChunk, ++chunks) {
                const uint32_t buf = chunks & 1u;
                ok = mbar_wait<SCOPE_CTA>(acc_full + 8 * buf, (chunks >> 1) & 1u, limit);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < HALF; c += 32) {
                    uint32_t v[32];
                    tmem_ld_x16(base + buf * TOKENS + c, v);
                    if (c + 16 < HALF) tmem_ld_x16(base + buf * TOKENS + c + 16, v + 16);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (c + j < HALF) acc[c + j] += __float2int_rn(__uint_as_float(v[j]));
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_leader_relaxed(acc_empty + 8 * buf);
            }
            if (!ok) break;
            int tn, tm;
            tc_tile(tile, tiles, tn, tm);
            const int n = (tn * 2 + rank) * kTcRows + row, m0 = tm * TOKENS + wg * HALF;
            if (n < p.n) {
                const float ws = p.w_scale[n], b = p.bias ? load_as(p.bias, n, p.dt) : 0.f;
                const float* const as = p.a_scale + m0;
                const int left = static_cast<int>(p.m) - m0, es = p.dt == DT_F32 ? 4 : 2;
                char* out = static_cast<char*>(p.out) + (m0 * p.n + n) * es;
                const long long pitch = p.n * es;
#pragma unroll
                for (int i = 0; i < HALF; ++i, out += pitch)
                    if (i < left) store_as(out, 0, p.dt, scaled(acc[i], as[i], ws, b, p.bias));
            }
        }
        if (!ok && lane == 0) atomicOr(p.err, ERRF_WAIT_TIMEOUT);
    }

    tc_fence_before();
    __syncthreads();
    // the MMAs in flight end, and their arrivals come, before either CTA frees its TMEM or leaves,
    // whichever role stopped waiting
    if (threadIdx.x == 0 && !mbar_wait<SCOPE_CTA>(drain, 0, drain_limit))
        atomicOr(p.err, ERRF_WAIT_TIMEOUT | ERRF_DRAIN_TIMEOUT);
    cluster_sync();                          // no CTA leaves while the other arrives on its barriers
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem));
    }
}

}  // namespace rmsq
