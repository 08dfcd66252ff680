// rmsq_fp4_pair.cuh -- the 4-bit product on the tensor cores for many tokens: a CTA pair per tile.
//
// As rmsq_fp4_tile_kernel, but two CTAs (a cluster of 2) share one MMA (cta_group::2) of 256 output channels by 256 tokens:
// each brings its own 128 channels, half of the tokens, its channels' scales and all of the tokens' (both
// tensor cores multiply by all columns), and holds the sums of its channels for all of the tokens.
//
// What bounds it is the power that the GPU may take (8192^3 runs at 1.8 GHz instead of 2.07, and at 1.6 where products follow
// one another), then how far the loads run ahead: a stage (256 elements of k, 38 KB a CTA) is 512 cycles of MMA, and from
// the MMAs that free a slot to the next ones that can use it pass about 2500 (word to the loading warps, the load, word
// to the MMA warp, its queue). 8192^3 takes 270 000 cycles, the MMAs alone 229 000. With five slots instead of six: 155 us instead
// of 150, with four 178; with three quarters of the MMAs 132. So
//   - the copies of both CTAs arrive on the leader's barrier themselves (passed on by a warp of the other CTA instead:
//     5 us more at 8192^3; that warp's arrival with release at cluster scope takes 1400 cycles: 357 us);
//   - codes have six slots, which leaves room for five of scales. Those are free earlier, once copied to TMEM: the
//     commit that follows a stage's scale copies and precedes its MMAs frees the codes of the stage before and the scales of
//     this one, so one barrier serves both;
//   - what runs per stage runs in converged warps that one lane issues from (a divergent loop takes 280 cycles to
//     start a stage's four loads, this one 120).
//
// TMEM has no room for two accumulators of 256 columns beside the scales, so they overlap by 96 columns: tiles take the
// columns from 0 and from 160 on in turn, the reading warps empty the shared columns first, and the next tile's
// products start when those are free.
//
//   warp 0       TMA loads into this CTA's slots
//   warp 1       rank 0: issues the copies of the scales and the MMAs
//   warp 2       where k ends inside an MMA's 64 elements: the scales of that end, the padding's cleared
//   warps 4-11   read the accumulator and write the output: two warps per 32 channels, taking every other 32 tokens
#pragma once

#include <type_traits>

#include "rmsq_fp4.cuh"
#include "rmsq_matmul_pair.cuh"

namespace rmsq {

constexpr int kFp4PairThreads = 384;
constexpr int kFp4PairTokens = 256;

template <bool NV> struct Fp4PairShape {
    static constexpr int CODES_W = kFp4Rows * kFp4Step / 2, CODES = 2 * CODES_W;      // as many tokens' as channels'
    static constexpr int SCALES_W = fp4_tiles<NV>() * kFp4ScaleTile, SCALES = 3 * SCALES_W;
    static constexpr int SLOTS = 6, SCALE_SLOTS = SLOTS - 1;
    static constexpr int AT_SCALES = SLOTS * CODES, AT_TAIL = AT_SCALES + SCALE_SLOTS * SCALES, AT_BARS = AT_TAIL + 3 * kFp4ScaleTile;
    static constexpr int SMEM = 1024 + AT_BARS + 256;                 // 1024 to align the codes
    static constexpr int SECOND = 160;                                // columns: the second accumulator's first
    static constexpr int COL_S = SECOND + 256, COLS_S = 4 * fp4_tiles<NV>() * 3;
    static_assert(COL_S + 2 * COLS_S <= 512, "accumulators and two stages' scales fit TMEM");
    static_assert(SMEM > 116 * 1024 && SMEM <= 232448, "one CTA per SM");
    static_assert(8 * (2 * SLOTS + 5) <= 256, "barriers");
};

// As tma_load_2d, arriving on a barrier of this CTA or of the pair's other one (bar: its address in the cluster).
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
        ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

// Address, in the cluster, of what lies at addr in the leader's shared memory.
__device__ __forceinline__ uint32_t leader_addr(uint32_t addr)
{
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(addr));
    return a;
}

template <bool NV>
__global__ void __launch_bounds__(kFp4PairThreads, 1) __cluster_dims__(2, 1, 1)
rmsq_fp4_pair_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_a,
                     const __grid_constant__ CUtensorMap map_sw, const __grid_constant__ CUtensorMap map_sa, const Fp4Params p,
                     const TcTiles tiles, const void* scales_w, const void* scales_a)
{
    using S = Fp4PairShape<NV>;
    constexpr int SLOTS = S::SLOTS, SCALE_SLOTS = S::SCALE_SLOTS;
    extern __shared__ unsigned char smem_raw[];
    __shared__ uint32_t tmem_slot;

    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t full = base + S::AT_BARS, empty = full + 8 * SLOTS, acc_full = empty + 8 * SLOTS;
    const uint32_t acc_free = acc_full + 16, tail_full = acc_free + 8, drain = tail_full + 8;

    const int lane = threadIdx.x & 31, warp = fp4_warp();
    const int rank = static_cast<int>(cluster_rank());

    const int steps = (p.k + kFp4Step - 1) / kFp4Step;
    const long long ntiles = static_cast<long long>(tiles.n_tiles) * tiles.m_tiles;
    const long long first = cluster_id(), stride = cluster_count();
    const bool tail = p.k % 64 != 0;              // the last MMA's 64 elements end half way

    // Stage s of a tile (one thread). The leader's barrier counts the bytes of both CTAs.
    auto fetch = [&](uint32_t slot, uint32_t scale_slot, int s, int tn, int tm) {
        const uint32_t bar = leader_addr(full + 8 * slot);
        if (rank == 0) mbar_arrive_expect_tx(full + 8 * slot, 2 * (S::CODES + S::SCALES));
        const uint32_t dst = base + slot * S::CODES, scales = base + S::AT_SCALES + scale_slot * S::SCALES;
        tma_load_2d_pair(dst, &map_w, s * (kFp4Step / 2), (tn * 2 + rank) * kFp4Rows, bar);
        tma_load_2d_pair(dst + S::CODES_W, &map_a, s * (kFp4Step / 2), tm * kFp4PairTokens + rank * (kFp4PairTokens / 2), bar);
        tma_load_2d_pair(scales, &map_sw, s * (S::SCALES_W / 8), tn * 2 + rank, bar);
        tma_load_2d_pair(scales + S::SCALES_W, &map_sa, s * (S::SCALES_W / 8), tm * 2, bar);
    };

    if (threadIdx.x == 0) {
        prefetch_map(&map_w);
        prefetch_map(&map_a);
        prefetch_map(&map_sw);
        prefetch_map(&map_sa);
        for (int i = 0; i < SLOTS; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) mbar_init(acc_full + 8 * i, 1);
        mbar_init(acc_free, 16);
        mbar_init(tail_full, 2);
        mbar_init(drain, 1);
        fence_mbar_init();
        fence_proxy_async_smem();
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
    pdl_wait();

    const uint32_t limit = min(p.wait, kWaitMost), drain_limit = min(p.drain, 2 * kWaitMost);
    bool ok = true;

    if (warp == 0) {
        const bool one = elect_one();
        uint32_t slot = 0, phase = 0, scale_slot = 0;
        long long it = 0;
        for (long long tile = first; tile < ntiles && ok; tile += stride) {
            int tn, tm;
            tc_tile(tile, tiles, tn, tm);
            for (int s = 0; s < steps; ++s, ++it) {
                // (a slot's codes are free from the start; the last slot's first word is of the first stage's scales)
                ok = mbar_wait<SCOPE_CTA>(empty + 8 * slot, slot == SLOTS - 1 ? phase : phase ^ 1u, limit);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                if (one) fetch(slot, scale_slot, s, tn, tm);
                __syncwarp();
                if (++scale_slot == SCALE_SLOTS) scale_slot = 0;
                if (++slot == SLOTS) {
                    slot = 0;
                    phase ^= 1u;
                }
            }
        }
        if (lane == 0) {
            // The copies in flight end before a CTA does, whichever role stopped waiting: the leader waits for both
            // CTAs' (for the whole bound, where the other one started fewer), and the other one for the leader.
            bool drained = true;
            for (long long i = it > SLOTS ? it - SLOTS : 0; rank == 0 && i < it; ++i)
                drained &= mbar_wait<SCOPE_CTA>(full + 8 * static_cast<int>(i % SLOTS), static_cast<uint32_t>(i / SLOTS) & 1u,
                                                drain_limit);
            if (!ok || !drained) atomicOr(p.err, drained ? ERRF_WAIT_TIMEOUT : ERRF_WAIT_TIMEOUT | ERRF_DRAIN_TIMEOUT);
        }
        __syncwarp();
    } else if (warp == 1 && rank == 0) {
        constexpr uint32_t idesc = fp4_idesc<NV>(2 * kFp4Rows, kFp4PairTokens);
        const bool one = elect_one();
        const uint32_t codes = fp4_desc(base), scales = fp4_desc(base + S::AT_SCALES);
        uint32_t slot = 0, phase = 0, scale_slot = 0, before = SLOTS - 1, done = 0, buffer = 0;    // done: tiles
        bool there = false;                                          // the next stage, asked ahead
        for (long long tile = first; tile < ntiles && ok; tile += stride, ++done) {
            const uint32_t acc = tmem + (done & 1u) * S::SECOND;
            for (int left = p.k; left > 0; left -= kFp4Step) {
                if (!there) {
                    ok = mbar_wait<SCOPE_CTA>(full + 8 * slot, phase, limit);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) break;
                }
                const uint32_t next = slot + 1 == SLOTS ? 0 : slot + 1, next_phase = slot + 1 == SLOTS ? phase ^ 1u : phase;
                const bool peek = mbar_test<SCOPE_CTA>(full + 8 * next, next_phase);
                const bool cut = tail && left <= kFp4Step;
                if (cut) {
                    ok = mbar_wait<SCOPE_CLUSTER>(tail_full, done & 1u, limit);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) break;
                }
                const auto copy = [&]() {
                    const uint32_t from = scales + scale_slot * (S::SCALES / 16), to = tmem + S::COL_S + buffer * S::COLS_S;
                    if (cut)
                        fp4_scales_cut<NV, 2, true>(from, from + S::SCALES_W / 16, to, Fp4Tail<NV>(p.k).tile, fp4_desc(base + S::AT_TAIL));
                    else
                        fp4_scales<NV, 2, true>(from, from + S::SCALES_W / 16, to);
                    tc_commit_pair(empty + 8 * before);
                };
                const auto multiply = [&]() {
                    const uint32_t a = codes + slot * (S::CODES / 16);
                    fp4_mmas<NV, 2, true>(acc, a, a + S::CODES_W / 16, tmem + S::COL_S + buffer * S::COLS_S, 0, idesc, (left + 63) / 64, left == p.k);
                    if (left <= kFp4Step) tc_commit_pair(acc_full + 8 * (done & 1u));
                };
                tc_fence_after();
                if (left == p.k && done > 0) {
                    // a tile's first scales are copied while the shared columns of the last accumulator are read
                    if (one) copy();
                    __syncwarp();
                    ok = mbar_wait<SCOPE_CTA>(acc_free, (done - 1) & 1u, limit);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) break;
                    tc_fence_after();
                    if (one) multiply();
                } else if (one) {
                    copy();
                    multiply();
                }
                __syncwarp();
                there = __all_sync(0xFFFFFFFFu, peek);
                buffer ^= 1u;
                if (++scale_slot == SCALE_SLOTS) scale_slot = 0;
                before = slot;
                slot = next;
                phase = next_phase;
            }
        }
        if (one) tc_commit_pair(drain);
        if (!ok && lane == 0) atomicOr(p.err, ERRF_WAIT_TIMEOUT);
        __syncwarp();
    } else if (warp == 2 && tail) {
        // the tile of scales that k ends in, of this CTA's channels and of all the tokens, for each output tile
        const Fp4Tail<NV> end(p.k);
        const long long k_tiles = (p.k / (NV ? 16 : 32) + 3) / 4;
        uint32_t done = 0;
        for (long long tile = first; tile < ntiles && ok; tile += stride, ++done) {
            int tn, tm;
            tc_tile(tile, tiles, tn, tm);
            if (done > 0) {
                ok = mbar_wait<SCOPE_CTA>(acc_full + 8 * ((done - 1) & 1u), ((done - 1) >> 1) & 1u, limit);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
            }
#pragma unroll
            for (int r = 0; r < 3; ++r) {
                const long long row_tile = r == 0 ? tn * 2LL + rank : tm * 2LL + r - 1;
                const bool in = row_tile * 128 < (r == 0 ? p.n : p.m);
                const unsigned char* const from = static_cast<const unsigned char*>(r == 0 ? scales_w : scales_a) +
                                                  (row_tile * k_tiles + k_tiles - 1) * kFp4ScaleTile + lane * 16;
                st_shared_v4(base + S::AT_TAIL + r * kFp4ScaleTile + lane * 16, in ? end.cut(ld_v4(from)) : make_uint4(0, 0, 0, 0));
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive_leader(tail_full);
        }
        if (!ok && lane == 0) atomicOr(p.err, ERRF_WAIT_TIMEOUT);
    } else if (warp >= 4) {
        const int wg = (warp - 4) >> 2, row = threadIdx.x & 127;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(warp & 3) << 21);
        const Fp4Factor factor = NV ? fp4_factor(p.a_gs, p.w_gs) : Fp4Factor{1.f, 0.f, 1.f, 0.f};
        // (twice, for the few calls whose factor is split: a test for each 32 columns takes 2 % longer at 8192 x 8192 x 1024)
        const auto read = [&](auto split) {
            constexpr bool SPLIT = decltype(split)::value;
            uint32_t done = 0;
            for (long long tile = first; tile < ntiles && ok; tile += stride, ++done) {
                const uint32_t b = done & 1u;
                int tn, tm;
                tc_tile(tile, tiles, tn, tm);
                const long long n = (static_cast<long long>(tn) * 2 + rank) * kFp4Rows + row;
                const float bias = p.bias != nullptr && n < p.n ? load_as(p.bias, n, p.dt) : 0.f;
                ok = mbar_wait<SCOPE_CTA>(acc_full + 8 * b, (done >> 1) & 1u, limit);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                tc_fence_after();
                // 32 columns at a time, the shared ones first: the first accumulator's last 96, the second's first 96
#pragma unroll 1
                for (int i = 0; i < 4; i += 2) {
                    const int c0 = b == 0 ? 6 + wg - 2 * i : wg + 2 * i, c1 = b == 0 ? c0 - 2 : c0 + 2;
                    uint32_t v[64];
                    const uint32_t at = lanes + b * S::SECOND;
                    tmem_ld_x16(at + 32 * c0, v);
                    tmem_ld_x16(at + 32 * c0 + 16, v + 16);
                    tmem_ld_x16(at + 32 * c1, v + 32);
                    tmem_ld_x16(at + 32 * c1 + 16, v + 48);
                    tmem_wait_ld();
                    if (i == 0) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_leader_relaxed(acc_free);
                    }
                    const long long m0 = static_cast<long long>(tm) * kFp4PairTokens;
                    const int left = static_cast<int>(min(static_cast<long long>(kFp4PairTokens), p.m - m0));
                    if constexpr (SPLIT) fp4_first<64>(v, p.a_gs, p.w_gs);
                    fp4_store<32, NV>(p, v, m0 + 32 * c0, n, left - 32 * c0, factor, bias);
                    fp4_store<32, NV>(p, v + 32, m0 + 32 * c1, n, left - 32 * c1, factor, bias);
                }
            }
        };
        if (NV && factor.split()) read(std::true_type());
        else read(std::false_type());
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
