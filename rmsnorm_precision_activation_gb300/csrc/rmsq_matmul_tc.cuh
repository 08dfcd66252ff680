// rmsq_matmul_tc.cuh -- the int8 product on the tensor cores.
//
// sm_103a's tcgen05 has no 8-bit-integer kind, so the codes go through its fp16 kind: a code is
// exact in fp16, a product of two is at most 2^14, and fp32 sums of up to 1024 products are whole
// numbers of at most 2^24, so exact. The fp32 accumulator is therefore read out and added to 32-bit
// integers every 1024 elements of k (kTcChunk code stages), which makes every sum exact.
//
// A CTA takes 128 output channels (the MMA's rows) and NT tokens (its columns):
//   warp 0       TMA loads the codes of both tiles into a ring, 128 elements of k per stage (a copy's cost is
//                per row of its box: boxes of 64 took 1153 us at 8192^3, these 1002, in the pair kernel)
//   warps 4-11   two warpgroups, each a half of every code stage, turn codes into fp16, one operand
//                stage of 64 elements of k: the channels' straight into TMEM (the MMA takes its
//                first operand from there, which spares shared memory a write and a read), the
//                tokens' into shared memory
//   warp 1       one thread issues tcgen05.mma, four per operand stage
//   warps 12-    one or two warpgroups read the accumulator out and write the output
// The weight is read as codes, so a call with few tokens streams one byte per weight; CTAs of a
// cluster then share a tile's k and add their integer sums through distributed shared memory.
//
// Every wait is bounded: a role whose wait runs out leaves its loop, and so then do the others. At their
// end the MMA and copy roles always wait (bounded again) for what they have in flight, because they can
// have issued everything when another role's wait runs out; then the CTA frees its TMEM and ends.
#pragma once

#include <cuda.h>

#include "rmsq_matmul.cuh"

namespace rmsq {

constexpr int kTcThreads = 640;
constexpr int kTcCodes = 128;            // elements of k per code stage
constexpr int kTcStep = 64;              // elements of k per operand stage
constexpr int kTcChunk = 1024 / kTcCodes; // code stages per read-out of the accumulator
constexpr int kTcRows = 128;             // output channels per CTA

template <int NT> struct TcShape {
    // Few tokens leave room for two CTAs on an SM, each with half of TMEM: a stage's hand-overs from
    // role to role take about 1000 cycles whatever its size, and a second CTA fills them (CTAS
    // hold up to 32 tokens, so that one warpgroup reads the sums).
    static constexpr int CTAS = NT <= 32 ? 2 : 1;
    static constexpr int READERS = 8 / CTAS;                          // warps that read the accumulator
    static constexpr int THREADS = 32 * (12 + READERS);
    static constexpr int COLS = 512 / CTAS;                           // TMEM columns
    static constexpr int ACC = NT <= 32 ? 64 : 256;                   // of these, before the operand stages
    static constexpr int RAW_A = kTcRows * kTcCodes;
    static constexpr int RAW_B = NT * kTcCodes;
    static constexpr int RAW = RAW_A + RAW_B;
    static constexpr int OP = NT * kTcStep * 2;
    static constexpr int OPS = NT >= 128 || NT <= 32 ? 6 : 8;         // operand stages
    static constexpr int RAWS = NT >= 128 ? 4 : NT >= 64 ? 6 : 4;    // code stages
    // 1024 bytes to align the ring, 1024 for barriers
    static constexpr int SMEM = 2048 + RAWS * RAW + OPS * OP;
    // no more CTAs on an SM than TMEM has columns for, or its allocation would wait for one to end
    static_assert(CTAS == 2 ? SMEM > 78 * 1024 && SMEM <= 112 * 1024 : SMEM > 116 * 1024 && SMEM <= 232448, "CTAs per SM");
    static_assert(NT <= ACC && ACC + 32 * OPS <= COLS, "accumulator and operand stages in TMEM");
    static_assert(RAWS * RAW + OPS * OP >= NT * kTcRows * 4, "the cluster's sums reuse the ring");
};

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
        ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Arrives on bar when every MMA this thread has issued is done.
__device__ __forceinline__ void tc_commit(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// One operand stage: d (+)= a b^T over 64 elements of k, four MMAs. a is fp16 in TMEM (128 lanes, 8
// columns per MMA), b fp16 in shared memory (K-major, 32 bytes per MMA; desc_lo: the descriptor's
// low word, which holds the address). fresh: overwrite d. PAIR: with the other CTA (cta_group::2).
template <bool PAIR>
__device__ __forceinline__ void tc_mma_step(uint32_t d, uint32_t a, uint32_t desc_lo, uint32_t idesc, bool fresh)
{
    constexpr uint32_t hi = 64u | (1u << 14) | (2u << 29);
#pragma unroll
    for (int k = 0; k < kTcStep / 16; ++k) {
        const uint32_t add = k > 0 || !fresh;
        if constexpr (PAIR)
            asm volatile(
                "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tsetp.ne.u32 p, %5, 0;\n\tmov.b64 b, {%2, %3};\n\t"
                "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], b, %4, p;\n\t}"
                ::"r"(d), "r"(a + 8 * k), "r"(desc_lo + 2 * k), "r"(hi), "r"(idesc), "r"(add) : "memory");
        else
            asm volatile(
                "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tsetp.ne.u32 p, %5, 0;\n\tmov.b64 b, {%2, %3};\n\t"
                "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}"
                ::"r"(d), "r"(a + 8 * k), "r"(desc_lo + 2 * k), "r"(hi), "r"(idesc), "r"(add) : "memory");
    }
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one()
{
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one != 0;
}

// Low word of the descriptor of a K-major operand with 128-byte swizzle, whose groups of 8 rows are
// 1024 bytes apart (the high word is constant: that pitch, the version, the swizzle).
__device__ __forceinline__ uint32_t tc_desc_lo(uint32_t addr) { return ((addr & 0x3FFFFu) >> 4) | (1u << 16); }

__device__ __forceinline__ void tmem_st_x16(uint32_t addr, const uint32_t (&v)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16};" ::"r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]),
        "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}

// 16 columns of this warp's lanes; the values are valid after tmem_wait_ld.
__device__ __forceinline__ void tmem_ld_x16(uint32_t addr, uint32_t* v)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
        "[%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
          "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ int4 ld_cluster_i4(uint32_t addr, uint32_t rank)
{
    uint32_t raddr;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(raddr) : "r"(addr), "r"(rank));
    int4 v;
    asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(raddr) : "memory");
    return v;
}

struct TcTiles {
    int n_tiles, m_tiles;
};

// Tiles in groups of 8 channel tiles, tokens fastest within a group's column, so that the CTAs
// running at one time share both operands in L2.
__device__ __forceinline__ void tc_tile(long long i, const TcTiles& t, int& n, int& m)
{
    const long long per = 8LL * t.m_tiles;
    const int group = static_cast<int>(i / per), in = static_cast<int>(i % per);
    const int first = group * 8, width = t.n_tiles - first < 8 ? t.n_tiles - first : 8;
    n = first + in % width;
    m = in / width;
}

template <int NT>
__global__ void __launch_bounds__(TcShape<NT>::THREADS, TcShape<NT>::CTAS)
rmsq_matmul_tc_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_a,
                      const MatmulParams p, const TcTiles tiles)
{
    using S = TcShape<NT>;
    constexpr int OPS = S::OPS, RAWS = S::RAWS;
    extern __shared__ unsigned char smem_raw[];
    __shared__ uint32_t tmem_slot;

    unsigned char* const smem = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    unsigned char* const raw = smem;
    unsigned char* const ops = smem + RAWS * S::RAW;
    const uint32_t bars = smem_u32(ops + OPS * S::OP);
    const uint32_t raw_full = bars, raw_empty = raw_full + 8 * RAWS;
    const uint32_t op_full = raw_empty + 8 * RAWS, op_empty = op_full + 8 * OPS;
    const uint32_t acc_full = op_empty + 8 * OPS, acc_empty = acc_full + 8, drain = acc_empty + 8;

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t nc = cluster_size(), rank = cluster_rank();

    const int steps_all = (p.k + kTcCodes - 1) / kTcCodes;      // code stages
    const int k0 = static_cast<int>(static_cast<long long>(steps_all) * rank / nc);
    const int steps = static_cast<int>(static_cast<long long>(steps_all) * (rank + 1) / nc) - k0;
    const long long ntiles = static_cast<long long>(tiles.n_tiles) * tiles.m_tiles;
    const long long first = cluster_id(), stride = cluster_count();

    // Code stage s of a tile into the ring (one thread).
    auto fetch = [&](uint32_t slot, int s, int tn, int tm) {
        const uint32_t full = raw_full + 8 * slot, dst = smem_u32(raw) + slot * S::RAW;
        mbar_arrive_expect_tx(full, S::RAW);
        tma_load_2d(dst, &map_w, (k0 + s) * kTcCodes, tn * kTcRows, full);
        tma_load_2d(dst + S::RAW_A, &map_a, (k0 + s) * kTcCodes, tm * NT, full);
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
            mbar_init(op_full + 8 * i, 4);
            mbar_init(op_empty + 8 * i, 1);
        }
        mbar_init(acc_full, 1);
        mbar_init(acc_empty, S::READERS);
        mbar_init(drain, 1);
        fence_mbar_init();
        fence_proxy_async_smem();
        // the first loads run while the CTA sets itself up
        pdl_wait_alone();
        int tn, tm;
        tc_tile(first, tiles, tn, tm);
        for (; started < RAWS && started < steps; ++started) fetch(started, started, tn, tm);
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)),
                     "r"(S::COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    const uint32_t tmem_a = tmem + S::ACC;   // operand stages of 32 columns behind the accumulator
    pdl_wait();

    const uint32_t limit = p.wait, drain_limit = p.drain;
    bool ok = true;

    if (warp == 0) {
        if (lane == 0) {
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
        }
        __syncwarp();
    } else if (warp == 1) {
        // The whole warp runs the loop and one lane issues: addresses and descriptors then stay in
        // uniform registers (from divergent code an MMA took 60 cycles to issue).
        constexpr uint32_t idesc = (1u << 4) | (static_cast<uint32_t>(NT / 8) << 17) | ((kTcRows / 16u) << 24);
        const bool one = elect_one();
        const uint32_t desc0 = tc_desc_lo(smem_u32(ops));
        uint32_t slot = 0, phase = 0, chunks = 0;        // a code stage fills operand stages slot and slot + 1
        bool ready0 = false, ready1 = false;             // asked a stage ahead
        for (long long tile = first; tile < ntiles && ok; tile += stride) {
            int left = 0;                                // code stages until the read-out
            for (int s = 0; s < steps; ++s) {
                const bool fresh = left == 0;
                if (fresh) {
                    left = kTcChunk;
                    ok = mbar_wait<SCOPE_CTA>(acc_empty, (chunks & 1u) ^ 1u, limit);
                    ++chunks;
                }
                const bool tail = --left == 0 || s == steps - 1;
                const uint32_t next = slot + 2 == OPS ? 0 : slot + 2, next_phase = slot + 2 == OPS ? phase ^ 1u : phase;
                if (!ready0) ok = ok && mbar_wait<SCOPE_CTA>(op_full + 8 * slot, phase, limit);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                tc_fence_after();
                if (one) {
                    tc_mma_step<false>(tmem, tmem_a + slot * 32, desc0 + slot * (S::OP / 16), idesc, fresh);
                    tc_commit(op_empty + 8 * slot);
                }
                __syncwarp();
                if (!ready1) ok = mbar_wait<SCOPE_CTA>(op_full + 8 * slot + 8, phase, limit);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                tc_fence_after();
                const bool peek0 = mbar_test<SCOPE_CTA>(op_full + 8 * next, next_phase);
                const bool peek1 = mbar_test<SCOPE_CTA>(op_full + 8 * next + 8, next_phase);
                if (one) {
                    tc_mma_step<false>(tmem, tmem_a + slot * 32 + 32, desc0 + (slot + 1) * (S::OP / 16), idesc, false);
                    tc_commit(op_empty + 8 * slot + 8);
                    if (tail) tc_commit(acc_full);
                }
                __syncwarp();
                ready0 = __all_sync(0xFFFFFFFFu, peek0);
                ready1 = __all_sync(0xFFFFFFFFu, peek1);
                slot = next;
                phase = next_phase;
            }
        }
        if (one) {
            // the MMAs in flight end before TMEM is freed, whichever role stopped waiting
            tc_commit(drain);
            const bool drained = mbar_wait<SCOPE_CTA>(drain, 0, drain_limit);
            if (!ok || !drained) atomicOr(p.err, drained ? ERRF_WAIT_TIMEOUT : ERRF_WAIT_TIMEOUT | ERRF_DRAIN_TIMEOUT);
        }
        __syncwarp();
    } else if (warp >= 4 && warp < 12) {
        const int wg = (warp - 4) >> 2, t = (threadIdx.x - 128) & 127;
        const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;     // this warp's TMEM lanes, in bits 16+
        constexpr int PB = (NT * 4 + 127) / 128;      // a thread's pieces of the tokens' NT x 4
        uint32_t rs = 0, rphase = 0, os = wg, ophase = 0;
        bool ready = false;                  // the next code stage, asked ahead
        for (long long tile = first; tile < ntiles && ok; tile += stride) {
            for (int s = 0; s < steps; ++s) {
                if (!ready) ok = mbar_wait<SCOPE_CTA>(raw_full + 8 * rs, rphase, limit);
                const uint32_t rnext = rs + 1 == RAWS ? 0 : rs + 1, rnext_phase = rs + 1 == RAWS ? rphase ^ 1u : rphase;
                const uint32_t ra = smem_u32(raw) + rs * S::RAW, rb = ra + S::RAW_A;
                const uint32_t ob = smem_u32(ops) + os * S::OP;
                uint4 va[4], vb[PB];                  // all loads first, to overlap
#pragma unroll
                for (int c = 0; c < 4; ++c) va[c] = ld_shared_v4(ra + t * 128 + (((4 * wg + c) ^ (t & 7)) << 4));
#pragma unroll
                for (int j = 0; j < PB; ++j) {
                    const int i = j * 128 + t, r = i % NT, c = i / NT;
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
                    const int i = j * 128 + t, r = i % NT, c = i / NT;
                    if (c < 4) {
                        uint4 lo, hi;
                        codes_to_half(vb[j].x, lo.x, lo.y);
                        codes_to_half(vb[j].y, lo.z, lo.w);
                        codes_to_half(vb[j].z, hi.x, hi.y);
                        codes_to_half(vb[j].w, hi.z, hi.w);
                        st_shared_v4(ob + r * 128 + (((2 * c) ^ (r & 7)) << 4), lo);
                        st_shared_v4(ob + r * 128 + (((2 * c + 1) ^ (r & 7)) << 4), hi);
                    }
                }
                fence_proxy_async_smem();
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(raw_empty + 8 * rs);
                    mbar_arrive(op_full + 8 * os);
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
    } else if (warp >= 12) {
        constexpr int HALF = NT * 4 / S::READERS, LD = HALF < 32 ? HALF : 32;     // columns of a warp, and of one read
        const int wg = (warp - 12) >> 2, row = threadIdx.x & 127;
        const uint32_t base = tmem + (static_cast<uint32_t>(warp & 3) << 21) + wg * HALF;
        long long chunks = 0;
        for (long long tile = first; tile < ntiles && ok; tile += stride) {
            int acc[HALF];
#pragma unroll
            for (int i = 0; i < HALF; ++i) acc[i] = 0;
            for (int s = 0; s < steps; s += kTcChunk, ++chunks) {
                ok = mbar_wait<SCOPE_CTA>(acc_full, static_cast<uint32_t>(chunks & 1), limit);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < HALF; c += LD) {
                    uint32_t v[LD];
                    tmem_ld_x16(base + c, v);
                    if constexpr (LD == 32) tmem_ld_x16(base + c + 16, v + 16);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < LD; ++j) acc[c + j] += __float2int_rn(__uint_as_float(v[j]));
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(acc_empty);
            }
            if (!ok) break;
            int tn, tm;
            tc_tile(tile, tiles, tn, tm);
            if (nc == 1) {
                const long long n = static_cast<long long>(tn) * kTcRows + row;
                if (n < p.n) {
                    const float ws = p.w_scale[n], b = p.bias ? load_as(p.bias, n, p.dt) : 0.f;
#pragma unroll
                    for (int i = 0; i < HALF; ++i) {
                        const long long m = static_cast<long long>(tm) * NT + wg * HALF + i;
                        if (m < p.m) store_as(p.out, m * p.n + n, p.dt, scaled(acc[i], p.a_scale[m], ws, b, p.bias));
                    }
                }
            } else {
                // one tile per cluster: the ring is free, and takes the sums, [token][channel]
                int* const sums = reinterpret_cast<int*>(raw);
#pragma unroll
                for (int i = 0; i < HALF; ++i) sums[(wg * HALF + i) * kTcRows + row] = acc[i];
            }
        }
        if (!ok && lane == 0) atomicOr(p.err, ERRF_WAIT_TIMEOUT);
    }

    if (nc > 1) {
        // tokens rank, rank + nc, ... of the tile: add the CTAs' sums and write
        cluster_sync();
        int tn, tm;
        tc_tile(first, tiles, tn, tm);
        const uint32_t sums = smem_u32(raw);
        for (int e = threadIdx.x; e < (NT + static_cast<int>(nc) - 1) / static_cast<int>(nc) * 32; e += S::THREADS) {
            const int i = (e >> 5) * static_cast<int>(nc) + static_cast<int>(rank);
            const long long m = static_cast<long long>(tm) * NT + i, n = static_cast<long long>(tn) * kTcRows + lane * 4;
            if (i >= NT || m >= p.m || n >= p.n) continue;
            int4 v = make_int4(0, 0, 0, 0);
            for (uint32_t r = 0; r < nc; ++r) {
                const int4 o = ld_cluster_i4(sums + (i * kTcRows + lane * 4) * 4, r);
                v.x += o.x;
                v.y += o.y;
                v.z += o.z;
                v.w += o.w;
            }
            const int a[4] = {v.x, v.y, v.z, v.w};
            const float as = p.a_scale[m];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (n + j < p.n)
                    store_as(p.out, m * p.n + n + j, p.dt,
                             scaled(a[j], as, p.w_scale[n + j], p.bias ? load_as(p.bias, n + j, p.dt) : 0.f, p.bias));
        }
        cluster_sync();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(S::COLS));
    }
}

}  // namespace rmsq
