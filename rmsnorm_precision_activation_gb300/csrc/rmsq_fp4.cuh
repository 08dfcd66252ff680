// rmsq_fp4.cuh -- product of 4-bit codes with block scales on the tensor cores, a CTA per tile.
//
//   out[m][n] = RN(sum_k (a[m][k] sa[m][k / B]) (w[n][k] sw[n][k / B]) / (gs_a gs_w) + bias[n])
//   NVFP4: B = 16, scales E4M3;  MXFP4: B = 32, scales UE8M0
//
// tcgen05.mma's block-scaled kinds take the codes as they are, K-major in shared memory, and the scales from TMEM. The
// swizzled 128x4 scale layout is made for that: a tile of 128 rows x 4 scales is 512 bytes, [row % 32][row / 32][4],
// which tcgen05.cp (32x128b.warpx4) puts into 4 TMEM columns, each the scales of 32 rows. So nothing stands between
// memory and the tensor cores but TMA and that copy.
//
// A CTA takes 128 output channels (the MMA's rows) and NT tokens (its columns); with few tokens, CTAs of a cluster
// share a tile's k. Each token's sums then go to one of them, which adds them up in rank order: threads send four tokens'
// values at a time straight into that CTA's shared memory, whose barrier counts the bytes (sums left in shared memory for others to read
// between two cluster barriers took 2 us, 3.5 at 128 tokens).
//   warps 0-3 (0-7 from 64 tokens on)   read the accumulator and write the output (a lane is a channel: 32 neighbours
//               of a token's row)
//   the next    TMA loads codes and scales of both tiles into a ring, 256 elements of k per stage
//   the last    one thread issues the copies of the scales and the MMAs, four of 64 elements per stage
//
// k is a multiple of 32, so the last MMA's 64 elements may end half way: TMA fills the codes behind the end with zeros,
// but the scales there are the padding's, which may be a NaN; they are cleared in shared memory before the copy.
//
// Every wait is bounded: a role whose wait runs out leaves its loop, and so then do the others. At their end the MMA and
// copy roles always wait (bounded again) for what they have in flight; then the CTA frees its TMEM and ends.
#pragma once

#include "rmsq_matmul_tc.cuh"

namespace rmsq {

struct Fp4Params {
    const float* a_gs;         // or null (1)
    const float* w_gs;
    const void* bias;          // [n] of the output's type, or null
    void* out;                 // [m x n]
    unsigned int* err;
    long long m, n;
    int k;
    int dt;                    // output's type
    uint32_t wait, drain;      // bounds of waits, and of what a stopping CTA has in flight (rmsq_ops_plan.h)
};

constexpr int kFp4Step = 256;                    // elements of k per stage: 128 bytes of codes a row
constexpr int kFp4Rows = 128;                    // output channels per CTA
constexpr int kFp4ScaleTile = 512;               // bytes of 128 rows x 4 scales

// Tiles of scales per 128 rows and stage.
template <bool NV> __host__ __device__ constexpr int fp4_tiles() { return NV ? 4 : 2; }

template <bool NV, int NT> struct Fp4Shape {
    static constexpr int ROW_TILES = (NT + 127) / 128;
    static constexpr int CODES_W = kFp4Rows * kFp4Step / 2, CODES_A = NT * kFp4Step / 2;
    static constexpr int SCALES_W = fp4_tiles<NV>() * kFp4ScaleTile, SCALES_A = ROW_TILES * SCALES_W;
    static constexpr int AT_A = CODES_W, AT_SW = AT_A + CODES_A, AT_SA = AT_SW + SCALES_W;
    static constexpr int STAGE = AT_SA + SCALES_A;
    static constexpr int CTAS = NT <= 32 ? 2 : 1;                     // on an SM
    static constexpr int READERS = NT <= 32 ? 4 : 8;                  // warps that read the accumulator
    static constexpr int THREADS = 32 * (READERS + 2);
    // sums from the cluster's CTAs, [rank][four tokens][channel][4]
    static constexpr int SUM_ROWS = NT + 16, SUMS = SUM_ROWS * kFp4Rows * 4;
    static constexpr int MOST = (CTAS == 2 ? 113 : 226) * 1024;
    // stages of the ring, and shared memory in all (1024 to align the ring, 1024 for barriers): a CTA that has a tile's k
    // to itself needs no room for sums
    static __host__ __device__ constexpr int stages(bool alone) { return (MOST - 2048 - (alone ? 0 : SUMS)) / STAGE; }
    static __host__ __device__ constexpr int smem(bool alone) { return 2048 + stages(alone) * STAGE + (alone ? 0 : SUMS); }
    // TMEM: the accumulator, then two buffers of scales (the channels', the tokens')
    static constexpr int ACC = NT < 32 ? 32 : NT;
    static constexpr int COLS_S = 4 * fp4_tiles<NV>() * (1 + ROW_TILES);
    static constexpr int NEED = ACC + 2 * COLS_S;
    static constexpr int COLS = NEED <= 128 ? 128 : NEED <= 256 ? 256 : 512;
    static_assert(STAGE % 1024 == 0 && AT_A % 1024 == 0 && AT_SW % 1024 == 0, "swizzle atoms");
    static_assert(MOST <= 232448 && COLS * CTAS <= 512, "fits the SM");
    static_assert((smem(true) < smem(false) ? smem(true) : smem(false)) * (CTAS + 1) > 233472 - 1024 * CTAS,
                  "no more CTAs on an SM than TMEM has columns for");
};

// The low word of a descriptor of what lies at a shared-memory address (the high words are constant; both kinds of
// operand take the same low word, and 16 bytes on are one more).
__device__ __forceinline__ uint32_t fp4_desc(uint32_t addr) { return tc_desc_lo(addr); }

// 512 bytes of scales from shared memory to 4 TMEM columns (all four lane quarters): no swizzle, groups of 8 rows of 16
// bytes 128 bytes apart.
template <bool PAIR> __device__ __forceinline__ void fp4_copy_scales(uint32_t tmem, uint32_t lo)
{
    constexpr uint32_t hi = 8u | (1u << 14);
    if constexpr (PAIR)
        asm volatile("{\n\t.reg .b64 d;\n\tmov.b64 d, {%1, %2};\n\ttcgen05.cp.cta_group::2.32x128b.warpx4 [%0], d;\n\t}"
                     ::"r"(tmem), "r"(lo), "r"(hi) : "memory");
    else
        asm volatile("{\n\t.reg .b64 d;\n\tmov.b64 d, {%1, %2};\n\ttcgen05.cp.cta_group::1.32x128b.warpx4 [%0], d;\n\t}"
                     ::"r"(tmem), "r"(lo), "r"(hi) : "memory");
}

// d (+)= a b^T over 64 elements of k, with scales at sa and sb in TMEM.
template <bool NV, bool PAIR>
__device__ __forceinline__ void fp4_mma(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t sa, uint32_t sb, uint32_t add)
{
    constexpr uint32_t hi = 64u | (1u << 14) | (2u << 29);            // as in tc_mma_step
#define RMSQ_FP4_MMA(GROUP, KIND)                                                                              \
    asm volatile(                                                                                              \
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.u32 p, %7, 0;\n\tmov.b64 a, {%1, %3};\n\t"            \
        "mov.b64 b, {%2, %3};\n\ttcgen05.mma.cta_group::" GROUP ".kind::" KIND " [%0], a, b, %4, [%5], [%6], p;\n\t}" \
        ::"r"(d), "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(sa), "r"(sb), "r"(add) : "memory")
    if constexpr (NV && PAIR) RMSQ_FP4_MMA("2", "mxf4nvf4.block_scale.scale_vec::4X");
    else if constexpr (NV) RMSQ_FP4_MMA("1", "mxf4nvf4.block_scale.scale_vec::4X");
    else if constexpr (PAIR) RMSQ_FP4_MMA("2", "mxf4.block_scale.scale_vec::2X");
    else RMSQ_FP4_MMA("1", "mxf4.block_scale.scale_vec::2X");
#undef RMSQ_FP4_MMA
}

// Instruction descriptor: both operands E2M1, K-major; E4M3 or UE8M0 scales.
template <bool NV> __host__ __device__ constexpr uint32_t fp4_idesc(int rows, int cols)
{
    return (1u << 7) | (1u << 10) | (static_cast<uint32_t>(cols / 8) << 17) | (NV ? 0u : 1u << 23) |
           (static_cast<uint32_t>(rows / 16) << 24);
}

// The copies of a stage's scales. weight, tokens: low words of the descriptors of their tiles in shared memory; to: the TMEM
// columns, the channels' first. The tokens' row tiles lie T tiles apart.
template <bool NV, int ROW_TILES, bool PAIR>
__device__ __forceinline__ void fp4_scales(uint32_t weight, uint32_t tokens, uint32_t to)
{
    constexpr int T = fp4_tiles<NV>(), D = kFp4ScaleTile / 16;
#pragma unroll
    for (int i = 0; i < T; ++i) {
        fp4_copy_scales<PAIR>(to + 4 * i, weight + i * D);
#pragma unroll
        for (int r = 0; r < ROW_TILES; ++r) fp4_copy_scales<PAIR>(to + 4 * (T + i * ROW_TILES + r), tokens + (r * T + i) * D);
    }
}

// The same where the last stage's tile `end` is taken from elsewhere: the channels' at `tail`, then the tokens' row tiles.
template <bool NV, int ROW_TILES, bool PAIR>
__device__ __forceinline__ void fp4_scales_cut(uint32_t weight, uint32_t tokens, uint32_t to, int end, uint32_t tail)
{
    constexpr int T = fp4_tiles<NV>(), D = kFp4ScaleTile / 16;
#pragma unroll 1
    for (int i = 0; i < T; ++i) {
        fp4_copy_scales<PAIR>(to + 4 * i, i == end ? tail : weight + i * D);
#pragma unroll
        for (int r = 0; r < ROW_TILES; ++r)
            fp4_copy_scales<PAIR>(to + 4 * (T + i * ROW_TILES + r), i == end ? tail + (1 + r) * D : tokens + (r * T + i) * D);
    }
}

// A stage's MMAs: `quarters` of 64 elements have codes; a whole stage's four are issued without a test. a, b: low words of
// the descriptors of the codes, which advance by 32 bytes an MMA. tokens_from: the column of the tokens' scales that the tile
// starts at (a column holds 32 tokens').
template <bool NV, int ROW_TILES, bool PAIR>
__device__ __forceinline__ void fp4_mmas(uint32_t d, uint32_t a, uint32_t b, uint32_t scales, uint32_t tokens_from, uint32_t idesc,
                                         int quarters, bool fresh)
{
    constexpr int T = fp4_tiles<NV>(), PER = 4 / T;                   // MMAs per tile of scales
    const auto mma = [&](int j) {
        const uint32_t id = j % PER * 2;                              // MXFP4: which two of a tile's four scales
        fp4_mma<NV, PAIR>(d, a + 2 * j, b + 2 * j, idesc | (id << 29) | (id << 4), scales + 4 * (j / PER),
                          scales + 4 * (T + ROW_TILES * (j / PER)) + tokens_from, j > 0 || !fresh);
    };
    if (quarters >= 4) {
#pragma unroll
        for (int j = 0; j < 4; ++j) mma(j);
    } else {
#pragma unroll
        for (int j = 0; j < 3; ++j)
            if (j < quarters) mma(j);
    }
}

// Scales in the tile of four that k ends in, and which tile of its stage that is (k % 64 == 32: there are 1 to 3).
template <bool NV> struct Fp4Tail {
    int tile;
    uint32_t keep;
    __device__ __forceinline__ explicit Fp4Tail(int k)
    {
        const int held = (k % kFp4Step + (NV ? 15 : 31)) / (NV ? 16 : 32);
        tile = held / 4;
        keep = (1u << (8 * (held % 4))) - 1u;
    }
    __device__ __forceinline__ uint4 cut(uint4 v) const { return make_uint4(v.x & keep, v.y & keep, v.z & keep, v.w & keep); }
};

// Clears the scales behind the end of k in the last stage (one warp, after the stage's copies have landed).
template <bool NV, int ROW_TILES, int AT_SW, int AT_SA>
__device__ __forceinline__ void fp4_clear_tail(uint32_t stage, int k, int lane)
{
    constexpr int T = fp4_tiles<NV>();
    const Fp4Tail<NV> tail(k);
#pragma unroll
    for (int r = 0; r < 1 + ROW_TILES; ++r) {
        const uint32_t at = stage + (r == 0 ? AT_SW : AT_SA + (r - 1) * T * kFp4ScaleTile) + tail.tile * kFp4ScaleTile + lane * 16;
        st_shared_v4(at, tail.cut(ld_shared_v4(at)));
    }
    fence_proxy_async_smem();
    __syncwarp();
}

// 1 / (gs_a gs_w) as a sum of two floats, high + low, so that the product of a sum with it is rounded once, in effect. Where it is past
// 2^99 or below 2^-98 a factor before it, first + rest, takes a part: below, the power of two that is left of 2^-100, which is
// exact (a sum is 0, or between 2^-20 and 2^41 in size); past, all but 2^100, so that the two parts of a product are never infinite
// with opposite signs. So a sum of 0 stays 0, and no bits are lost but where results are subnormal. (Powers past 2^200 need not
// be told from it: results are infinite, or 0.) Scales that are 0 or not finite: the plain quotients.
struct Fp4Factor {
    float high, low, first, rest;
    // (from high alone: first and rest are formed again where they are needed, and take no registers elsewhere)
    __device__ __forceinline__ bool split() const { return !(fabsf(high) > 1.6e-30f && fabsf(high) < 1.2e30f); }
};

// A float's significand, in [1, 2) and with its sign, and its power of two (a finite float other than 0).
__device__ __forceinline__ float fp4_significand(float v, int& power)
{
    if (fabsf(v) < 1.17549435e-38f) {
        v *= 16777216.0f;
        power -= 24;
    }
    power += static_cast<int>((__float_as_uint(v) >> 23) & 0xFFu) - 127;
    return __uint_as_float((__float_as_uint(v) & 0x807FFFFFu) | 0x3F800000u);
}

__device__ __forceinline__ float fp4_power(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

__device__ __forceinline__ Fp4Factor fp4_factor(const float* a_gs, const float* w_gs)
{
    const float a = a_gs != nullptr ? *a_gs : 1.0f, w = w_gs != nullptr ? *w_gs : 1.0f;
    const float most = 3.402823466e38f;
    if (!(fabsf(a) > 0.f && fabsf(a) <= most && fabsf(w) > 0.f && fabsf(w) <= most))
        return {__fmul_rn(__fdiv_rn(1.0f, a), __fdiv_rn(1.0f, w)), 0.f, 1.0f, 0.f};
    int power = 0;
    const float ma = fp4_significand(a, power), mw = fp4_significand(w, power), p = __fmul_rn(ma, mw);
    const float high = __fdiv_rn(1.0f, p);
    const float low = __fmul_rn(high, __fsub_rn(__fmaf_rn(-high, p, 1.0f), __fmul_rn(high, __fmaf_rn(ma, mw, -p))));
    power = max(-200, min(200, -power));
    if (power > 99) return {fp4_power(100), 0.f, __fmul_rn(high, fp4_power(power - 100)), __fmul_rn(low, fp4_power(power - 100))};
    const int left = power < -96 ? power + 100 : 0;
    return {__fmul_rn(high, fp4_power(power - left)), __fmul_rn(low, fp4_power(power - left)), fp4_power(left), 0.f};
}

// Sums times the factor before the factor, where it is split.
template <int N> __device__ __forceinline__ void fp4_first(uint32_t* v, const float* a_gs, const float* w_gs)
{
    const Fp4Factor f = fp4_factor(a_gs, w_gs);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float sum = __uint_as_float(v[i]);
        v[i] = __float_as_uint(__fmaf_rn(sum, f.first, __fmul_rn(sum, f.rest)));
    }
}

// Tokens that each CTA of a cluster of nc adds up: whole fours, which a thread sends together.
__host__ __device__ constexpr int fp4_share(int tokens, int nc) { return (tokens + 4 * nc - 1) / (4 * nc) * 4; }

// Four values to another CTA's shared memory (both addresses in the cluster); its barrier counts the 16 bytes.
__device__ __forceinline__ void fp4_send(uint32_t addr, uint32_t bar, const uint32_t* v)
{
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];"
                 ::"r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(bar) : "memory");
}

__device__ __forceinline__ uint32_t fp4_peer(uint32_t addr, uint32_t rank)
{
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
    return a;
}

// N columns (tokens) of a lane's channel to the output: out is where the first goes, pitch the bytes to the next token's
// row, `left` the tokens that there are, in: the channel is one. Neighbouring lanes have neighbouring channels, so
// where their two 16-bit values are a word (the output's width is even) lanes of a pair exchange two tokens' values and each
// writes one token's: half the stores. (An accumulator's 128 columns a warp take longer here than short products' MMAs,
// so instructions count: two columns at a time in packed arithmetic. MXFP4 has no factor.)
template <int DT, int N, bool NV, bool ALL>
__device__ __forceinline__ void fp4_store(const uint32_t* v, char* out, uint32_t pitch, int left, float2 high, float2 low, float2 bias, bool in, bool words)
{
    const bool odd = threadIdx.x & 1;
    const uint32_t half = odd ? 0x3276u : 0x5410u;
    char* const pair = odd ? out + pitch - 2 : out;
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        const float2 sum = make_float2(__uint_as_float(v[i]), __uint_as_float(v[i + 1]));
        const float2 f = add2(NV ? fma2(sum, high, mul2(sum, low)) : sum, bias);
        if constexpr (DT == DT_F32) {
            if (in && (ALL || i < left)) st_u32(out + static_cast<unsigned long long>(pitch) * i, __float_as_uint(f.x));
            if (in && (ALL || i + 1 < left)) st_u32(out + static_cast<unsigned long long>(pitch) * (i + 1), __float_as_uint(f.y));
        } else {
            const uint32_t w = Scalar<DT>::put2(f.x, f.y);
            if (words) {
                const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, w, 1);
                if (in && (ALL || i + odd < left)) st_u32(pair + static_cast<unsigned long long>(pitch) * i, __byte_perm(w, other, half));
            } else {
                if (in && (ALL || i < left)) st_u16(out + static_cast<unsigned long long>(pitch) * i, static_cast<uint16_t>(w));
                if (in && (ALL || i + 1 < left)) st_u16(out + static_cast<unsigned long long>(pitch) * (i + 1), static_cast<uint16_t>(w >> 16));
            }
        }
    }
}

template <int DT, int N, bool NV>
__device__ __forceinline__ void fp4_store(const uint32_t* v, char* out, uint32_t pitch, int left, float2 high, float2 low, float2 bias, bool in, bool words)
{
    if (left >= N && words) fp4_store<DT, N, NV, true>(v, out, pitch, left, high, low, bias, in, true);
    else fp4_store<DT, N, NV, false>(v, out, pitch, left, high, low, bias, in, words);
}

template <int N, bool NV>
__device__ __forceinline__ void fp4_store(const Fp4Params& p, const uint32_t* v, long long m, long long n, int left, Fp4Factor factor, float bias)
{
    const uint32_t es = p.dt == DT_F32 ? 4 : 2, pitch = static_cast<uint32_t>(p.n) * es;
    char* const out = static_cast<char*>(p.out) + (m * p.n + n) * es;
    const bool in = n < p.n, words = p.n % 2 == 0;
    if (p.dt == DT_BF16) fp4_store<DT_BF16, N, NV>(v, out, pitch, left, splat(factor.high), splat(factor.low), splat(bias), in, words);
    else if (p.dt == DT_FP16) fp4_store<DT_FP16, N, NV>(v, out, pitch, left, splat(factor.high), splat(factor.low), splat(bias), in, words);
    else fp4_store<DT_F32, N, NV>(v, out, pitch, left, splat(factor.high), splat(factor.low), splat(bias), in, words);
}

// This thread's warp, from a lane of it: a number that the compiler knows to be the warp's own. What a warp does alone then stays
// in its uniform registers, which descriptors and barriers are taken from (by threadIdx alone every operand is moved
// there first: 610 cycles instead of 530 to issue a stage at 128 tokens, 8192^3 155 us instead of 151).
__device__ __forceinline__ int fp4_warp() { return __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x >> 5), 0); }

template <bool NV, int NT>
__global__ void __launch_bounds__(Fp4Shape<NV, NT>::THREADS, Fp4Shape<NV, NT>::CTAS)
rmsq_fp4_tile_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_a,
                     const __grid_constant__ CUtensorMap map_sw, const __grid_constant__ CUtensorMap map_sa, const Fp4Params p,
                     const TcTiles tiles)
{
    using S = Fp4Shape<NV, NT>;
    constexpr int LOADER = S::READERS, ISSUER = LOADER + 1;
    extern __shared__ unsigned char smem_raw[];
    __shared__ uint32_t tmem_slot;

    const int lane = threadIdx.x & 31, warp = fp4_warp();
    const uint32_t nc = cluster_size(), rank = cluster_rank();
    constexpr int joined = S::stages(false), alone = S::stages(true);
    const int stages = nc == 1 ? alone : joined;

    const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t sums = ring + stages * S::STAGE, full = sums + (nc == 1 ? 0 : S::SUMS);
    const uint32_t empty = full + 8 * stages, acc_full = empty + 8 * stages, drain = acc_full + 8, received = drain + 8;

    int tn, tm;
    tc_tile(cluster_id(), tiles, tn, tm);

    // this CTA's stages of k
    const int steps_all = (p.k + kFp4Step - 1) / kFp4Step;
    const int s0 = static_cast<int>(static_cast<long long>(steps_all) * rank / nc);
    const int steps = static_cast<int>(static_cast<long long>(steps_all) * (rank + 1) / nc) - s0;
    // the tile's tokens, and those of them that this CTA adds up: per from first on
    const int tokens = static_cast<int>(min(static_cast<long long>(NT), p.m - static_cast<long long>(tm) * NT));
    const int per = fp4_share(tokens, static_cast<int>(nc)), fours = per / 4;
    const int own = max(0, min(per, tokens - static_cast<int>(rank) * per)), own_fours = (own + 3) / 4;

    // (Fewer tokens than a tile's columns: the map's boxes have as many rows, and the columns behind them hold what was there.
    // Rows outside a tensor, which TMA fills, take longer than rows that it reads: 48 of 128 tokens x 11008 x 4096 10.0 us
    // with whole boxes, 8.3 so.)
    const uint32_t stage_bytes = S::STAGE - (p.m < NT ? (NT - static_cast<int>(p.m)) * (kFp4Step / 2) : 0);
    auto fetch = [&](uint32_t slot, int s) {
        const uint32_t bar = full + 8 * slot, dst = ring + slot * S::STAGE;
        mbar_arrive_expect_tx(bar, stage_bytes);
        tma_load_2d(dst, &map_w, (s0 + s) * (kFp4Step / 2), tn * kFp4Rows, bar);
        tma_load_2d(dst + S::AT_SW, &map_sw, (s0 + s) * (S::SCALES_W / 8), tn, bar);
        tma_load_2d(dst + S::AT_A, &map_a, (s0 + s) * (kFp4Step / 2), tm * NT, bar);
        tma_load_2d(dst + S::AT_SA, &map_sa, (s0 + s) * (S::SCALES_W / 8), tm * NT / 128, bar);
    };
    int started = 0;                          // stages fetched ahead

    if (warp == LOADER) {
        // (the whole warp runs the loop and one lane issues: a stage's loads take 120 cycles then, from divergent code 330)
        const bool one = elect_one();
        if (one) {
            prefetch_map(&map_w);
            prefetch_map(&map_a);
            prefetch_map(&map_sw);
            prefetch_map(&map_sa);
            for (int i = 0; i < stages; ++i) {
                mbar_init(full + 8 * i, 1);
                mbar_init(empty + 8 * i, 1);
            }
            mbar_init(acc_full, 1);
            mbar_init(drain, 1);
            mbar_init(received, 1);
            fence_mbar_init();
            fence_proxy_async_smem();
            if (nc > 1) mbar_arrive_expect_tx(received, (nc - 1) * static_cast<uint32_t>(own_fours * kFp4Rows * 16));
        }
        __syncwarp();
        // the first loads run while the CTA sets itself up
        pdl_wait_alone();
        for (; started < stages && started < steps; ++started)
            if (one) fetch(static_cast<uint32_t>(started), started);
        __syncwarp();
    }
    if (warp == ISSUER) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)),
                     "r"(S::COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        tc_fence_before();
    }
    __syncthreads();
    if (nc > 1) cluster_arrive_as(false);     // this CTA's barriers are set up
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    pdl_wait();

    const uint32_t limit = p.wait, drain_limit = p.drain;
    bool ok = true;

    if (warp == LOADER) {
        const bool one = elect_one();
        int s = started, slot = 0;
        uint32_t phase = 0;
        for (; s < steps; ++s) {                                       // (only where the first loads filled the ring)
            ok = mbar_wait<SCOPE_CTA>(empty + 8 * slot, phase, limit);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            if (one) fetch(slot, s);
            __syncwarp();
            if (++slot == stages) {
                slot = 0;
                phase ^= 1u;
            }
        }
        if (lane == 0) {
            // the copies in flight end before the CTA does, whichever role stopped waiting
            bool drained = true;
            for (int i = s > stages ? s - stages : 0; i < s; ++i)
                drained &= mbar_wait<SCOPE_CTA>(full + 8 * (i % stages), static_cast<uint32_t>(i / stages) & 1u, drain_limit);
            if (!ok || !drained) atomicOr(p.err, drained ? ERRF_WAIT_TIMEOUT : ERRF_WAIT_TIMEOUT | ERRF_DRAIN_TIMEOUT);
        }
        __syncwarp();
        if (nc > 1) {
            cluster_wait();
            cluster_arrive_as(false);
        }
    } else if (warp == ISSUER) {
        constexpr uint32_t idesc = fp4_idesc<NV>(kFp4Rows, NT);
        // 0 or 2: an MMA takes the scales from even columns only, so tiles of fewer tokens are for the first alone
        const uint32_t tokens_from = NT == 64 ? (static_cast<uint32_t>(tm) & 1u) * 2u : 0u;
        const bool one = elect_one();
        int slot = 0;
        uint32_t phase = 0;
        bool there = false;                                           // the next stage, asked ahead
        for (int s = 0; s < steps; ++s) {
            if (!there) {
                ok = mbar_wait<SCOPE_CTA>(full + 8 * slot, phase, limit);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
            }
            const int next = slot + 1 == stages ? 0 : slot + 1;
            const uint32_t next_phase = next == 0 ? phase ^ 1u : phase;
            const bool peek = mbar_test<SCOPE_CTA>(full + 8 * next, next_phase);
            const uint32_t stage = ring + slot * S::STAGE;
            const int left = p.k - (s0 + s) * kFp4Step;               // elements of k from this stage on
            if (left < kFp4Step && left % 64 != 0) fp4_clear_tail<NV, S::ROW_TILES, S::AT_SW, S::AT_SA>(stage, p.k, lane);
            tc_fence_after();
            if (one) {
                const uint32_t desc = fp4_desc(stage), scales = tmem + S::ACC + (s & 1) * S::COLS_S;
                fp4_scales<NV, S::ROW_TILES, false>(desc + S::AT_SW / 16, desc + S::AT_SA / 16, scales);
                fp4_mmas<NV, S::ROW_TILES, false>(tmem, desc, desc + S::AT_A / 16, scales, tokens_from, idesc, (left + 63) / 64,
                                                  s == 0);
                tc_commit(empty + 8 * slot);
                if (s == steps - 1) tc_commit(acc_full);
            }
            __syncwarp();
            there = __all_sync(0xFFFFFFFFu, peek);
            slot = next;
            phase = next_phase;
        }
        if (one) {
            // the MMAs in flight end before TMEM is freed, whichever role stopped waiting
            tc_commit(drain);
            const bool drained = mbar_wait<SCOPE_CTA>(drain, 0, drain_limit);
            if (!ok || !drained) atomicOr(p.err, drained ? ERRF_WAIT_TIMEOUT : ERRF_WAIT_TIMEOUT | ERRF_DRAIN_TIMEOUT);
        }
        __syncwarp();
        if (nc > 1) {
            cluster_wait();
            cluster_arrive_as(false);
        }
    } else {
        const uint32_t acc = tmem + (static_cast<uint32_t>(warp & 3) << 21);
        constexpr int PARTS = S::READERS / 4;                         // of the columns
        const int row = threadIdx.x & 127, part = warp >> 2;
        const long long n = static_cast<long long>(tn) * kFp4Rows + row, m0 = static_cast<long long>(tm) * NT;
        const Fp4Factor factor = NV ? fp4_factor(p.a_gs, p.w_gs) : Fp4Factor{1.f, 0.f, 1.f, 0.f};
        const float bias = p.bias != nullptr && n < p.n ? load_as(p.bias, n, p.dt) : 0.f;
        if (nc > 1) cluster_wait();
        ok = mbar_wait<SCOPE_CTA>(acc_full, 0, limit);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (ok) {
            tc_fence_after();
            constexpr int COLS = NT / PARTS, LD = COLS < 32 ? COLS : 32;       // of a part, and of one read
            // the CTA that adds up the next four tokens, and their place there
            int to = part * (COLS / 4) / fours, at = part * (COLS / 4) - to * fours;
#pragma unroll 1
            for (int c = part * COLS; c < (part + 1) * COLS && c < tokens; c += LD) {
                uint32_t v[LD];
                tmem_ld_x16(acc + c, v);
                if constexpr (LD == 32) tmem_ld_x16(acc + c + 16, v + 16);
                tmem_wait_ld();
                if (nc == 1) {
                    if (NV && factor.split()) fp4_first<LD>(v, p.a_gs, p.w_gs);
                    fp4_store<LD, NV>(p, v, m0 + c, n, tokens - c, factor, bias);
                } else {
#pragma unroll
                    for (int i = 0; i < LD / 4; ++i) {
                        if (c + 4 * i < tokens) {
                            const uint32_t addr = sums + ((rank * fours + at) * kFp4Rows + row) * 16;
                            if (to == static_cast<int>(rank)) st_shared_v4(addr, make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]));
                            else fp4_send(fp4_peer(addr, to), fp4_peer(received, to), v + 4 * i);
                        }
                        if (++at == fours) {
                            at = 0;
                            ++to;
                        }
                    }
                }
            }
        }
        if (nc > 1) {
            cluster_arrive_as(false);                                 // this thread sends no more
            if (own > 0) {
                ok = ok && mbar_wait<SCOPE_CLUSTER>(received, 0, limit);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (PARTS > 1) asm volatile("bar.sync 1, %0;" ::"n"(32 * S::READERS) : "memory");   // this CTA's own
                const uint32_t stride = static_cast<uint32_t>(fours) * kFp4Rows * 16;
                for (int i = part; ok && i < own_fours; i += PARTS) {
                    uint4 o[8];
#pragma unroll
                    for (uint32_t r = 0; r < 8; ++r)
                        o[r] = r < nc ? ld_shared_v4(sums + r * stride + (i * kFp4Rows + row) * 16) : make_uint4(0, 0, 0, 0);
                    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (uint32_t r = 0; r < 8; ++r) {
                        v.x += __uint_as_float(o[r].x);
                        v.y += __uint_as_float(o[r].y);
                        v.z += __uint_as_float(o[r].z);
                        v.w += __uint_as_float(o[r].w);
                    }
                    uint32_t four[4] = {__float_as_uint(v.x), __float_as_uint(v.y), __float_as_uint(v.z), __float_as_uint(v.w)};
                    if (NV && factor.split()) fp4_first<4>(four, p.a_gs, p.w_gs);
                    fp4_store<4, NV>(p, four, m0 + static_cast<int>(rank) * per + 4 * i, n, own - 4 * i, factor, bias);
                }
            }
        }
        if (!ok && lane == 0) atomicOr(p.err, ERRF_WAIT_TIMEOUT);
    }

    if (nc > 1) cluster_wait();                                       // nobody sends to a CTA that has left
    tc_fence_before();
    if (__syncthreads_or(!ok) && nc > 1) {
        // what was sent here lands before the CTA leaves, which takes about a microsecond
        const uint32_t t0 = time_units();
        while (time_units() - t0 < 1000) __nanosleep(100000);
    }
    if (warp == ISSUER) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(S::COLS));
    }
}

}  // namespace rmsq
