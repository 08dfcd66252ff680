// rmsq_fp4.cu -- C ABI of the 4-bit products: argument checks and the choice of kernel.
#include <cstdint>

#include "rmsq_fp4_pair.cuh"
#include "rmsq_ops.h"
#include "rmsq_tensor_map.h"

namespace rmsq {

static bool aligned(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(bytes) == 0; }

struct Fp4Operands {
    const void *a, *sa, *w, *sw;
};

// Codes [rows x k] in boxes of box_rows x 256 elements, and their scales in boxes of a stage's tiles of box_tiles x 128 rows.
template <bool NV>
static bool encode(CUtensorMap* codes_map, CUtensorMap* scales_map, const void* codes, const void* scales, long long rows, int k,
                   int box_rows, int box_tiles)
{
    const long long k_tiles = (k / (NV ? 16 : 32) + 3) / 4;
    return encode_map(codes_map, codes, 1, rows, k / 2, box_rows, kFp4Step / 2, CU_TENSOR_MAP_SWIZZLE_128B) &&
           encode_map(scales_map, scales, 8, (rows + 127) / 128, k_tiles * (kFp4ScaleTile / 8), box_tiles,
                      fp4_tiles<NV>() * kFp4ScaleTile / 8, CU_TENSOR_MAP_SWIZZLE_NONE);
}

template <bool NV, int NT> static cudaError_t launch_tile(Fp4Params& p, const Fp4Operands& o, int cluster, cudaStream_t stream)
{
    using S = Fp4Shape<NV, NT>;
    CUtensorMap map_w, map_a, map_sw, map_sa;
    if (!encode<NV>(&map_w, &map_sw, o.w, o.sw, p.n, p.k, kFp4Rows, 1) ||
        !encode<NV>(&map_a, &map_sa, o.a, o.sa, p.m, p.k, p.m < NT ? static_cast<int>(p.m) : NT, S::ROW_TILES))
        return cudaErrorUnknown;
    TcTiles t;
    t.n_tiles = static_cast<int>((p.n + kFp4Rows - 1) / kFp4Rows);
    t.m_tiles = static_cast<int>((p.m + NT - 1) / NT);
    const long long ctas = static_cast<long long>(t.n_tiles) * t.m_tiles * cluster;
    if (ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
    void* args[] = {&map_w, &map_a, &map_sw, &map_sa, &p, &t};
    return launch_kernel(reinterpret_cast<const void*>(&rmsq_fp4_tile_kernel<NV, NT>), dim3(static_cast<unsigned>(ctas)), S::THREADS,
                         S::smem(cluster == 1), cluster, stream, args);
}

template <bool NV> static cudaError_t launch_pair(Fp4Params& p, const Fp4Operands& o, const DeviceView& dv, cudaStream_t stream)
{
    using S = Fp4PairShape<NV>;
    CUtensorMap map_w, map_a, map_sw, map_sa;
    if (!encode<NV>(&map_w, &map_sw, o.w, o.sw, p.n, p.k, kFp4Rows, 1) ||
        !encode<NV>(&map_a, &map_sa, o.a, o.sa, p.m, p.k, kFp4PairTokens / 2, 2))
        return cudaErrorUnknown;
    TcTiles t;
    t.n_tiles = static_cast<int>((p.n + 2 * kFp4Rows - 1) / (2 * kFp4Rows));
    t.m_tiles = static_cast<int>((p.m + kFp4PairTokens - 1) / kFp4PairTokens);
    const long long tiles = static_cast<long long>(t.n_tiles) * t.m_tiles;
    const long long pairs = tiles < dv.sms / 2 ? tiles : dv.sms / 2;
    const void *sw = o.sw, *sa = o.sa;
    void* args[] = {&map_w, &map_a, &map_sw, &map_sa, &p, &t, &sw, &sa};
    return launch_kernel(reinterpret_cast<const void*>(&rmsq_fp4_pair_kernel<NV>), dim3(static_cast<unsigned>(2 * pairs)),
                         kFp4PairThreads, S::SMEM, 2, stream, args);
}

// What a call takes in each kernel, in cycles, by the parts of its time that were measured (GB300, 2.07 GHz), and with
// it the choice of kernel, tile and cluster. Sizes only: the same call always takes the same one.
//   - Before the first product and after the last 2500 to 3500 cycles pass in every wave of CTAs (pairs 9500).
//   - A stage takes as long as its bytes (60 a cycle and SM), as its issue (450; pairs 600), or, where there are more than
//     the ring has slots, as a load's latency under load over the stages in flight (3600, so three stages of 32 tokens are
//     slower than six of 64).
//   - The weight comes from HBM at 3200 bytes a cycle at most, and at 32 to an SM.
//   - CTAs that share a tile's k spend 1500 cycles on joining their sums, and 24 for every token they send.
// Measured, in us, NVFP4, tokens x channels x k, tokens of a tile / CTAs that share its k:
//   1 x 1024 x 4096: 16/8 2.8, 16/4 3.2, 16/1 5.6;  1 x 7168 x 8192: 16/4 7.9, 16/2 8.9, 16/1 10.6
//   24 x 8192 x 8192: 64/2 9.1, 32/2 10.3;  24 x 28672 x 8192: 32/1 22.9, 64/1 26.9
//   128 x 1024 x 4096: 64/6 4.3, 128/6 5.0, pair 9.2;  128 x 8192 x 8192: 64/1 10.9, 128/2 11.8, pair 14.5
//   256 x 8192 x 8192: 128/1 11.6, pair 13.7, 64/1 20.6;  256 x 28672 x 8192: pair 30.9, 128/1 37.3
//   512 x 1024 x 4096: 64/2 6.0, pair 8.4;  512 x 8192 x 8192: pair 14.5, 128/1 21.8
// Over 154 such sizes in both formats the choice takes 1 % longer than the best one on average, 10 % at most.
struct Fp4Plan {
    long long cycles;
    int tokens, cluster;              // tokens of a tile; 0: none yet
};

static long long most(long long a, long long b) { return a > b ? a : b; }

static long long weight_cycles(const Fp4Params& p, bool nv) { return p.n * (p.k / 2 + p.k / (nv ? 16 : 32)) / 3200; }

template <bool NV, int NT> static void plan_tile(const Fp4Params& p, const DeviceView& dv, Fp4Plan* best)
{
    using S = Fp4Shape<NV, NT>;
    const void* fn = reinterpret_cast<const void*>(&rmsq_fp4_tile_kernel<NV, NT>);
    const long long tiles = (p.n + kFp4Rows - 1) / kFp4Rows * ((p.m + NT - 1) / NT), slots = static_cast<long long>(dv.sms) * S::CTAS;
    const int steps = (p.k + kFp4Step - 1) / kFp4Step, tokens = p.m < NT ? static_cast<int>(p.m) : NT;
    for (int c = 1; c <= 8 && c <= steps && (c == 1 || c * tiles <= slots); ++c) {
        if (c > 1 && c * fp4_share(tokens, c) > S::SUM_ROWS) continue;
        const long long waves = (tiles * c + slots - 1) / slots, each = (tiles * c + dv.sms - 1) / dv.sms;   // CTAs of an SM
        const int mine = (steps + c - 1) / c, ring = S::stages(c == 1);
        const long long stage = most(most(S::STAGE * (each < S::CTAS ? each : S::CTAS) / 60, 450), mine > ring ? 3600 / ring : 0);
        const long long join = c > 1 ? 1500 + 24LL * tokens * (c - 1) / c : 8LL * tokens;
        // (tiles of other tokens find the weight in L2)
        const long long weight = most(weight_cycles(p, NV), p.m <= NT ? each * mine * (S::CODES_W + S::SCALES_W) / 32 : 0);
        const long long cycles = (NT < 64 ? 2500 : NT < 128 ? 3000 : 3500) * waves + most(waves * mine * stage, weight) + join;
        if (best->tokens != 0 && cycles >= best->cycles) continue;
        // (what fits goes by the device's clusters of SMs, not by SMs alone; they are counted with one CTA on an SM)
        if (c > 1 && tiles > static_cast<long long>(S::CTAS) * resident_clusters(fn, S::THREADS, S::smem(false), c)) continue;
        *best = {cycles, NT, c};
    }
}

template <bool NV> static cudaError_t launch_fp4(Fp4Params& p, const Fp4Operands& o, const DeviceView& dv, cudaStream_t stream)
{
    Fp4Plan t = {0, 0, 0};
    // (tiles of 16 and 32 tokens are for the only tile: the kernel says why)
    if (p.m <= 16) plan_tile<NV, 16>(p, dv, &t);
    else {
        if (p.m <= 32) plan_tile<NV, 32>(p, dv, &t);
        plan_tile<NV, 64>(p, dv, &t);
        if (p.m > 64) plan_tile<NV, 128>(p, dv, &t);
    }
    if (p.m > 64) {
        const long long tiles = (p.n + 2 * kFp4Rows - 1) / (2 * kFp4Rows) * ((p.m + kFp4PairTokens - 1) / kFp4PairTokens);
        const long long waves = (tiles + dv.sms / 2 - 1) / (dv.sms / 2), steps = (p.k + kFp4Step - 1) / kFp4Step;
        if (9500 + most(waves * steps * 600, weight_cycles(p, NV)) < t.cycles) return launch_pair<NV>(p, o, dv, stream);
    }
    switch (t.tokens) {
    case 16: return launch_tile<NV, 16>(p, o, t.cluster, stream);
    case 32: return launch_tile<NV, 32>(p, o, t.cluster, stream);
    case 64: return launch_tile<NV, 64>(p, o, t.cluster, stream);
    default: return launch_tile<NV, 128>(p, o, t.cluster, stream);
    }
}

template <bool NV>
static rmsq_status matmul_fp4(const Fp4Operands& o, const float* a_gs, const float* w_gs, const void* bias, int64_t m, int64_t n,
                              int64_t k, void* output, int output_dtype, void* stream)
{
    if (output_dtype != RMSQ_BF16 && output_dtype != RMSQ_FP16 && output_dtype != RMSQ_F32) return RMSQ_ERR_DTYPE;
    if (m < 0 || n < 0 || m > RMSQ_MATMUL_MAX_ROWS || n > RMSQ_MATMUL_MAX_ROWS || k < 32 || k % 32 != 0 ||
        k > RMSQ_MATMUL_FP4_MAX_K)
        return RMSQ_ERR_SHAPE;
    if (m == 0 || n == 0) return RMSQ_OK;
    if (!o.a || !o.sa || !o.w || !o.sw || !output) return RMSQ_ERR_NULL;
    if (!aligned(o.a, 16) || !aligned(o.sa, 16) || !aligned(o.w, 16) || !aligned(o.sw, 16) || !aligned(a_gs, 4) ||
        !aligned(w_gs, 4) || !aligned(bias, 16) || !aligned(output, 16))
        return RMSQ_ERR_ALIGN;
    DeviceView dv;
    if (!device_view(&dv)) return RMSQ_ERR_DEVICE;
    Fp4Params p = {};
    p.a_gs = a_gs;
    p.w_gs = w_gs;
    p.bias = bias;
    p.out = output;
    p.err = dv.err;
    p.m = m;
    p.n = n;
    p.k = static_cast<int>(k);
    p.dt = output_dtype;
    p.wait = dv.wait;
    p.drain = dv.drain;
    const cudaError_t e = launch_fp4<NV>(p, o, dv, static_cast<cudaStream_t>(stream));
    if (e == cudaSuccess) return RMSQ_OK;
    cudaGetLastError();
    return RMSQ_ERR_LAUNCH;
}

}  // namespace rmsq

using namespace rmsq;

extern "C" rmsq_status matmul_nvfp4(const void* input, const void* input_scale, const float* input_gs, const void* weight,
                                    const void* weight_scale, const float* weight_gs, const void* bias, int64_t m, int64_t n,
                                    int64_t k, void* output, int output_dtype, void* stream)
{
    return matmul_fp4<true>({input, input_scale, weight, weight_scale}, input_gs, weight_gs, bias, m, n, k, output,
                            output_dtype, stream);
}

extern "C" rmsq_status matmul_mxfp4(const void* input, const void* input_scale, const void* weight, const void* weight_scale,
                                    const void* bias, int64_t m, int64_t n, int64_t k, void* output, int output_dtype,
                                    void* stream)
{
    return matmul_fp4<false>({input, input_scale, weight, weight_scale}, nullptr, nullptr, bias, m, n, k, output,
                             output_dtype, stream);
}
