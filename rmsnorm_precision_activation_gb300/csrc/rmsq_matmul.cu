// rmsq_matmul.cu -- C ABI of the int8 product: argument checks and the choice of kernel.
#include <atomic>
#include <cstdint>

#include "rmsq_matmul_pair.cuh"
#include "rmsq_ops.h"
#include "rmsq_tensor_map.h"

namespace rmsq {

static bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <int NB, int ROWS> static cudaError_t launch_stream(MatmulParams& p, cudaStream_t stream)
{
    void* args[] = {&p};
    return launch_kernel(reinterpret_cast<const void*>(&rmsq_matmul_stream_kernel<NB, ROWS>),
                         dim3(static_cast<unsigned>((p.n + ROWS - 1) / ROWS)), kStreamWarps * 32, 0, 1, stream, args);
}

// 16 channels per CTA where all of the CTAs run at a time then, else 32 (GB300, 1 token, n x k: 7168 x 8192
// 12.1 us against 13.2, 1024 x 4096 3.3 against 4.3, 300 x 16384 7.4 against 10.6; 8192 x 8192, which
// takes more than one wave of 16, 15.9 against 14.0; 16 tokens 5000 x 8192 14.6 against 15.5).
template <int NB> static cudaError_t launch_stream(MatmulParams& p, const DeviceView& dv, cudaStream_t stream)
{
    if (p.n <= static_cast<long long>(dv.sms) * kStreamHalves * 16) return launch_stream<NB, 16>(p, stream);
    return launch_stream<NB, 32>(p, stream);
}

// Codes [rows x k], read in boxes of box_rows x 128 elements.
static bool encode(CUtensorMap* map, const void* codes, long long rows, int k, int box_rows)
{
    return encode_map(map, codes, 1, rows, k, box_rows, kTcCodes, CU_TENSOR_MAP_SWIZZLE_128B);
}

// CTAs that share a tile's k: as many as let all tiles run at a time, each with at least 2 code stages.
// What fits goes by the device's clusters of SMs, not by SMs alone: 100 x 2400 x 8192 (19 tiles of 128
// tokens) takes 15.9 us in clusters of 6, of which 23 fit, and 26.2 in clusters of 8, of which 15 do.
template <int NT> static int tc_cluster(long long tiles, int steps, const DeviceView& dv)
{
    const void* fn = reinterpret_cast<const void*>(&rmsq_matmul_tc_kernel<NT>);
    int best = 1;
    for (int c = 2; c <= 8 && c * 2 <= steps && c * tiles <= dv.sms * TcShape<NT>::CTAS; ++c)
        if (tiles <= resident_clusters(fn, TcShape<NT>::THREADS, TcShape<NT>::SMEM, c)) best = c;
    return best;
}

template <int NT> static cudaError_t launch_tc(MatmulParams& p, const DeviceView& dv, cudaStream_t stream)
{
    CUtensorMap map_w, map_a;
    if (!encode(&map_w, p.w, p.n, p.k, kTcRows) || !encode(&map_a, p.a, p.m, p.k, NT)) return cudaErrorUnknown;
    TcTiles t;
    t.n_tiles = static_cast<int>((p.n + kTcRows - 1) / kTcRows);
    t.m_tiles = static_cast<int>((p.m + NT - 1) / NT);
    const long long tiles = static_cast<long long>(t.n_tiles) * t.m_tiles;
    const long long slots = static_cast<long long>(dv.sms) * TcShape<NT>::CTAS;
    const int steps = (p.k + kTcCodes - 1) / kTcCodes;
    const int cluster = tc_cluster<NT>(tiles, steps, dv);
    const long long grid = cluster > 1 ? tiles * cluster : tiles < slots ? tiles : slots;
    void* args[] = {&map_w, &map_a, &p, &t};
    return launch_kernel(reinterpret_cast<const void*>(&rmsq_matmul_tc_kernel<NT>),
                         dim3(static_cast<unsigned>(grid)), TcShape<NT>::THREADS, TcShape<NT>::SMEM,
                         static_cast<int>(cluster), stream, args);
}

template <int TOKENS> static cudaError_t launch_pair(MatmulParams& p, const DeviceView& dv, cudaStream_t stream)
{
    // setmaxnreg moves registers that the launch must have
    static std::atomic<int> regs{0};
    const void* fn = reinterpret_cast<const void*>(&rmsq_matmul_pair_kernel<TOKENS>);
    if (regs.load() == 0) {
        cudaFuncAttributes fa;
        const cudaError_t e = cudaFuncGetAttributes(&fa, fn);
        if (e != cudaSuccess) return e;
        regs.store(fa.numRegs);
    }
    if (regs.load() < kPairRegs) return cudaErrorInvalidConfiguration;
    CUtensorMap map_w, map_a;
    if (!encode(&map_w, p.w, p.n, p.k, kTcRows) || !encode(&map_a, p.a, p.m, p.k, PairShape<TOKENS>::HALF)) return cudaErrorUnknown;
    TcTiles t;
    t.n_tiles = static_cast<int>((p.n + 2 * kTcRows - 1) / (2 * kTcRows));
    t.m_tiles = static_cast<int>((p.m + TOKENS - 1) / TOKENS);
    const long long tiles = static_cast<long long>(t.n_tiles) * t.m_tiles;
    const long long pairs = tiles < dv.sms / 2 ? tiles : dv.sms / 2;
    void* args[] = {&map_w, &map_a, &p, &t};
    return launch_kernel(fn, dim3(static_cast<unsigned>(2 * pairs)), kTcThreads, PairShape<TOKENS>::SMEM, 2, stream, args);
}

// The kernel, by tokens (GB300, weights from HBM, n x k = 8192 x 8192 where not given):
//   up to 16: mma.sync, 16.8 us at 16 tokens (tcgen05: 20.4), but 23.9 at 32 (tcgen05: 20.7)
//   up to 32, up to 64: tiles of 32 and 64 tokens, 20.7 and 21.8 us (of 128: 27.8)
//   more: what takes least by the time of a step of 128 elements of k in each kernel (hundredths of a
//   us, with a CTA or pair on every SM) and the steps its CTAs take one after another. Measured, in the
//   order tiles of 128, pairs of 128, pairs of 192:  128 tokens 29.3, 33.3, 40.9 us;  200 47.0, 34.2, 42.3;
//   512 87, 60, 74;  768 128, 87, 76;  4096 570, 376, 337;  1024 x 1024 x 8192 28.5, 32.9, 40.2.
static cudaError_t launch_matmul(MatmulParams& p, const DeviceView& dv, cudaStream_t stream)
{
    if (p.m <= 8) return launch_stream<1>(p, dv, stream);
    if (p.m <= 16) return launch_stream<2>(p, dv, stream);
    if (p.m <= 32) return launch_tc<32>(p, dv, stream);
    if (p.m <= 64) return launch_tc<64>(p, dv, stream);
    const int steps = (p.k + kTcCodes - 1) / kTcCodes;
    const auto tiles = [&](int channels, int tokens) {
        return (p.n + channels - 1) / channels * ((p.m + tokens - 1) / tokens);
    };
    const auto waves = [](long long work, int places) { return (work + places - 1) / places; };
    const long long one = tiles(kTcRows, 128);
    const int cluster = tc_cluster<128>(one, steps, dv);
    const long long t1 = waves(one, dv.sms) * ((steps + cluster - 1) / cluster) * 58;
    const long long t128 = waves(tiles(2 * kTcRows, 128), dv.sms / 2) * steps * 42;
    const long long t192 = waves(tiles(2 * kTcRows, 192), dv.sms / 2) * steps * 52;
    if (t1 < t128 && t1 < t192) return launch_tc<128>(p, dv, stream);
    return t128 < t192 ? launch_pair<128>(p, dv, stream) : launch_pair<192>(p, dv, stream);
}

}  // namespace rmsq

using namespace rmsq;

extern "C" rmsq_status matmul_int8(const void* input, const float* input_scale, const void* weight,
                                   const float* weight_scale, const void* bias, int64_t m, int64_t n,
                                   int64_t k, void* output, int output_dtype, void* stream)
{
    if (output_dtype != RMSQ_BF16 && output_dtype != RMSQ_FP16 && output_dtype != RMSQ_F32)
        return RMSQ_ERR_DTYPE;
    if (m < 0 || n < 0 || m > RMSQ_MATMUL_MAX_ROWS || n > RMSQ_MATMUL_MAX_ROWS || k < 16 || k % 16 != 0 ||
        k > RMSQ_MATMUL_MAX_K)
        return RMSQ_ERR_SHAPE;
    if (m == 0 || n == 0) return RMSQ_OK;
    if (!input || !input_scale || !weight || !weight_scale || !output) return RMSQ_ERR_NULL;
    if (!aligned16(input) || !aligned16(input_scale) || !aligned16(weight) || !aligned16(weight_scale) ||
        !aligned16(bias) || !aligned16(output))
        return RMSQ_ERR_ALIGN;
    DeviceView dv;
    if (!device_view(&dv)) return RMSQ_ERR_DEVICE;
    MatmulParams p = {};
    p.a = static_cast<const signed char*>(input);
    p.a_scale = input_scale;
    p.w = static_cast<const signed char*>(weight);
    p.w_scale = weight_scale;
    p.bias = bias;
    p.out = output;
    p.err = dv.err;
    p.m = m;
    p.n = n;
    p.k = static_cast<int>(k);
    p.dt = output_dtype;
    p.wait = dv.wait;
    p.drain = dv.drain;
    const cudaError_t e = launch_matmul(p, dv, static_cast<cudaStream_t>(stream));
    if (e == cudaSuccess) return RMSQ_OK;
    cudaGetLastError();
    return RMSQ_ERR_LAUNCH;
}
