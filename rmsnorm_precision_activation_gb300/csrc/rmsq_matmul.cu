// rmsq_matmul.cu -- C ABI of the int8 product: argument checks and the choice of kernel.
#include <cstdint>

#include "rmsq_matmul.cuh"
#include "rmsq_ops.h"

namespace rmsq {

static bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

static cudaError_t launch_few(MatmulParams& p, const DeviceView& dv, cudaStream_t stream)
{
    const int mt = p.m <= 1 ? 1 : p.m <= 2 ? 2 : p.m <= 4 ? 4 : 8;
    const void* fn = mt == 1 ? reinterpret_cast<const void*>(&rmsq_matmul_few_kernel<1>)
                   : mt == 2 ? reinterpret_cast<const void*>(&rmsq_matmul_few_kernel<2>)
                   : mt == 4 ? reinterpret_cast<const void*>(&rmsq_matmul_few_kernel<4>)
                             : reinterpret_cast<const void*>(&rmsq_matmul_few_kernel<8>);
    const long long tiles = (p.n + kFewRows - 1) / kFewRows, mtiles = (p.m + mt - 1) / mt;
    // warps sharing a channel: until there are 32 warps per SM, or a warp has two pieces left
    p.ksplit = 1;
    while (p.ksplit < kFewWarps && tiles * mtiles * p.ksplit < 32LL * dv.sms && p.k > 1024 * p.ksplit) p.ksplit *= 2;
    const long long per = kFewWarps / p.ksplit;
    void* args[] = {&p};
    return launch_kernel(fn, dim3(static_cast<unsigned>((tiles + per - 1) / per), static_cast<unsigned>(mtiles)),
                         kFewWarps * 32, 0, 1, stream, args);
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
    p.timeout_ns = dv.timeout_ns;
    const cudaError_t e = launch_few(p, dv, static_cast<cudaStream_t>(stream));
    if (e == cudaSuccess) return RMSQ_OK;
    cudaGetLastError();
    return RMSQ_ERR_LAUNCH;
}
