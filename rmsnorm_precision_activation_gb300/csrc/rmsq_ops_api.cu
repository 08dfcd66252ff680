// rmsq_ops_api.cu -- C ABI of layer norm, its gradient and the norms to int8: argument checks,
// launch plans and entry points (declared in include/rmsq.h).
#include <climits>
#include <cmath>
#include <cstdint>

#include "rmsq_norm_bwd.cuh"
#include "rmsq_ops.h"

namespace rmsq {

static bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

static bool known_dtype(int dtype)
{
    return dtype == RMSQ_BF16 || dtype == RMSQ_FP16 || dtype == RMSQ_F32;
}

static bool known_hidden(int64_t hidden, int dtype)
{
    return hidden >= 1 && hidden <= (dtype == RMSQ_F32 ? RMSQ_MAX_HIDDEN / 2 : RMSQ_MAX_HIDDEN);
}

static int elem_bytes(int dtype) { return dtype == RMSQ_F32 ? 4 : 2; }

static rmsq_status status_of(cudaError_t e)
{
    if (e == cudaSuccess) return RMSQ_OK;
    cudaGetLastError();
    return RMSQ_ERR_LAUNCH;
}

// Elements of a row that one CTA takes: 512 threads of 32 elements forward, of 16 backward (whose
// threads also hold two column sums per element). Wider rows are split evenly over the smallest
// cluster of 2, 4, 8 or 16 CTAs, in whole vectors where the row has them.
static int cluster_slice(int hidden, int most, int vec, int* cluster)
{
    int c = 1;
    while (static_cast<long long>(c) * most < hidden) c *= 2;
    *cluster = c;
    const int slice = (hidden + c - 1) / c;
    return (slice + vec - 1) / vec * vec;
}

// A warp per row up to 1024 elements (no block barrier), a CTA per row up to 16384, a cluster
// beyond. CTAs take 16 elements per thread up to 8192 elements, then 32.
static rmsq_status launch_norm(cudaError_t (*go)(const NormPlan&, const NormParams&, cudaStream_t),
                               NormParams& p, int64_t rows, int dtype, cudaStream_t stream)
{
    const int per16 = 16 / elem_bytes(dtype);
    NormPlan pl;
    pl.dt = dtype;
    pl.vec = p.hidden % per16 == 0;
    pl.cluster = 1;
    p.rows = rows;
    p.slice = p.hidden;
    if (p.hidden <= 1024) {
        pl.scope = SCOPE_WARP;
        pl.elems = p.hidden <= 256 ? 8 : p.hidden <= 512 ? 16 : 32;
        pl.threads = 256;
        pl.grid = static_cast<unsigned>((rows + 7) / 8);
    } else {
        p.slice = cluster_slice(p.hidden, 512 * 32, pl.vec ? per16 : 1, &pl.cluster);
        pl.scope = pl.cluster > 1 ? SCOPE_CLUSTER : SCOPE_CTA;
        pl.elems = p.slice > 512 * 16 || pl.cluster > 1 ? 32 : 16;
        pl.threads = ((p.slice + pl.elems - 1) / pl.elems + 31) / 32 * 32;
        pl.grid = static_cast<unsigned>(rows * pl.cluster);
    }
    return status_of(go(pl, p, stream));
}

// Checks shared by the forward norms; *empty for a valid rows == 0 call.
static rmsq_status check_norm(const void* input, const void* residual, const void* residual_output,
                              const void* gamma, const void* beta, const void* output, int64_t rows,
                              int64_t hidden, int dtype, float epsilon, float weight_offset, bool* empty)
{
    *empty = false;
    if (!known_dtype(dtype)) return RMSQ_ERR_DTYPE;
    if (rows < 0 || !known_hidden(hidden, dtype) || rows > INT32_MAX / 16) return RMSQ_ERR_SHAPE;
    if (!(epsilon >= 0.0f) || !std::isfinite(epsilon) || !std::isfinite(weight_offset))
        return RMSQ_ERR_VALUE;
    if (rows == 0) {
        *empty = true;
        return RMSQ_OK;
    }
    if (!input || !gamma || !output) return RMSQ_ERR_NULL;
    if ((residual == nullptr) != (residual_output == nullptr)) return RMSQ_ERR_NULL;
    if (!aligned16(input) || !aligned16(gamma) || !aligned16(beta) || !aligned16(residual) ||
        !aligned16(residual_output) || !aligned16(output))
        return RMSQ_ERR_ALIGN;
    return RMSQ_OK;
}

static NormParams norm_params(const void* input, const void* residual, void* residual_output,
                              const void* gamma, const void* beta, int64_t hidden, float epsilon,
                              float weight_offset, void* output)
{
    NormParams p = {};
    p.x = input;
    p.res = residual;
    p.res_out = residual_output;
    p.gamma = gamma;
    p.beta = beta;
    p.out = output;
    p.hidden = static_cast<int>(hidden);
    p.eps = epsilon;
    p.offset = weight_offset;
    return p;
}

static rmsq_status norm_int8(cudaError_t (*go)(const NormPlan&, const NormParams&, cudaStream_t),
                             const void* input, const void* residual, void* residual_output,
                             const void* gamma, const void* beta, int64_t rows, int64_t hidden,
                             int dtype, float epsilon, float weight_offset, void* output,
                             float* scale_output, void* stream)
{
    bool empty = false;
    rmsq_status st = check_norm(input, residual, residual_output, gamma, beta, output, rows, hidden,
                                dtype, epsilon, weight_offset, &empty);
    if (st != RMSQ_OK || empty) return st;
    if (!scale_output) return RMSQ_ERR_NULL;
    if (!aligned16(scale_output)) return RMSQ_ERR_ALIGN;
    DeviceView dv;
    if (!device_view(&dv)) return RMSQ_ERR_DEVICE;
    NormParams p = norm_params(input, residual, residual_output, gamma, beta, hidden, epsilon,
                               weight_offset, output);
    p.scale = scale_output;
    return launch_norm(go, p, rows, dtype, static_cast<cudaStream_t>(stream));
}

}  // namespace rmsq

using namespace rmsq;

extern "C" rmsq_status layernorm(const void* input, const void* residual, void* residual_output,
                                 const void* gamma, const void* beta, int64_t rows, int64_t hidden,
                                 int dtype, float epsilon, float weight_offset, void* output,
                                 float* mean, float* rstd, void* stream)
{
    bool empty = false;
    rmsq_status st = check_norm(input, residual, residual_output, gamma, beta, output, rows, hidden,
                                dtype, epsilon, weight_offset, &empty);
    if (st != RMSQ_OK || empty) return st;
    if (!aligned16(mean) || !aligned16(rstd)) return RMSQ_ERR_ALIGN;
    DeviceView dv;
    if (!device_view(&dv)) return RMSQ_ERR_DEVICE;
    NormParams p = norm_params(input, residual, residual_output, gamma, beta, hidden, epsilon,
                               weight_offset, output);
    p.mean = mean;
    p.rstd = rstd;
    return launch_norm(&norm_layer, p, rows, dtype, static_cast<cudaStream_t>(stream));
}

extern "C" rmsq_status layernorm_quant_int8(const void* input, const void* residual,
                                            void* residual_output, const void* gamma,
                                            const void* beta, int64_t rows, int64_t hidden, int dtype,
                                            float epsilon, float weight_offset, void* output,
                                            float* scale_output, void* stream)
{
    return norm_int8(&norm_layer_int8, input, residual, residual_output, gamma, beta, rows, hidden,
                     dtype, epsilon, weight_offset, output, scale_output, stream);
}

extern "C" rmsq_status rmsnorm_quant_int8(const void* input, const void* residual,
                                          void* residual_output, const void* gamma, int64_t rows,
                                          int64_t hidden, int dtype, float epsilon,
                                          float weight_offset, void* output, float* scale_output,
                                          void* stream)
{
    return norm_int8(&norm_rms_int8, input, residual, residual_output, gamma, nullptr, rows, hidden,
                     dtype, epsilon, weight_offset, output, scale_output, stream);
}

// Partial rows of the column sums: at most one per CTA of a GB300 (152), and no more than rows.
static int64_t bwd_parts(int64_t rows)
{
    return rows < RMSQ_LAYERNORM_PARTS ? rows : RMSQ_LAYERNORM_PARTS;
}

extern "C" int64_t layernorm_backward_workspace(int64_t rows, int64_t hidden)
{
    if (rows <= 0 || hidden <= 0 || hidden > RMSQ_MAX_HIDDEN) return 0;
    return bwd_parts(rows) * 2 * hidden * static_cast<int64_t>(sizeof(float));
}

extern "C" rmsq_status layernorm_backward(const void* grad_output, const void* grad_residual,
                                          const void* input, const void* gamma, const float* mean,
                                          const float* rstd, int64_t rows, int64_t hidden, int dtype,
                                          float weight_offset, void* grad_input, void* grad_gamma,
                                          void* grad_beta, int param_grad_dtype, void* workspace,
                                          int64_t workspace_bytes, void* stream)
{
    if (!known_dtype(dtype)) return RMSQ_ERR_DTYPE;
    if (param_grad_dtype != dtype && param_grad_dtype != RMSQ_F32) return RMSQ_ERR_DTYPE;
    if (rows < 0 || rows > INT32_MAX / 16 || !known_hidden(hidden, dtype)) return RMSQ_ERR_SHAPE;
    if (!std::isfinite(weight_offset)) return RMSQ_ERR_VALUE;
    if (!grad_gamma) return RMSQ_ERR_NULL;
    if (!aligned16(grad_gamma) || !aligned16(grad_beta)) return RMSQ_ERR_ALIGN;
    if (rows > 0) {
        if (!grad_output || !input || !gamma || !mean || !rstd || !grad_input || !workspace)
            return RMSQ_ERR_NULL;
        if (!aligned16(grad_output) || !aligned16(grad_residual) || !aligned16(input) ||
            !aligned16(gamma) || !aligned16(mean) || !aligned16(rstd) || !aligned16(grad_input) ||
            !aligned16(workspace))
            return RMSQ_ERR_ALIGN;
        if (workspace_bytes < layernorm_backward_workspace(rows, hidden)) return RMSQ_ERR_SHAPE;
    }
    DeviceView dv;
    if (!device_view(&dv)) return RMSQ_ERR_DEVICE;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);

    NormBwdReduceParams r = {};
    r.part = static_cast<const float*>(workspace);
    r.dgamma = grad_gamma;
    r.dbeta = grad_beta;
    r.hidden = static_cast<int>(hidden);
    r.dt = param_grad_dtype;

    if (rows > 0) {
        NormBwdParams p = {};
        p.in[0] = grad_output;
        p.in[1] = input;
        p.in[2] = grad_residual;
        p.gamma = gamma;
        p.mean = mean;
        p.rstd = rstd;
        p.ds = grad_input;
        p.part = static_cast<float*>(workspace);
        p.err = dv.err;
        p.rows = rows;
        p.hidden = static_cast<int>(hidden);
        p.offset = weight_offset;
        p.timeout_ns = dv.timeout_ns;

        const int es = elem_bytes(dtype), per16 = 16 / es;
        const bool vec = hidden % per16 == 0;
        int cluster = 1;
        p.slice = cluster_slice(p.hidden, kBwdThreads * 16, vec ? per16 : 1, &cluster);
        const int elems = p.slice <= 256 ? 8 : 16;
        p.T = ((p.slice + elems - 1) / elems + 31) / 32 * 32;
        // Row groups: as many as 512 threads hold, but no more than it takes to give every CTA
        // of the device a row.
        p.groups = cluster > 1 ? 1 : kBwdThreads / p.T;
        const int64_t spread = (rows + dv.sms - 1) / dv.sms;
        if (p.groups > spread) p.groups = static_cast<int>(spread);
        p.slot = vec ? p.slice * es : (p.slice * es + 30) / 16 * 16;
        const int64_t stage = static_cast<int64_t>(p.slot) * (grad_residual ? 3 : 2) * p.groups;
        int64_t stages = (dv.smem_optin - kBwdHead) / stage;
        if (stages < 1) return RMSQ_ERR_LAUNCH;
        p.stages = static_cast<int>(stages > kBwdMaxStages ? kBwdMaxStages : stages);
        int64_t ring = p.stages * stage;
        if (p.groups > 1 && ring < 8LL * p.slice) ring = 8LL * p.slice;   // the groups' sums
        int64_t parts = (rows + p.groups - 1) / p.groups;
        const int64_t resident = dv.sms / cluster;
        if (parts > resident) parts = resident;
        if (parts > bwd_parts(rows)) parts = bwd_parts(rows);
        if (parts < 1) return RMSQ_ERR_LAUNCH;
        r.parts = static_cast<int>(parts);
        void* args[] = {&p};
        const rmsq_status e = status_of(launch_kernel(
            norm_bwd_fn(dtype, elems, vec), static_cast<unsigned>(parts * cluster),
            static_cast<unsigned>(p.T * p.groups), static_cast<int>(kBwdHead + ring), cluster, st, args));
        if (e != RMSQ_OK) return e;
    }
    void* args[] = {&r};
    return status_of(launch_kernel(norm_bwd_reduce_fn(), static_cast<unsigned>((2 * hidden + 31) / 32), 512, 0,
                                   1, st, args));
}
