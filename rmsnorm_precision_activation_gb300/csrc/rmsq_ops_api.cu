// rmsq_ops_api.cu -- C ABI of layer norm, its gradient and the norms to int8: argument checks,
// launch plans and entry points (declared in include/rmsq.h).
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

// Launch of a forward norm. Who takes a row, and in what shares (GB300, rows x hidden, bf16):
//  - up to 1024 columns a warp, of 8, 16 or 32 elements a thread;
//  - up to 16384 a CTA, of 32 elements a thread as fp32 (16 elements: 16384 x 8192 117 us, 32: 86);
//  - wider 16-bit rows a CTA of 64 elements a thread, packed: 4096 x 20000 58.5 us (clusters of fp32
//    shares: 83), 4096 x 32768 89 us (131); and rows from 8193 on without a residual and off no 16-byte
//    boundary: 8192 x 12000 65 us (fp32 shares: 82), but with a residual 123 (118), 8192 x 14001 136 (132),
//    to int8 96 (93), which forms y twice then. (100 x 12000 takes 4.7 us packed, 3.5 not; the choice does
//    not go by the number of rows, so that a row's bits do not depend on the others.)
//  - rows wider than a CTA takes a cluster of 4 or 8: 2048 x 65536 106 us, in clusters of 2 some 5 % more.
static rmsq_status launch_norm(cudaError_t (*go)(const NormPlan&, const NormParams&, cudaStream_t),
                               NormParams& p, int64_t rows, int dtype, cudaStream_t stream)
{
    NormPlan pl;
    const int hidden = p.hidden, vw = 16 / elem_bytes(dtype);
    p.rows = static_cast<int>(rows);
    pl.dt = dtype;
    pl.vec = hidden % vw == 0;
    const int columns = pl.vec ? hidden : hidden + vw - 1;      // from a row's 16-byte boundary on
    const bool packed = dtype != RMSQ_F32 &&
                        (columns > 16384 || (columns > 8192 && pl.vec && p.residual == nullptr && p.scale == nullptr));
    pl.elems = columns <= 256 ? 8 : columns <= 512 ? 16 : packed ? 64 : 32;
    const int most = 512 * pl.elems;                            // of a CTA
    pl.cluster = columns <= most ? 1 : columns < 2 * most + vw ? 4 : 8;
    pl.scope = columns <= 1024 ? SCOPE_WARP : pl.cluster == 1 ? SCOPE_CTA : SCOPE_CLUSTER;
    p.slice = ((columns + pl.cluster - 1) / pl.cluster + vw - 1) / vw * vw;
    const int T = (p.slice + 32 * pl.elems - 1) / (32 * pl.elems) * 32;
    pl.full = T * pl.elems == p.slice && p.slice * pl.cluster == hidden;
    pl.threads = pl.scope == SCOPE_WARP ? 256 : T;
    pl.grid = static_cast<unsigned>(pl.scope == SCOPE_WARP ? (rows + 7) / 8 : rows * pl.cluster);
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
    p.residual = residual;
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

// How a row is dealt out in the backward pass: split evenly, in whole vectors, over the smallest cluster of
// 1, 2, 4, 8 or 16 CTAs whose slices take at most kRingSlice bytes (off 16-byte boundaries a vector more); a
// slice takes T threads of `elems` elements. (Clusters of other sizes fill the SMs worse: 4096 x 20000 bf16
// 137 us in clusters of 4, 191 of 3. Halved slices and two CTAs on an SM: 8192 x 16384 236 us against 164.)
struct RowGeometry {
    int cluster, slice, elems, T, slot;
    int period;      // rows after which the shift off 16-byte boundaries repeats
};

static RowGeometry row_geometry(int hidden, int dtype)
{
    const int es = elem_bytes(dtype), vw = 16 / es;
    RowGeometry g;
    g.period = 1;
    while (static_cast<long long>(g.period) * hidden % vw != 0) ++g.period;
    const int columns = g.period == 1 ? hidden : hidden + vw - 1;
    const int most = kRingSlice / es + (g.period == 1 ? 0 : vw);
    g.cluster = 1;
    while (g.cluster < 16 && g.cluster * most < columns) g.cluster *= 2;
    g.slice = ((columns + g.cluster - 1) / g.cluster + vw - 1) / vw * vw;
    g.elems = g.slice <= 256 ? 8 : g.slice <= row_warps(16) * 32 * 16 ? 16 : 24;
    g.T = ((g.slice + g.elems - 1) / g.elems + 31) / 32 * 32;
    g.slot = g.slice * es;
    return g;
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
        p.r.in[0] = grad_output;
        p.r.in[1] = input;
        p.r.in[2] = grad_residual;
        p.gamma = gamma;
        p.mean = mean;
        p.rstd = rstd;
        p.ds = grad_input;
        p.part = static_cast<float*>(workspace);
        p.err = dv.err;
        p.r.ntens = grad_residual != nullptr ? 3 : 2;
        p.r.rows = static_cast<int>(rows);
        p.r.hidden = static_cast<int>(hidden);
        p.r.total = rows * hidden * elem_bytes(dtype);
        p.offset = weight_offset;
        p.wait = dv.wait;
        p.drain = dv.drain;

        const RowGeometry g = row_geometry(p.r.hidden, dtype);
        p.r.slice = g.slice;
        p.r.slot = g.slot;
        p.T = g.T;
        const int cluster = g.cluster;
        // short rows leave room for several row groups in a CTA, which takes no more than give every SM a row
        const int64_t spread = (rows + dv.sms - 1) / dv.sms;
        p.groups = cluster > 1 ? 1 : row_warps(g.elems) * 32 / g.T;
        if (p.groups > spread) p.groups = static_cast<int>(spread);
        // at least two pairs of rows in the ring: one is refilled while the other is worked on
        auto slots = [&]() {
            return (dv.smem_optin - kBwdHead) / (static_cast<int64_t>(p.r.slot) * p.r.ntens * p.groups);
        };
        while (p.groups > 1 && slots() < 4) --p.groups;
        const int64_t stages = slots();
        if (stages < 4) return RMSQ_ERR_LAUNCH;
        p.r.stages = static_cast<int>(stages > kRingStages ? kRingStages : stages) & ~1;
        // (4 stages of 2 tensors at least, so the groups' sums, 8 bytes an element, fit where the ring was)
        const int64_t ring = static_cast<int64_t>(p.r.stages) * p.r.slot * p.r.ntens * p.groups;
        const void* fn = norm_bwd_fn(dtype, g.elems, g.T * g.elems == g.slice && g.slice * cluster == hidden, g.period == 1,
                                     cluster > 1);
        const unsigned threads = static_cast<unsigned>(p.T * p.groups + 32);
        const int smem = static_cast<int>(kBwdHead + ring);
        int64_t resident = cluster == 1 ? dv.sms : resident_clusters(fn, threads, smem, cluster);
        if (resident < 1) resident = dv.sms / cluster;                  // not known
        const int64_t parts = bwd_clusters(rows, p.groups, g.period, resident, bwd_parts(rows));
        r.parts = static_cast<int>(parts);
        void* args[] = {&p};
        const rmsq_status e = status_of(launch_kernel(
            fn, static_cast<unsigned>(parts * cluster), threads, smem, cluster, st, args));
        if (e != RMSQ_OK) return e;
    }
    void* args[] = {&r};
    return status_of(launch_kernel(norm_bwd_reduce_fn(), static_cast<unsigned>((2 * hidden + 31) / 32), 512, 0,
                                   1, st, args));
}
