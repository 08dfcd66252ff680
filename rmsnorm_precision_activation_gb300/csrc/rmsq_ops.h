// rmsq_ops.h -- host-side plumbing of the layer-norm and int8 operators: what they share with the
// quantising RMS-norm entry points (device facts, launches), and their dispatch.
#pragma once

#include <cuda_runtime.h>

#include "rmsq.h"
#include "rmsq_norm.cuh"
#include "rmsq_ops_plan.h"

namespace rmsq {

// Facts about the current device and the process's settings (rmsq_api.cu).
struct DeviceView {
    int sms;
    int smem_optin;
    unsigned int* err;                // device error word
    uint32_t wait, drain;             // bounds of device-side waits (rmsq_ops_plan.h)
};
// False: no usable device.
bool device_view(DeviceView* v);

// Launches fn on the stream with programmatic dependent launch (as rmsq_set_pdl says), in clusters
// of `cluster` CTAs when that is over 1, and counts the launch. Sets the function's attributes on
// its first launch on a device.
cudaError_t launch_kernel(const void* fn, dim3 grid, unsigned threads, int smem, int cluster,
                          cudaStream_t stream, void** args);

// How many clusters of that size (1 to 16 CTAs) the current device runs at a time; 0: not known.
int resident_clusters(const void* fn, unsigned threads, int smem, int cluster);

struct NormPlan {
    int dt;
    int elems;      // per thread: 8 or 16 (short rows), 32, or 64 (16-bit types, packed)
    bool vec;       // rows are whole vectors of 16 bytes
    bool full;      // the threads' shares cover the row exactly
    int scope;      // SCOPE_*
    int threads;
    unsigned grid;
    int cluster;
};

cudaError_t norm_layer(const NormPlan& pl, const NormParams& p, cudaStream_t stream);
cudaError_t norm_layer_int8(const NormPlan& pl, const NormParams& p, cudaStream_t stream);
cudaError_t norm_rms_int8(const NormPlan& pl, const NormParams& p, cudaStream_t stream);

// Backward pass (rmsq_norm_bwd.cu): the row kernel for a type, elements per thread (8, 16, or 24 for
// slices of more than 7680 elements of 16 bits), whether the threads cover the slices exactly, whether
// rows are whole vectors and whether they are split over clusters, and the column reduction.
struct NormBwdParams;
const void* norm_bwd_fn(int dt, int elems, bool full, bool vec, bool cluster);
const void* norm_bwd_reduce_fn();

#define RMSQ_DEFINE_NORM_DISPATCH(NAME, KIND)                                                     \
    template <int DT, bool EDGE, bool FULL, int E, int SCOPE> static const void* NAME##_at()      \
    {                                                                                             \
        return reinterpret_cast<const void*>(&rmsq_norm_kernel<DT, E, FULL, EDGE, SCOPE, KIND>);  \
    }                                                                                             \
    template <int DT, bool EDGE, bool FULL> static const void* NAME##_pick(const NormPlan& pl)    \
    {                                                                                             \
        constexpr int WIDE = DT == DT_F32 ? 32 : 64;                                              \
        if (pl.scope == SCOPE_CLUSTER) return NAME##_at<DT, EDGE, FULL, WIDE, SCOPE_CLUSTER>();   \
        if (pl.scope == SCOPE_CTA)                                                                \
            return pl.elems == WIDE ? NAME##_at<DT, EDGE, FULL, WIDE, SCOPE_CTA>()                \
                                    : NAME##_at<DT, EDGE, FULL, 32, SCOPE_CTA>();                 \
        return pl.elems == 8    ? NAME##_at<DT, EDGE, FULL, 8, SCOPE_WARP>()                      \
               : pl.elems == 16 ? NAME##_at<DT, EDGE, FULL, 16, SCOPE_WARP>()                     \
                                : NAME##_at<DT, EDGE, FULL, 32, SCOPE_WARP>();                    \
    }                                                                                             \
    template <int DT> static const void* NAME##_fn(const NormPlan& pl)                            \
    {                                                                                             \
        if (!pl.vec) return NAME##_pick<DT, true, false>(pl);                                     \
        return pl.full ? NAME##_pick<DT, false, true>(pl) : NAME##_pick<DT, false, false>(pl);    \
    }                                                                                             \
    cudaError_t NAME(const NormPlan& pl, const NormParams& p, cudaStream_t stream)                \
    {                                                                                             \
        const void* fn = pl.dt == DT_BF16 ? NAME##_fn<DT_BF16>(pl)                                \
                       : pl.dt == DT_FP16 ? NAME##_fn<DT_FP16>(pl) : NAME##_fn<DT_F32>(pl);       \
        NormParams q = p;                                                                         \
        void* args[] = {&q};                                                                      \
        return launch_kernel(fn, pl.grid, pl.threads, 0, pl.cluster, stream, args);         \
    }

}  // namespace rmsq
