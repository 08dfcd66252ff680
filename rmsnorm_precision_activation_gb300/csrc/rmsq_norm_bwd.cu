// rmsq_norm_bwd.cu -- instantiations of layer norm's backward kernels.
#include "rmsq_norm_bwd.cuh"
#include "rmsq_ops.h"

namespace rmsq {

template <int DT, int E, bool FULL, bool EDGE, bool CLUSTER> static const void* kernel()
{
    return reinterpret_cast<const void*>(&rmsq_norm_bwd_kernel<DT, E, FULL, EDGE, CLUSTER>);
}

template <int DT, bool FULL, bool EDGE> static const void* pick(int elems, bool cluster)
{
    // (slices of more than 7680 elements are no multiple of 32 x 24, and fp32 slices have 4100 at most)
    if constexpr (!FULL && DT != DT_F32) {
        if (elems == 24) return kernel<DT, 24, FULL, EDGE, true>();
    }
    if (cluster) return kernel<DT, 16, FULL, EDGE, true>();
    return elems == 8 ? kernel<DT, 8, FULL, EDGE, false>() : kernel<DT, 16, FULL, EDGE, false>();
}

template <int DT> static const void* pick(int elems, bool full, bool vec, bool cluster)
{
    if (!vec) return pick<DT, false, true>(elems, cluster);
    return full ? pick<DT, true, false>(elems, cluster) : pick<DT, false, false>(elems, cluster);
}

const void* norm_bwd_fn(int dt, int elems, bool full, bool vec, bool cluster)
{
    return dt == DT_BF16 ? pick<DT_BF16>(elems, full, vec, cluster)
         : dt == DT_FP16 ? pick<DT_FP16>(elems, full, vec, cluster)
                         : pick<DT_F32>(elems, full, vec, cluster);
}

const void* norm_bwd_reduce_fn() { return reinterpret_cast<const void*>(&rmsq_norm_bwd_reduce_kernel); }

}  // namespace rmsq
