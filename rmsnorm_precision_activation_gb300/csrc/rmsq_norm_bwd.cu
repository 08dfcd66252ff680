// rmsq_norm_bwd.cu -- instantiations of layer norm's backward kernels.
#include "rmsq_norm_bwd.cuh"
#include "rmsq_ops.h"

namespace rmsq {

template <int DT, bool FULL, bool EDGE> static const void* pick(int elems)
{
    // (slices of more than 7680 elements are no multiple of 32 x 24, and fp32 slices have 4100 at most)
    if constexpr (!FULL && DT != DT_F32) {
        if (elems == 24) return reinterpret_cast<const void*>(&rmsq_norm_bwd_kernel<DT, 24, FULL, EDGE>);
    }
    return elems == 8 ? reinterpret_cast<const void*>(&rmsq_norm_bwd_kernel<DT, 8, FULL, EDGE>)
                      : reinterpret_cast<const void*>(&rmsq_norm_bwd_kernel<DT, 16, FULL, EDGE>);
}

template <int DT> static const void* pick(int elems, bool full, bool vec)
{
    if (!vec) return pick<DT, false, true>(elems);
    return full ? pick<DT, true, false>(elems) : pick<DT, false, false>(elems);
}

const void* norm_bwd_fn(int dt, int elems, bool full, bool vec)
{
    return dt == DT_BF16 ? pick<DT_BF16>(elems, full, vec) : dt == DT_FP16 ? pick<DT_FP16>(elems, full, vec)
                                                                           : pick<DT_F32>(elems, full, vec);
}

const void* norm_bwd_reduce_fn() { return reinterpret_cast<const void*>(&rmsq_norm_bwd_reduce_kernel); }

}  // namespace rmsq
