// rmsq_norm_bwd.cu -- instantiations of layer norm's backward kernels.
#include "rmsq_norm_bwd.cuh"
#include "rmsq_ops.h"

namespace rmsq {

template <int DT> static const void* pick(int elems, bool vec)
{
    if (elems == 8)
        return vec ? reinterpret_cast<const void*>(&rmsq_norm_bwd_kernel<DT, 8, true>)
                   : reinterpret_cast<const void*>(&rmsq_norm_bwd_kernel<DT, 8, false>);
    return vec ? reinterpret_cast<const void*>(&rmsq_norm_bwd_kernel<DT, 16, true>)
               : reinterpret_cast<const void*>(&rmsq_norm_bwd_kernel<DT, 16, false>);
}

const void* norm_bwd_fn(int dt, int elems, bool vec)
{
    return dt == DT_BF16 ? pick<DT_BF16>(elems, vec) : dt == DT_FP16 ? pick<DT_FP16>(elems, vec)
                                                                     : pick<DT_F32>(elems, vec);
}

const void* norm_bwd_reduce_fn() { return reinterpret_cast<const void*>(&rmsq_norm_bwd_reduce_kernel); }

}  // namespace rmsq
