// rmsq_norm_rms_int8.cu -- instantiations of the register-row norm kernel for NORM_RMS_INT8.
#include "rmsq_ops.h"

namespace rmsq {
RMSQ_DEFINE_NORM_DISPATCH(norm_rms_int8, NORM_RMS_INT8)
}  // namespace rmsq
