// rmsq_norm_layer_int8.cu -- instantiations of the register-row norm kernel for NORM_LAYER_INT8.
#include "rmsq_ops.h"

namespace rmsq {
RMSQ_DEFINE_NORM_DISPATCH(norm_layer_int8, NORM_LAYER_INT8)
}  // namespace rmsq
