// rmsq_norm_layer.cu -- instantiations of the register-row norm kernel for NORM_LAYER.
#include "rmsq_ops.h"

namespace rmsq {
RMSQ_DEFINE_NORM_DISPATCH(norm_layer, NORM_LAYER)
}  // namespace rmsq
