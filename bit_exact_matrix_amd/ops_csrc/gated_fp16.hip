// gated_fp16.hip -- the FP16 kernels of gated.h
#include "gated.h"

namespace mmaops {

GatedLaunches gated_fp16() { return gated_launches<kFP16>(); }

}  // namespace mmaops
