// gated_bf16.hip -- the BF16 kernels of gated.h
#include "gated.h"

namespace mmaops {

GatedLaunches gated_bf16() { return gated_launches<kBF16>(); }

}  // namespace mmaops
