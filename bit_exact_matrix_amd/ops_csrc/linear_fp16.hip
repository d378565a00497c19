// linear_fp16.hip -- the FP16 products of linear.h
#include "linear.h"

namespace mmaops {

hipError_t linear_launch_fp16(int tile, bool direct, int la, int lb, const LinearArgs& g,
                             hipStream_t s) {
  return linear_launch<kFP16>(tile, direct, la, lb, g, s);
}

}  // namespace mmaops
