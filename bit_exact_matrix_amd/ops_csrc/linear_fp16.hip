// linear_fp16.hip -- the FP16 products of linear.h
#include "linear.h"

namespace mmaops {

hipError_t linear_launch_fp16(int tile, bool direct, int la, int lb, const LinearArgs& g,
                             hipStream_t s) {
  return linear_launch<kFP16>(tile, direct, la, lb, g, s);
}

hipError_t pair_launch_fp16(int lb, const PairArgs& p, hipStream_t s) {
  return pair_launch<kFP16>(lb, p, s);
}

}  // namespace mmaops
