// linear_bf16.hip -- the BF16 products of linear.h
#include "linear.h"

namespace mmaops {

hipError_t linear_launch_bf16(int tile, bool direct, int la, int lb, const LinearArgs& g,
                             hipStream_t s) {
  return linear_launch<kBF16>(tile, direct, la, lb, g, s);
}

hipError_t pair_launch_bf16(int lb, const PairArgs& p, hipStream_t s) {
  return pair_launch<kBF16>(lb, p, s);
}

}  // namespace mmaops
