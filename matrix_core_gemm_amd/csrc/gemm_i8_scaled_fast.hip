// gemm_i8_scaled_fast.hip -- the 256 x 256 instances of the pipelined kernel
// (gemm_fast_kernel.hpp) for the int8 product with scales, whole tiles and stream-K.
#include "gemm_fast_kernel.hpp"

namespace mcg {

hipError_t launch_scaled_fast(int layoutB, const ScaledArgs& a, hipStream_t s) {
  using Op = fast::I8Scaled;
  if (a.sk_tiles > 0)
    return layoutB == LAYOUT_K ? fast::launch_one<Op, LAYOUT_K, LAYOUT_K, 256, true>(a, s)
                               : fast::launch_one<Op, LAYOUT_K, LAYOUT_MN, 256, true>(a, s);
  return layoutB == LAYOUT_K ? fast::launch_one<Op, LAYOUT_K, LAYOUT_K, 256>(a, s)
                             : fast::launch_one<Op, LAYOUT_K, LAYOUT_MN, 256>(a, s);
}

}  // namespace mcg
