// gemm_i8_scaled_mid.hip -- the 128 x 128 instances of the pipelined kernel
// (gemm_fast_kernel.hpp) for the int8 product with scales, whole tiles and stream-K.
#include "gemm_fast_kernel.hpp"

namespace mcg {

hipError_t launch_scaled_mid(int layoutB, const ScaledArgs& a, hipStream_t s) {
  using Op = fast::I8Scaled;
  if (a.sk_tiles > 0)
    return layoutB == LAYOUT_K ? fast::launch_one<Op, LAYOUT_K, LAYOUT_K, 128, true>(a, s)
                               : fast::launch_one<Op, LAYOUT_K, LAYOUT_MN, 128, true>(a, s);
  return layoutB == LAYOUT_K ? fast::launch_one<Op, LAYOUT_K, LAYOUT_K, 128>(a, s)
                             : fast::launch_one<Op, LAYOUT_K, LAYOUT_MN, 128>(a, s);
}

}  // namespace mcg
