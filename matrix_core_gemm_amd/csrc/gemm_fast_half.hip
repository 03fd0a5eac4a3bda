// gemm_fast_half.hip -- the 64 x 128 instances of the pipelined kernel
// (gemm_fast_kernel.hpp), for products of the 8-bit linear layer with too few
// 128 x 128 tiles to give every compute unit one.
#include "gemm_fast_kernel.hpp"

namespace mcg {

hipError_t launch_scaled_half(int layoutB, const ScaledArgs& a, hipStream_t s) {
  using Op = fast::I8Scaled;
  return layoutB == LAYOUT_K ? fast::launch_one<Op, LAYOUT_K, LAYOUT_K, 128, false, 64>(a, s)
                             : fast::launch_one<Op, LAYOUT_K, LAYOUT_MN, 128, false, 64>(a, s);
}

template <class Op>
static hipError_t launch_op(int layoutA, const DenseArgs& a, hipStream_t s) {
  return layoutA == LAYOUT_K ? fast::launch_one<Op, LAYOUT_K, LAYOUT_MN, 128, false, 64>(a, s)
                             : fast::launch_one<Op, LAYOUT_MN, LAYOUT_MN, 128, false, 64>(a, s);
}
hipError_t launch_fast_half(int dtA, int layoutA, const DenseArgs& a, hipStream_t s) {
  return dtA == DT_BF16 ? launch_op<fast::BF16>(layoutA, a, s) : launch_op<fast::F16>(layoutA, a, s);
}

}  // namespace mcg
