// f8_blocks.hip -- the 256 x 256 instances of f8_blocks_kernel.hpp.
#include "f8_blocks_kernel.hpp"

namespace mcg {

hipError_t launch_f8_blocks_256(int dtA, int la, int lb, const GroupArgs& a, hipStream_t s) {
  return dtA == DT_E4M3 ? f8b::launch_kinds<f8b::Native<0>, 256, 256>(la, lb, a, s)
                        : f8b::launch_kinds<f8b::Native<1>, 256, 256>(la, lb, a, s);
}

}  // namespace mcg
