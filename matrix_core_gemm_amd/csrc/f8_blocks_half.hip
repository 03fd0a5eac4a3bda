// f8_blocks_half.hip -- the 64 x 128 instances of f8_blocks_kernel.hpp.
#include "f8_blocks_kernel.hpp"

namespace mcg {

hipError_t launch_f8_blocks_64(int dtA, int la, int lb, bool wide, const GroupArgs& a, hipStream_t s) {
  if (wide)
    return dtA == DT_E4M3 ? f8b::launch_kinds<f8b::Wide<0>, 64, 128>(la, lb, a, s)
                          : f8b::launch_kinds<f8b::Wide<1>, 64, 128>(la, lb, a, s);
  return dtA == DT_E4M3 ? f8b::launch_kinds<f8b::Native<0>, 64, 128>(la, lb, a, s)
                        : f8b::launch_kinds<f8b::Native<1>, 64, 128>(la, lb, a, s);
}

}  // namespace mcg
