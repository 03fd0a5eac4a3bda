// group_pipe.hip -- the instances of group_pipe_kernel.hpp.
#include "group_pipe_kernel.hpp"

namespace mcg {

hipError_t launch_group_pipe(int dt, int lb, bool grad, int tile, const GroupArgs& a, hipStream_t s) {
  return dt == DT_BF16 ? gpipe::launch_op<fast::BF16>(lb, grad, tile, a, s) : gpipe::launch_op<fast::F16>(lb, grad, tile, a, s);
}

}  // namespace mcg
