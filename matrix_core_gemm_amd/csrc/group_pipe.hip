// group_pipe.hip -- the instances of group_pipe_kernel.hpp.
#include "group_pipe_kernel.hpp"

namespace mcg {

hipError_t launch_group_pipe(int dt, int lb, bool grad, int tile, const GroupArgs& a, hipStream_t s) {
  if (dt == DT_BF16)
    return tile == 256 ? gpipe::launch_kinds<fast::BF16, 256>(lb, grad, a, s) : gpipe::launch_kinds<fast::BF16, 128>(lb, grad, a, s);
  return tile == 256 ? gpipe::launch_kinds<fast::F16, 256>(lb, grad, a, s) : gpipe::launch_kinds<fast::F16, 128>(lb, grad, a, s);
}

}  // namespace mcg
