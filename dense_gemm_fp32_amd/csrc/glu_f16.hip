// glu_f16.hip -- gated blocks of halves of many rows, forward and [dG dU] of the
// backward pass (proj_tile.hpp).
#include "proj_tile.hpp"

namespace dgemm {

hipError_t launch_glu_f16(const ProjParams &e, bool slopes, hipStream_t stream) {
  return slopes ? launch_tiles<2, kSlopes, _Float16>(e, stream)
                : launch_tiles<2, kGated, _Float16>(e, stream);
}

}  // namespace dgemm
