// glu_f32.hip -- gated blocks of floats of many rows, forward and [dG dU] of the
// backward pass (proj_tile.hpp).
#include "proj_tile.hpp"

namespace dgemm {

hipError_t launch_glu_f32(const ProjParams &e, bool slopes, hipStream_t stream) {
  return slopes ? launch_tiles<4, kSlopes, float>(e, stream)
                : launch_tiles<4, kGated, float>(e, stream);
}

}  // namespace dgemm
