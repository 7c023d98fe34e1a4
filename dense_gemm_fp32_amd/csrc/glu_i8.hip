// glu_i8.hip -- gated blocks of 8-bit integers of many rows (proj_tile.hpp).
#include "proj_tile.hpp"

namespace dgemm {

hipError_t launch_glu_i8(const ProjParams &e, bool half, hipStream_t stream) {
  return half ? launch_tiles<1, kGated, _Float16>(e, stream)
              : launch_tiles<1, kGated, float>(e, stream);
}

}  // namespace dgemm
