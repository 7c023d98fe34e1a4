// gemm_i8.hip -- products of 8-bit integers with scales for each row of X and of
// W, of many rows (proj_tile.hpp).
#include "proj_tile.hpp"

namespace dgemm {

hipError_t launch_proj_i8(const ProjParams &e, bool half, hipStream_t stream) {
  return half ? launch_tiles<1, kScaled, _Float16>(e, stream)
              : launch_tiles<1, kScaled, float>(e, stream);
}

}  // namespace dgemm
