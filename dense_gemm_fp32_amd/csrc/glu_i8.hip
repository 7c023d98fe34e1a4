// glu_i8.hip -- gated blocks of 8-bit integers of many rows (proj_tile.hpp).
#include "proj_tile.hpp"

namespace dgemm {

typedef H16Tile<256, 256, 128, 2, 4, 2, 4, 16, 1> I8Big;
typedef H16Tile<128, 128, 64, 2, 2, 4, 8, 32, 1> I8Mid;
typedef H16Tile<64, 128, 64, 1, 2, 4, 8, 32, 1> I8Small;

hipError_t launch_glu_i8(const ProjParams &e, bool half, hipStream_t stream) {
  return half ? launch_tiles<I8Big, I8Mid, I8Small, kGated, _Float16>(e, stream)
              : launch_tiles<I8Big, I8Mid, I8Small, kGated, float>(e, stream);
}

}  // namespace dgemm
