// gemm_i8.hip -- products of 8-bit integers with scales for each row of X and of
// W, of many rows (proj_tile.hpp).
#include "proj_tile.hpp"

namespace dgemm {

typedef H16Tile<256, 256, 128, 2, 4, 2, 4, 16, 1> I8Big;   // 8 waves, 128 KB LDS
typedef H16Tile<128, 128, 64, 2, 2, 4, 8, 32, 1> I8Mid;    // 4 waves,  64 KB LDS
typedef H16Tile<64, 128, 64, 1, 2, 4, 8, 32, 1> I8Small;   // 2 waves,  48 KB LDS

hipError_t launch_proj_i8(const ProjParams &e, bool half, hipStream_t stream) {
  return half ? launch_tiles<I8Big, I8Mid, I8Small, kScaled, _Float16>(e, stream)
              : launch_tiles<I8Big, I8Mid, I8Small, kScaled, float>(e, stream);
}

}  // namespace dgemm
