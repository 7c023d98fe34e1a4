// gemm_f16_lora.hip -- the fp16 GEMM on top of a low-rank term of each row's own
// adapter (low_rank_start and LowRankTerm of gemm_f16_kernel.hpp).  The term
// costs a tile ceil(rank/32) more K steps of 64 for each adapter among its
// rows, and no pass over C of its own.
#include "gemm_f16_kernel.hpp"

namespace dgemm {

hipError_t launch_f16_lora(const Call &c) {
  return run_packed(c, 2, plan_f16, launch_f16_as_is<true>);
}

}  // namespace dgemm
