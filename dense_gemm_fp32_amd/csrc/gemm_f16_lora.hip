// gemm_f16_lora.hip -- the fp16 GEMM on top of a low-rank term of each row's own
// adapter: the kernel of gemm_f16_kernel.hpp with its accumulators started by
// low_rank_init.  The term costs ceil(rank/16) more steps of 32 k per tile
// than the product's K/32, and no pass over C of its own.
#include "gemm_f16_kernel.hpp"

namespace dgemm {

hipError_t launch_f16_lora(const Call &c) { return launch_f16_as_is<true>(c); }

}  // namespace dgemm
