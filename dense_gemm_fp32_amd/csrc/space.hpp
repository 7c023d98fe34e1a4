// space.hpp -- the workspace of one call of the entry points that take one from
// their caller or from the library's pool.
#pragma once

#include "../../include/gemm.h"
#include "internal.hpp"

namespace dgemm {

// A workspace of `bytes` for one call on `stream`: the caller's, or one from
// the library's pool, given back in stream order by close().  A caller's that
// is not 256-byte aligned gives status `base`, one too small `base` - 1.  A
// stream that is being captured gets none from the pool: it would become an
// allocation node of the graph, and graphs of such calls have faulted when two
// were alive and replayed in turn.
class Space {
 public:
  int open(void *given, size_t given_bytes, size_t bytes, hipStream_t stream, int base) {
    if (bytes == 0) return 0;
    if (given != nullptr) {
      if (!aligned_to(given, 256)) return base;
      if (given_bytes < bytes) return base - 1;
      ptr_ = given;
      return 0;
    }
    if (capturing(stream)) return GEMM_ERR_NO_WORKSPACE;
    pool_.ws_limit = workspace_limit();
    pool_.stream = stream;
    if (workspace_alloc(pool_, bytes, &ptr_) != hipSuccess) return GEMM_ERR_NO_WORKSPACE;
    pooled_ = true;
    return 0;
  }
  hipError_t close() { return pooled_ ? workspace_free(pool_, ptr_) : hipSuccess; }
  void *get() const { return ptr_; }

 private:
  Call pool_ = {};
  void *ptr_ = nullptr;
  bool pooled_ = false;
};

}  // namespace dgemm
