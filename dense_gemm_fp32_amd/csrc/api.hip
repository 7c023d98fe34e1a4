// api.hip -- the extern "C" entry points declared in include/gemm.h:
// argument checks, quick returns, variant choice and launch.
//
// Argument checks follow the BLAS convention (return -i for the first invalid
// argument i) and run before any HIP call.  The operation is
// C := alpha*A*B + beta*C on row-major matrices with leading dimensions (the
// SGEMM summary: definition and memory-layout section).
#include <stdio.h>
#include <string.h>

#include <atomic>

#include "../../include/gemm.h"
#include "internal.hpp"

namespace {

std::atomic<int> g_load_mode{0};
std::atomic<int> g_tile_config{0};
std::atomic<int> g_split_mode{0};
std::atomic<int> g_tail_mode{0};
std::atomic<long long> g_ws_limit{-1};
std::atomic<int> g_pack_mode{0};
std::atomic<int> g_streamk_mode{0};

// Shared argument checks.  ta / tb: A is stored transposed (K x M, so its
// rows hold M elements) / B is (N x K, rows of K); otherwise A is M x K and B
// K x N.  Every matrix is row-major.
int check_args_t(bool ta, bool tb, int M, int N, int K, float alpha, const void *A, int lda,
                 const void *B, int ldb, float beta, const void *C, int ldc) {
  if (M < 0) return -1;
  if (N < 0) return -2;
  if (K < 0) return -3;
  const int row_a = ta ? M : K, row_b = tb ? K : N;
  if (lda < (row_a > 1 ? row_a : 1)) return -6;
  if (ldb < (row_b > 1 ? row_b : 1)) return -8;
  if (ldc < (N > 1 ? N : 1)) return -11;
  const bool empty = (M == 0 || N == 0);
  const bool reads_ab = !empty && K > 0 && alpha != 0.0f;
  if (reads_ab && A == nullptr) return -5;
  if (reads_ab && B == nullptr) return -7;
  const bool touches_c = !empty && !((alpha == 0.0f || K == 0) && beta == 1.0f);
  if (touches_c && C == nullptr) return -10;
  return 0;
}

int check_args(int M, int N, int K, float alpha, const void *A, int lda, const void *B, int ldb,
               float beta, const void *C, int ldc) {
  return check_args_t(false, false, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc);
}

// The same checks for column-major operands (BLAS layout: X(i, j) at
// X[i + j*ldX]), with the argument indices of the column-major entry points.
int check_args_colmajor(int M, int N, int K, float alpha, const void *A, int lda, const void *B,
                        int ldb, float beta, const void *C, int ldc) {
  if (M < 0) return -1;
  if (N < 0) return -2;
  if (K < 0) return -3;
  if (lda < (M > 1 ? M : 1)) return -6;
  if (ldb < (K > 1 ? K : 1)) return -8;
  if (ldc < (M > 1 ? M : 1)) return -11;
  const bool empty = (M == 0 || N == 0);
  const bool reads_ab = !empty && K > 0 && alpha != 0.0f;
  if (reads_ab && A == nullptr) return -5;
  if (reads_ab && B == nullptr) return -7;
  const bool touches_c = !empty && !((alpha == 0.0f || K == 0) && beta == 1.0f);
  if (touches_c && C == nullptr) return -10;
  return 0;
}

enum class Route { kNothing, kScale, kGemm };

Route route(int M, int N, int K, float alpha, float beta) {
  if (M == 0 || N == 0) return Route::kNothing;
  if (alpha == 0.0f || K == 0) return beta == 1.0f ? Route::kNothing : Route::kScale;
  return Route::kGemm;
}

dgemm::Call make_call(int M, int N, int K, float alpha, const void *A, int lda, const void *B,
                      int ldb, float beta, void *C, int ldc, void *stream, bool out32 = false,
                      bool ta = false, bool tb = false) {
  dgemm::Call c = {};
  c.out32 = out32;
  c.ta = ta;
  c.tb = tb;
  c.M = M;
  c.N = N;
  c.K = K;
  c.alpha = alpha;
  c.beta = beta;
  c.A = A;
  c.lda = lda;
  c.B = B;
  c.ldb = ldb;
  c.C = C;
  c.ldc = ldc;
  c.force_scalar = g_load_mode.load(std::memory_order_relaxed) == 1;
  c.tile_config = g_tile_config.load(std::memory_order_relaxed);
  c.split_mode = g_split_mode.load(std::memory_order_relaxed);
  c.splits = 1;
  c.k_chunk = 0;
  c.split_stride = 0;
  c.tile_base = 0;
  c.tile_count = 0;
  c.c_tiles = false;
  c.tail_mode = g_tail_mode.load(std::memory_order_relaxed);
  c.ws_limit = g_ws_limit.load(std::memory_order_relaxed);
  c.ws_fixed = nullptr;
  c.ws_fixed_bytes = 0;
  c.pack_mode = g_pack_mode.load(std::memory_order_relaxed);
  c.streamk_mode = g_streamk_mode.load(std::memory_order_relaxed);
  c.term = nullptr;
  c.stream = static_cast<hipStream_t>(stream);
  return c;
}

// One call of any type and layout: checks, quick returns, launch.
// kind: 0 = fp32, 1 = fp16 in and out, 2 = fp16 in, fp32 C.
int run_gemm(int kind, bool ta, bool tb, int M, int N, int K, float alpha, const void *A, int lda,
             const void *B, int ldb, float beta, void *C, int ldc, void *stream) {
  const int rc = check_args_t(ta, tb, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc);
  if (rc != 0) return rc;
  hipError_t e = hipSuccess;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  switch (route(M, N, K, alpha, beta)) {
    case Route::kNothing:
      return GEMM_SUCCESS;
    case Route::kScale:
      e = kind == 1 ? dgemm::launch_scale_f16(M, N, beta, static_cast<uint16_t *>(C), ldc, s)
                    : dgemm::launch_scale_f32(M, N, beta, static_cast<float *>(C), ldc, s);
      break;
    case Route::kGemm: {
      const dgemm::Call c = make_call(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream,
                                      kind == 2, ta, tb);
      e = kind == 0 ? dgemm::launch_f32(c) : dgemm::launch_f16(c);
      break;
    }
  }
  return e == hipSuccess ? GEMM_SUCCESS : (int)e;
}

}  // namespace

namespace dgemm {
long long workspace_limit() { return g_ws_limit.load(std::memory_order_relaxed); }
}  // namespace dgemm

extern "C" {

int gemm_f32(int M, int N, int K, float alpha, const float *A, int lda, const float *B, int ldb,
             float beta, float *C, int ldc, void *stream) {
  return run_gemm(0, false, false, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream);
}

int gemm_f16(int M, int N, int K, float alpha, const gemm_half_t *A, int lda, const gemm_half_t *B,
             int ldb, float beta, gemm_half_t *C, int ldc, void *stream) {
  return run_gemm(1, false, false, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream);
}

int gemm_f16f32(int M, int N, int K, float alpha, const gemm_half_t *A, int lda,
                const gemm_half_t *B, int ldb, float beta, float *C, int ldc, void *stream) {
  return run_gemm(2, false, false, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream);
}

// Transposed operands (row-major storage): the first letter gives A's
// operation, the second B's; "t": the operand is stored transposed (A as
// K x M, B as N x K) and multiplied as its transpose.
int gemm_f32_nt(int M, int N, int K, float alpha, const float *A, int lda, const float *B,
                int ldb, float beta, float *C, int ldc, void *stream) {
  return run_gemm(0, false, true, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream);
}

int gemm_f32_tn(int M, int N, int K, float alpha, const float *A, int lda, const float *B,
                int ldb, float beta, float *C, int ldc, void *stream) {
  return run_gemm(0, true, false, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream);
}

int gemm_f32_tt(int M, int N, int K, float alpha, const float *A, int lda, const float *B,
                int ldb, float beta, float *C, int ldc, void *stream) {
  return run_gemm(0, true, true, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream);
}

int gemm_f16_nt(int M, int N, int K, float alpha, const gemm_half_t *A, int lda,
                const gemm_half_t *B, int ldb, float beta, gemm_half_t *C, int ldc, void *stream) {
  return run_gemm(1, false, true, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream);
}

int gemm_f16_tn(int M, int N, int K, float alpha, const gemm_half_t *A, int lda,
                const gemm_half_t *B, int ldb, float beta, gemm_half_t *C, int ldc, void *stream) {
  return run_gemm(1, true, false, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream);
}

int gemm_f16_tt(int M, int N, int K, float alpha, const gemm_half_t *A, int lda,
                const gemm_half_t *B, int ldb, float beta, gemm_half_t *C, int ldc, void *stream) {
  return run_gemm(1, true, true, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream);
}

int gemm_f16f32_nt(int M, int N, int K, float alpha, const gemm_half_t *A, int lda,
                   const gemm_half_t *B, int ldb, float beta, float *C, int ldc, void *stream) {
  return run_gemm(2, false, true, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream);
}

int gemm_f16f32_tn(int M, int N, int K, float alpha, const gemm_half_t *A, int lda,
                   const gemm_half_t *B, int ldb, float beta, float *C, int ldc, void *stream) {
  return run_gemm(2, true, false, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream);
}

int gemm_f16f32_tt(int M, int N, int K, float alpha, const gemm_half_t *A, int lda,
                   const gemm_half_t *B, int ldb, float beta, float *C, int ldc, void *stream) {
  return run_gemm(2, true, true, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream);
}

// gemm_f32 for callers that cannot allocate: the same checks, plan and
// kernels, with the workspace (operand copies, split K) taken from the
// library's fixed scratch region instead of its memory pool.  A call whose plan needs more workspace
// than the region holds is refused before anything is enqueued.
int gemm_f32_noalloc(int M, int N, int K, float alpha, const float *A, int lda, const float *B,
                     int ldb, float beta, float *C, int ldc, void *stream) {
  const int rc = check_args(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc);
  if (rc != 0) return rc;
  hipError_t e = hipSuccess;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  switch (route(M, N, K, alpha, beta)) {
    case Route::kNothing:
      return GEMM_SUCCESS;
    case Route::kScale:
      e = dgemm::launch_scale_f32(M, N, beta, C, ldc, s);
      break;
    case Route::kGemm: {
      dgemm::Call c = make_call(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream);
      // The plan sees the region's size (copies of unaligned operands are
      // made only where they fit in it beside the split-K workspace); the
      // refusal comes before any HIP call.
      c.ws_fixed_bytes = dgemm::kScratchBytes;
      const dgemm::Plan p = dgemm::plan_f32(c);
      if (p.ws_bytes > dgemm::kScratchBytes) return GEMM_ERR_SCRATCH_LIMIT;
      e = dgemm::scratch_region(dgemm::stream_device(s), &c.ws_fixed);
      if (e != hipSuccess) return (int)e;
      e = dgemm::launch_f32(c);
      break;
    }
  }
  return e == hipSuccess ? GEMM_SUCCESS : (int)e;
}

int gemm_f32_valu(int M, int N, int K, float alpha, const float *A, int lda, const float *B,
                  int ldb, float beta, float *C, int ldc, void *stream) {
  const int rc = check_args(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc);
  if (rc != 0) return rc;
  hipError_t e = hipSuccess;
  switch (route(M, N, K, alpha, beta)) {
    case Route::kNothing:
      return GEMM_SUCCESS;
    case Route::kScale:
      e = dgemm::launch_scale_f32(M, N, beta, C, ldc, static_cast<hipStream_t>(stream));
      break;
    case Route::kGemm:
      e = dgemm::launch_f32_valu(make_call(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream));
      break;
  }
  return e == hipSuccess ? GEMM_SUCCESS : (int)e;
}

// Column-major calls.  A column-major M x N matrix with leading dimension ld
// is, byte for byte, the row-major N x M matrix of its transpose with the same
// ld.  So C = A*B (all column-major) is the row-major product
// C^T = B^T * A^T: the row-major entry point with M and N exchanged and A and
// B exchanged, on the same buffers (the SGEMM summary's layout section:
// column-major use swaps A and B).  Arguments are checked first with the
// column-major rules and indices.
int gemm_f32_colmajor(int M, int N, int K, float alpha, const float *A, int lda, const float *B,
                      int ldb, float beta, float *C, int ldc, void *stream) {
  const int rc = check_args_colmajor(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc);
  if (rc != 0) return rc;
  return gemm_f32(N, M, K, alpha, B, ldb, A, lda, beta, C, ldc, stream);
}

int gemm_f16_colmajor(int M, int N, int K, float alpha, const gemm_half_t *A, int lda,
                      const gemm_half_t *B, int ldb, float beta, gemm_half_t *C, int ldc,
                      void *stream) {
  const int rc = check_args_colmajor(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc);
  if (rc != 0) return rc;
  return gemm_f16(N, M, K, alpha, B, ldb, A, lda, beta, C, ldc, stream);
}

int gemm_f16f32_colmajor(int M, int N, int K, float alpha, const gemm_half_t *A, int lda,
                         const gemm_half_t *B, int ldb, float beta, float *C, int ldc,
                         void *stream) {
  const int rc = check_args_colmajor(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc);
  if (rc != 0) return rc;
  return gemm_f16f32(N, M, K, alpha, B, ldb, A, lda, beta, C, ldc, stream);
}

const char *gemm_status_string(int status) {
  switch (status) {
    case 0: return "success";
    case -1: return "invalid argument 1: M < 0";
    case -2: return "invalid argument 2: N < 0";
    case -3: return "invalid argument 3: K < 0";
    case -5: return "invalid argument 5: A is NULL";
    case -6: return "invalid argument 6: lda < max(1, row length of A as stored: K, or M when A is stored transposed or column-major)";
    case -7: return "invalid argument 7: B is NULL";
    case -8: return "invalid argument 8: ldb < max(1, row length of B as stored: N, or K when B is stored transposed or column-major)";
    case -10: return "invalid argument 10: C is NULL";
    case -11: return "invalid argument 11: ldc < max(1, N) (row-major) or max(1, M) (column-major)";
    case GEMM_ERR_SCRATCH_LIMIT: return "gemm_f32_noalloc: the call's workspace (split K) would exceed the library's fixed scratch region (64 MiB); nothing was enqueued";
    case GEMM_ERR_NO_WORKSPACE: return "the call's workspace could not be had from the library's pool (gemm_set_workspace_limit, a stream that is being captured, or out of memory); nothing was enqueued";
    case -101: return "invalid probe argument 1: dtype is not 0 (fp32) or 1 (fp16)";
    case -102: return "invalid probe argument 2: iters < 1";
    case -103: return "invalid probe argument 3: operands is NULL";
    case -104: return "invalid probe argument 4: operand buffer smaller than 65536 bytes";
    case -105: return "invalid probe argument 5: out is NULL";
    case -106: return "invalid probe argument 6: out buffer smaller than 1 MiB";
    case -107: return "invalid probe argument 7: flops is NULL";
    case -301: return "gemm_lora: invalid argument 1: M < 0";
    case -302: return "gemm_lora: invalid argument 2: N < 0";
    case -303: return "gemm_lora: invalid argument 3: K < 0";
    case -305: return "gemm_lora: invalid argument 5: X is NULL";
    case -306: return "gemm_lora: invalid argument 6: ldx < max(1, K)";
    case -307: return "gemm_lora: invalid argument 7: W is NULL";
    case -308: return "gemm_lora: invalid argument 8: ldw < max(1, K)";
    case -310: return "gemm_lora: invalid argument 10: Y is NULL";
    case -311: return "gemm_lora: invalid argument 11: ldy < max(1, N)";
    case -312: return "gemm_lora: invalid argument 12: L outside 0 .. 65535";
    case -313: return "gemm_lora: invalid argument 13: R outside 0 .. 256";
    case -314: return "gemm_lora: invalid argument 14: A is NULL";
    case -315: return "gemm_lora: invalid argument 15: lda < max(1, K)";
    case -316: return "gemm_lora: invalid argument 16: stride_a < 0";
    case -317: return "gemm_lora: invalid argument 17: B is NULL";
    case -318: return "gemm_lora: invalid argument 18: ldb < max(1, R)";
    case -319: return "gemm_lora: invalid argument 19: stride_b < 0";
    case -322: return "gemm_lora: invalid argument 22: rows is NULL";
    case -323: return "gemm_lora: invalid argument 23: workspace not 256-byte aligned";
    case -324: return "gemm_lora: invalid argument 24: workspace_bytes too small (gemm_lora_workspace)";
    case -401: return "gemm_lora_grad: invalid argument 1: M < 0";
    case -402: return "gemm_lora_grad: invalid argument 2: N < 0";
    case -403: return "gemm_lora_grad: invalid argument 3: K < 0";
    case -405: return "gemm_lora_grad: invalid argument 5: dY is NULL";
    case -406: return "gemm_lora_grad: invalid argument 6: lddy < max(1, N)";
    case -407: return "gemm_lora_grad: invalid argument 7: X is NULL";
    case -408: return "gemm_lora_grad: invalid argument 8: ldx < max(1, K)";
    case -409: return "gemm_lora_grad: invalid argument 9: W is NULL";
    case -410: return "gemm_lora_grad: invalid argument 10: ldw < max(1, K)";
    case -411: return "gemm_lora_grad: invalid argument 11: L outside 0 .. 65535";
    case -412: return "gemm_lora_grad: invalid argument 12: R outside 0 .. 256";
    case -413: return "gemm_lora_grad: invalid argument 13: A is NULL";
    case -414: return "gemm_lora_grad: invalid argument 14: lda < max(1, K)";
    case -415: return "gemm_lora_grad: invalid argument 15: stride_a < 0";
    case -416: return "gemm_lora_grad: invalid argument 16: B is NULL";
    case -417: return "gemm_lora_grad: invalid argument 17: ldb < max(1, R)";
    case -418: return "gemm_lora_grad: invalid argument 18: stride_b < 0";
    case -421: return "gemm_lora_grad: invalid argument 21: rows is NULL";
    case -424: return "gemm_lora_grad: invalid argument 24: lddx < max(1, K)";
    case -427: return "gemm_lora_grad: invalid argument 27: ldda < max(1, K)";
    case -428: return "gemm_lora_grad: invalid argument 28: stride_da less than one matrix";
    case -430: return "gemm_lora_grad: invalid argument 30: lddb < max(1, R)";
    case -431: return "gemm_lora_grad: invalid argument 31: stride_db less than one matrix";
    case -432: return "gemm_lora_grad: invalid argument 32: workspace not 256-byte aligned";
    case -433: return "gemm_lora_grad: invalid argument 33: workspace_bytes too small (gemm_lora_grad_workspace)";
    case -601: return "gemm_quant_i8: invalid argument 1: M outside 0 .. 16777216";
    case -602: return "gemm_quant_i8: invalid argument 2: K outside 0 .. 16777216";
    case -603: return "gemm_quant_i8: invalid argument 3: X is NULL";
    case -604: return "gemm_quant_i8: invalid argument 4: ldx < max(1, K)";
    case -605: return "gemm_quant_i8: invalid argument 5: Q is NULL";
    case -606: return "gemm_quant_i8: invalid argument 6: ldq < max(1, K)";
    case -607: return "gemm_quant_i8: invalid argument 7: scale is NULL";
    case -701: return "gemm_i8: invalid argument 1: M outside 0 .. 16777216";
    case -702: return "gemm_i8: invalid argument 2: N outside 0 .. 16777216";
    case -703: return "gemm_i8: invalid argument 3: K outside 0 .. 131071";
    case -705: return "gemm_i8: invalid argument 5: X is NULL";
    case -706: return "gemm_i8: invalid argument 6: ldx < max(1, K)";
    case -708: return "gemm_i8: invalid argument 8: W is NULL";
    case -709: return "gemm_i8: invalid argument 9: ldw < max(1, K)";
    case -712: return "gemm_i8: invalid argument 12: Y is NULL";
    case -713: return "gemm_i8: invalid argument 13: ldy < max(1, N)";
    case -714: return "gemm_i8: invalid argument 14: workspace not 256-byte aligned";
    case -715: return "gemm_i8: invalid argument 15: workspace_bytes too small (gemm_i8_workspace)";
    case -801: return "gemm_glu: invalid argument 1: M outside 0 .. 16777216";
    case -802: return "gemm_glu: invalid argument 2: F outside 0 .. 8388608";
    case -803: return "gemm_glu: invalid argument 3: K outside 0 .. 16777216";
    case -804: return "gemm_glu: invalid argument 4: act is no GEMM_ACT_*";
    case -805: return "gemm_glu: invalid argument 5: X is NULL";
    case -806: return "gemm_glu: invalid argument 6: ldx < max(1, K)";
    case -807: return "gemm_glu: invalid argument 7: W is NULL";
    case -808: return "gemm_glu: invalid argument 8: ldw < max(1, K)";
    case -809: return "gemm_glu: invalid argument 9: H is NULL";
    case -810: return "gemm_glu: invalid argument 10: ldh < max(1, F)";
    case -812: return "gemm_glu: invalid argument 12: ldz < max(1, 2F)";
    case -813: return "gemm_glu: invalid argument 13: workspace not 256-byte aligned";
    case -814: return "gemm_glu: invalid argument 14: workspace_bytes too small (gemm_glu_workspace)";
    case -901: return "gemm_glu_i8: invalid argument 1: M outside 0 .. 16777216";
    case -902: return "gemm_glu_i8: invalid argument 2: F outside 0 .. 8388608";
    case -903: return "gemm_glu_i8: invalid argument 3: K outside 0 .. 131071";
    case -904: return "gemm_glu_i8: invalid argument 4: act is no GEMM_ACT_*";
    case -905: return "gemm_glu_i8: invalid argument 5: X is NULL";
    case -906: return "gemm_glu_i8: invalid argument 6: ldx < max(1, K)";
    case -908: return "gemm_glu_i8: invalid argument 8: W is NULL";
    case -909: return "gemm_glu_i8: invalid argument 9: ldw < max(1, K)";
    case -911: return "gemm_glu_i8: invalid argument 11: H is NULL";
    case -912: return "gemm_glu_i8: invalid argument 12: ldh < max(1, F)";
    case -913: return "gemm_glu_i8: invalid argument 13: workspace not 256-byte aligned";
    case -914: return "gemm_glu_i8: invalid argument 14: workspace_bytes too small (gemm_glu_workspace)";
    case -1001: return "gemm_glu_grad: invalid argument 1: M outside 0 .. 16777216";
    case -1002: return "gemm_glu_grad: invalid argument 2: F outside 0 .. 8388608";
    case -1003: return "gemm_glu_grad: invalid argument 3: K outside 0 .. 16777216";
    case -1004: return "gemm_glu_grad: invalid argument 4: act is no GEMM_ACT_*";
    case -1005: return "gemm_glu_grad: invalid argument 5: dH is NULL";
    case -1006: return "gemm_glu_grad: invalid argument 6: lddh < max(1, F)";
    case -1007: return "gemm_glu_grad: invalid argument 7: X is NULL";
    case -1008: return "gemm_glu_grad: invalid argument 8: ldx < max(1, K)";
    case -1009: return "gemm_glu_grad: invalid argument 9: W is NULL";
    case -1010: return "gemm_glu_grad: invalid argument 10: ldw < max(1, K)";
    case -1012: return "gemm_glu_grad: invalid argument 12: ldz < max(1, 2F)";
    case -1015: return "gemm_glu_grad: invalid argument 15: lddx < max(1, K)";
    case -1018: return "gemm_glu_grad: invalid argument 18: lddw < max(1, K)";
    case -1019: return "gemm_glu_grad: invalid argument 19: workspace not 256-byte aligned";
    case -1020: return "gemm_glu_grad: invalid argument 20: workspace_bytes too small (gemm_glu_grad_workspace)";
    case -501: return "gemm_moe: invalid argument 1: M outside 0 .. 256";
    case -502: return "gemm_moe: invalid argument 2: D < 1";
    case -503: return "gemm_moe: invalid argument 3: F < 1";
    case -504: return "gemm_moe: invalid argument 4: E outside 1 .. 1024";
    case -505: return "gemm_moe: invalid argument 5: top_k outside 1 .. min(E, 64)";
    case -506: return "gemm_moe: invalid argument 6: renorm is not 0 or 1";
    case -508: return "gemm_moe: invalid argument 8: X is NULL";
    case -509: return "gemm_moe: invalid argument 9: ldx < D";
    case -510: return "gemm_moe: invalid argument 10: Wr is NULL";
    case -511: return "gemm_moe: invalid argument 11: ldr < D";
    case -512: return "gemm_moe: invalid argument 12: W1 is NULL";
    case -513: return "gemm_moe: invalid argument 13: ld1 < D";
    case -514: return "gemm_moe: invalid argument 14: stride1 < 0";
    case -515: return "gemm_moe: invalid argument 15: W2 is NULL";
    case -516: return "gemm_moe: invalid argument 16: ld2 < F";
    case -517: return "gemm_moe: invalid argument 17: stride2 < 0";
    case -519: return "gemm_moe: invalid argument 19: Y is NULL";
    case -520: return "gemm_moe: invalid argument 20: ldy < D";
    case -523: return "gemm_moe: invalid argument 23: workspace not 256-byte aligned";
    case -524: return "gemm_moe: invalid argument 24: workspace_bytes too small (gemm_moe_workspace)";
    default: break;
  }
  if (status > 0) return hipGetErrorString(static_cast<hipError_t>(status));
  return "unknown status";
}

int gemm_describe(int dtype, int M, int N, int K, float alpha, const void *A, int lda,
                  const void *B, int ldb, float beta, const void *C, int ldc, char *buf, int len) {
  const int rc = check_args(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc);
  char text[256];
  if (rc != 0) {
    snprintf(text, sizeof text, "invalid: %s", gemm_status_string(rc));
  } else if (dtype < 0 || dtype > 2) {
    snprintf(text, sizeof text, "invalid: unknown dtype %d", dtype);
  } else {
    static const char *const kNames[3] = {"f32", "f16", "f16f32"};
    const char *dn = kNames[dtype];
    switch (route(M, N, K, alpha, beta)) {
      case Route::kNothing:
        snprintf(text, sizeof text, "%s no-op", dn);
        break;
      case Route::kScale:
        snprintf(text, sizeof text, "%s scale C := beta*C%s", dn,
                 beta == 0.0f ? " (zero fill, C not read)" : "");
        break;
      case Route::kGemm: {
        dgemm::Call c = make_call(M, N, K, alpha, A, lda, B, ldb, beta, const_cast<void *>(C), ldc,
                                  nullptr, dtype == 2);
        dgemm::Plan p = dtype ? dgemm::plan_f16(c) : dgemm::plan_f32(c);
        char split[48] = "";
        if (p.streamk && p.sk_whole > 0)
          snprintf(split, sizeof split, " stream-K after %lld whole tiles", p.sk_whole);
        else if (p.streamk) snprintf(split, sizeof split, " stream-K");
        else if (p.splits > 1) snprintf(split, sizeof split, " split-K %d", p.splits);
        else if (p.tail > 1) snprintf(split, sizeof split, " last round split-K %d", p.tail);
        char ws[48] = "";
        if (p.ws_bytes > 0) snprintf(ws, sizeof ws, " workspace %zu bytes", p.ws_bytes);
        const char *packed = p.packed_a ? (p.packed_b ? " copies A B" : " copies A")
                                        : (p.packed_b ? " copies B" : "");
        snprintf(text, sizeof text, "%s loads A:%s%d B:%s%d C:%s%d%s blocks %lld threads %d%s%s%s",
                 p.name, p.vec_a > 2 ? "vec" : (p.vec_a == 2 ? "pair" : "scalar"), p.vec_a,
                 p.vec_b > 2 ? "vec" : (p.vec_b == 2 ? "pair" : "scalar"), p.vec_b,
                 p.vec_c > 1 ? "vec" : "scalar", p.vec_c, packed, p.blocks, p.threads, split, ws,
                 beta == 0.0f ? " beta0 (C not read)" : "");
        break;
      }
    }
  }
  if (buf && len > 0) {
    strncpy(buf, text, (size_t)len - 1);
    buf[len - 1] = '\0';
  }
  return rc;
}

int gemm_probe_mfma(int dtype, int iters, const void *operands, size_t operand_bytes, float *out,
                    size_t out_bytes, double *flops, void *stream) {
  if (dtype != 0 && dtype != 1) return -101;
  if (iters < 1) return -102;
  if (operands == nullptr) return -103;
  if (operand_bytes < dgemm::probe_operand_bytes()) return -104;
  if (out == nullptr) return -105;
  if (out_bytes < dgemm::probe_out_bytes()) return -106;
  if (flops == nullptr) return -107;
  *flops = dgemm::probe_flops(dtype, iters);
  const hipError_t e = dgemm::launch_probe(dtype, iters, operands, out, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? GEMM_SUCCESS : (int)e;
}

int gemm_set_load_mode(int mode) {
  if (mode != 0 && mode != 1) return -1;
  return g_load_mode.exchange(mode);
}

int gemm_set_split(int mode) {
  if (mode < 0 || mode > 64) return -1;
  return g_split_mode.exchange(mode);
}

int gemm_set_tail_split(int mode) {
  if (mode < 0 || mode > 64) return -1;
  return g_tail_mode.exchange(mode);
}

int gemm_set_tile_config(int config) {
  if (config < 0 || config > 10) return -1;
  return g_tile_config.exchange(config);
}

int gemm_set_pack(int mode) {
  if (mode < 0 || mode > 2) return -1;
  return g_pack_mode.exchange(mode);
}

int gemm_set_stream_k(int mode) {
  if (mode < 0 || mode > 6) return -1;
  return g_streamk_mode.exchange(mode);
}

long long gemm_set_workspace_limit(long long bytes) {
  if (bytes < -1) return -2;
  return g_ws_limit.exchange(bytes);
}

}  // extern "C"
