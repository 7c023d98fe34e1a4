// rows_api.hip -- the extern "C" entry points of the products whose rows
// choose their own weights (include/gemm.h): argument checks, quick returns,
// workspace.  Checks run before any HIP call; the first failure wins.
#include "../../include/gemm.h"
#include "internal.hpp"
#include "space.hpp"

namespace {

using dgemm::LoraCall;
using dgemm::MoeCall;
using dgemm::Space;

int at_least_one(int n) { return n > 1 ? n : 1; }

// Grids and 32-bit indices hold up to the limit with room to spare.
bool bad_size(int n) { return n < 0 || n > GEMM_ROWS_MAX_SIZE; }

int status(hipError_t e) { return e == hipSuccess ? GEMM_SUCCESS : (int)e; }

// The product of a call without adapters, A op(B), as gemm_* would run it: its
// copies and K parts take the caller's workspace as far as that reaches, or the
// library's pool where the caller gave none and the stream is not being captured.
hipError_t shared_product(bool half, bool tb, int M, int N, int K, float alpha, const void *A,
                          int lda, const void *B, int ldb, float beta, void *C, int ldc, void *ws,
                          size_t ws_bytes, hipStream_t stream) {
  dgemm::Call c = {};
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
  c.tb = tb;
  c.splits = 1;
  c.stream = stream;
  if (ws != nullptr) {
    c.ws_fixed = ws;
    c.ws_fixed_bytes = dgemm::aligned_to(ws, 256) ? ws_bytes : 0;
  } else {
    c.ws_limit = dgemm::capturing(stream) ? 0 : dgemm::workspace_limit();
  }
  return half ? dgemm::launch_f16(c) : dgemm::launch_f32(c);
}

int lora(bool half, int M, int N, int K, float alpha, const void *X, int ldx, const void *W,
         int ldw, float beta, void *Y, int ldy, int L, int R, const void *A, int lda,
         long long stride_a, const void *B, int ldb, long long stride_b, const float *scale,
         const int *ranks, const int *rows, void *ws, size_t ws_bytes, void *stream) {
  if (bad_size(M)) return -301;
  if (bad_size(N)) return -302;
  if (bad_size(K)) return -303;
  if (ldx < at_least_one(K)) return -306;
  if (ldw < at_least_one(K)) return -308;
  if (ldy < at_least_one(N)) return -311;
  if (L < 0 || L > GEMM_LORA_MAX_ADAPTERS) return -312;
  if (R < 0 || R > GEMM_LORA_MAX_RANK) return -313;
  if (lda < at_least_one(K)) return -315;
  if (stride_a < 0) return -316;
  if (ldb < at_least_one(R)) return -318;
  if (stride_b < 0) return -319;
  if (M == 0 || N == 0) return GEMM_SUCCESS;
  const bool product = K > 0 && alpha != 0.0f;
  const bool adapters = product && L > 0 && R > 0;
  if (product && X == nullptr) return -305;
  if (product && W == nullptr) return -307;
  if (!product && beta == 1.0f) return GEMM_SUCCESS;
  if (Y == nullptr) return -310;
  if (adapters && A == nullptr) return -314;
  if (adapters && B == nullptr) return -317;
  if (adapters && rows == nullptr) return -322;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if (!product)
    return status(half ? dgemm::launch_scale_f16(M, N, beta, static_cast<uint16_t *>(Y), ldy, s)
                       : dgemm::launch_scale_f32(M, N, beta, static_cast<float *>(Y), ldy, s));
  if (!adapters)
    return status(shared_product(half, true, M, N, K, alpha, X, ldx, W, ldw, beta, Y, ldy, ws,
                                 ws_bytes, s));
  LoraCall c = {};
  c.half = half;
  c.M = M;
  c.N = N;
  c.K = K;
  c.alpha = alpha;
  c.X = X;
  c.ldx = ldx;
  c.W = W;
  c.ldw = ldw;
  c.beta = beta;
  c.Y = Y;
  c.ldy = ldy;
  c.L = L;
  c.R = R;
  c.A = A;
  c.lda = lda;
  c.stride_a = stride_a;
  c.B = B;
  c.ldb = ldb;
  c.stride_b = stride_b;
  c.scale = scale;
  c.ranks = ranks;
  c.rows = rows;
  c.stream = s;
  Space space;
  const int rc = space.open(ws, ws_bytes, dgemm::lora_workspace(c), s, -323);
  if (rc != 0) return rc;
  const hipError_t e = dgemm::launch_lora(c, space.get());
  const hipError_t f = space.close();
  return status(e != hipSuccess ? e : f);
}

int lora_grad(bool half, int M, int N, int K, float alpha, const void *dY, int lddy,
              const void *X, int ldx, const void *W, int ldw, int L, int R, const void *A, int lda,
              long long stride_a, const void *B, int ldb, long long stride_b, const float *scale,
              const int *ranks, const int *rows, float beta_x, void *dX, int lddx, float beta_ab,
              float *dA, int ldda, long long stride_da, float *dB, int lddb, long long stride_db,
              void *ws, size_t ws_bytes, void *stream) {
  if (bad_size(M)) return -401;
  if (bad_size(N)) return -402;
  if (bad_size(K)) return -403;
  if (lddy < at_least_one(N)) return -406;
  if (ldx < at_least_one(K)) return -408;
  if (dX != nullptr && ldw < at_least_one(K)) return -410;
  if (L < 0 || L > GEMM_LORA_MAX_ADAPTERS) return -411;
  if (R < 0 || R > GEMM_LORA_MAX_RANK) return -412;
  if (lda < at_least_one(K)) return -414;
  if (stride_a < 0) return -415;
  if (ldb < at_least_one(R)) return -417;
  if (stride_b < 0) return -418;
  if (dX != nullptr && lddx < at_least_one(K)) return -424;
  if (dA != nullptr && ldda < at_least_one(K)) return -427;
  // the gradients of two adapters must not overlap
  if (dA != nullptr && L > 1 && R > 0 && stride_da < (long long)(R - 1) * ldda + K) return -428;
  if (dB != nullptr && lddb < at_least_one(R)) return -430;
  if (dB != nullptr && L > 1 && N > 0 && stride_db < (long long)(N - 1) * lddb + R) return -431;
  const bool adapters = L > 0 && R > 0;
  const bool want_x = dX != nullptr && M > 0 && K > 0;
  const bool want_a = dA != nullptr && adapters && K > 0;
  const bool want_b = dB != nullptr && adapters && N > 0;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if (!want_x && !want_a && !want_b) return GEMM_SUCCESS;
  if (M == 0 || N == 0 || K == 0 || alpha == 0.0f) {
    // every sum is empty: each output is scaled
    hipError_t e = hipSuccess;
    if (want_x && beta_x != 1.0f)
      e = half ? dgemm::launch_scale_f16(M, K, beta_x, static_cast<uint16_t *>(dX), lddx, s)
               : dgemm::launch_scale_f32(M, K, beta_x, static_cast<float *>(dX), lddx, s);
    if (e == hipSuccess && want_a && beta_ab != 1.0f)
      e = dgemm::launch_scale_batch_f32(L, R, K, beta_ab, dA, ldda, stride_da, s);
    if (e == hipSuccess && want_b && beta_ab != 1.0f)
      e = dgemm::launch_scale_batch_f32(L, N, R, beta_ab, dB, lddb, stride_db, s);
    return status(e);
  }
  if (dY == nullptr) return -405;
  if (X == nullptr && (want_a || want_b)) return -407;
  if (W == nullptr && want_x) return -409;
  if (adapters && A == nullptr && (want_x || want_b)) return -413;
  if (adapters && B == nullptr && (want_x || want_a)) return -416;
  if (adapters && rows == nullptr) return -421;
  if (!adapters)
    return status(shared_product(half, false, M, K, N, alpha, dY, lddy, W, ldw, beta_x, dX, lddx,
                                 ws, ws_bytes, s));
  LoraCall c = {};
  c.half = half;
  c.M = M;
  c.N = N;
  c.K = K;
  c.alpha = alpha;
  c.X = X;
  c.ldx = ldx;
  c.W = W;
  c.ldw = ldw;
  c.L = L;
  c.R = R;
  c.A = A;
  c.lda = lda;
  c.stride_a = stride_a;
  c.B = B;
  c.ldb = ldb;
  c.stride_b = stride_b;
  c.scale = scale;
  c.ranks = ranks;
  c.rows = rows;
  c.dY = dY;
  c.lddy = lddy;
  c.beta_x = beta_x;
  c.dX = want_x ? dX : nullptr;
  c.lddx = lddx;
  c.beta_ab = beta_ab;
  c.dA = want_a ? dA : nullptr;
  c.ldda = ldda;
  c.stride_da = stride_da;
  c.dB = want_b ? dB : nullptr;
  c.lddb = lddb;
  c.stride_db = stride_db;
  c.stream = s;
  Space space;
  const int rc = space.open(ws, ws_bytes, dgemm::lora_grad_workspace(c), s, -432);
  if (rc != 0) return rc;
  const hipError_t e = dgemm::launch_lora_grad(c, space.get());
  const hipError_t f = space.close();
  return status(e != hipSuccess ? e : f);
}

int moe(bool half, int M, int D, int F, int E, int top_k, int renorm, float alpha, const void *X,
        int ldx, const void *Wr, int ldr, const void *W1, int ld1, long long stride1,
        const void *W2, int ld2, long long stride2, float beta, void *Y, int ldy, int *ids,
        float *weights, void *ws, size_t ws_bytes, void *stream) {
  if (M < 0 || M > GEMM_MOE_MAX_TOKENS) return -501;
  if (D < 1 || bad_size(D)) return -502;
  if (F < 1 || bad_size(F)) return -503;
  if (E < 1 || E > GEMM_MOE_MAX_EXPERTS) return -504;
  if (top_k < 1 || top_k > E || top_k > GEMM_MOE_MAX_CHOICES) return -505;
  if (renorm != 0 && renorm != 1) return -506;
  if (ldx < D) return -509;
  if (ldr < D) return -511;
  if (ld1 < D) return -513;
  if (stride1 < 0) return -514;
  if (ld2 < F) return -516;
  if (stride2 < 0) return -517;
  if (ldy < D) return -520;
  if (M == 0) return GEMM_SUCCESS;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if (alpha == 0.0f && beta == 1.0f) return GEMM_SUCCESS;
  if (alpha != 0.0f) {
    if (X == nullptr) return -508;
    if (Wr == nullptr) return -510;
    if (W1 == nullptr) return -512;
    if (W2 == nullptr) return -515;
  }
  if (Y == nullptr) return -519;
  if (alpha == 0.0f)
    return status(half ? dgemm::launch_scale_f16(M, D, beta, static_cast<uint16_t *>(Y), ldy, s)
                       : dgemm::launch_scale_f32(M, D, beta, static_cast<float *>(Y), ldy, s));
  MoeCall c = {};
  c.half = half;
  c.M = M;
  c.D = D;
  c.F = F;
  c.E = E;
  c.k = top_k;
  c.renorm = renorm != 0;
  c.alpha = alpha;
  c.X = X;
  c.ldx = ldx;
  c.Wr = Wr;
  c.ldr = ldr;
  c.W1 = W1;
  c.ld1 = ld1;
  c.stride1 = stride1;
  c.W2 = W2;
  c.ld2 = ld2;
  c.stride2 = stride2;
  c.beta = beta;
  c.Y = Y;
  c.ldy = ldy;
  c.ids = ids;
  c.weights = weights;
  c.stream = s;
  Space space;
  const int rc = space.open(ws, ws_bytes, dgemm::moe_workspace(c), s, -523);
  if (rc != 0) return rc;
  const hipError_t e = dgemm::launch_moe(c, space.get());
  const hipError_t f = space.close();
  return status(e != hipSuccess ? e : f);
}

}  // namespace

extern "C" {

int gemm_lora_f16(int M, int N, int K, float alpha, const gemm_half_t *X, int ldx,
                  const gemm_half_t *W, int ldw, float beta, gemm_half_t *Y, int ldy, int L, int R,
                  const gemm_half_t *A, int lda, long long stride_a, const gemm_half_t *B, int ldb,
                  long long stride_b, const float *scale, const int *ranks, const int *rows,
                  void *workspace, size_t workspace_bytes, void *stream) {
  return lora(true, M, N, K, alpha, X, ldx, W, ldw, beta, Y, ldy, L, R, A, lda, stride_a, B, ldb,
              stride_b, scale, ranks, rows, workspace, workspace_bytes, stream);
}

int gemm_lora_f32(int M, int N, int K, float alpha, const float *X, int ldx, const float *W,
                  int ldw, float beta, float *Y, int ldy, int L, int R, const float *A, int lda,
                  long long stride_a, const float *B, int ldb, long long stride_b,
                  const float *scale, const int *ranks, const int *rows, void *workspace,
                  size_t workspace_bytes, void *stream) {
  return lora(false, M, N, K, alpha, X, ldx, W, ldw, beta, Y, ldy, L, R, A, lda, stride_a, B, ldb,
              stride_b, scale, ranks, rows, workspace, workspace_bytes, stream);
}

size_t gemm_lora_workspace(int dtype, int M, int N, int K, int L, int R) {
  if ((dtype != 0 && dtype != 1) || M <= 0 || N <= 0 || K <= 0 || L <= 0 || bad_size(M) ||
      bad_size(N) || bad_size(K) || L > GEMM_LORA_MAX_ADAPTERS || R <= 0 || R > GEMM_LORA_MAX_RANK)
    return 0;
  LoraCall c = {};
  c.half = dtype == 1;
  c.M = M;
  c.N = N;
  c.K = K;
  c.L = L;
  c.R = R;
  return dgemm::lora_workspace(c);
}

int gemm_lora_grad_f16(int M, int N, int K, float alpha, const gemm_half_t *dY, int lddy,
                       const gemm_half_t *X, int ldx, const gemm_half_t *W, int ldw, int L, int R,
                       const gemm_half_t *A, int lda, long long stride_a, const gemm_half_t *B,
                       int ldb, long long stride_b, const float *scale, const int *ranks,
                       const int *rows, float beta_x, gemm_half_t *dX, int lddx, float beta_ab,
                       float *dA, int ldda, long long stride_da, float *dB, int lddb,
                       long long stride_db, void *workspace, size_t workspace_bytes,
                       void *stream) {
  return lora_grad(true, M, N, K, alpha, dY, lddy, X, ldx, W, ldw, L, R, A, lda, stride_a, B, ldb,
                   stride_b, scale, ranks, rows, beta_x, dX, lddx, beta_ab, dA, ldda, stride_da,
                   dB, lddb, stride_db, workspace, workspace_bytes, stream);
}

int gemm_lora_grad_f32(int M, int N, int K, float alpha, const float *dY, int lddy, const float *X,
                       int ldx, const float *W, int ldw, int L, int R, const float *A, int lda,
                       long long stride_a, const float *B, int ldb, long long stride_b,
                       const float *scale, const int *ranks, const int *rows, float beta_x,
                       float *dX, int lddx, float beta_ab, float *dA, int ldda,
                       long long stride_da, float *dB, int lddb, long long stride_db,
                       void *workspace, size_t workspace_bytes, void *stream) {
  return lora_grad(false, M, N, K, alpha, dY, lddy, X, ldx, W, ldw, L, R, A, lda, stride_a, B, ldb,
                   stride_b, scale, ranks, rows, beta_x, dX, lddx, beta_ab, dA, ldda, stride_da,
                   dB, lddb, stride_db, workspace, workspace_bytes, stream);
}

size_t gemm_lora_grad_workspace(int dtype, int M, int N, int K, int L, int R) {
  if ((dtype != 0 && dtype != 1) || M <= 0 || N <= 0 || K <= 0 || L <= 0 || bad_size(M) ||
      bad_size(N) || bad_size(K) || L > GEMM_LORA_MAX_ADAPTERS || R <= 0 || R > GEMM_LORA_MAX_RANK)
    return 0;
  static float some;   // only tells which outputs are wanted: all of them
  LoraCall c = {};
  c.half = dtype == 1;
  c.M = M;
  c.N = N;
  c.K = K;
  c.L = L;
  c.R = R;
  c.dX = &some;
  c.dA = &some;
  c.dB = &some;
  return dgemm::lora_grad_workspace(c);
}

int gemm_moe_f16(int M, int D, int F, int E, int top_k, int renorm, float alpha,
                 const gemm_half_t *X, int ldx, const gemm_half_t *Wr, int ldr,
                 const gemm_half_t *W1, int ld1, long long stride1, const gemm_half_t *W2, int ld2,
                 long long stride2, float beta, gemm_half_t *Y, int ldy, int *ids, float *weights,
                 void *workspace, size_t workspace_bytes, void *stream) {
  return moe(true, M, D, F, E, top_k, renorm, alpha, X, ldx, Wr, ldr, W1, ld1, stride1, W2, ld2,
             stride2, beta, Y, ldy, ids, weights, workspace, workspace_bytes, stream);
}

int gemm_moe_f32(int M, int D, int F, int E, int top_k, int renorm, float alpha, const float *X,
                 int ldx, const float *Wr, int ldr, const float *W1, int ld1, long long stride1,
                 const float *W2, int ld2, long long stride2, float beta, float *Y, int ldy,
                 int *ids, float *weights, void *workspace, size_t workspace_bytes, void *stream) {
  return moe(false, M, D, F, E, top_k, renorm, alpha, X, ldx, Wr, ldr, W1, ld1, stride1, W2, ld2,
             stride2, beta, Y, ldy, ids, weights, workspace, workspace_bytes, stream);
}

size_t gemm_moe_workspace(int dtype, int M, int D, int F, int E, int top_k) {
  if ((dtype != 0 && dtype != 1) || M <= 0 || M > GEMM_MOE_MAX_TOKENS || D < 1 || F < 1 || E < 1 ||
      bad_size(D) || bad_size(F) ||
      E > GEMM_MOE_MAX_EXPERTS || top_k < 1 || top_k > E || top_k > GEMM_MOE_MAX_CHOICES)
    return 0;
  MoeCall c = {};
  c.half = dtype == 1;
  c.M = M;
  c.D = D;
  c.F = F;
  c.E = E;
  c.k = top_k;
  return dgemm::moe_workspace(c);
}

}  // extern "C"
