// proj_api.hip -- the extern "C" entry points of products of 8-bit integers and
// gated blocks (include/gemm.h): argument checks, quick returns, workspace.
// Checks run before any HIP call; the first failure wins.
#include "../../include/gemm.h"
#include "internal.hpp"
#include "space.hpp"

namespace {

using dgemm::GluGradCall;
using dgemm::ProjCall;
using dgemm::rows_at_16;
using dgemm::rows_for_tiles;
using dgemm::Space;

int at_least_one(int n) { return n > 1 ? n : 1; }

bool bad_size(int n) { return n < 0 || n > GEMM_ROWS_MAX_SIZE; }
bool bad_half_size(int n) { return n < 0 || n > GEMM_ROWS_MAX_SIZE / 2; }
bool bad_act(int act) { return act < GEMM_ACT_SILU || act > GEMM_ACT_RELU; }

int status(hipError_t e) { return e == hipSuccess ? GEMM_SUCCESS : (int)e; }

hipStream_t stream_of(void *s) { return static_cast<hipStream_t>(s); }

hipError_t scale(bool half, int M, int N, float beta, void *C, int ldc, hipStream_t s) {
  return half ? dgemm::launch_scale_f16(M, N, beta, static_cast<uint16_t *>(C), ldc, s)
              : dgemm::launch_scale_f32(M, N, beta, static_cast<float *>(C), ldc, s);
}

int run(ProjCall &c, void *ws, size_t ws_bytes, int base) {
  const int eb = c.i8 ? 1 : (c.half ? 2 : 4);
  c.aligned = rows_for_tiles(c.X, c.ldx, eb) && rows_for_tiles(c.W, c.ldw, eb);
  Space space;
  const int rc = space.open(ws, ws_bytes, dgemm::proj_workspace(c), c.stream, base);
  if (rc != 0) return rc;
  const hipError_t e = dgemm::launch_proj(c, space.get());
  const hipError_t f = space.close();
  return status(e != hipSuccess ? e : f);
}

int quant(bool half, int M, int K, const void *X, int ldx, int8_t *Q, int ldq, float *scale,
          void *stream) {
  if (bad_size(M)) return -601;
  if (bad_size(K)) return -602;
  if (ldx < at_least_one(K)) return -604;
  if (ldq < at_least_one(K)) return -606;
  if (M == 0) return GEMM_SUCCESS;
  if (K > 0 && X == nullptr) return -603;
  if (K > 0 && Q == nullptr) return -605;
  if (scale == nullptr) return -607;
  return status(dgemm::launch_quant(half, M, K, X, ldx, Q, ldq, scale, stream_of(stream)));
}

int product(bool half, int M, int N, int K, float alpha, const int8_t *X, int ldx,
            const float *xs, const int8_t *W, int ldw, const float *wsc, float beta, void *Y,
            int ldy, void *ws, size_t ws_bytes, void *stream) {
  if (bad_size(M)) return -701;
  if (bad_size(N)) return -702;
  if (K < 0 || K > GEMM_I8_MAX_K) return -703;
  if (ldx < at_least_one(K)) return -706;
  if (ldw < at_least_one(K)) return -709;
  if (ldy < at_least_one(N)) return -713;
  if (M == 0 || N == 0) return GEMM_SUCCESS;
  const bool sums = K > 0 && alpha != 0.0f;
  if (sums && X == nullptr) return -705;
  if (sums && W == nullptr) return -708;
  if (!sums && beta == 1.0f) return GEMM_SUCCESS;
  if (Y == nullptr) return -712;
  if (!sums) return status(scale(half, M, N, beta, Y, ldy, stream_of(stream)));
  ProjCall c = {};
  c.i8 = true;
  c.half = half;
  c.M = M;
  c.N = N;
  c.K = K;
  c.alpha = alpha;
  c.beta = beta;
  c.X = X;
  c.ldx = ldx;
  c.xs = xs;
  c.W = W;
  c.ldw = ldw;
  c.ws = wsc;
  c.Y = Y;
  c.ldy = ldy;
  c.stream = stream_of(stream);
  return run(c, ws, ws_bytes, -714);
}

int glu(bool half, int M, int F, int K, int act, const void *X, int ldx, const void *W, int ldw,
        void *H, int ldh, void *Z, int ldz, void *ws, size_t ws_bytes, void *stream) {
  if (bad_size(M)) return -801;
  if (bad_half_size(F)) return -802;
  if (bad_size(K)) return -803;
  if (bad_act(act)) return -804;
  if (ldx < at_least_one(K)) return -806;
  if (ldw < at_least_one(K)) return -808;
  if (ldh < at_least_one(F)) return -810;
  if (Z != nullptr && ldz < at_least_one(2 * F)) return -812;
  if (M == 0 || F == 0) return GEMM_SUCCESS;
  if (K > 0 && X == nullptr) return -805;
  if (K > 0 && W == nullptr) return -807;
  if (H == nullptr) return -809;
  if (K == 0) {
    hipError_t e = scale(half, M, F, 0.0f, H, ldh, stream_of(stream));
    if (e == hipSuccess && Z != nullptr) e = scale(half, M, 2 * F, 0.0f, Z, ldz, stream_of(stream));
    return status(e);
  }
  ProjCall c = {};
  c.half = half;
  c.gated = true;
  c.M = M;
  c.N = F;
  c.K = K;
  c.act = act;
  c.X = X;
  c.ldx = ldx;
  c.W = W;
  c.ldw = ldw;
  c.Y = H;
  c.ldy = ldh;
  c.Z = Z;
  c.ldz = ldz;
  c.stream = stream_of(stream);
  return run(c, ws, ws_bytes, -813);
}

int glu_i8(bool half, int M, int F, int K, int act, const int8_t *X, int ldx, const float *xs,
           const int8_t *W, int ldw, const float *wsc, void *H, int ldh, void *ws,
           size_t ws_bytes, void *stream) {
  if (bad_size(M)) return -901;
  if (bad_half_size(F)) return -902;
  if (K < 0 || K > GEMM_I8_MAX_K) return -903;
  if (bad_act(act)) return -904;
  if (ldx < at_least_one(K)) return -906;
  if (ldw < at_least_one(K)) return -909;
  if (ldh < at_least_one(F)) return -912;
  if (M == 0 || F == 0) return GEMM_SUCCESS;
  if (K > 0 && X == nullptr) return -905;
  if (K > 0 && W == nullptr) return -908;
  if (H == nullptr) return -911;
  if (K == 0) return status(scale(half, M, F, 0.0f, H, ldh, stream_of(stream)));
  ProjCall c = {};
  c.i8 = true;
  c.half = half;
  c.gated = true;
  c.M = M;
  c.N = F;
  c.K = K;
  c.act = act;
  c.X = X;
  c.ldx = ldx;
  c.xs = xs;
  c.W = W;
  c.ldw = ldw;
  c.ws = wsc;
  c.Y = H;
  c.ldy = ldh;
  c.stream = stream_of(stream);
  return run(c, ws, ws_bytes, -913);
}

int glu_grad(bool half, bool dw32, int M, int F, int K, int act, const void *dH, int lddh,
             const void *X, int ldx, const void *W, int ldw, const void *Z, int ldz, float beta_x,
             void *dX, int lddx, float beta_w, void *dW, int lddw, void *ws, size_t ws_bytes,
             void *stream) {
  if (bad_size(M)) return -1001;
  if (bad_half_size(F)) return -1002;
  if (bad_size(K)) return -1003;
  if (bad_act(act)) return -1004;
  if (lddh < at_least_one(F)) return -1006;
  const bool reads_x = dW != nullptr || Z == nullptr, reads_w = dX != nullptr || Z == nullptr;
  if (reads_x && ldx < at_least_one(K)) return -1008;
  if (reads_w && ldw < at_least_one(K)) return -1010;
  if (Z != nullptr && ldz < at_least_one(2 * F)) return -1012;
  if (dX != nullptr && lddx < at_least_one(K)) return -1015;
  if (dW != nullptr && lddw < at_least_one(K)) return -1018;
  const bool want_x = dX != nullptr && M > 0 && K > 0;
  const bool want_w = dW != nullptr && F > 0 && K > 0;
  const hipStream_t s = stream_of(stream);
  if (!want_x && !want_w) return GEMM_SUCCESS;
  if (M == 0 || F == 0) {
    // every sum is empty: what there is of the outputs is scaled
    hipError_t e = hipSuccess;
    if (want_x && beta_x != 1.0f) e = scale(half, M, K, beta_x, dX, lddx, s);
    if (e == hipSuccess && want_w && beta_w != 1.0f)
      e = scale(half && !dw32, 2 * F, K, beta_w, dW, lddw, s);
    return status(e);
  }
  if (dH == nullptr) return -1005;
  if (X == nullptr && (want_w || Z == nullptr)) return -1007;
  if (W == nullptr && (want_x || Z == nullptr)) return -1009;
  GluGradCall c = {};
  c.half = half;
  c.dw32 = dw32;
  const int eb = half ? 2 : 4;
  c.aligned = (X == nullptr || rows_for_tiles(X, ldx, eb)) &&
              (W == nullptr || rows_for_tiles(W, ldw, eb));
  c.at_16 = (X == nullptr || rows_at_16(X, ldx, eb)) && (W == nullptr || rows_at_16(W, ldw, eb));
  c.M = M;
  c.F = F;
  c.K = K;
  c.act = act;
  c.dH = dH;
  c.lddh = lddh;
  c.X = X;
  c.ldx = ldx;
  c.W = W;
  c.ldw = ldw;
  c.Z = Z;
  c.ldz = ldz;
  c.beta_x = beta_x;
  c.dX = want_x ? dX : nullptr;
  c.lddx = lddx;
  c.beta_w = beta_w;
  c.dW = want_w ? dW : nullptr;
  c.lddw = lddw;
  c.stream = s;
  Space space;
  const int rc = space.open(ws, ws_bytes, dgemm::glu_grad_workspace(c), s, -1019);
  if (rc != 0) return rc;
  const hipError_t e = dgemm::launch_glu_grad(c, space.get());
  const hipError_t f = space.close();
  return status(e != hipSuccess ? e : f);
}

}  // namespace

extern "C" {

int gemm_quant_i8_f16(int M, int K, const gemm_half_t *X, int ldx, int8_t *Q, int ldq,
                      float *scale, void *stream) {
  return quant(true, M, K, X, ldx, Q, ldq, scale, stream);
}

int gemm_quant_i8_f32(int M, int K, const float *X, int ldx, int8_t *Q, int ldq, float *scale,
                      void *stream) {
  return quant(false, M, K, X, ldx, Q, ldq, scale, stream);
}

int gemm_i8_f16(int M, int N, int K, float alpha, const int8_t *X, int ldx, const float *x_scale,
                const int8_t *W, int ldw, const float *w_scale, float beta, gemm_half_t *Y,
                int ldy, void *workspace, size_t workspace_bytes, void *stream) {
  return product(true, M, N, K, alpha, X, ldx, x_scale, W, ldw, w_scale, beta, Y, ldy, workspace,
                 workspace_bytes, stream);
}

int gemm_i8_f32(int M, int N, int K, float alpha, const int8_t *X, int ldx, const float *x_scale,
                const int8_t *W, int ldw, const float *w_scale, float beta, float *Y, int ldy,
                void *workspace, size_t workspace_bytes, void *stream) {
  return product(false, M, N, K, alpha, X, ldx, x_scale, W, ldw, w_scale, beta, Y, ldy, workspace,
                 workspace_bytes, stream);
}

size_t gemm_i8_workspace(int M, int N, int K, int aligned) {
  if (M <= 0 || N <= 0 || K <= 0 || bad_size(M) || bad_size(N) || K > GEMM_I8_MAX_K) return 0;
  ProjCall c = {};
  c.i8 = true;
  c.half = true;
  c.aligned = aligned != 0;
  c.M = M;
  c.N = N;
  c.K = K;
  return dgemm::proj_workspace(c);
}

int gemm_glu_f16(int M, int F, int K, int act, const gemm_half_t *X, int ldx, const gemm_half_t *W,
                 int ldw, gemm_half_t *H, int ldh, gemm_half_t *Z, int ldz, void *workspace,
                 size_t workspace_bytes, void *stream) {
  return glu(true, M, F, K, act, X, ldx, W, ldw, H, ldh, Z, ldz, workspace, workspace_bytes,
             stream);
}

int gemm_glu_f32(int M, int F, int K, int act, const float *X, int ldx, const float *W, int ldw,
                 float *H, int ldh, float *Z, int ldz, void *workspace, size_t workspace_bytes,
                 void *stream) {
  return glu(false, M, F, K, act, X, ldx, W, ldw, H, ldh, Z, ldz, workspace, workspace_bytes,
             stream);
}

int gemm_glu_i8_f16(int M, int F, int K, int act, const int8_t *X, int ldx, const float *x_scale,
                    const int8_t *W, int ldw, const float *w_scale, gemm_half_t *H, int ldh,
                    void *workspace, size_t workspace_bytes, void *stream) {
  return glu_i8(true, M, F, K, act, X, ldx, x_scale, W, ldw, w_scale, H, ldh, workspace,
                workspace_bytes, stream);
}

int gemm_glu_i8_f32(int M, int F, int K, int act, const int8_t *X, int ldx, const float *x_scale,
                    const int8_t *W, int ldw, const float *w_scale, float *H, int ldh,
                    void *workspace, size_t workspace_bytes, void *stream) {
  return glu_i8(false, M, F, K, act, X, ldx, x_scale, W, ldw, w_scale, H, ldh, workspace,
                workspace_bytes, stream);
}

size_t gemm_glu_workspace(int dtype, int M, int F, int K, int aligned) {
  if (dtype < 0 || dtype > 2 || M <= 0 || F <= 0 || K <= 0 || bad_size(M) || bad_half_size(F) ||
      bad_size(K) || (dtype == 2 && K > GEMM_I8_MAX_K))
    return 0;
  ProjCall c = {};
  c.i8 = dtype == 2;
  c.half = dtype != 0;
  c.gated = true;
  c.aligned = aligned != 0;
  c.M = M;
  c.N = F;
  c.K = K;
  return dgemm::proj_workspace(c);
}

int gemm_glu_grad_f16(int M, int F, int K, int act, const gemm_half_t *dH, int lddh,
                      const gemm_half_t *X, int ldx, const gemm_half_t *W, int ldw,
                      const gemm_half_t *Z, int ldz, float beta_x, gemm_half_t *dX, int lddx,
                      float beta_w, gemm_half_t *dW, int lddw, void *workspace,
                      size_t workspace_bytes, void *stream) {
  return glu_grad(true, false, M, F, K, act, dH, lddh, X, ldx, W, ldw, Z, ldz, beta_x, dX, lddx,
                  beta_w, dW, lddw, workspace, workspace_bytes, stream);
}

int gemm_glu_grad_f16f32(int M, int F, int K, int act, const gemm_half_t *dH, int lddh,
                         const gemm_half_t *X, int ldx, const gemm_half_t *W, int ldw,
                         const gemm_half_t *Z, int ldz, float beta_x, gemm_half_t *dX, int lddx,
                         float beta_w, float *dW, int lddw, void *workspace,
                         size_t workspace_bytes, void *stream) {
  return glu_grad(true, true, M, F, K, act, dH, lddh, X, ldx, W, ldw, Z, ldz, beta_x, dX, lddx,
                  beta_w, dW, lddw, workspace, workspace_bytes, stream);
}

int gemm_glu_grad_f32(int M, int F, int K, int act, const float *dH, int lddh, const float *X,
                      int ldx, const float *W, int ldw, const float *Z, int ldz, float beta_x,
                      float *dX, int lddx, float beta_w, float *dW, int lddw, void *workspace,
                      size_t workspace_bytes, void *stream) {
  return glu_grad(false, true, M, F, K, act, dH, lddh, X, ldx, W, ldw, Z, ldz, beta_x, dX, lddx,
                  beta_w, dW, lddw, workspace, workspace_bytes, stream);
}

size_t gemm_glu_grad_workspace(int dtype, int M, int F, int K, int aligned) {
  if (dtype < 0 || dtype > 1 || M <= 0 || F <= 0 || K <= 0 || bad_size(M) || bad_half_size(F) ||
      bad_size(K))
    return 0;
  GluGradCall c = {};
  c.half = dtype == 1;
  c.M = M;
  c.F = F;
  c.K = K;
  // also what a call takes whose rows allow more
  size_t bytes = 0;
  for (int least = aligned != 0 ? 1 : 0; least <= 2; ++least) {
    c.aligned = least >= 1;
    c.at_16 = least >= 2;
    const size_t n = dgemm::glu_grad_workspace(c);
    bytes = n > bytes ? n : bytes;
  }
  return bytes;
}

}  // extern "C"
