// proj.hpp -- a projection X W^T with what follows it in the same kernel: the
// scales of a product of 8-bit integers, or a gated block's activation and
// product (forward, and [dG dU] of its backward pass).
//
// This file holds what every form shares: the arguments, what becomes of an
// element, and the kernel for few rows.
#pragma once

#include "act.hpp"
#include "common.hpp"
#include "internal.hpp"
#include "rows.hpp"

namespace dgemm {

// What becomes of the sums.
//   kScaled  Y[m, n] := alpha * xs[m] ws[n] * sum + beta * Y[m, n]
//   kGated   H[m, f] := act(g) * u, and Z[m, f], Z[m, F + f] := g, u where
//            wanted; g and u: the sums of W's rows f and F + f (times their
//            scales)
//   kSlopes  Z[m, f], Z[m, F + f] := dH[m, f] * u * act'(g), dH[m, f] * act(g)
enum ProjOut { kScaled, kGated, kSlopes };

struct ProjParams {
  const void *X, *W;
  const float *xs, *ws;   // scales of X's rows and of W's (NULL: 1)
  void *Y, *Z;            // kGated: H and Z (may be NULL)
  const void *dH;
  int ldx, ldw, ldy, ldz, lddh;
  int M, N, K;            // gated: N = F, W has 2N rows
  int act;
  float alpha, beta;
};

// The sum in 32-bit integers as a number with its scales: one rounding of the
// sum and two of the scales.
__device__ __forceinline__ float with_scales(float v, const ProjParams &p, float xs, int row) {
  if (p.xs != nullptr) v *= xs;
  if (p.ws != nullptr) v *= p.ws[row];
  return v;
}

// Element (m, n), from the sums of rows n and (gated) N + n of W.
template <int OUT, typename TO>
__device__ __forceinline__ void finish(const ProjParams &p, int m, int n, float a, float b) {
  const float xs = p.xs != nullptr ? p.xs[m] : 1.0f;
  a = with_scales(a, p, xs, n);
  if constexpr (OUT == kScaled) {
    TO *y = static_cast<TO *>(p.Y) + (size_t)m * (size_t)p.ldy + n;
    float o = p.alpha * a;
    if (p.beta != 0.0f) o = __builtin_fmaf(p.beta, (float)*y, o);
    *y = (TO)o;
  } else {
    b = with_scales(b, p, xs, p.N + n);
    TO *z = static_cast<TO *>(p.Z) + (size_t)m * (size_t)p.ldz + n;
    if constexpr (OUT == kGated) {
      static_cast<TO *>(p.Y)[(size_t)m * (size_t)p.ldy + n] = (TO)(act_value(p.act, a) * b);
      if (p.Z != nullptr) {
        z[0] = (TO)a;
        z[p.N] = (TO)b;
      }
    } else {
      const float d = (float)static_cast<const TO *>(p.dH)[(size_t)m * (size_t)p.lddh + n];
      float value, slope;
      act_both(p.act, a, value, slope);
      z[0] = (TO)(d * b * slope);
      z[p.N] = (TO)(d * value);
    }
  }
}

// Kernels of many rows (gemm_i8.hip, glu_f16.hip, glu_i8.hip): rows of X and W
// start at 16 bytes and are less than kTileRowBytes apart, so that a tile's
// offsets fit 32 bits.  half: outputs of fp16, else fp32; slopes: kSlopes.
constexpr long long kTileRowBytes = 1 << 23;
hipError_t launch_proj_i8(const ProjParams &p, bool half, hipStream_t stream);
hipError_t launch_glu_i8(const ProjParams &p, bool half, hipStream_t stream);
hipError_t launch_glu_f16(const ProjParams &p, bool slopes, hipStream_t stream);

// ---------------------------------------------------------------- few rows

// grid: (columns / BC, rows / BT).  A workgroup's waves divide K among
// themselves; each wave streams its stretch of the weights' rows from memory
// into matrix-core fragments (stream_mac), then the waves' sums meet in LDS.
// NF blocks of 16 / P weight rows (gated: the first half gate rows, the rest up
// rows), NB blocks of 16 / P rows of X, P stretches of k in one instruction.
template <typename T, typename TO, int OUT, int NF, int NB, int P, int WAVES>
__global__ __launch_bounds__(WAVES *kWave) void proj_skinny(ProjParams p) {
  typedef typename El<T>::Acc Acc;
  typedef typename std::remove_reference<decltype(Acc{}[0])>::type Sum;
  constexpr bool GATED = OUT != kScaled;
  constexpr int BR = 16 / P;
  constexpr int BC = GATED ? BR * NF / 2 : BR * NF;   // columns of the result
  constexpr int BT = BR * NB;                         // rows of it
  static_assert(!GATED || NF % 2 == 0, "gate and up rows in pairs of blocks");
  __shared__ Sum red[WAVES][BR * NF][BR + 1];
  const int lane = threadIdx.x % kWave, wave = wave_id();
  const int li = lane % 16, lg = lane / 16;
  const int n0 = blockIdx.x * BC, m0 = blockIdx.y * BT;
  const T *w[NF];
#pragma unroll
  for (int f = 0; f < NF; ++f) {
    const int r = BR * f + li / P;
    const int n = n0 + (r < BC ? r : r - BC);
    w[f] = static_cast<const T *>(p.W) +
           (size_t)((r < BC ? 0 : p.N) + (n < p.N ? n : p.N - 1)) * (size_t)p.ldw;
  }
  constexpr int G = 2 * El<T>::KSTEP * P;
  const int part = ((p.K + WAVES - 1) / WAVES + G - 1) / G * G;
  const int k0 = wave * part < p.K ? wave * part : p.K;
  const int k1 = k0 + part < p.K ? k0 + part : p.K;
  RowLoader<T, NB> x;
  x.lim = k1;
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const int m = m0 + BR * b + li / P;
    x.row[b] = static_cast<const T *>(p.X) + (size_t)(m < p.M ? m : p.M - 1) * (size_t)p.ldx;
  }
  Acc acc[NF][NB];
#pragma unroll
  for (int f = 0; f < NF; ++f)
#pragma unroll
    for (int b = 0; b < NB; ++b) acc[f][b] = Acc{0, 0, 0, 0};
  stream_mac<T, (NF * NB >= 8 ? 2 : 4), P>(w, k0, k1, k1, k1, x, acc);
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    if (m0 + BR * b >= p.M) break;
    if (b > 0) __syncthreads();
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      Sum v[4 / P];
      diagonal_sum<P>(acc[f][b], v);
      if (li % P == 0)
#pragma unroll
        for (int j = 0; j < 4 / P; ++j) red[wave][BR * f + 4 / P * lg + j][li / P] = v[j];
    }
    __syncthreads();
    for (int q = threadIdx.x; q < BC * BR; q += WAVES * kWave) {
      const int c = q % BC, t = q / BC;
      const int n = n0 + c, m = m0 + BR * b + t;
      Sum s = 0, u = 0;
#pragma unroll
      for (int v = 0; v < WAVES; ++v) {
        s += red[v][c][t];
        if constexpr (GATED) u += red[v][BC + c][t];
      }
      if (n < p.N && m < p.M) finish<OUT, TO>(p, m, n, (float)s, (float)u);
    }
  }
}

}  // namespace dgemm
