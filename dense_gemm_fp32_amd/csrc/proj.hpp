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
//   kScaled  Y[m, n] := alpha * (ws[n] * (xs[m] * sum)) + beta * Y[m, n]
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

// Kernels of many rows (gemm_i8.hip, glu_f16.hip, glu_f32.hip, glu_i8.hip): rows of X and W
// start at 16 bytes (of floats anywhere) and are less than kTileRowBytes apart, so
// that a tile's offsets fit 32 bits.  half: outputs of fp16, else fp32; slopes: kSlopes.
constexpr long long kTileRowBytes = 1 << 23;
hipError_t launch_proj_i8(const ProjParams &p, bool half, hipStream_t stream);
hipError_t launch_glu_i8(const ProjParams &p, bool half, hipStream_t stream);
hipError_t launch_glu_f16(const ProjParams &p, bool slopes, hipStream_t stream);
hipError_t launch_glu_f32(const ProjParams &p, bool slopes, hipStream_t stream);

// One of the two products of a gated block's backward pass (glu_products.hip):
// C := A B + beta * C, B's rows along k, and A's in the second product.  Rows of
// both start at 16 bytes, but for B's of floats.
struct ProductJob {
  const void *A, *B;
  void *C;                // NULL: not wanted
  int lda, ldb, ldc, M, N, K;
  float beta;
  bool odd;               // fp32: not every row of B starts at 16 bytes
  int splits, chunk;      // K in parts of `chunk`; more than one: their sums to
  float *slab;            // slab, part after part, in rows of N rounded up to 4
};
struct ProductPlan {
  bool mid;               // 128x128 tiles, else 64x64
  double us;              // estimate
};
ProductPlan plan_products(bool half, ProductJob &a, ProductJob &b);   // sets splits, chunk
// half: A and B hold fp16 (and C, but b's fp32 with b32), else fp32
hipError_t launch_products(bool half, bool b32, bool mid, const ProductJob &a, const ProductJob &b,
                           hipStream_t stream);

// ---------------------------------------------------------------- few rows

// A block of 16 rows as a lane loads it: 256 consecutive bytes of each row, in
// four loads of four rows each, in which the four lanes of a quad read 64
// consecutive bytes.  (The texture unit takes a load quad by quad, a cycle for
// each line that a quad touches.  Loads in the fragments' own layout, where each
// lane of a quad reads another row, take it four times as long: 64 rows of 4096
// bytes beside 16 rows of weights on each of 64 CUs, 8.5 us beyond a launch's own
// time; in all 11.7 us so, 7.0 in quads.)  Offsets are 32 bits wide: rows less than kQuadRowBytes apart.
constexpr long long kQuadRowBytes = 1 << 27;

template <typename T>
struct QuadRows {
  const T *base;
  uint32_t at[4];      // byte offsets of load j: row 4 * (lane % 16 / 4) + j

  // first: the block's first row, in a matrix that ends after `rows` rows
  __device__ __forceinline__ void set(const void *m, int first, int rows, int ld) {
    const int lane = threadIdx.x % kWave;
    const int f = first < rows ? first : rows - 1;
    base = static_cast<const T *>(m) + (size_t)f * (size_t)ld;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = lane % 16 / 4 * 4 + j, last = rows - 1 - f;
      at[j] = (uint32_t)(r < last ? r : last) * (uint32_t)ld * (uint32_t)sizeof(T) +
              (uint32_t)(lane / 16 * 64 + lane % 4 * 16);
    }
  }
  __device__ __forceinline__ typename El<T>::Frag load(int j, int k) const {
    const char *p = reinterpret_cast<const char *>(base + k);
    return load_whole(reinterpret_cast<const T *>(p + at[j]));
  }
};

// Four loads as four fragments: element j of lane t of a quad changes places with
// element t of lane j.  Fragment i then holds, in lane l, bytes 64 * (l / 16) + 16 i
// .. +15 of row l % 16's 256: the same k in all rows of a group of 16 lanes, as
// the matrix instruction wants it, whose order over k is its own.
template <class F>
__device__ __forceinline__ void quad_transpose(F (&v)[4]) {
  const bool odd = (threadIdx.x & 1) != 0, high = (threadIdx.x & 2) != 0;
  i32x4 r[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) r[j] = __builtin_bit_cast(i32x4, v[j]);
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    int s[4];
#pragma unroll
    for (int j = 0; j < 4; j += 2) {
      const int x = __builtin_amdgcn_mov_dpp(r[j + 1][d], 0xB1, 0xf, 0xf, true);   // lane ^ 1
      const int y = __builtin_amdgcn_mov_dpp(r[j][d], 0xB1, 0xf, 0xf, true);
      s[j] = odd ? x : r[j][d];
      s[j + 1] = odd ? r[j + 1][d] : y;
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int x = __builtin_amdgcn_mov_dpp(s[j + 2], 0x4E, 0xf, 0xf, true);      // lane ^ 2
      const int y = __builtin_amdgcn_mov_dpp(s[j], 0x4E, 0xf, 0xf, true);
      r[j][d] = high ? x : s[j];
      r[j + 2][d] = high ? s[j + 2] : y;
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = __builtin_bit_cast(F, r[j]);
}

// acc[f][b] += U chunks of 256 bytes a row from element k on.
template <typename T, int U, int NF, int NB>
__device__ __forceinline__ void quad_steps(const QuadRows<T> (&w)[NF], const QuadRows<T> (&x)[NB],
                                           int k, typename El<T>::Acc (&acc)[NF][NB]) {
  typedef typename El<T>::Frag Frag;
  constexpr int CH = 16 * El<T>::VEC;
  Frag wf[U][NF][4], xf[U][NB][4];
#pragma unroll
  for (int u = 0; u < U; ++u) {
#pragma unroll
    for (int f = 0; f < NF; ++f)
#pragma unroll
      for (int j = 0; j < 4; ++j) wf[u][f][j] = w[f].load(j, k + u * CH);
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int j = 0; j < 4; ++j) xf[u][b][j] = x[b].load(j, k + u * CH);
  }
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int u = 0; u < U; ++u) {
#pragma unroll
    for (int f = 0; f < NF; ++f) quad_transpose(wf[u][f]);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      quad_transpose(xf[u][b]);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int f = 0; f < NF; ++f) acc[f][b] = mma16(wf[u][f][i], xf[u][b][i], acc[f][b]);
    }
  }
}

// grid: (columns / BC, rows / BT).  A workgroup's waves divide K among
// themselves; each wave streams its stretch of the weights' rows from memory
// into matrix-core fragments, then the waves' sums meet in LDS.  NF blocks of BR
// weight rows (gated: the first half gate rows, the rest up rows), NB blocks of
// BR rows of X.  P > 1: blocks of 16 / P rows, P stretches of k in one
// instruction (stream_mac); P == 1: blocks of 16 rows (quad_steps).
template <typename T, typename TO, int OUT, int NF, int NB, int P, int WAVES, int U>
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
  auto w_row = [&](int r) {      // row r of the workgroup's
    const int n = n0 + (r < BC ? r : r - BC);
    return static_cast<const T *>(p.W) +
           (size_t)((r < BC ? 0 : p.N) + (n < p.N ? n : p.N - 1)) * (size_t)p.ldw;
  };
  auto x_row = [&](int r) {
    const int m = m0 + r;
    return static_cast<const T *>(p.X) + (size_t)(m < p.M ? m : p.M - 1) * (size_t)p.ldx;
  };
  // each wave a stretch of whole chunks (of at least 256 bytes a row)
  constexpr int G = P == 1 ? 16 * El<T>::VEC : 2 * El<T>::KSTEP * P;
  const int part = ((p.K + WAVES - 1) / WAVES + G - 1) / G * G;
  const int k0 = wave * part < p.K ? wave * part : p.K;
  const int k1 = k0 + part < p.K ? k0 + part : p.K;
  Acc acc[NF][NB];
#pragma unroll
  for (int f = 0; f < NF; ++f)
#pragma unroll
    for (int b = 0; b < NB; ++b) acc[f][b] = Acc{0, 0, 0, 0};
  int k = k0;
  if constexpr (P == 1) {
    QuadRows<T> w[NF], x[NB];
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      const bool up = GATED && f >= NF / 2;
      w[f].set(static_cast<const T *>(p.W) + (up ? (size_t)p.N * (size_t)p.ldw : 0),
               n0 + 16 * (up ? f - NF / 2 : f), p.N, p.ldw);
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) x[b].set(p.X, m0 + 16 * b, p.M, p.ldx);
    for (; k + U * G <= k1; k += U * G) quad_steps<T, U>(w, x, k, acc);
    if constexpr (U > 1)
      for (; k + G <= k1; k += G) quad_steps<T, 1>(w, x, k, acc);
  }
  if (P > 1 || k < k1) {
    const T *w[NF];
#pragma unroll
    for (int f = 0; f < NF; ++f) w[f] = w_row(BR * f + li / P);
    RowLoader<T, NB> x;
    x.lim = k1;
#pragma unroll
    for (int b = 0; b < NB; ++b) x.row[b] = x_row(BR * b + li / P);
    stream_mac<T, (P == 1 ? 1 : U), P>(w, k, k1, k1, k1, x, acc);
  }
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
