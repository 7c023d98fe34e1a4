// rows.hpp -- device-side pieces shared by the products whose rows choose
// their own weights (lora.hip, moe.hip).
//
// Both are skinny products: 16 rows of activations at a time against rows of
// weights that are read once, so the operands go from global memory straight
// into matrix-core fragments, without a stop in LDS.  One fragment holds, in
// lane l, VEC consecutive k of row l % 16 (16 bytes: 8 halves or 4 floats), k
// group l / 16; the 16x16 result holds, in lane l, column l % 16 (the second
// operand's row) and rows 4*(l/16) .. +3 (the first operand's).
#pragma once

#include "common.hpp"

namespace dgemm {

template <typename T>
struct El;

template <>
struct El<_Float16> {
  static constexpr int VEC = 8;      // elements per 16 bytes: k per lane of a fragment
  static constexpr int KSTEP = 32;   // k per fragment (4 lane groups)
  typedef f16x8 Frag;
};

template <>
struct El<float> {
  static constexpr int VEC = 4;
  static constexpr int KSTEP = 16;
  typedef f32x4 Frag;
};

__device__ __forceinline__ f32x4 mma16(f16x8 a, f16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// Four v_mfma_f32_16x16x4_f32: the j-th takes element j of every lane, so the
// k order is the same for both operands and the sum covers all 16 k.
__device__ __forceinline__ f32x4 mma16(f32x4 a, f32x4 b, f32x4 c) {
#pragma unroll
  for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[j], b[j], c, 0, 0, 0);
  return c;
}

// A row's values as two halves each: hi + lo holds 22 bits.
struct Halves {
  f16x8 hi, lo;
};

// An infinity or NaN among the weights meets the high parts only: a low part,
// of either sign or zero, would make a NaN of an infinity.
__device__ __forceinline__ f32x4 mma16(f16x8 w, const Halves &x, f32x4 c) {
  return mma16(finite(w), x.lo, mma16(w, x.hi, c));
}

// VEC consecutive elements at any element's address.  Global loads of 16
// bytes need no more than the element's own alignment on this target, so rows
// of any length, padding and offset take the same path; only the last, partly
// filled step of a row is loaded element by element, since what lies behind a
// row is never read.
template <typename T>
__device__ __forceinline__ typename El<T>::Frag load_whole(const T *p) {
  typedef T Any __attribute__((ext_vector_type(El<T>::VEC), aligned(sizeof(T))));
  return *reinterpret_cast<const Any *>(p);
}

// The first n of VEC elements, the others 0: one at a time, since this is for
// the ends of rows only and unrolled it costs a kernel that has several of
// them in flight the registers of every element's address.
__device__ __forceinline__ f16x8 load_part(const _Float16 *p, int n) {
  unsigned long long lo = 0, hi = 0;
#pragma unroll 1
  for (int e = (n < 8 ? n : 8) - 1; e >= 0; --e) {
    hi = (hi << 16) | (lo >> 48);
    lo = (lo << 16) | __builtin_bit_cast(uint16_t, p[e]);
  }
  typedef unsigned long long u64x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(f16x8, u64x2{lo, hi});
}

__device__ __forceinline__ f32x4 load_part(const float *p, int n) {
  f32x4 f = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
  for (int e = (n < 4 ? n : 4) - 1; e >= 0; --e) f = f32x4{p[e], f[0], f[1], f[2]};
  return f;
}

// v's elements moved down by s places (none for s <= 0, all out for s >= VEC),
// zeros behind them.
__device__ __forceinline__ f16x8 move_down(f16x8 v, int s) {
  typedef unsigned long long u64x2 __attribute__((ext_vector_type(2)));
  const u64x2 w = __builtin_bit_cast(u64x2, v);
  unsigned long long lo = w[0], hi = w[1];
  s = s > 0 ? s : 0;
  if (s & 4) lo = hi, hi = 0;
  if (s & 2) lo = (lo >> 32) | (hi << 32), hi >>= 32;
  if (s & 1) lo = (lo >> 16) | (hi << 48), hi >>= 16;
  if (s >= 8) lo = hi = 0;
  return __builtin_bit_cast(f16x8, u64x2{lo, hi});
}

__device__ __forceinline__ f32x4 move_down(f32x4 v, int s) {
  s = s > 0 ? s : 0;
  if (s & 2) v = f32x4{v[2], v[3], 0.0f, 0.0f};
  if (s & 1) v = f32x4{v[1], v[2], v[3], 0.0f};
  if (s >= 4) v = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  return v;
}

// Elements k .. k+VEC-1 of a row of K >= VEC elements, 0 beyond its end: one
// load that stays inside the row, whatever k, and is moved into place, so that
// several can be on their way together.
template <typename T>
__device__ __forceinline__ typename El<T>::Frag load_end(const T *row, int k, int K) {
  const int last = K - El<T>::VEC;
  return move_down(load_whole(row + (k < last ? k : last)), k - last);
}

// The same for a row of any length.
template <typename T>
__device__ __forceinline__ typename El<T>::Frag load_frag(const T *row, int k, int K) {
  return K < El<T>::VEC ? load_part(row + k, K - k) : load_end(row, k, K);
}

// acc[f][b] += W block f (16 rows, this lane's at w[f]) times activation block
// b over k in [k0, k1).  Activations come from `x`: x.whole(b, kk) loads this
// lane's values at kk = k + VEC * lane group, x.masked(b, kk) the same with 0
// at and beyond this lane's end of the row, x.frag makes a fragment (or Halves)
// of them.
// Steps that end at or before `kw` are whole for every lane; `lim` is this
// lane's end of the weights' rows.  The loads of U steps are issued together,
// ahead of their products (the scheduling barrier keeps the compiler from
// pairing each load with its use, which left too few bytes in flight).  k0 is
// a multiple of KSTEP.
//
// P > 1 puts P neighbouring stretches of k into one instruction: lane l % 16
// holds row l % 16 / P of 16 / P rows, stretch l % P, so that P neighbouring
// lanes read 16 P consecutive bytes; a step then covers P * KSTEP k, and of the
// 16 x 16 products those whose row and column hold the same stretch count
// (diagonal_sum adds them up).
template <typename T, int U, int P, int NF, int NB, class X>
__device__ __forceinline__ void stream_steps(const T *const (&w)[NF], int k, const X &x,
                                             f32x4 (&acc)[NF][NB]) {
  typedef typename El<T>::Frag Frag;
  constexpr int KS = P * El<T>::KSTEP;
  Frag wf[U][NF];
  typename X::Raw xr[U][NB];
#pragma unroll
  for (int u = 0; u < U; ++u) {
#pragma unroll
    for (int f = 0; f < NF; ++f) wf[u][f] = load_whole(w[f] + k + u * KS);
#pragma unroll
    for (int b = 0; b < NB; ++b) xr[u][b] = x.whole(b, k + u * KS);
  }
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const auto xf = x.frag(b, xr[u][b]);
#pragma unroll
      for (int f = 0; f < NF; ++f) acc[f][b] = mma16(wf[u][f], xf, acc[f][b]);
    }
}

template <typename T, int U, int P, int NF, int NB, class X>
__device__ __forceinline__ void stream_mac(const T *const (&w)[NF], int k0, int k1, int kw,
                                           int lim, const X &x, f32x4 (&acc)[NF][NB]) {
  typedef typename El<T>::Frag Frag;
  constexpr int KS = P * El<T>::KSTEP;
  const int lane = threadIdx.x % kWave;
  const int lk = (lane / 16 * P + lane % P) * El<T>::VEC;
  int k = k0;
  for (; k + U * KS <= kw; k += U * KS) stream_steps<T, U, P>(w, k + lk, x, acc);
  // what is left of the whole steps, in halves, so that it too is loaded together
  if constexpr (U >= 8)
    if (k + 4 * KS <= kw) {
      stream_steps<T, 4, P>(w, k + lk, x, acc);
      k += 4 * KS;
    }
  if constexpr (U >= 4)
    if (k + 2 * KS <= kw) {
      stream_steps<T, 2, P>(w, k + lk, x, acc);
      k += 2 * KS;
    }
  for (; k + KS <= kw; k += KS) stream_steps<T, 1, P>(w, k + lk, x, acc);
  for (; k < k1; k += KS) {
    Frag wf[NF];
#pragma unroll
    for (int f = 0; f < NF; ++f) wf[f] = load_frag(w[f], k + lk, lim);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const auto xf = x.frag(b, x.masked(b, k + lk));
#pragma unroll
      for (int f = 0; f < NF; ++f) acc[f][b] = mma16(wf[f], xf, acc[f][b]);
    }
  }
}

// The sums of a product made with P stretches (above): element q of the result
// is row lane/16 * 4/P + q, column lane % 16 / P, in every lane.
template <int P>
__device__ __forceinline__ void diagonal_sum(const f32x4 &v, float (&out)[4 / P]) {
  const int p = threadIdx.x % P;
#pragma unroll
  for (int q = 0; q < 4 / P; ++q) {
    float s = v[q * P];
#pragma unroll
    for (int j = 1; j < P; ++j) s = p == j ? v[q * P + j] : s;
#pragma unroll
    for (int o = 1; o < P; o <<= 1) s += __shfl_xor(s, o);
    out[q] = s;
  }
}

// Activations of the weights' own type: this lane's row of block b at row[b].
template <typename T, int NB>
struct RowLoader {
  typedef typename El<T>::Frag Raw;
  const T *row[NB];
  int lim;
  __device__ __forceinline__ Raw whole(int b, int k) const { return load_whole(row[b] + k); }
  __device__ __forceinline__ Raw masked(int b, int k) const { return load_frag(row[b], k, lim); }
  __device__ __forceinline__ Raw frag(int, const Raw &r) const { return r; }
};

// Exponent of the power of two that a row is divided by so that its largest
// finite magnitude, of these bits, comes to [2^14, 2^15) as fp16 (at least -100;
// 0 for a row without a normal number): what is not finite must not decide it,
// or the finite values beside an infinity would become infinities themselves.
__device__ __forceinline__ int row_exponent(unsigned bits) {
  const int e = (int)(bits >> 23);
  if (e == 0) return 0;
  return e - 141 > -100 ? e - 141 : -100;
}

// The adapter of a row: -1 when it has none (or an index out of range).
__device__ __forceinline__ int adapter_of(const int *rows, int row, int M, int L) {
  if (row >= M) return -1;
  const int a = rows[row];
  return a >= 0 && a < L ? a : -1;
}

__device__ __forceinline__ int rank_of(const int *ranks, int a, int R) {
  if (ranks == nullptr) return R;
  const int r = ranks[a];
  return r < 0 ? 0 : (r < R ? r : R);
}

}  // namespace dgemm
