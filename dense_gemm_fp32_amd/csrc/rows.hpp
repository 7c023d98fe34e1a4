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

template <typename T>
__device__ __forceinline__ typename El<T>::Frag zero_frag() {
  typename El<T>::Frag f;
#pragma unroll
  for (int e = 0; e < El<T>::VEC; ++e) f[e] = (T)0.0f;
  return f;
}

// Elements k .. k+VEC-1 of a row of K elements (0 beyond its end).  vec: the
// row starts 16-byte aligned and k is a multiple of VEC.
template <typename T>
__device__ __forceinline__ typename El<T>::Frag load_frag(const T *row, int k, int K, bool vec) {
  typedef typename El<T>::Frag Frag;
  if (vec && k + El<T>::VEC <= K) return *reinterpret_cast<const Frag *>(row + k);
  Frag f;
#pragma unroll
  for (int e = 0; e < El<T>::VEC; ++e) f[e] = k + e < K ? row[k + e] : (T)0.0f;
  return f;
}

// The same elements where consecutive k lie ld elements apart (col: the
// address of k = 0).
template <typename T>
__device__ __forceinline__ typename El<T>::Frag load_frag_strided(const T *col, size_t ld, int k,
                                                                  int K) {
  typename El<T>::Frag f;
#pragma unroll
  for (int e = 0; e < El<T>::VEC; ++e) f[e] = k + e < K ? col[(size_t)(k + e) * ld] : (T)0.0f;
  return f;
}

// The adapter of a row: -1 when it has none (or an index out of range), or
// when that adapter's rank is at most `r0` (nothing of it from rank r0 on).
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
