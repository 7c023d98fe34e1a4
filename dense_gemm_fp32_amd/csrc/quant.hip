// quant.hip -- rows to 8-bit integers with a scale each:
//
//     s = fl32(max_k |x_k| / 127),  q_k = the whole number nearest to x_k / s,
//
// ties to the even one, the exact quotient decides; s = 0 gives q = 0, and a
// row with an infinity or NaN gets s = NaN and q = 0, so that what is made of it
// is NaN and no other row is touched.
//
// Bound by memory: X is read once and stays in registers while its largest
// element is found (rows too long for that are read twice, the second time from
// the cache), Q is written once, in pieces of 8 bytes (4 of fp32 rows).
#include "rows.hpp"
#include "internal.hpp"

namespace dgemm {

namespace {

constexpr int kQuantThreads = 256;
constexpr int kQuantGrid = 1 << 20;     // rows to a grid's x: a dimension's threads fit 32 bits

// A row's scale s and what its elements are divided by it with.
struct Divisor {
  float up;      // a power of two that x and s are taken times of: keeps 1/s finite
  float s, inv;  // s * up and its reciprocal
  bool zero;     // every q is 0
};

// q of x, whatever x / s is.  The quotient by way of the reciprocal is at most one
// step off, and x - q s is exact (its bits fit 24: q has 7, and the difference is
// at most about s), so its size against s / 2 tells.
__device__ __forceinline__ int quantized(float x, const Divisor &d) {
  x *= d.up;
  float q = rintf(x * d.inv);
  const float e = 2.0f * __builtin_fmaf(-q, d.s, x);
  const bool odd = ((int)q & 1) != 0;
  if (e > d.s || (e == d.s && odd)) q += 1.0f;
  else if (-e > d.s || (-e == d.s && odd)) q -= 1.0f;
  return (int)fminf(fmaxf(q, -127.0f), 127.0f);
}

// A fragment's q, as bytes.  x times the reciprocal is within 127 * 2^-22 of the
// quotient: only where one of the elements lies that near to the border of two
// whole numbers (2^-14 here; 1 in 16 waves at a time) the exact way is taken.
// Adding 1.5 * 2^23 leaves the whole number in the low bits, ties to even.
template <typename T>
__device__ __forceinline__ void quantize_frag(const typename El<T>::Frag &f, const Divisor &d,
                                              uint32_t (&out)[El<T>::VEC / 4]) {
  constexpr int VEC = El<T>::VEC;
  constexpr float kWhole = 12582912.0f;
  float far = 0.0f;
  uint32_t b[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    const float t = (float)f[e] * d.inv;
    const float r = t + kWhole;
    far = fmaxf(far, fabsf(t - (r - kWhole)));
    b[e] = __builtin_bit_cast(uint32_t, r);
  }
  if (far > 0.5f - 0x1p-14f || d.up != 1.0f)
#pragma unroll
    for (int e = 0; e < VEC; ++e) b[e] = (uint32_t)quantized((float)f[e], d);
#pragma unroll
  for (int w = 0; w < VEC / 4; ++w) {
    const uint32_t lo = __builtin_amdgcn_perm(b[4 * w + 1], b[4 * w], 0x0c0c0400u);
    const uint32_t hi = __builtin_amdgcn_perm(b[4 * w + 3], b[4 * w + 2], 0x0c0c0400u);
    out[w] = d.zero ? 0u : __builtin_amdgcn_perm(hi, lo, 0x05040100u);
  }
}

// Elements k .. k+VEC-1 of a row of Q, as far as it goes.
template <typename T>
__device__ __forceinline__ void store_frag(int8_t *q, int k, int K,
                                           const uint32_t (&w)[El<T>::VEC / 4]) {
  constexpr int VEC = El<T>::VEC;
  if (k + VEC <= K) {
    if constexpr (VEC == 8) {
      typedef uint32_t Any __attribute__((ext_vector_type(2), aligned(1)));
      *reinterpret_cast<Any *>(q + k) = u32x2{w[0], w[1]};
    } else {
      typedef uint32_t Any __attribute__((aligned(1)));
      *reinterpret_cast<Any *>(q + k) = w[0];
    }
  } else {
    for (int e = 0; k + e < K; ++e) q[k + e] = (int8_t)(w[e / 4] >> (8 * (e % 4)));
  }
}

template <typename T>
__device__ __forceinline__ unsigned top_bits(unsigned top, const typename El<T>::Frag &f) {
#pragma unroll
  for (int e = 0; e < El<T>::VEC; ++e) {
    const unsigned b = __builtin_bit_cast(unsigned, fabsf((float)f[e]));
    top = b > top ? b : top;
  }
  return top;
}

// A workgroup a row.  NV: pieces of a row that a thread holds; 0: rows of any
// length, read twice.
template <typename T, int NV>
__global__ __launch_bounds__(kQuantThreads) void quant_rows(const T *X, int ldx, int M, int K,
                                                            int8_t *Q, int ldq, float *scale) {
  constexpr int STEP = kQuantThreads * El<T>::VEC;
  __shared__ unsigned part[kQuantThreads / kWave];
  const int row = (int)(blockIdx.y * kQuantGrid + blockIdx.x);
  if (row >= M) return;
  const T *x = X + (size_t)row * (size_t)ldx;
  int8_t *q = Q + (size_t)row * (size_t)ldq;
  const int k0 = threadIdx.x * El<T>::VEC;
  typename El<T>::Frag f[NV > 0 ? NV : 1];
  unsigned top = 0;
  if constexpr (NV > 0) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (k0 + i * STEP < K) f[i] = load_frag(x, k0 + i * STEP, K);
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (k0 + i * STEP < K) top = top_bits<T>(top, f[i]);
  } else {
    for (int k = k0; k < K; k += STEP) top = top_bits<T>(top, load_frag(x, k, K));
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    const unsigned b = __shfl_xor(top, o);
    top = b > top ? b : top;
  }
  if (threadIdx.x % kWave == 0) part[wave_id()] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kQuantThreads / kWave; ++w) top = part[w] > top ? part[w] : top;
  const bool bad = top >= 0x7f800000u;
  const float s = __builtin_bit_cast(float, top) / 127.0f;
  if (threadIdx.x == 0) scale[row] = bad ? __builtin_nanf("") : s;
  Divisor d;
  d.zero = bad || s == 0.0f;
  d.up = s < 0x1p-60f ? 0x1p64f : 1.0f;
  d.s = s * d.up;
  d.inv = d.zero ? 0.0f : 1.0f / d.s;
  uint32_t w[El<T>::VEC / 4];
  if constexpr (NV > 0) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (k0 + i * STEP < K) {
        quantize_frag<T>(f[i], d, w);
        store_frag<T>(q, k0 + i * STEP, K, w);
      }
  } else {
    for (int k = k0; k < K; k += STEP) {
      quantize_frag<T>(load_frag(x, k, K), d, w);
      store_frag<T>(q, k, K, w);
    }
  }
}

template <typename T, int NV>
void launch(int M, int K, const void *X, int ldx, int8_t *Q, int ldq, float *scale,
            hipStream_t stream) {
  const dim3 grid((unsigned)(M < kQuantGrid ? M : kQuantGrid),
                  (unsigned)((M + kQuantGrid - 1) / kQuantGrid));
  hipLaunchKernelGGL((quant_rows<T, NV>), grid, dim3(kQuantThreads), 0, stream,
                     static_cast<const T *>(X), ldx, M, K, Q, ldq, scale);
}

template <typename T>
hipError_t run(int M, int K, const void *X, int ldx, int8_t *Q, int ldq, float *scale,
               hipStream_t stream) {
  const int pieces = (K + kQuantThreads * El<T>::VEC - 1) / (kQuantThreads * El<T>::VEC);
  if (pieces <= 1) launch<T, 1>(M, K, X, ldx, Q, ldq, scale, stream);
  else if (pieces <= 2) launch<T, 2>(M, K, X, ldx, Q, ldq, scale, stream);
  else if (pieces <= 4) launch<T, 4>(M, K, X, ldx, Q, ldq, scale, stream);
  else if (pieces <= 8) launch<T, 8>(M, K, X, ldx, Q, ldq, scale, stream);
  else launch<T, 0>(M, K, X, ldx, Q, ldq, scale, stream);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quant(bool half, int M, int K, const void *X, int ldx, int8_t *Q, int ldq,
                        float *scale, hipStream_t stream) {
  return half ? run<_Float16>(M, K, X, ldx, Q, ldq, scale, stream)
              : run<float>(M, K, X, ldx, Q, ldq, scale, stream);
}

}  // namespace dgemm
