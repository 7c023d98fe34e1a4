// quant.hip -- rows to 8-bit integers with a scale each:
//
//     s = fl32(max_k |x_k| / 127),  q_k = the whole number nearest to x_k / s,
//
// ties to the even one, the exact quotient decides; s = 0 gives q = 0, and a
// row with an infinity or NaN gets s = NaN and q = 0, so that what is made of it
// is NaN and no other row is touched.
//
// Bound by memory: one read of X (the second pass finds it in the cache), one
// write of Q.
#include "rows.hpp"
#include "internal.hpp"

namespace dgemm {

namespace {

constexpr int kQuantThreads = 256;

// q of x for a scale s.  The quotient by way of s's reciprocal is at most one
// step off, and x - q s is exact (its bits fit 24: q has 7, and the
// difference is at most about s), so its size against s / 2 tells.  x and s come
// times a power of two that keeps s's reciprocal finite.
__device__ __forceinline__ int quantized(float x, float s, float inv) {
  float q = rintf(x * inv);
  const float e = 2.0f * __builtin_fmaf(-q, s, x);
  const bool odd = ((int)q & 1) != 0;
  if (e > s || (e == s && odd)) q += 1.0f;
  else if (-e > s || (-e == s && odd)) q -= 1.0f;
  return (int)fminf(fmaxf(q, -127.0f), 127.0f);
}

template <typename T>
__device__ __forceinline__ unsigned top_bits(const typename El<T>::Frag &f) {
  unsigned top = 0;
#pragma unroll
  for (int e = 0; e < El<T>::VEC; ++e) {
    const unsigned b = __builtin_bit_cast(unsigned, fabsf((float)f[e]));
    top = b > top ? b : top;
  }
  return top;
}

template <typename T>
__global__ __launch_bounds__(kQuantThreads) void quant_rows(const T *X, int ldx, int K, int8_t *Q,
                                                            int ldq, float *scale) {
  constexpr int VEC = El<T>::VEC;
  __shared__ unsigned part[kQuantThreads / kWave];
  const T *x = X + (size_t)blockIdx.x * (size_t)ldx;
  int8_t *q = Q + (size_t)blockIdx.x * (size_t)ldq;
  unsigned top = 0;
  for (int k = threadIdx.x * VEC; k < K; k += kQuantThreads * VEC) {
    const unsigned b = top_bits<T>(load_frag(x, k, K));
    top = b > top ? b : top;
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
  if (threadIdx.x == 0) scale[blockIdx.x] = bad ? __builtin_nanf("") : s;
  const float up = s < 0x1p-60f ? 0x1p64f : 1.0f;
  const float su = s * up;
  const bool none = bad || s == 0.0f;
  const float inv = none ? 0.0f : 1.0f / su;
  for (int k = threadIdx.x * VEC; k < K; k += kQuantThreads * VEC) {
    const typename El<T>::Frag f = load_frag(x, k, K);
#pragma unroll
    for (int e = 0; e < VEC; ++e)
      if (k + e < K) q[k + e] = none ? (int8_t)0 : (int8_t)quantized((float)f[e] * up, su, inv);
  }
}

}  // namespace

hipError_t launch_quant(bool half, int M, int K, const void *X, int ldx, int8_t *Q, int ldq,
                        float *scale, hipStream_t stream) {
  if (half)
    hipLaunchKernelGGL((quant_rows<_Float16>), dim3((unsigned)M), dim3(kQuantThreads), 0, stream,
                       static_cast<const _Float16 *>(X), ldx, K, Q, ldq, scale);
  else
    hipLaunchKernelGGL((quant_rows<float>), dim3((unsigned)M), dim3(kQuantThreads), 0, stream,
                       static_cast<const float *>(X), ldx, K, Q, ldq, scale);
  return hipGetLastError();
}

}  // namespace dgemm
