// moe.hip -- a mixture-of-experts layer for a few tokens.
//
//     l = Wr x,  e_1..e_k = the k largest l (ties: lowest index first),
//     w = softmax over the k chosen (renorm) or over all E,
//     Y := alpha * sum_j w_j W2_e (silu(G_e x) * (U_e x)) + beta * Y,
//
// G_e, U_e the first and last F rows of W1_e.  Three launches:
//   logits  l in 64-bit sums (two logits may lie closer than 32-bit sums
//           tell apart, and which expert a token takes hangs on it);
//   up      a workgroup per expert and 16 rows of F finds the tokens that
//           chose its expert -- those whose rank among the logits is below k:
//           a count of the larger ones, no search -- and writes
//           silu(g) * u for each (token, choice) pair;
//   down    a workgroup per 16 outputs walks all chosen experts in order,
//           so the weighted sum over a token's experts needs no atomics and
//           no second pass.
#include "../../include/gemm.h"
#include "internal.hpp"
#include "rows.hpp"

namespace dgemm {

namespace {

// ---------------------------------------------------------------- router

// l[t, e] for 4 experts (one a wave) x 4 tokens a workgroup.  Products of
// halves are exact in fp32, products of floats in fp64.
template <typename T>
__global__ __launch_bounds__(256) void moe_logits(const T *X, int ldx, const T *Wr, int ldr, int M,
                                                  int D, int E, int vec, double *logits) {
  const int lane = threadIdx.x % kWave, wave = wave_id();
  const int e = blockIdx.x * 4 + wave, t0 = blockIdx.y * 4;
  if (e >= E) return;
  const T *w = Wr + (size_t)e * (size_t)ldr;
  const T *x[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = X + (size_t)(t0 + i < M ? t0 + i : M - 1) * (size_t)ldx;
  double s[4] = {0.0, 0.0, 0.0, 0.0};
  for (int k = lane * El<T>::VEC; k < D; k += kWave * El<T>::VEC) {
    const typename El<T>::Frag wf = load_frag<T>(w, k, D, vec);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const typename El<T>::Frag xf = load_frag<T>(x[i], k, D, vec);
#pragma unroll
      for (int j = 0; j < El<T>::VEC; ++j) s[i] += (double)wf[j] * (double)xf[j];
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) s[i] += __shfl_xor(s[i], o);
    if (lane == 0 && t0 + i < M) logits[(size_t)(t0 + i) * E + e] = s[i];
  }
}

// A NaN logit ranks below every number.
__device__ __forceinline__ double logit_key(double l) { return l == l ? l : -__builtin_inf(); }

struct MoeParams {
  const void *X, *W1, *W2;
  const double *logits;   // M x E
  float *prob;            // M x k: each choice's exp(l - max), over their sum unless renorm
  int *count, *list;      // tokens of expert e; their pairs t*k + choice: list[e*M ..]
  float *H;               // M*k x F
  void *Y;
  int *ids;
  float *weights;
  long long stride1, stride2;
  int M, D, F, E, k, renorm;
  int ldx, ld1, ld2, ldy;
  int vec_x, vec_1, vec_2;
  float alpha, beta;
};

// ---------------------------------------------------------------- gate and up

// grid: (ceil(F/16), E), 4 waves.
template <typename T>
__global__ __launch_bounds__(256) void moe_up(MoeParams p) {
  __shared__ int rank[kMoeMaxTokens];
  __shared__ int pairs[kMoeMaxTokens];
  __shared__ int total;
  __shared__ float red[2][4][16][17];
  typedef typename El<T>::Frag Frag;
  constexpr int KS = El<T>::KSTEP;
  const int lane = threadIdx.x % kWave, wave = wave_id();
  const int li = lane % 16, lg = lane / 16;
  const int f0 = blockIdx.x * 16, e = blockIdx.y;
  for (int t = wave; t < p.M; t += 4) {
    const double *l = p.logits + (size_t)t * p.E;
    const double mine = logit_key(l[e]);
    int larger = 0;
    for (int j0 = 0; j0 < p.E; j0 += kWave) {
      const int j = j0 + lane;
      const double v = j < p.E ? logit_key(l[j]) : 0.0;
      larger += __popcll(__ballot(j < p.E && (v > mine || (v == mine && j < e))));
    }
    if (lane == 0) rank[t] = larger < p.k ? larger : -1;
  }
  __syncthreads();
  if (wave == 0) {
    int n = 0;
    for (int t0 = 0; t0 < p.M; t0 += kWave) {
      const int t = t0 + lane;
      const bool in = t < p.M && rank[t] >= 0;
      const unsigned long long m = __ballot(in);
      if (in) pairs[n + __popcll(m & ((1ull << lane) - 1))] = t * p.k + rank[t];
      n += __popcll(m);
    }
    if (lane == 0) total = n;
  }
  __syncthreads();
  const int n = total;
  if (blockIdx.x == 0) {
    if (threadIdx.x == 0) p.count[e] = n;
    for (int i = threadIdx.x; i < n; i += 256) p.list[(size_t)e * p.M + i] = pairs[i];
    for (int i = wave; i < n; i += 4) {
      const int t = pairs[i] / p.k;
      const double *l = p.logits + (size_t)t * p.E;
      double top = -__builtin_inf();
      for (int j = lane; j < p.E; j += kWave) top = fmax(top, logit_key(l[j]));
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) top = fmax(top, __shfl_xor(top, o));
      float w = expf((float)(logit_key(l[e]) - top));
      if (!p.renorm) {
        float all = 0.0f;
        for (int j = lane; j < p.E; j += kWave) all += expf((float)(logit_key(l[j]) - top));
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) all += __shfl_xor(all, o);
        w /= all;
      }
      if (lane == 0) {
        p.prob[pairs[i]] = w;
        if (p.ids) p.ids[pairs[i]] = e;
      }
    }
  }
  if (n == 0) return;
  const int f = f0 + li < p.F ? f0 + li : p.F - 1;
  const T *w1 = static_cast<const T *>(p.W1) + (size_t)e * (size_t)p.stride1;
  const T *wg = w1 + (size_t)f * (size_t)p.ld1;
  const T *wu = w1 + (size_t)(p.F + f) * (size_t)p.ld1;
  for (int i0 = 0; i0 < n; i0 += 16) {
    const int t = pairs[i0 + li < n ? i0 + li : n - 1] / p.k;
    const T *x = static_cast<const T *>(p.X) + (size_t)t * (size_t)p.ldx;
    f32x4 g = f32x4{0.0f, 0.0f, 0.0f, 0.0f}, u = g;
#pragma unroll 4
    for (int k = wave * KS; k < p.D; k += 4 * KS) {
      const int kk = k + lg * El<T>::VEC;
      const Frag xf = load_frag<T>(x, kk, p.D, p.vec_x);
      g = mma16(load_frag<T>(wg, kk, p.D, p.vec_1), xf, g);
      u = mma16(load_frag<T>(wu, kk, p.D, p.vec_1), xf, u);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      red[0][wave][li][4 * lg + j] = g[j];
      red[1][wave][li][4 * lg + j] = u[j];
    }
    __syncthreads();
    const int c = threadIdx.x / 16, r = threadIdx.x % 16;
    if (i0 + c < n && f0 + r < p.F) {
      float gs = 0.0f, us = 0.0f;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        gs += red[0][w][c][r];
        us += red[1][w][c][r];
      }
      p.H[(size_t)pairs[i0 + c] * p.F + f0 + r] = gs / (1.0f + expf(-gs)) * us;
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------- down and weighted sum

// grid: ceil(D/16), 4 waves; dynamic LDS: 4 x M x 16 floats.
template <typename T>
__global__ __launch_bounds__(256) void moe_down(MoeParams p) {
  __shared__ int act[kMoeMaxExperts];
  __shared__ int n_act;
  __shared__ float den[kMoeMaxTokens];
  extern __shared__ float y[];
  const int lane = threadIdx.x % kWave, wave = wave_id();
  const int li = lane % 16, lg = lane / 16;
  const int d0 = blockIdx.x * 16;
  if (wave == 0) {
    int n = 0;
    for (int e0 = 0; e0 < p.E; e0 += kWave) {
      const int e = e0 + lane;
      const bool in = e < p.E && p.count[e] > 0;
      const unsigned long long m = __ballot(in);
      if (in) act[n + __popcll(m & ((1ull << lane) - 1))] = e;
      n += __popcll(m);
    }
    if (lane == 0) n_act = n;
  }
  for (int t = threadIdx.x; t < p.M; t += 256) {
    float s = 1.0f;
    if (p.renorm) {
      s = 0.0f;
      for (int j = 0; j < p.k; ++j) s += p.prob[t * p.k + j];
    }
    den[t] = s;
    if (blockIdx.x == 0 && p.weights)
      for (int j = 0; j < p.k; ++j) p.weights[t * p.k + j] = p.prob[t * p.k + j] / s;
  }
  for (int i = threadIdx.x; i < 4 * p.M * 16; i += 256) y[i] = 0.0f;
  __syncthreads();
  const int na = n_act;
  const int parts = na < 4 ? 4 / na : 1;             // parts of F per expert
  const int chunk = ((p.F + parts - 1) / parts + 15) / 16 * 16;
  const int d = d0 + li < p.D ? d0 + li : p.D - 1;
  float *yw = y + (size_t)wave * p.M * 16;
  for (int i = wave; i < na * parts; i += 4) {
    const int e = act[i / parts];
    const int k0 = i % parts * chunk;
    const int k1 = k0 + chunk < p.F ? k0 + chunk : p.F;
    const int n = p.count[e];
    const T *w2 = static_cast<const T *>(p.W2) + (size_t)e * (size_t)p.stride2 +
                  (size_t)d * (size_t)p.ld2;
    for (int i0 = 0; i0 < n; i0 += 16) {
      const int pair = p.list[(size_t)e * p.M + (i0 + li < n ? i0 + li : n - 1)];
      const float *h = p.H + (size_t)pair * p.F;
      f32x4 acc = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      for (int k = k0; k < k1; k += 16) {
        const int kk = k + 4 * lg;
        f32x4 wf, hf;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          wf[j] = kk + j < p.F ? (float)w2[kk + j] : 0.0f;
          hf[j] = kk + j < p.F ? h[kk + j] : 0.0f;
        }
        acc = mma16(wf, hf, acc);
      }
      if (i0 + li < n) {
        const int t = pair / p.k;
        const float w = p.prob[pair] / den[t];
#pragma unroll
        for (int j = 0; j < 4; ++j) yw[t * 16 + 4 * lg + j] += w * acc[j];
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < p.M * 16; i += 256) {
    const int t = i / 16, c = d0 + i % 16;
    if (c >= p.D) continue;
    float s = 0.0f;
    for (int w = 0; w < 4; ++w) s += y[((size_t)w * p.M + t) * 16 + i % 16];
    T *out = static_cast<T *>(p.Y) + (size_t)t * (size_t)p.ldy + c;
    float o = p.alpha * s;
    if (p.beta != 0.0f) o = __builtin_fmaf(p.beta, (float)*out, o);
    *out = (T)o;
  }
}

// ---------------------------------------------------------------- host side

struct MoeSpace {
  double *logits;
  float *prob, *H;
  int *count, *list;
};

size_t carve(const MoeCall &c, void *base, MoeSpace *s) {
  char *b = static_cast<char *>(base);
  size_t used = 0;
  auto take = [&](size_t bytes) {
    char *p = b ? b + used : nullptr;
    used += (bytes + 255) / 256 * 256;
    return p;
  };
  s->logits = reinterpret_cast<double *>(take((size_t)c.M * c.E * sizeof(double)));
  s->prob = reinterpret_cast<float *>(take((size_t)c.M * c.k * sizeof(float)));
  s->H = reinterpret_cast<float *>(take((size_t)c.M * c.k * (size_t)c.F * sizeof(float)));
  s->count = reinterpret_cast<int *>(take((size_t)c.E * sizeof(int)));
  s->list = reinterpret_cast<int *>(take((size_t)c.E * c.M * sizeof(int)));
  return used;
}

template <typename T>
bool rows16(const void *p, int ld, long long stride = 0) {
  return ld % El<T>::VEC == 0 && stride % El<T>::VEC == 0 && aligned_to(p, 16);
}

template <typename T>
hipError_t run(const MoeCall &c, const MoeSpace &s) {
  const bool vec_x = !c.force_scalar && rows16<T>(c.X, c.ldx);
  const bool vec_r = !c.force_scalar && rows16<T>(c.Wr, c.ldr);
  hipLaunchKernelGGL((moe_logits<T>), dim3((unsigned)((c.E + 3) / 4), (unsigned)((c.M + 3) / 4)),
                     dim3(256), 0, c.stream, static_cast<const T *>(c.X), c.ldx,
                     static_cast<const T *>(c.Wr), c.ldr, c.M, c.D, c.E, vec_x && vec_r, s.logits);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  MoeParams p;
  p.X = c.X;
  p.W1 = c.W1;
  p.W2 = c.W2;
  p.logits = s.logits;
  p.prob = s.prob;
  p.count = s.count;
  p.list = s.list;
  p.H = s.H;
  p.Y = c.Y;
  p.ids = c.ids;
  p.weights = c.weights;
  p.stride1 = c.stride1;
  p.stride2 = c.stride2;
  p.M = c.M;
  p.D = c.D;
  p.F = c.F;
  p.E = c.E;
  p.k = c.k;
  p.renorm = c.renorm;
  p.ldx = c.ldx;
  p.ld1 = c.ld1;
  p.ld2 = c.ld2;
  p.ldy = c.ldy;
  p.vec_x = vec_x;
  p.vec_1 = !c.force_scalar && rows16<T>(c.W1, c.ld1, c.stride1);
  p.vec_2 = !c.force_scalar && rows16<T>(c.W2, c.ld2, c.stride2);
  p.alpha = c.alpha;
  p.beta = c.beta;
  hipLaunchKernelGGL((moe_up<T>), dim3((unsigned)((c.F + 15) / 16), (unsigned)c.E), dim3(256), 0,
                     c.stream, p);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((moe_down<T>), dim3((unsigned)((c.D + 15) / 16)), dim3(256),
                     (size_t)4 * c.M * 16 * sizeof(float), c.stream, p);
  return hipGetLastError();
}

}  // namespace

size_t moe_workspace(const MoeCall &c) {
  MoeSpace s;
  return carve(c, nullptr, &s);
}

hipError_t launch_moe(const MoeCall &c, void *ws) {
  MoeSpace s;
  carve(c, ws, &s);
  return c.half ? run<_Float16>(c, s) : run<float>(c, s);
}

}  // namespace dgemm
