// moe.hip -- a mixture-of-experts layer for a few tokens.
//
//     l = Wr x,  e_1..e_k = the k largest l (ties: lowest index first),
//     w = softmax over the k chosen (renorm) or over all E,
//     Y := alpha * sum_j w_j W2_e (silu(G_e x) * (U_e x)) + beta * Y,
//
// G_e, U_e the first and last F rows of W1_e.  Three or four launches:
//   logits  l in 64-bit sums (two logits may lie closer than 32-bit sums
//           tell apart, and which expert a token takes hangs on it);
//   up      a workgroup per expert and 4 to 32 rows of F finds the tokens that
//           chose its expert -- those whose rank among the logits is below k:
//           a count of the larger ones, no search -- and writes
//           silu(g) * u for each (token, choice) pair;
//   down    few tokens an expert: a workgroup per 4 or 8 outputs walks all
//           chosen experts in order, so the weighted sum over a token's experts
//           needs no atomics and no second pass;
//           more: a workgroup per expert and 16 to 64 outputs writes each
//           pair's own, and
//   combine adds up each token's choices in order.
#include "../../include/gemm.h"
#include "internal.hpp"
#include "rows.hpp"

namespace dgemm {

namespace {

// ---------------------------------------------------------------- router

// l[t, e] for one expert and 4 tokens a workgroup, whose 4 waves divide D.
// Products of halves are exact in fp32, products of floats in fp64.  The
// workgroups also clear `top` for the next launch.
template <typename T>
__global__ __launch_bounds__(256) void moe_logits(const T *X, int ldx, const T *Wr, int ldr, int M,
                                                  int D, int E, double *logits, unsigned *top,
                                                  int pairs) {
  __shared__ double part[4][4];
  if (blockIdx.x == 0 && blockIdx.y == 0)
    for (int i = threadIdx.x; i < pairs; i += 256) top[i] = 0u;
  const int lane = threadIdx.x % kWave, wave = wave_id();
  const int e = blockIdx.x, t0 = blockIdx.y * 4;
  const T *w = Wr + (size_t)e * (size_t)ldr;
  const T *x[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = X + (size_t)(t0 + i < M ? t0 + i : M - 1) * (size_t)ldx;
  double s[4] = {0.0, 0.0, 0.0, 0.0};
  constexpr int VEC = El<T>::VEC;
  auto add = [&](const typename El<T>::Frag &wf, const typename El<T>::Frag (&xf)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) s[i] += (double)wf[j] * (double)xf[i][j];
  };
  int k = threadIdx.x * VEC;
#pragma unroll 2
  for (; k - (int)threadIdx.x * VEC + 256 * VEC <= D; k += 256 * VEC) {
    const typename El<T>::Frag wf = load_whole(w + k);
    typename El<T>::Frag xf[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) xf[i] = load_whole(x[i] + k);
    add(wf, xf);
  }
  if (k < D) {
    const typename El<T>::Frag wf = load_frag(w, k, D);
    typename El<T>::Frag xf[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) xf[i] = load_frag(x[i], k, D);
    add(wf, xf);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) s[i] += __shfl_xor(s[i], o);
    if (lane == 0) part[wave][i] = s[i];
  }
  __syncthreads();
  if (threadIdx.x < 4 && t0 + (int)threadIdx.x < M) {
    const int i = threadIdx.x;
    logits[(size_t)(t0 + i) * E + e] = (part[0][i] + part[1][i]) + (part[2][i] + part[3][i]);
  }
}

// A NaN logit weighs what minus infinity does, and ranks below it.
__device__ __forceinline__ double logit_key(double l) { return l == l ? l : -__builtin_inf(); }

// Whether expert j with logit a comes before expert e with logit b.
__device__ __forceinline__ bool logit_before(double a, int j, double b, int e) {
  return a > b || (b != b && a == a) || ((a == b || (a != a && b != b)) && j < e);
}

struct MoeParams {
  const void *X, *W1, *W2;
  const double *logits;   // M x E
  float *prob;            // M x k: each choice's exp(l - max), over their sum unless renorm
  int *count, *list;      // tokens of expert e; their pairs t*k + choice: list[e*M ..]
  float *H;               // M*k x F
  unsigned *top;          // M*k: bits of the largest finite |H| of the row
  float *O;               // M*k x D (many tokens only)
  void *Y;
  int *ids;
  float *weights;
  long long stride1, stride2;
  int M, D, F, E, k, renorm;
  int ldx, ld1, ld2, ldy;
  float alpha, beta;
};

// ---------------------------------------------------------------- gate and up

constexpr int kUpWaves = 4;

// grid: (ceil(F / FS), E), 4 waves that divide D.  NF blocks of 16 / P weight
// rows: FS = 8 NF / P of the gate's and as many of the up projection's; NB
// blocks of 16 / P tokens at a time, with P stretches of k in one instruction
// (stream_mac).
template <typename T, int NF, int NB, int P>
__global__ __launch_bounds__(kUpWaves *kWave) void moe_up(MoeParams p) {
  __shared__ int rank[kMoeMaxTokens];
  __shared__ int pairs[kMoeMaxTokens];
  __shared__ int total;
  constexpr int BR = 16 / P;           // rows, and tokens, of a block
  constexpr int FS = BR * NF / 2;
  __shared__ float red[kUpWaves][BR * NF][17];
  const int lane = threadIdx.x % kWave, wave = wave_id();
  const int li = lane % 16, lg = lane / 16;
  const int f0 = blockIdx.x * FS, e = blockIdx.y;
  constexpr int TB = 4;
  // four tokens a wave at a time, so that their logits are on the way together
  for (int t0 = TB * wave; t0 < p.M; t0 += TB * kUpWaves) {
    const double *l[TB];
    double mine[TB];
    int larger[TB];
#pragma unroll
    for (int i = 0; i < TB; ++i) {
      l[i] = p.logits + (size_t)(t0 + i < p.M ? t0 + i : p.M - 1) * p.E;
      mine[i] = l[i][e];
      larger[i] = 0;
    }
    for (int j0 = 0; j0 < p.E; j0 += kWave) {
      const int j = j0 + lane;
      double v[TB];
#pragma unroll
      for (int i = 0; i < TB; ++i) v[i] = l[i][j < p.E ? j : p.E - 1];
#pragma unroll
      for (int i = 0; i < TB; ++i)
        larger[i] += __popcll(__ballot(j < p.E && logit_before(v[i], j, mine[i], e)));
    }
#pragma unroll
    for (int i = 0; i < TB; ++i)
      if (lane == 0 && t0 + i < p.M) rank[t0 + i] = larger[i] < p.k ? larger[i] : -1;
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
    for (int i = threadIdx.x; i < n; i += kUpWaves * kWave) p.list[(size_t)e * p.M + i] = pairs[i];
    for (int i = wave; i < n; i += kUpWaves) {
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
  const T *w1 = static_cast<const T *>(p.W1) + (size_t)e * (size_t)p.stride1;
  const T *w[NF];
#pragma unroll
  for (int b = 0; b < NF; ++b) {
    // row r of the workgroup's: the first half gate rows, the rest up rows
    const int r = BR * b + li / P;
    const int f = f0 + (r < FS ? r : r - FS);
    w[b] = w1 + (size_t)((r < FS ? 0 : p.F) + (f < p.F ? f : p.F - 1)) * (size_t)p.ld1;
  }
  // each wave a stretch of D, whole steps (of at least 128 bytes a row) long
  constexpr int G = 2 * El<T>::KSTEP * P;
  const int part = ((p.D + kUpWaves - 1) / kUpWaves + G - 1) / G * G;
  const int k0 = wave * part;
  const int k1 = k0 + part < p.D ? k0 + part : p.D;
  for (int i0 = 0; i0 < n; i0 += BR * NB) {
    RowLoader<T, NB> x;
    x.lim = k1;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int i = i0 + BR * b + li / P;
      x.row[b] =
          static_cast<const T *>(p.X) + (size_t)(pairs[i < n ? i : n - 1] / p.k) * (size_t)p.ldx;
    }
    f32x4 acc[NF][NB];
#pragma unroll
    for (int f = 0; f < NF; ++f)
#pragma unroll
      for (int b = 0; b < NB; ++b) acc[f][b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    stream_mac<T, (NF * NB >= 8 ? 2 : 4), P>(w, k0, k1, k1, k1, x, acc);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      if (i0 + BR * b >= n) break;
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        float v[4 / P];
        diagonal_sum<P>(acc[f][b], v);
        if (li % P == 0)
#pragma unroll
          for (int j = 0; j < 4 / P; ++j) red[wave][BR * f + 4 / P * lg + j][li / P] = v[j];
      }
      __syncthreads();
      // RG lanes share a token: a row's largest |h| takes one atomic per RG f
      constexpr int RG = FS < 8 ? FS : 8;
      for (int q = threadIdx.x; q < BR * FS; q += kUpWaves * kWave) {
        const int c = q / RG % BR, r = q % RG + q / (RG * BR) * RG;
        float g = 0.0f, u = 0.0f;
#pragma unroll
        for (int v = 0; v < kUpWaves; ++v) {
          g += red[v][r][c];
          u += red[v][FS + r][c];
        }
        const int i = i0 + BR * b + c;
        const bool ok = i < n && f0 + r < p.F;
        const float h = g / (1.0f + expf(-g)) * u;
        const int pair = pairs[i < n ? i : n - 1];
        if (ok) p.H[(size_t)pair * p.F + f0 + r] = h;
        if constexpr (sizeof(T) == 2) {
          unsigned m = __builtin_bit_cast(unsigned, fabsf(h));
          m = ok && m < 0x7f800000u ? m : 0u;
#pragma unroll
          for (int o = RG / 2; o > 0; o >>= 1) {
            const unsigned v = __shfl_xor(m, o);
            m = m > v ? m : v;
          }
          if (r % RG == 0 && m != 0u) atomicMax(&p.top[pair], m);
        }
      }
      __syncthreads();
    }
  }
}

// ---------------------------------------------------------------- down and weighted sum

// A row of H as fragments of T: for fp16, scaled by the row's power of two
// and held as two halves, 22 bits of every value within 2^-17 of the row's
// largest (to 2^-39 of that below).  The low halves' instruction stands behind the
// weights' loads: at most 1% of a call (16 tokens of 2048, 64 experts of 1024, 132
// and 133.5 us without and with it; 256 tokens of 4096, 32 experts of 2048, 535).
template <typename T, int NB>
struct HiddenLoader;

template <int NB>
struct HiddenLoader<_Float16, NB> {
  struct Raw {
    f32x4 a, b;
  };
  const float *row[NB];
  float down[NB];
  int lim;
  __device__ __forceinline__ Raw whole(int b, int k) const {
    return Raw{load_whole(row[b] + k), load_whole(row[b] + k + 4)};
  }
  __device__ __forceinline__ Raw masked(int b, int k) const {
    return Raw{load_frag(row[b], k, lim), load_frag(row[b], k + 4, lim)};
  }
  __device__ __forceinline__ Halves frag(int b, const Raw &r) const {
    typedef float f32x8 __attribute__((ext_vector_type(8)));
    const f32x8 h = f32x8{r.a[0], r.a[1], r.a[2], r.a[3], r.b[0], r.b[1], r.b[2], r.b[3]} * down[b];
    const f16x8 hi = __builtin_convertvector(h, f16x8);
    const f32x8 rest = h - __builtin_convertvector(hi, f32x8);
    // an infinity's rest is a NaN
    return Halves{hi, finite(__builtin_convertvector(rest, f16x8))};
  }
};

template <int NB>
struct HiddenLoader<float, NB> {
  typedef f32x4 Raw;
  const float *row[NB];
  float down[NB];
  int lim;
  __device__ __forceinline__ Raw whole(int b, int k) const { return load_whole(row[b] + k); }
  __device__ __forceinline__ Raw masked(int b, int k) const { return load_frag(row[b], k, lim); }
  __device__ __forceinline__ f32x4 frag(int, const Raw &r) const { return r; }
};

// grid: ceil(D/ROWS), NW waves.  The work items are (chosen expert, part of F),
// dealt to the waves in turn; a wave multiplies its rows of W2 by the expert's
// tokens and adds the weighted result to its own copy of the ROWS x M outputs
// in LDS, which are summed in wave order at the end.
//
// The experts here have few tokens, so an instruction holds 8 rows and 2
// stretches of k, or 4 and 4 (stream_mac): neighbouring lanes then read
// neighbouring pieces of a row, and there are more workgroups.
// Dynamic LDS: NW x M x ROWS floats, then M*k pair numbers.
constexpr int kDownWaves = 16;
constexpr int kNarrowTokens = 64;   // their copies of the outputs fit the LDS

template <typename T, int ROWS>
__global__ __launch_bounds__(kDownWaves *kWave) void moe_down(MoeParams p) {
  constexpr int NW = kDownWaves;
  __shared__ unsigned short act[kMoeMaxExperts];
  __shared__ unsigned short first[kMoeMaxExperts + 1];
  __shared__ int n_act;
  __shared__ float den[kNarrowTokens];
  extern __shared__ __attribute__((aligned(16))) float y[];
  unsigned short *pl = reinterpret_cast<unsigned short *>(y + (size_t)NW * p.M * ROWS);
  const int lane = threadIdx.x % kWave, wave = wave_id();
  const int li = lane % 16, lg = lane / 16;
  const int d0 = blockIdx.x * ROWS;
  if (wave == 0) {
    int n = 0, at = 0;
    for (int e0 = 0; e0 < p.E; e0 += kWave) {
      const int e = e0 + lane;
      const int c = e < p.E ? p.count[e] : 0;
      const unsigned long long m = __ballot(c > 0);
      const int pos = n + __popcll(m & ((1ull << lane) - 1));
      int upto = c;
#pragma unroll
      for (int o = 1; o < kWave; o <<= 1) {
        const int v = __shfl_up(upto, o);
        if (lane >= o) upto += v;
      }
      if (c > 0) {
        act[pos] = (unsigned short)e;
        first[pos] = (unsigned short)(at + upto - c);
      }
      n += __popcll(m);
      at += __shfl(upto, kWave - 1);
    }
    if (lane == 0) {
      n_act = n;
      first[n] = (unsigned short)at;
    }
  }
  for (int t = threadIdx.x; t < p.M; t += NW * kWave) {
    float s = 1.0f;
    if (p.renorm) {
      s = 0.0f;
      for (int j = 0; j < p.k; ++j) s += p.prob[t * p.k + j];
    }
    den[t] = s;
    if (blockIdx.x == 0 && p.weights)
      for (int j = 0; j < p.k; ++j) p.weights[t * p.k + j] = p.prob[t * p.k + j] / s;
  }
  for (int i = threadIdx.x; i < NW * p.M * (ROWS / 4); i += NW * kWave)
    reinterpret_cast<f32x4 *>(y)[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  __syncthreads();
  const int na = n_act;
  for (int i = threadIdx.x / 16; i < na; i += NW * 4) {
    const int at = first[i], n = first[i + 1] - at;
    for (int j = li; j < n; j += 16)
      pl[at + j] = (unsigned short)p.list[(size_t)act[i] * p.M + j];
  }
  __syncthreads();
  // enough items that the last round's idle waves cost little, each a whole
  // number of steps that are loaded together
  constexpr int U = 4;
  constexpr int P = 16 / ROWS;
  constexpr int G = U * P * El<T>::KSTEP;
  const int want = (8 * NW + na - 1) / na;
  const int len = p.F / want / G * G > G ? p.F / want / G * G : G;   // k per item
  const int parts = (p.F + len - 1) / len;
  const int lr = li / P;
  const int d = d0 + lr < p.D ? d0 + lr : p.D - 1;
  float *yw = y + (size_t)wave * p.M * ROWS;
  for (int i = wave; i < na * parts; i += NW) {
    const int ia = i / parts;
    const int k0 = i % parts * len;
    const int k1 = k0 + len < p.F ? k0 + len : p.F;
    const int e = act[ia], at = first[ia], n = first[ia + 1] - at;
    const T *w[1] = {static_cast<const T *>(p.W2) + (size_t)e * (size_t)p.stride2 +
                     (size_t)d * (size_t)p.ld2};
    for (int i0 = 0; i0 < n; i0 += ROWS) {
      const int pair = pl[at + (i0 + lr < n ? i0 + lr : n - 1)];
      const int t = pair / p.k;
      const float pr = p.prob[pair];
      int ex = 0;
      if constexpr (sizeof(T) == 2) ex = row_exponent(p.top[pair]);
      const HiddenLoader<T, 1> h = {{p.H + (size_t)pair * p.F}, {ldexpf(1.0f, -ex)}, k1};
      f32x4 acc[1][1] = {{f32x4{0.0f, 0.0f, 0.0f, 0.0f}}};
      stream_mac<T, U, P>(w, k0, k1, k1, k1, h, acc);
      float sum[4 / P];
      diagonal_sum<P>(acc[0][0], sum);
      if (li % P == 0 && i0 + lr < n) {
        const float wt = ldexpf(pr / den[t], ex);
        float *o = yw + t * ROWS + 4 / P * lg;
#pragma unroll
        for (int j = 0; j < 4 / P; ++j) o[j] += wt * sum[j];
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < p.M * ROWS; i += NW * kWave) {
    const int t = i / ROWS, c = d0 + i % ROWS;
    if (c >= p.D) continue;
    float s = 0.0f;
    for (int v = 0; v < NW; ++v) s += y[((size_t)v * p.M + t) * ROWS + i % ROWS];
    T *out = static_cast<T *>(p.Y) + (size_t)t * (size_t)p.ldy + c;
    float o = p.alpha * s;
    if (p.beta != 0.0f) o = __builtin_fmaf(p.beta, (float)*out, o);
    *out = (T)o;
  }
}

// ---------------------------------------------------------------- down, many tokens

constexpr int kWideWaves = 4;

// O[pair, d] = the pair's unweighted output.  grid: (ceil(D / (16 NF)), E), 4
// waves that divide F; NB blocks of 16 tokens at a time.
template <typename T, int NF, int NB>
__global__ __launch_bounds__(kWideWaves *kWave) void moe_down_wide(MoeParams p) {
  __shared__ float red[kWideWaves][16 * NF][17];
  const int e = blockIdx.y;
  const int n = p.count[e];
  if (n == 0) return;
  const int lane = threadIdx.x % kWave, wave = wave_id();
  const int li = lane % 16, lg = lane / 16;
  const int d0 = blockIdx.x * 16 * NF;
  const int *list = p.list + (size_t)e * p.M;
  const T *w[NF];
#pragma unroll
  for (int b = 0; b < NF; ++b) {
    const int d = d0 + 16 * b + li;
    w[b] = static_cast<const T *>(p.W2) + (size_t)e * (size_t)p.stride2 +
           (size_t)(d < p.D ? d : p.D - 1) * (size_t)p.ld2;
  }
  constexpr int G = 2 * El<T>::KSTEP;
  const int part = ((p.F + kWideWaves - 1) / kWideWaves + G - 1) / G * G;
  const int k0 = wave * part;
  const int k1 = k0 + part < p.F ? k0 + part : p.F;
  for (int i0 = 0; i0 < n; i0 += 16 * NB) {
    HiddenLoader<T, NB> h;
    h.lim = k1;
    int ex[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int i = i0 + 16 * b + li;
      const int pair = list[i < n ? i : n - 1];
      h.row[b] = p.H + (size_t)pair * p.F;
      ex[b] = 0;
      if constexpr (sizeof(T) == 2) ex[b] = row_exponent(p.top[pair]);
      h.down[b] = ldexpf(1.0f, -ex[b]);
    }
    f32x4 acc[NF][NB];
#pragma unroll
    for (int f = 0; f < NF; ++f)
#pragma unroll
      for (int b = 0; b < NB; ++b) acc[f][b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    stream_mac<T, (NF * NB >= 8 ? 2 : 4), 1>(w, k0, k1, k1, k1, h, acc);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      if (i0 + 16 * b >= n) break;
#pragma unroll
      for (int f = 0; f < NF; ++f)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          red[wave][16 * f + 4 * lg + j][li] = ldexpf(acc[f][b][j], ex[b]);
      __syncthreads();
      for (int q = threadIdx.x; q < 256 * NF; q += kWideWaves * kWave) {
        const int c = q / (16 * NF), r = q % (16 * NF);
        const int i = i0 + 16 * b + c;
        if (i >= n || d0 + r >= p.D) continue;
        float s = 0.0f;
#pragma unroll
        for (int v = 0; v < kWideWaves; ++v) s += red[v][r][c];
        p.O[(size_t)list[i] * p.D + d0 + r] = s;
      }
      __syncthreads();
    }
  }
}

// Y[t] := alpha * sum_j w_j O[t, j] + beta * Y[t], choices in order.  grid:
// (ceil(D/256), M).
template <typename T>
__global__ __launch_bounds__(256) void moe_combine(MoeParams p) {
  const int t = blockIdx.y, d = blockIdx.x * 256 + threadIdx.x;
  const float *prob = p.prob + t * p.k;
  float den = 1.0f;
  if (p.renorm) {
    den = 0.0f;
    for (int j = 0; j < p.k; ++j) den += prob[j];
  }
  if (blockIdx.x == 0 && p.weights && (int)threadIdx.x < p.k)
    p.weights[t * p.k + threadIdx.x] = prob[threadIdx.x] / den;
  if (d >= p.D) return;
  const float *o = p.O + (size_t)t * p.k * p.D + d;
  float s = 0.0f;
  for (int j = 0; j < p.k; ++j) s += prob[j] / den * o[(size_t)j * p.D];
  T *out = static_cast<T *>(p.Y) + (size_t)t * (size_t)p.ldy + d;
  s *= p.alpha;
  if (p.beta != 0.0f) s = __builtin_fmaf(p.beta, (float)*out, s);
  *out = (T)s;
}

// ---------------------------------------------------------------- host side

struct MoeSpace {
  double *logits;
  float *prob, *H, *O;
  unsigned *top;
  int *count, *list;
};

// One pass over the outputs (moe_down) where an expert's tokens are likely to
// fit the 8 of its blocks, else by expert with a pass that combines them.
bool narrow(const MoeCall &c) {
  return c.M <= 8 || (c.M <= kNarrowTokens && (long long)c.M * c.k <= 4LL * c.E);
}

size_t carve(const MoeCall &c, void *base, MoeSpace *s) {
  Carve w(base);
  const size_t pairs = (size_t)c.M * c.k;
  s->logits = w.take<double>((size_t)c.M * c.E);
  s->prob = w.take<float>(pairs);
  s->top = w.take<unsigned>(pairs);
  s->H = w.take<float>(pairs * (size_t)c.F);
  s->O = narrow(c) ? nullptr : w.take<float>(pairs * (size_t)c.D);
  s->count = w.take<int>((size_t)c.E);
  s->list = w.take<int>((size_t)c.E * c.M);
  return w.used;
}

// Blocks of 16 weight rows a workgroup takes: 4 where that still makes two
// workgroups per CU of the experts that some token is likely to choose, else
// 2 or 1 (an expert has `blocks` of them).
int row_blocks(const MoeCall &c, int blocks) {
  const long long active = (long long)c.M * c.k < c.E ? (long long)c.M * c.k : c.E;
  if (active * ((blocks + 3) / 4) >= 2 * kCUs) return 4;
  return active * ((blocks + 1) / 2) >= 2 * kCUs ? 2 : 1;
}

// Whether workgroups take several blocks of 16 tokens at a time, so that the
// weights are read once for them: more than 8 tokens per expert on average.
bool several_blocks(const MoeCall &c) {
  return c.M > 16 && (long long)c.M * c.k > 8LL * c.E;
}

template <typename T, int NF, int NB, int P>
void launch_up(const MoeCall &c, const MoeParams &p) {
  constexpr int FS = 8 * NF / P;
  hipLaunchKernelGGL((moe_up<T, NF, NB, P>), dim3((unsigned)((c.F + FS - 1) / FS), (unsigned)c.E),
                     dim3(kUpWaves * kWave), 0, c.stream, p);
}

template <typename T, int NF>
void launch_up(const MoeCall &c, const MoeParams &p) {
  if (several_blocks(c)) launch_up<T, NF, 4, 1>(c, p);
  else launch_up<T, NF, 1, 1>(c, p);
}

template <typename T>
void launch_up(const MoeCall &c, const MoeParams &p) {
  if (narrow(c)) {
    switch (row_blocks(c, (2 * c.F + 7) / 8)) {
      case 4: return launch_up<T, 4, 1, 2>(c, p);
      case 2: return launch_up<T, 2, 1, 2>(c, p);
      default: return launch_up<T, 1, 1, 2>(c, p);
    }
  }
  switch (row_blocks(c, (2 * c.F + 15) / 16)) {
    case 4: return launch_up<T, 4>(c, p);
    case 2: return launch_up<T, 2>(c, p);
    default: return launch_up<T, 1>(c, p);
  }
}

template <typename T, int ROWS>
void launch_narrow(const MoeCall &c, const MoeParams &p) {
  hipLaunchKernelGGL((moe_down<T, ROWS>), dim3((unsigned)((c.D + ROWS - 1) / ROWS)),
                     dim3(kDownWaves * kWave),
                     (size_t)kDownWaves * c.M * ROWS * 4 + (size_t)c.M * c.k * 2, c.stream, p);
}

template <typename T, int NF>
void launch_wide(const MoeCall &c, const MoeParams &p) {
  const dim3 g((unsigned)((c.D + 16 * NF - 1) / (16 * NF)), (unsigned)c.E), b(kWideWaves * kWave);
  if (several_blocks(c)) hipLaunchKernelGGL((moe_down_wide<T, NF, 4>), g, b, 0, c.stream, p);
  else hipLaunchKernelGGL((moe_down_wide<T, NF, 1>), g, b, 0, c.stream, p);
}

template <typename T>
hipError_t launch_down(const MoeCall &c, const MoeParams &p) {
  if (narrow(c)) {
    // 4 rows where 8 would leave CUs without a workgroup and 4 tokens are
    // likely to be all that an expert has
    if (c.D < 8 * kCUs && (c.M <= 4 || (long long)c.M * c.k <= c.E)) launch_narrow<T, 4>(c, p);
    else launch_narrow<T, 8>(c, p);
    return hipGetLastError();
  }
  switch (row_blocks(c, (c.D + 15) / 16)) {
    case 4: launch_wide<T, 4>(c, p); break;
    case 2: launch_wide<T, 2>(c, p); break;
    default: launch_wide<T, 1>(c, p); break;
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((moe_combine<T>), dim3((unsigned)((c.D + 255) / 256), (unsigned)c.M),
                     dim3(256), 0, c.stream, p);
  return hipGetLastError();
}

template <typename T>
hipError_t run(const MoeCall &c, const MoeSpace &s) {
  hipLaunchKernelGGL((moe_logits<T>), dim3((unsigned)c.E, (unsigned)((c.M + 3) / 4)), dim3(256),
                     0, c.stream, static_cast<const T *>(c.X), c.ldx,
                     static_cast<const T *>(c.Wr), c.ldr, c.M, c.D, c.E, s.logits, s.top,
                     c.M * c.k);
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
  p.top = s.top;
  p.O = s.O;
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
  p.alpha = c.alpha;
  p.beta = c.beta;
  launch_up<T>(c, p);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  return launch_down<T>(c, p);
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
