// lora.hip -- low-rank adapters of many requests beside a shared projection,
// and their gradients.
//
//     Y := alpha * (X W^T + s_a (X A_a^T) B_a^T) + beta * Y
//
// with a = rows[i] the adapter of row i (none: no second term).  Two steps:
//   shrink  V[i, :] = A_a x_i, R numbers a row, fp32 sums kept in fp32;
//   expand  the M x N term s_a V B_a^T, next to the shared product.
// Gradients, for dY the gradient of alpha * (...):
//     G = s_a dY B_a,  dX := alpha (dY W + G A_a) + beta_x dX,
//     dA_a := alpha sum_i G_i^T x_i + beta_ab dA_a,
//     dB_a := alpha s_a sum_i dY_i^T V_i + beta_ab dB_a.
//
// A row's adapter only ever touches that row: products with another
// adapter's weights are dropped by selection, never multiplied by zero, so an
// infinity or NaN in one adapter stays with its own rows.
#include "../../include/gemm.h"
#include "internal.hpp"
#include "rows.hpp"

namespace dgemm {

namespace {

constexpr int kShrinkWaves = 8;
constexpr int kShrinkThreads = kShrinkWaves * kWave;

// ---------------------------------------------------------------- shrink

struct ShrinkParams {
  const void *X;          // M x K
  const void *W;          // L adapters: R x K rows (KMAJ) or K x R (k down the rows)
  float *V;               // M x Rp
  const int *rows, *ranks;
  long long stride;
  int M, K, L, R, Rp, ldx, ldw;
};

// V[16 rows, 16 ranks] for the distinct adapters z, z + Z, ... among the rows:
// the workgroup's waves divide K and their sums meet in LDS.
template <typename T, bool KMAJ>
__device__ __forceinline__ void shrink_block(const ShrinkParams &p, int row0, int r0, int z, int Z,
                                             float (*red)[16][17]) {
  typedef typename El<T>::Frag Frag;
  constexpr int KS = El<T>::KSTEP;
  const int lane = threadIdx.x % kWave, wave = wave_id();
  const int li = lane % 16, lg = lane / 16;
  const int row = row0 + li;
  int id = adapter_of(p.rows, row, p.M, p.L);
  if (id >= 0 && rank_of(p.ranks, id, p.R) <= r0) id = -1;
  unsigned left = (unsigned)(__ballot(id >= 0) & 0xffffu);
  const int tr = threadIdx.x / 16, tc = threadIdx.x % 16;
  if (z == 0 && threadIdx.x < 256 && row0 + tr < p.M && !((left >> tr) & 1))
    p.V[(size_t)(row0 + tr) * p.Rp + r0 + tc] = 0.0f;
  // each wave a stretch of K, whole steps of at least 128 bytes a row long
  constexpr int G = 2 * KS;
  const int part = ((p.K + kShrinkWaves - 1) / kShrinkWaves + G - 1) / G * G;
  const int k0 = wave * part;
  const int k1 = k0 + part < p.K ? k0 + part : p.K;
  RowLoader<T, 1> x;
  x.row[0] = static_cast<const T *>(p.X) + (size_t)(row < p.M ? row : p.M - 1) * p.ldx;
  x.lim = k1;
  for (int d = 0; left != 0; ++d) {
    const int a = __builtin_amdgcn_readlane(id, __builtin_ctz(left));
    const unsigned same = (unsigned)(__ballot(id == a) & 0xffffu);
    left &= ~same;
    if (d % Z != z) continue;
    const int rk = rank_of(p.ranks, a, p.R);
    const int r = r0 + li < rk ? r0 + li : rk - 1;
    const T *w = static_cast<const T *>(p.W) + (size_t)a * (size_t)p.stride;
    f32x4 acc[1][1] = {{f32x4{0.0f, 0.0f, 0.0f, 0.0f}}};
    if constexpr (KMAJ) {
      const T *wr[1] = {w + (size_t)r * p.ldw};
      stream_mac<T, 4, 1>(wr, k0, k1, k1, k1, x, acc);
    } else {
#pragma unroll 4
      for (int k = k0; k < k1; k += KS) {
        const int kk = k + lg * El<T>::VEC;
        const Frag wf = load_frag_strided<T>(w + r, p.ldw, kk, k1);
        acc[0][0] = mma16(wf, x.masked(0, kk), acc[0][0]);
      }
    }
    // the result holds ranks down its rows, activations across its columns
#pragma unroll
    for (int j = 0; j < 4; ++j) red[wave][li][4 * lg + j] = acc[0][0][j];
    __syncthreads();
    if (threadIdx.x < 256 && ((same >> tr) & 1)) {
      float s = 0.0f;
#pragma unroll
      for (int v = 0; v < kShrinkWaves; ++v) s += red[v][tr][tc];
      p.V[(size_t)(row0 + tr) * p.Rp + r0 + tc] = r0 + tc < rk ? s : 0.0f;
    }
    __syncthreads();
  }
}

// grid: (row blocks, rank blocks, Z).
template <typename T, bool KMAJ>
__global__ __launch_bounds__(kShrinkThreads) void lora_shrink(ShrinkParams p) {
  __shared__ float red[kShrinkWaves][16][17];
  shrink_block<T, KMAJ>(p, blockIdx.x * 16, blockIdx.y * 16, blockIdx.z, gridDim.z, red);
}

// ---------------------------------------------------------------- few rows

// Rows up to which the shared product is done here (a stream over W) rather
// than by the tiled kernels.
constexpr int kSkinnyRows = 64;

struct SkinnyParams {
  ShrinkParams shrink;
  const void *W;          // N x K
  float *S;               // parts x M x N: sums over a part of K each
  int N, ldw, tiles, parts, chunk;
  int blocks, ranks16, z; // the shrink workgroups, first in the grid
};

// The shared product X W^T over parts of K and, in the same launch, the
// shrink step: neither needs the other.  A workgroup takes 16 NF / P rows of W
// against NB blocks of 16 / P rows of X (all there are), its 8 waves dividing
// its part of K.
template <typename T, int NF, int NB, int P>
__global__ __launch_bounds__(kShrinkThreads) void lora_skinny(SkinnyParams p) {
  constexpr int BR = 16 / P;
  constexpr int ROWS = BR * NF;
  __shared__ float red[kShrinkWaves][ROWS < 16 ? 16 : ROWS][17];
  int bid = blockIdx.x;
  const int shrinks = p.blocks * p.ranks16 * p.z;
  if (bid < shrinks) {
    const int z = bid % p.z, q = bid / p.z;
    shrink_block<T, true>(p.shrink, q % p.blocks * 16, q / p.blocks * 16, z, p.z,
                          reinterpret_cast<float (*)[16][17]>(red));
    return;
  }
  bid -= shrinks;
  const int M = p.shrink.M, K = p.shrink.K;
  const int n0 = bid % p.tiles * ROWS, part = bid / p.tiles;
  const int lane = threadIdx.x % kWave, wave = wave_id();
  const int li = lane % 16, lg = lane / 16;
  const T *w[NF];
#pragma unroll
  for (int f = 0; f < NF; ++f) {
    const int n = n0 + BR * f + li / P;
    w[f] = static_cast<const T *>(p.W) + (size_t)(n < p.N ? n : p.N - 1) * (size_t)p.ldw;
  }
  RowLoader<T, NB> x;
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const int i = BR * b + li / P;
    x.row[b] = static_cast<const T *>(p.shrink.X) + (size_t)(i < M ? i : M - 1) * p.shrink.ldx;
  }
  const int k0 = (part * kShrinkWaves + wave) * p.chunk;
  const int k1 = k0 + p.chunk < K ? k0 + p.chunk : K;
  x.lim = k1;
  f32x4 acc[NF][NB];
#pragma unroll
  for (int f = 0; f < NF; ++f)
#pragma unroll
    for (int b = 0; b < NB; ++b) acc[f][b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  stream_mac<T, (NF * NB >= 8 ? 2 : 4), P>(w, k0, k1, k1, k1, x, acc);
  float *out = p.S + (size_t)part * M * p.N;
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    if (b > 0) __syncthreads();
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      float v[4 / P];
      diagonal_sum<P>(acc[f][b], v);
      if (li % P == 0)
#pragma unroll
        for (int j = 0; j < 4 / P; ++j) red[wave][BR * f + 4 / P * lg + j][li / P] = v[j];
    }
    __syncthreads();
    for (int q = threadIdx.x; q < BR * ROWS; q += kShrinkThreads) {
      const int c = q / ROWS, r = q % ROWS;
      const int i = BR * b + c, n = n0 + r;
      if (i >= M || n >= p.N) continue;
      float s = 0.0f;
#pragma unroll
      for (int v = 0; v < kShrinkWaves; ++v) s += red[v][r][c];
      out[(size_t)i * p.N + n] = s;
    }
  }
}

struct JoinParams {
  const float *S, *V;
  const void *B;
  void *Y;
  const int *rows, *ranks;
  const float *scale;
  long long stride;
  int M, N, L, R, Rp, ldb, ldy, parts;
  float alpha, beta;
};

// Y := alpha * (the parts' sums + s_a B_a V) + beta * Y, one output a thread.
// grid: (ceil(N/256), M).
template <typename T>
__global__ __launch_bounds__(256) void lora_join(JoinParams p) {
  const int i = blockIdx.y, n = blockIdx.x * 256 + threadIdx.x;
  if (n >= p.N) return;
  const float *s = p.S + (size_t)i * p.N + n;
  float sum = 0.0f;
  for (int q = 0; q < p.parts; ++q) sum += s[(size_t)q * p.M * p.N];
  const int a = adapter_of(p.rows, i, p.M, p.L);
  if (a >= 0) {
    const int rk = rank_of(p.ranks, a, p.R);
    const T *u = static_cast<const T *>(p.B) + (size_t)a * (size_t)p.stride +
                 (size_t)n * (size_t)p.ldb;
    const float *v = p.V + (size_t)i * p.Rp;
    float t = 0.0f;
    constexpr int VEC = El<T>::VEC;
    int r = 0;
    for (; r + VEC <= rk; r += VEC) {
      const typename El<T>::Frag f = load_whole(u + r);
#pragma unroll
      for (int e = 0; e < VEC; ++e) t = __builtin_fmaf((float)f[e], v[r + e], t);
    }
    for (; r < rk; ++r) t = __builtin_fmaf((float)u[r], v[r], t);
    if (rk > 0) sum = __builtin_fmaf(p.scale ? p.scale[a] : 1.0f, t, sum);
  }
  T *y = static_cast<T *>(p.Y) + (size_t)i * (size_t)p.ldy + n;
  float o = p.alpha * sum;
  if (p.beta != 0.0f) o = __builtin_fmaf(p.beta, (float)*y, o);
  *y = (T)o;
}

// ---------------------------------------------------------------- expand

struct ExpandParams {
  const float *V;         // M x Rp
  const void *B;          // L adapters: N x R rows (RMAJ) or R x N
  float *C;               // M x N
  const int *rows, *ranks;
  const float *scale;
  long long stride;
  int M, N, L, R, Rp, ldb, ldc;
  float alpha, beta;
};

// C := alpha * s_a V B_a^T + beta * C, fp32 products: 16 rows x 64 columns a
// wave.  grid: (ceil(N/256), row blocks, at most 65535 and strided over).
template <typename T, bool RMAJ>
__global__ __launch_bounds__(256) void lora_expand(ExpandParams p) {
  const int lane = threadIdx.x % kWave, wave = wave_id();
  const int li = lane % 16, lg = lane / 16;
  const int n0 = blockIdx.x * 256 + wave * 64;
  if (n0 >= p.N) return;
  for (int rb = blockIdx.y; rb < (p.M + 15) / 16; rb += gridDim.y) {
  const int row0 = rb * 16;
  const int row = row0 + li;
  const int id = adapter_of(p.rows, row, p.M, p.L);
  unsigned left = (unsigned)(__ballot(id >= 0) & 0xffffu);
  const float *vrow = p.V + (size_t)(row < p.M ? row : p.M - 1) * p.Rp;
  f32x4 out[4];
#pragma unroll
  for (int b = 0; b < 4; ++b) out[b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  while (left != 0) {
    const int a = __builtin_amdgcn_readlane(id, __builtin_ctz(left));
    const unsigned same = (unsigned)(__ballot(id == a) & 0xffffu);
    left &= ~same;
    const int rk = rank_of(p.ranks, a, p.R);
    const float s = p.scale ? p.scale[a] : 1.0f;
    const T *w = static_cast<const T *>(p.B) + (size_t)a * (size_t)p.stride;
    f32x4 t[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) t[b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int r = 4 * lg; r < rk + 4 * lg; r += 16) {
      f32x4 v;
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = r + e < rk ? vrow[r + e] : 0.0f;
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        int n = n0 + 16 * b + li;
        n = n < p.N ? n : p.N - 1;
        f32x4 u;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          u[e] = r + e < rk ? (float)(RMAJ ? w[(size_t)n * p.ldb + r + e]
                                           : w[(size_t)(r + e) * p.ldb + n])
                            : 0.0f;
        t[b] = mma16(v, u, t[b]);
      }
    }
#pragma unroll
    for (int b = 0; b < 4; ++b)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if ((same >> (4 * lg + j)) & 1) out[b][j] = s * t[b][j];
  }
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    const int n = n0 + 16 * b + li;
    if (n >= p.N) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = row0 + 4 * lg + j;
      if (i >= p.M) continue;
      float *c = p.C + (size_t)i * (size_t)p.ldc + n;
      const float o = p.alpha * out[b][j];
      *c = p.beta != 0.0f ? __builtin_fmaf(p.beta, *c, o) : o;
    }
  }
  }
}

// D_a := beta * D_a, L matrices of rows x cols.
__global__ __launch_bounds__(256) void scale_batch(int rows, int cols, float beta, float *D,
                                                   int ldd, long long stride) {
  const long long total = (long long)rows * cols;
  for (long long t = (long long)blockIdx.x * 256 + threadIdx.x; t < total;
       t += (long long)gridDim.x * 256) {
    const long long i = t / cols;
    float *d = D + (size_t)blockIdx.y * (size_t)stride + (size_t)i * (size_t)ldd + (t - i * cols);
    *d = beta != 0.0f ? beta * *d : 0.0f;
  }
}

// Y := alpha * T + beta * Y, T fp32 M x N dense, Y fp16.
__global__ __launch_bounds__(256) void lora_finish(const float *T, _Float16 *Y, int M, int N,
                                                   int ldy, float alpha, float beta) {
  const long long total = (long long)M * N;
  for (long long t = (long long)blockIdx.x * 256 + threadIdx.x; t < total;
       t += (long long)gridDim.x * 256) {
    const long long i = t / N;
    _Float16 *y = Y + (size_t)i * (size_t)ldy + (t - i * N);
    float o = alpha * T[t];
    if (beta != 0.0f) o = __builtin_fmaf(beta, (float)*y, o);
    *y = (_Float16)o;
  }
}

// ---------------------------------------------------------------- rows of each adapter

// perm[start[a] .. start[a+1]) := the rows of adapter a, in order.  One
// workgroup per adapter (grid: L): it counts the rows of smaller adapters and
// its own, then writes its own.
constexpr int kGroupThreads = 1024;

__global__ __launch_bounds__(kGroupThreads) void lora_group(const int *rows, int M, int L,
                                                            int *start, int *perm) {
  __shared__ int cnt[2][kGroupThreads / kWave];
  const int a = blockIdx.x;
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  int below = 0, mine = 0;
  for (int i = threadIdx.x; i < M; i += kGroupThreads) {
    const int id = rows[i];
    below += id >= 0 && id < a;
    mine += id == a;
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    below += __shfl_xor(below, o);
    mine += __shfl_xor(mine, o);
  }
  if (lane == 0) {
    cnt[0][wave] = below;
    cnt[1][wave] = mine;
  }
  __syncthreads();
  below = mine = 0;
  for (int w = 0; w < kGroupThreads / kWave; ++w) {
    below += cnt[0][w];
    mine += cnt[1][w];
  }
  if (threadIdx.x == 0) {
    start[a] = below;
    if (a == L - 1) start[L] = below + mine;
  }
  if (mine == 0) return;
  int at = below;
  for (int i0 = 0; i0 < M; i0 += kGroupThreads) {
    const int i = i0 + threadIdx.x;
    const bool is = i < M && rows[i] == a;
    const unsigned long long m = __ballot(is);
    __syncthreads();
    if (lane == 0) cnt[0][wave] = __popcll(m);
    __syncthreads();
    int before = 0, all = 0;
    for (int w = 0; w < kGroupThreads / kWave; ++w) {
      before += w < wave ? cnt[0][w] : 0;
      all += cnt[0][w];
    }
    if (is) perm[at + before + __popcll(m & ((1ull << lane) - 1))] = i;
    at += all;
  }
}

// ---------------------------------------------------------------- dA, dB

struct OuterParams {
  const float *V;         // M x Rp (G or V)
  const void *X;          // M x K (X or dY)
  float *P;               // partial sums: S x L x Rp x K
  const int *start, *perm;
  int K, L, Rp, ldx, S;
};

// P[s, a, r, k] = sum over part s of adapter a's rows of V[i, r] X[i, k]: fp32
// products.  grid: (L * Rp/16, ceil(K/256), S); 16 ranks x 64 columns a wave.
template <typename T>
__global__ __launch_bounds__(256) void lora_outer(OuterParams p) {
  const int lane = threadIdx.x % kWave, wave = wave_id();
  const int li = lane % 16, lg = lane / 16;
  const int rblocks = p.Rp / 16;
  const int a = blockIdx.x / rblocks, r0 = blockIdx.x % rblocks * 16;
  const int k0 = blockIdx.y * 256 + wave * 64;
  if (k0 >= p.K) return;
  const int b = p.start[a], n = p.start[a + 1] - b;
  const int chunk = (n + p.S - 1) / p.S;
  const int i0 = blockIdx.z * chunk;
  const int i1 = i0 + chunk < n ? i0 + chunk : n;
  f32x4 acc[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) acc[c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  for (int i = i0; i < i1; i += 4) {
    const bool ok = i + lg < i1;
    const int row = ok ? p.perm[b + i + lg] : 0;
    const float v = ok ? p.V[(size_t)row * p.Rp + r0 + li] : 0.0f;
    const T *x = static_cast<const T *>(p.X) + (size_t)row * (size_t)p.ldx;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int k = k0 + 16 * c + li;
      const float xv = ok && k < p.K ? (float)x[k] : 0.0f;
      acc[c] = __builtin_amdgcn_mfma_f32_16x16x4f32(v, xv, acc[c], 0, 0, 0);
    }
  }
  float *out = p.P + ((size_t)blockIdx.z * p.L + a) * (size_t)p.Rp * p.K;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const int k = k0 + 16 * c + li;
    if (k >= p.K) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j) out[(size_t)(r0 + 4 * lg + j) * p.K + k] = acc[c][j];
  }
}

// D_a[r, k] (or, TR, D_a[k, r]) := alpha * s_a * sum_s P[s, a, r, k] + beta * D.
template <bool TR>
__global__ __launch_bounds__(256) void lora_outer_sum(const float *P, float *D, int ldd,
                                                      long long stride, const float *scale,
                                                      const int *ranks, int K, int L, int R,
                                                      int Rp, int S, float alpha, float beta) {
  const int a = blockIdx.y;
  const int rk = rank_of(ranks, a, R);
  const float s = alpha * (scale ? scale[a] : 1.0f);
  const long long total = (long long)R * K;
  for (long long t = (long long)blockIdx.x * 256 + threadIdx.x; t < total;
       t += (long long)gridDim.x * 256) {
    const int r = TR ? (int)(t % R) : (int)(t / K);
    const int k = TR ? (int)(t / R) : (int)(t % K);
    float sum = 0.0f;
    if (r < rk)
      for (int q = 0; q < S; ++q) sum += P[(((size_t)q * L + a) * Rp + r) * K + k];
    float *d = D + (size_t)a * (size_t)stride +
               (TR ? (size_t)k * (size_t)ldd + r : (size_t)r * (size_t)ldd + k);
    const float o = r < rk ? s * sum : 0.0f;
    *d = beta != 0.0f ? __builtin_fmaf(beta, *d, o) : o;
  }
}

// ---------------------------------------------------------------- host side

int rank_pad(int R) { return (R + 15) / 16 * 16; }

ShrinkParams shrink_params(const LoraCall &c, const void *X, int ldx, int K, const void *W,
                           int ldw, long long stride, float *V) {
  ShrinkParams p;
  p.X = X;
  p.W = W;
  p.V = V;
  p.rows = c.rows;
  p.ranks = c.ranks;
  p.stride = stride;
  p.M = c.M;
  p.K = K;
  p.L = c.L;
  p.R = c.R;
  p.Rp = rank_pad(c.R);
  p.ldx = ldx;
  p.ldw = ldw;
  return p;
}

// Workgroups per block of 16 rows: one for each adapter that may be among
// them while the blocks are few, so that a decode batch's adapters are read
// side by side; longer batches mostly have one adapter per block.
int shrink_z(const LoraCall &c) {
  const int blocks = (c.M + 15) / 16;
  if (blocks > 64) return 1;
  const int z = c.L < 16 ? c.L : 16;
  return z < c.M ? z : c.M;
}

template <typename T, bool KMAJ>
hipError_t shrink(const LoraCall &c, const void *X, int ldx, int K, const void *W, int ldw,
                  long long stride, float *V) {
  const ShrinkParams p = shrink_params(c, X, ldx, K, W, ldw, stride, V);
  hipLaunchKernelGGL((lora_shrink<T, KMAJ>),
                     dim3((unsigned)((c.M + 15) / 16), (unsigned)(p.Rp / 16),
                          (unsigned)shrink_z(c)),
                     dim3(kShrinkThreads), 0, c.stream, p);
  return hipGetLastError();
}

// The shape of a skinny product: blocks of 16 rows of W a workgroup takes, and
// the parts K is divided into so that there are two workgroups per CU, each
// wave with at least two steps.
struct SkinnyPlan {
  int P, NB, NF, tiles, parts, chunk;
};

SkinnyPlan skinny_plan(const LoraCall &c) {
  SkinnyPlan s;
  s.P = c.M <= 4 ? 4 : (c.M <= 8 ? 2 : 1);
  const int br = 16 / s.P;
  s.NB = (c.M + br - 1) / br;
  const int kstep = (c.half ? 32 : 16) * s.P;
  const int steps = (c.K + kstep - 1) / kstep;
  const int most = steps / (2 * kShrinkWaves) > 1 ? steps / (2 * kShrinkWaves) : 1;
  for (s.NF = 4;; s.NF /= 2) {
    s.tiles = (c.N + br * s.NF - 1) / (br * s.NF);
    s.parts = (2 * kCUs + s.tiles - 1) / s.tiles;
    if (s.parts > most) s.parts = most;
    if (s.NF == 1 || s.tiles * s.parts >= kCUs) break;
  }
  const int waves = s.parts * kShrinkWaves;
  s.chunk = (steps + waves - 1) / waves * kstep;
  s.parts = (c.K + kShrinkWaves * s.chunk - 1) / (kShrinkWaves * s.chunk);
  return s;
}

template <typename T, int NF, int NB, int P>
void launch_skinny(const SkinnyParams &p, hipStream_t stream) {
  const unsigned wgs = (unsigned)(p.blocks * p.ranks16 * p.z + p.tiles * p.parts);
  hipLaunchKernelGGL((lora_skinny<T, NF, NB, P>), dim3(wgs), dim3(kShrinkThreads), 0, stream, p);
}

template <typename T, int NF>
void launch_skinny(const SkinnyPlan &s, const SkinnyParams &p, hipStream_t stream) {
  if (s.P == 4) launch_skinny<T, NF, 1, 4>(p, stream);
  else if (s.P == 2) launch_skinny<T, NF, 1, 2>(p, stream);
  else if (s.NB == 1) launch_skinny<T, NF, 1, 1>(p, stream);
  else if (s.NB == 2) launch_skinny<T, NF, 2, 1>(p, stream);
  else if (s.NB == 3) launch_skinny<T, NF, 3, 1>(p, stream);
  else launch_skinny<T, NF, 4, 1>(p, stream);
}

template <typename T>
hipError_t skinny(const LoraCall &c, float *V, float *S) {
  const SkinnyPlan s = skinny_plan(c);
  SkinnyParams p;
  p.shrink = shrink_params(c, c.X, c.ldx, c.K, c.A, c.lda, c.stride_a, V);
  p.W = c.W;
  p.S = S;
  p.N = c.N;
  p.ldw = c.ldw;
  p.tiles = s.tiles;
  p.parts = s.parts;
  p.chunk = s.chunk;
  p.blocks = (c.M + 15) / 16;
  p.ranks16 = p.shrink.Rp / 16;
  p.z = shrink_z(c);
  if (s.NF == 4) launch_skinny<T, 4>(s, p, c.stream);
  else if (s.NF == 2) launch_skinny<T, 2>(s, p, c.stream);
  else launch_skinny<T, 1>(s, p, c.stream);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  JoinParams j;
  j.S = S;
  j.V = V;
  j.B = c.B;
  j.Y = c.Y;
  j.rows = c.rows;
  j.ranks = c.ranks;
  j.scale = c.scale;
  j.stride = c.stride_b;
  j.M = c.M;
  j.N = c.N;
  j.L = c.L;
  j.R = c.R;
  j.Rp = p.shrink.Rp;
  j.ldb = c.ldb;
  j.ldy = c.ldy;
  j.parts = s.parts;
  j.alpha = c.alpha;
  j.beta = c.beta;
  hipLaunchKernelGGL((lora_join<T>), dim3((unsigned)((c.N + 255) / 256), (unsigned)c.M), dim3(256),
                     0, c.stream, j);
  return hipGetLastError();
}

template <typename T, bool RMAJ>
hipError_t expand(const LoraCall &c, const float *V, const void *B, int ldb, long long stride,
                  int N, float alpha, float beta, float *C, int ldc) {
  ExpandParams p;
  p.V = V;
  p.B = B;
  p.C = C;
  p.rows = c.rows;
  p.ranks = c.ranks;
  p.scale = c.scale;
  p.stride = stride;
  p.M = c.M;
  p.N = N;
  p.L = c.L;
  p.R = c.R;
  p.Rp = rank_pad(c.R);
  p.ldb = ldb;
  p.ldc = ldc;
  p.alpha = alpha;
  p.beta = beta;
  const int rb = (c.M + 15) / 16;
  hipLaunchKernelGGL((lora_expand<T, RMAJ>),
                     dim3((unsigned)((N + 255) / 256), (unsigned)(rb < 65535 ? rb : 65535)), dim3(256),
                     0, c.stream, p);
  return hipGetLastError();
}

unsigned flat_grid(long long total) {
  long long b = (total + 255) / 256;
  return (unsigned)(b < 1 ? 1 : (b > 8192 ? 8192 : b));
}

int outer_parts(const LoraCall &c, int K) {
  const long long wgs = (long long)((K + 255) / 256) * c.L * (rank_pad(c.R) / 16);
  int s = (int)((512 + wgs - 1) / wgs);
  const int most = (c.M + 63) / 64;
  if (s > most) s = most;
  return s < 1 ? 1 : s;
}

template <typename T, bool TR>
hipError_t outer(const LoraCall &c, const float *V, const void *X, int ldx, int K,
                 const int *start, const int *perm, float *P, float *D, int ldd,
                 long long stride_d) {
  OuterParams p;
  p.V = V;
  p.X = X;
  p.P = P;
  p.start = start;
  p.perm = perm;
  p.K = K;
  p.L = c.L;
  p.Rp = rank_pad(c.R);
  p.ldx = ldx;
  p.S = outer_parts(c, K);
  hipLaunchKernelGGL((lora_outer<T>),
                     dim3((unsigned)(c.L * (p.Rp / 16)), (unsigned)((K + 255) / 256),
                          (unsigned)p.S),
                     dim3(256), 0, c.stream, p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((lora_outer_sum<TR>),
                     dim3(flat_grid((long long)c.R * K), (unsigned)c.L), dim3(256), 0, c.stream, P,
                     D, ldd, stride_d, c.scale, c.ranks, K, c.L, c.R, p.Rp, p.S, c.alpha,
                     c.beta_ab);
  return hipGetLastError();
}

struct LoraSpace {
  float *V, *T;
};

size_t carve(const LoraCall &c, void *base, LoraSpace *s) {
  Carve w(base);
  s->V = w.take<float>((size_t)c.M * rank_pad(c.R));
  if (c.M <= kSkinnyRows)
    s->T = w.take<float>((size_t)skinny_plan(c).parts * c.M * (size_t)c.N);
  else s->T = c.half ? w.take<float>((size_t)c.M * (size_t)c.N) : nullptr;
  return w.used;
}

struct GradSpace {
  float *V, *G, *T, *P;
  int *start, *perm;
};

size_t carve_grad(const LoraCall &c, void *base, GradSpace *s) {
  Carve w(base);
  const size_t rp = (size_t)rank_pad(c.R);
  s->G = w.take<float>((size_t)c.M * rp);
  s->V = w.take<float>((size_t)c.M * rp);
  s->T = c.half && c.dX ? w.take<float>((size_t)c.M * (size_t)c.K) : nullptr;
  const size_t pa = c.dA ? (size_t)outer_parts(c, c.K) * c.L * rp * (size_t)c.K : 0;
  const size_t pb = c.dB ? (size_t)outer_parts(c, c.N) * c.L * rp * (size_t)c.N : 0;
  s->P = w.take<float>(pa > pb ? pa : pb);
  s->start = w.take<int>((size_t)c.L + 1);
  s->perm = w.take<int>((size_t)c.M);
  return w.used;
}

template <typename T>
hipError_t run(const LoraCall &c, const LoraSpace &s) {
  if (c.M <= kSkinnyRows) return skinny<T>(c, s.V, s.T);
  hipError_t e = shrink<T, true>(c, c.X, c.ldx, c.K, c.A, c.lda, c.stride_a, s.V);
  if (e != hipSuccess) return e;
  if (!c.half) {
    e = expand<T, true>(c, s.V, c.B, c.ldb, c.stride_b, c.N, c.alpha, c.beta,
                        static_cast<float *>(c.Y), c.ldy);
    if (e != hipSuccess) return e;
    return (hipError_t)gemm_f32_nt(c.M, c.N, c.K, c.alpha, static_cast<const float *>(c.X), c.ldx,
                                   static_cast<const float *>(c.W), c.ldw, 1.0f,
                                   static_cast<float *>(c.Y), c.ldy, c.stream);
  }
  e = expand<T, true>(c, s.V, c.B, c.ldb, c.stride_b, c.N, 1.0f, 0.0f, s.T, c.N);
  if (e != hipSuccess) return e;
  const int rc = gemm_f16f32_nt(c.M, c.N, c.K, 1.0f, static_cast<const gemm_half_t *>(c.X), c.ldx,
                                static_cast<const gemm_half_t *>(c.W), c.ldw, 1.0f, s.T, c.N,
                                c.stream);
  if (rc != 0) return (hipError_t)rc;
  hipLaunchKernelGGL(lora_finish, dim3(flat_grid((long long)c.M * c.N)), dim3(256), 0, c.stream,
                     s.T, static_cast<_Float16 *>(c.Y), c.M, c.N, c.ldy, c.alpha, c.beta);
  return hipGetLastError();
}

template <typename T>
hipError_t run_grad(const LoraCall &c, const GradSpace &s) {
  hipError_t e;
  const bool adapters = c.L > 0 && c.R > 0;
  if (adapters && (c.dX || c.dA)) {
    e = shrink<T, false>(c, c.dY, c.lddy, c.N, c.B, c.ldb, c.stride_b, s.G);
    if (e != hipSuccess) return e;
  }
  if (c.dX) {
    float *t = c.half ? s.T : static_cast<float *>(c.dX);
    const int ldt = c.half ? c.K : c.lddx;
    const float al = c.half ? 1.0f : c.alpha, be = c.half ? 0.0f : c.beta_x;
    e = expand<T, false>(c, s.G, c.A, c.lda, c.stride_a, c.K, al, be, t, ldt);
    if (e != hipSuccess) return e;
    const int rc =
        c.half ? gemm_f16f32(c.M, c.K, c.N, 1.0f, static_cast<const gemm_half_t *>(c.dY), c.lddy,
                             static_cast<const gemm_half_t *>(c.W), c.ldw, 1.0f, t, ldt, c.stream)
               : gemm_f32(c.M, c.K, c.N, c.alpha, static_cast<const float *>(c.dY), c.lddy,
                          static_cast<const float *>(c.W), c.ldw, 1.0f, t, ldt, c.stream);
    if (rc != 0) return (hipError_t)rc;
    if (c.half) {
      hipLaunchKernelGGL(lora_finish, dim3(flat_grid((long long)c.M * c.K)), dim3(256), 0,
                         c.stream, s.T, static_cast<_Float16 *>(c.dX), c.M, c.K, c.lddx, c.alpha,
                         c.beta_x);
      e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
  }
  if (!adapters || (!c.dA && !c.dB)) return hipSuccess;
  hipLaunchKernelGGL(lora_group, dim3((unsigned)c.L), dim3(kGroupThreads), 0, c.stream, c.rows,
                     c.M, c.L, s.start, s.perm);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (c.dA) {
    e = outer<T, false>(c, s.G, c.X, c.ldx, c.K, s.start, s.perm, s.P, c.dA, c.ldda, c.stride_da);
    if (e != hipSuccess) return e;
  }
  if (c.dB) {
    e = shrink<T, true>(c, c.X, c.ldx, c.K, c.A, c.lda, c.stride_a, s.V);
    if (e != hipSuccess) return e;
    e = outer<T, true>(c, s.V, c.dY, c.lddy, c.N, s.start, s.perm, s.P, c.dB, c.lddb,
                       c.stride_db);
  }
  return e;
}

}  // namespace

size_t lora_workspace(const LoraCall &c) {
  LoraSpace s;
  return carve(c, nullptr, &s);
}

hipError_t launch_lora(const LoraCall &c, void *ws) {
  LoraSpace s;
  carve(c, ws, &s);
  return c.half ? run<_Float16>(c, s) : run<float>(c, s);
}

hipError_t launch_scale_batch_f32(int L, int rows, int cols, float beta, float *D, int ldd,
                                  long long stride, hipStream_t s) {
  hipLaunchKernelGGL(scale_batch, dim3(flat_grid((long long)rows * cols), (unsigned)L), dim3(256),
                     0, s, rows, cols, beta, D, ldd, stride);
  return hipGetLastError();
}

size_t lora_grad_workspace(const LoraCall &c) {
  GradSpace s;
  return carve_grad(c, nullptr, &s);
}

hipError_t launch_lora_grad(const LoraCall &c, void *ws) {
  GradSpace s;
  carve_grad(c, ws, &s);
  return c.half ? run_grad<_Float16>(c, s) : run_grad<float>(c, s);
}

}  // namespace dgemm
