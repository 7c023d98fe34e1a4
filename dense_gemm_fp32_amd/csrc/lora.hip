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
  const void *W;          // L adapters of R x K
  float *V;               // M x Rp
  const int *rows, *ranks;
  long long stride;
  int M, K, L, R, Rp, ldx, ldw;
};

// V[16 rows, 16 ranks] for the distinct adapters z, z + Z, ... among the rows:
// the workgroup's waves divide K and their sums meet in LDS.
template <typename T>
__device__ __forceinline__ void shrink_block(const ShrinkParams &p, int row0, int r0, int z, int Z,
                                             float (*red)[16][17]) {
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
  // each wave a stretch of K, whole steps of 256 bytes a row long
  constexpr int G = 4 * KS;
  const int part = ((p.K + kShrinkWaves - 1) / kShrinkWaves + G - 1) / G * G;
  const int k0 = wave * part;
  const int k1 = k0 + part < p.K ? k0 + part : p.K;
  for (int d = 0; left != 0; ++d) {
    const int a = __builtin_amdgcn_readlane(id, __builtin_ctz(left));
    const unsigned same = (unsigned)(__ballot(id == a) & 0xffffu);
    left &= ~same;
    if (d % Z != z) continue;
    const int rk = rank_of(p.ranks, a, p.R);
    const T *w = static_cast<const T *>(p.W) + (size_t)a * (size_t)p.stride;
    const int n = __popc(same);
    if (n <= 4) {
      // few rows, as in a decode batch: 4 of them and 4 ranks by 4 stretches of
      // k in an instruction, so that the adapter is read in whole lines
      const int c = li / 4;
      unsigned m = same;
      for (int i = 0; i < c; ++i) m = (m & (m - 1)) ? m & (m - 1) : m;
      RowLoader<T, 1> x4;
      x4.row[0] = static_cast<const T *>(p.X) + (size_t)(row0 + __builtin_ctz(m)) * p.ldx;
      x4.lim = k1;
      const T *wr[4];
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        const int r = r0 + 4 * f + c;
        wr[f] = w + (size_t)(r < rk ? r : rk - 1) * p.ldw;
      }
      f32x4 acc[4][1];
#pragma unroll
      for (int f = 0; f < 4; ++f) acc[f][0] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      stream_mac<T, 2, 4>(wr, k0, k1, k1, k1, x4, acc);
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        float v[1];
        diagonal_sum<4>(acc[f][0], v);
        if (li % 4 == 0 && c < n) red[wave][__builtin_ctz(m)][4 * f + lg] = v[0];
      }
    } else {
      const int r = r0 + li < rk ? r0 + li : rk - 1;
      RowLoader<T, 1> x;
      x.row[0] = static_cast<const T *>(p.X) + (size_t)(row < p.M ? row : p.M - 1) * p.ldx;
      x.lim = k1;
      f32x4 acc[1][1] = {{f32x4{0.0f, 0.0f, 0.0f, 0.0f}}};
      const T *wr[1] = {w + (size_t)r * p.ldw};
      stream_mac<T, 4, 1>(wr, k0, k1, k1, k1, x, acc);
      // the result holds ranks down its rows, activations across its columns
#pragma unroll
      for (int j = 0; j < 4; ++j) red[wave][li][4 * lg + j] = acc[0][0][j];
    }
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

// ---------------------------------------------------------------- few rows

// Rows up to which the shared product is done here (a stream over W) rather
// than by the tiled kernels: all that four blocks of 16 hold.  4096 x 4096, rank
// 16, each row any of 64 adapters: 8 rows 12.7 against 26.6 us, 64 rows 20.1
// against 33.4; fp32 24.3 against 56.0 and 45.6 against 63.1.
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
__global__ __launch_bounds__(kShrinkThreads, 4) void lora_skinny(SkinnyParams p) {
  constexpr int BR = 16 / P;
  constexpr int ROWS = BR * NF;
  __shared__ float red[kShrinkWaves][ROWS < 16 ? 16 : ROWS][17];
  int bid = blockIdx.x;
  const int shrinks = p.blocks * p.ranks16 * p.z;
  if (bid < shrinks) {
    const int z = bid % p.z, q = bid / p.z;
    shrink_block<T>(p.shrink, q % p.blocks * 16, q / p.blocks * 16, z, p.z,
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
  // as many steps together as two workgroups' registers allow
  constexpr int U = NF * NB >= 12 ? 1 : (NF * NB >= 8 ? 2 : 4);
  stream_mac<T, U, P>(w, k0, k1, k1, k1, x, acc);
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
    const T *u = static_cast<const T *>(p.B) + (size_t)a * (size_t)p.stride +
                 (size_t)n * (size_t)p.ldb;
    const float *v = p.V + (size_t)i * p.Rp;
    constexpr int VEC = El<T>::VEC;
    // the first 16 ranks are on their way before the adapter's rank is known
    constexpr int AHEAD = 16 / VEC;
    typename El<T>::Frag f[AHEAD];
#pragma unroll
    for (int q = 0; q < AHEAD; ++q) f[q] = load_frag(u, q * VEC, p.R);
    const float scale = p.scale ? p.scale[a] : 1.0f;
    const int rk = rank_of(p.ranks, a, p.R);
    float t = 0.0f;
#pragma unroll
    for (int q = 0; q < AHEAD; ++q)
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        if (q * VEC + e < rk) t = __builtin_fmaf((float)f[q][e], v[q * VEC + e], t);
    for (int r = 16; r < rk; r += VEC) {
      const typename El<T>::Frag g = load_frag(u, r, p.R);
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        if (r + e < rk) t = __builtin_fmaf((float)g[e], v[r + e], t);
    }
    if (rk > 0) sum = __builtin_fmaf(scale, t, sum);
  }
  T *y = static_cast<T *>(p.Y) + (size_t)i * (size_t)p.ldy + n;
  float o = p.alpha * sum;
  if (p.beta != 0.0f) o = __builtin_fmaf(p.beta, (float)*y, o);
  *y = (T)o;
}

// ---------------------------------------------------------------- many rows: shrink

// One first product of a call: V = X A^T (kmaj) or G = dY B (B's rows run
// along the ranks).
struct ShrinkJob {
  const void *X;          // M x K
  const void *W;          // L adapters: R x K (kmaj) or K x R
  long long stride;
  int K, ldx, ldw, kmaj, chunk;
  float *S;               // parts x M x Rp: sums over a part of K each
  float *V;               // M x Rp (NULL: not wanted)
  _Float16 *split;        // M x 2 Rp: high and low parts (NULL: not wanted)
  float *scale;           // M: what a row of `split` is to be multiplied by
};

struct TileShrinkParams {
  ShrinkJob job[2];
  const int *rows, *ranks;
  const int *start, *perm, *owner;   // rows in adapter order (NULL: as they come)
  const float *ascale;
  int M, L, R, Rp, parts, z;
};

constexpr int kShrinkTile = 64;   // rows, and ranks, of a workgroup's tile

// S[part][rows, ranks] of 64 rows by 64 ranks over a part of K.  Both tiles go
// through LDS in steps of 512 bytes a row, 16-byte pieces XOR-swizzled by row:
// every piece of X is loaded once per adapter among the rows, in whole lines.
// A step's loads (up to 64 KB a workgroup, two workgroups per CU) are issued as
// soon as the registers of the last are in LDS and arrive behind its products;
// steps of 128 bytes left a quarter of that in flight (26.7 against 20.9 us at
// 4096 rows of 4096, rank 64).  Rows in adapter order (perm) have one adapter
// per tile but where two meet.  grid: (row tiles, rank tiles * parts * z,
// jobs); workgroup z takes the distinct adapters z, z + Z, ... of its rows.
constexpr int kStepBytes = 512;
constexpr int kTileThreads = 512;

// The tiles of one adapter's step in LDS, X's then W's: 64 rows of kStepBytes,
// piece c of row u at c ^ (u % 8).
template <typename T, bool KMAJ>
struct ShrinkTiles {
  typedef typename El<T>::Frag Frag;
  static constexpr int VEC = El<T>::VEC;
  static constexpr int BK = kStepBytes / (int)sizeof(T);
  static constexpr int CH = kStepBytes / 16;              // pieces of a row
  static constexpr int PER = kShrinkTile * CH / kTileThreads;   // pieces a thread loads of either tile
  static constexpr int RP = kShrinkTile / VEC;            // rank pieces of a k (not KMAJ)
  const ShrinkJob &j;
  char *lds;
  const T *w;                                             // the adapter's matrix
  int row, r0, rk, R, nb;                                 // row: of the tile, one a lane

  // This thread's number, from which each call below works out its addresses
  // anew: kept from one step to the next they would take the registers that two
  // workgroups per CU need.
  __device__ __forceinline__ static int thread() {
    int t = threadIdx.x;
    asm volatile("" : "+v"(t));
    return t;
  }
  // X: piece c of tile row u; W: piece v of rank u, or rank piece v of k u
  __device__ __forceinline__ const T *x_at(int t, int q, int k, int &u, int &c) const {
    c = t % CH;
    u = t / CH + kTileThreads / CH * q;
    return static_cast<const T *>(j.X) + (size_t)__shfl(row, u) * (size_t)j.ldx + k + c * VEC;
  }
  __device__ __forceinline__ void w_piece(int t, int q, int &u, int &v) const {
    const int i = t + kTileThreads * q;
    u = i / (KMAJ ? CH : RP);
    v = i % (KMAJ ? CH : RP);
  }
  // Whether any rank of this thread's piece q is in a block of 16 that the
  // adapter has (not KMAJ: the same for all q).
  __device__ __forceinline__ bool wanted(int q) const {
    return KMAJ ? kTileThreads / CH * q < 16 * nb : (int)threadIdx.x % RP * VEC < 16 * nb;
  }
  __device__ __forceinline__ void put_x(int u, int c, const Frag &f) const {
    *reinterpret_cast<Frag *>(lds + u * kStepBytes + 16 * (c ^ (u & 7))) = f;
  }
  __device__ __forceinline__ void put_w(int u, int v, const Frag &f) const {
    char *l = lds + kShrinkTile * kStepBytes;
    if constexpr (KMAJ) {
      *reinterpret_cast<Frag *>(l + u * kStepBytes + 16 * (v ^ (u & 7))) = f;
    } else {
      // k u of ranks v*VEC .. +VEC-1
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const int r = v * VEC + e;
        *reinterpret_cast<T *>(l + r * kStepBytes + 16 * ((u / VEC) ^ (r & 7)) +
                               u % VEC * sizeof(T)) = f[e];
      }
    }
  }

  // A step all of which lies inside the rows; ranks past the last are repeated
  // or, where they are there, taken as they are (their sums are dropped).
  __device__ __forceinline__ void load_whole_step(int k, Frag (&xr)[PER], Frag (&wr)[PER]) const {
    const int t = thread();
#pragma unroll
    for (int q = 0; q < PER; ++q) {
      int u, c;
      xr[q] = load_whole(x_at(t, q, k, u, c));
    }
#pragma unroll
    for (int q = 0; q < PER; ++q) {
      if (!wanted(q)) break;
      int u, v;
      w_piece(t, q, u, v);
      if (KMAJ) {
        const int r = r0 + u < rk ? r0 + u : rk - 1;
        wr[q] = load_whole(w + (size_t)r * (size_t)j.ldw + k + v * VEC);
      } else {
        const T *row = w + (size_t)(k + u) * (size_t)j.ldw;
        wr[q] = R < VEC ? load_part(row + v * VEC, R - v * VEC) : load_end(row, r0 + v * VEC, R);
      }
    }
  }
  // The step in which the rows end: zeros behind the end on both sides.
  __device__ __forceinline__ void load_last_step(int k, Frag (&xr)[PER], Frag (&wr)[PER]) const {
    const int t = thread();
#pragma unroll
    for (int q = 0; q < PER; ++q) {
      int u, c;
      const T *x = x_at(t, q, 0, u, c) - c * VEC;
      xr[q] = load_end(x, k + c * VEC, j.K);
    }
#pragma unroll
    for (int q = 0; q < PER; ++q) {
      if (!wanted(q)) break;
      int u, v;
      w_piece(t, q, u, v);
      if (KMAJ) {
        const int r = r0 + u < rk ? r0 + u : rk - 1;
        wr[q] = load_end(w + (size_t)r * (size_t)j.ldw, k + v * VEC, j.K);
      } else {
        const bool in = k + u < j.K;
        const int r = r0 + v * VEC, last = R - VEC;
        if (R < VEC) {
          wr[q] = load_part(w + (size_t)(in ? k + u : j.K - 1) * (size_t)j.ldw + v * VEC,
                            in ? R - v * VEC : 0);
          continue;
        }
        wr[q] = move_down(load_whole(w + (size_t)(in ? k + u : j.K - 1) * (size_t)j.ldw +
                                     (r < last ? r : last)),
                          in ? r - last : VEC);
      }
    }
  }
  // Rows shorter than a piece, which no such load fits.
  __device__ __forceinline__ bool tiny() const { return j.K < VEC; }
  __device__ __forceinline__ void load(int k, Frag (&xr)[PER], Frag (&wr)[PER]) const {
    if (tiny()) return;
    if (k + BK <= j.K) load_whole_step(k, xr, wr);
    else load_last_step(k, xr, wr);
  }
  // Their steps, piece by piece straight into LDS.
  __device__ __forceinline__ void fill(int k) const {
    const int t = thread();
#pragma unroll 1
    for (int q = 0; q < PER; ++q) {
      int u, c;
      const T *x = x_at(t, q, 0, u, c) - c * VEC;
      put_x(u, c, load_part(x + k + c * VEC, j.K - k - c * VEC));
      if (!wanted(q)) continue;
      int v;
      w_piece(t, q, u, v);
      put_w(u, v, KMAJ ? load_part(w + (size_t)(r0 + u) * (size_t)j.ldw + k + v * VEC,
                                   r0 + u < rk ? j.K - k - v * VEC : 0)
                       : load_part(w + (size_t)(k + u) * (size_t)j.ldw + r0 + v * VEC,
                                   k + u < j.K ? R - r0 - v * VEC : 0));
    }
  }
  __device__ __forceinline__ void store(const Frag (&xr)[PER], const Frag (&wr)[PER]) const {
    const int t = thread();
#pragma unroll
    for (int q = 0; q < PER; ++q) {
      put_x(t / CH + kTileThreads / CH * q, t % CH, xr[q]);
    }
#pragma unroll
    for (int q = 0; q < PER; ++q) {
      if (!wanted(q)) break;
      int u, v;
      w_piece(t, q, u, v);
      put_w(u, v, wr[q]);
    }
  }
};

template <typename T, bool KMAJ>
__device__ __forceinline__ void shrink_tile(const TileShrinkParams &p, const ShrinkJob &j,
                                            char *lds) {
  typedef ShrinkTiles<T, KMAJ> Tiles;
  typedef typename El<T>::Frag Frag;
  const int lane = threadIdx.x % kWave, wave = wave_id();
  const int li = lane % 16, lg = lane / 16;
  const int zi = blockIdx.y % p.z, part = blockIdx.y / p.z % p.parts;
  const int r0 = blockIdx.y / p.z / p.parts * kShrinkTile;
  const int k0 = part * j.chunk;
  const int k1 = k0 + j.chunk < j.K ? k0 + j.chunk : j.K;
  if (k0 >= j.K) return;
  const int count = p.perm ? p.start[p.L] : p.M;
  const int pos0 = blockIdx.x * kShrinkTile;
  if (pos0 >= count) return;
  // the row at each position of the tile, one a lane
  const int pos = pos0 + lane < count ? pos0 + lane : count - 1;
  const int row = p.perm ? p.perm[pos] : pos;
  int id = p.perm ? p.owner[pos] : adapter_of(p.rows, row, p.M, p.L);
  if (pos0 + lane >= count || (id >= 0 && rank_of(p.ranks, id, p.R) <= r0)) id = -1;
  unsigned long long left = __ballot(id >= 0);
  for (int d = 0; left != 0; ++d) {
    const int a = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
    const unsigned long long same = __ballot(id == a);
    left &= ~same;
    if (d % p.z != zi) continue;
    const int rk = rank_of(p.ranks, a, p.R);
    const int nr = rk - r0 < kShrinkTile ? rk - r0 : kShrinkTile;   // ranks of this tile
    const int nb = (nr + 15) / 16;
    const Tiles tiles = {j, lds, static_cast<const T *>(j.W) + (size_t)a * (size_t)j.stride, row,
                         r0, rk, p.R, nb};
    Frag xr[Tiles::PER], wr[Tiles::PER];
    // waves 0-3 take a block of 16 rows and ranks 0-31 each, waves 4-7 ranks 32-63
    const int wrow0 = 16 * (wave & 3), b0 = wave >> 2 << 1;
    f32x4 acc[2];
#pragma unroll
    for (int b = 0; b < 2; ++b) acc[b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    tiles.load(k0, xr, wr);
    for (int k = k0; k < k1; k += Tiles::BK) {
      if (tiles.tiny()) tiles.fill(k);
      else tiles.store(xr, wr);
      __syncthreads();
      if (k + Tiles::BK < k1) tiles.load(k + Tiles::BK, xr, wr);
#pragma unroll 2
      for (int s = 0; s < Tiles::CH / 4; ++s) {
        const int xrow = wrow0 + li;
        const Frag xf = *reinterpret_cast<const Frag *>(lds + xrow * kStepBytes +
                                                        16 * ((4 * s + lg) ^ (xrow & 7)));
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          if (b0 + b >= nb) break;
          const int wrow = kShrinkTile + 16 * (b0 + b) + li;
          const Frag wf = *reinterpret_cast<const Frag *>(lds + wrow * kStepBytes +
                                                          16 * ((4 * s + lg) ^ (wrow & 7)));
          acc[b] = mma16(xf, wf, acc[b]);
        }
      }
      __syncthreads();
    }
    // rows wrow0 + 4 lg + e of the tile, ranks r0 + 16 (b0 + b) + li
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = wrow0 + 4 * lg + e;
      const int m = __shfl(row, i);
      if (!((same >> i) & 1)) continue;
      float *out = j.S + ((size_t)part * p.M + m) * p.Rp + r0 + li;
#pragma unroll
      for (int b = 0; b < 2; ++b)
        if (b0 + b < nb) out[16 * (b0 + b)] = acc[b][e];
    }
  }
}

template <typename T>
__global__ __launch_bounds__(kTileThreads, 4) void lora_shrink_tile(TileShrinkParams p) {
  __shared__ __attribute__((aligned(16))) char lds[2 * kShrinkTile * kStepBytes];
  const ShrinkJob &j = p.job[blockIdx.z];
  if (j.kmaj) shrink_tile<T, true>(p, j, lds);
  else shrink_tile<T, false>(p, j, lds);
}

// Sums the parts of each row's V, a wave a row: as fp32, and as the pairs of
// halves that the fp16 product takes, scaled to [2^14, 2^15) by the row's power
// of two so that neither range nor the low part is lost (22 bits of every
// number within 2^-17 of the row's largest).  grid: (ceil(M/4), jobs).
__global__ __launch_bounds__(256) void lora_shrink_sum(TileShrinkParams p) {
  const ShrinkJob j = p.job[blockIdx.y];
  const int lane = threadIdx.x % kWave, row = blockIdx.x * 4 + wave_id();
  if (row >= p.M) return;
  const int a = adapter_of(p.rows, row, p.M, p.L);
  const int rk = a >= 0 ? rank_of(p.ranks, a, p.R) : 0;
  const int used = (j.K + j.chunk - 1) / j.chunk;
  float v[4];
  float top = 0.0f;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int r = lane + 64 * q;
    v[q] = 0.0f;
    if (r < rk) {
      const float *s = j.S + (size_t)row * p.Rp + r;
      for (int u = 0; u < used; ++u) v[q] += s[(size_t)u * p.M * p.Rp];
    }
    top = fmaxf(top, __builtin_isfinite(v[q]) ? fabsf(v[q]) : 0.0f);
    if (j.V && r < p.Rp) j.V[(size_t)row * p.Rp + r] = v[q];
  }
  if (!j.split) return;
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
  const int e = row_exponent(__builtin_bit_cast(unsigned, top));
  const float down = ldexpf(1.0f, -e);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int r = lane + 64 * q;
    if (r >= p.Rp) continue;
    const float f = v[q] * down;
    const _Float16 hi = (_Float16)f;
    const float rest = f - (float)hi;
    _Float16 *o = j.split + (size_t)row * (2 * p.Rp) + r / 16 * 32 + r % 16;
    o[0] = hi;
    o[16] = (_Float16)(rest == rest ? rest : 0.0f);   // an infinity has no rest
  }
  // (of an adapter without a rank nothing is to be scaled)
  if (lane == 0) j.scale[row] = ldexpf(rk > 0 && p.ascale ? p.ascale[a] : 1.0f, e);
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

// C := alpha * s_a V B_a^T + beta * C in fp32: 16 rows x 16 NB columns a wave.
// grid: (ceil(N / (64 NB)), row blocks, at most 65535 and strided over).
template <bool RMAJ, int NB>
__global__ __launch_bounds__(256) void lora_expand(ExpandParams p) {
  const int lane = threadIdx.x % kWave, wave = wave_id();
  const int li = lane % 16, lg = lane / 16;
  const int n0 = (blockIdx.x * 4 + wave) * 16 * NB;
  if (n0 >= p.N) return;
  for (int rb = blockIdx.y; rb < (p.M + 15) / 16; rb += gridDim.y) {
    const int row0 = rb * 16;
    const int row = row0 + li;
    const int id = adapter_of(p.rows, row, p.M, p.L);
    unsigned left = (unsigned)(__ballot(id >= 0) & 0xffffu);
    const float *vrow = p.V + (size_t)(row < p.M ? row : p.M - 1) * p.Rp;
    f32x4 out[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) out[b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    while (left != 0) {
      const int a = __builtin_amdgcn_readlane(id, __builtin_ctz(left));
      const unsigned same = (unsigned)(__ballot(id == a) & 0xffffu);
      left &= ~same;
      const int rk = rank_of(p.ranks, a, p.R);
      if (rk == 0) continue;
      const float s = p.scale ? p.scale[a] : 1.0f;
      const float *w = static_cast<const float *>(p.B) + (size_t)a * (size_t)p.stride;
      f32x4 t[NB];
#pragma unroll
      for (int b = 0; b < NB; ++b) t[b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      for (int r = 4 * lg; r < rk + 4 * lg; r += 16) {
        const f32x4 v = load_whole(vrow + r);     // zeros from the rank on
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          int n = n0 + 16 * b + li;
          n = n < p.N ? n : p.N - 1;
          f32x4 u;
          if constexpr (RMAJ) u = load_frag(w + (size_t)n * p.ldb, r, p.R);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            u[e] = r + e < rk ? (RMAJ ? u[e] : w[(size_t)(r + e) * p.ldb + n]) : 0.0f;
          t[b] = mma16(v, u, t[b]);
        }
      }
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if ((same >> (4 * lg + j)) & 1) out[b][j] = s * t[b][j];
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
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

// ---------------------------------------------------------------- rows of each adapter

// perm[start[a] .. start[a+1]) := the rows of adapter a, in order, and
// owner[...] := a.  One workgroup per adapter (grid: L): it counts the rows of
// smaller adapters and its own, then writes its own.
constexpr int kGroupThreads = 1024;

__global__ __launch_bounds__(kGroupThreads) void lora_group(const int *rows, int M, int L,
                                                            int *start, int *perm, int *owner) {
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
    if (is) {
      const int pos = at + before + __popcll(m & ((1ull << lane) - 1));
      perm[pos] = i;
      owner[pos] = a;
    }
    at += all;
  }
}

// ---------------------------------------------------------------- dA, dB

// One gradient of a call: D_a[r, k] (or, tr, D_a[k, r]) := alpha * s_a * sum
// over a's rows of V[i, r] X[i, k] + beta * D_a.
struct OuterJob {
  const float *V;         // M x Rp
  const void *X;          // M x K
  float *D;
  long long stride;
  int K, ldx, ldd, tr;
  float *P;               // partial sums: part_slots(M) x Rp x K (tr: K x Rp)
};

struct OuterParams {
  OuterJob job[2];
  const int *ranks, *start, *perm;
  const float *scale;
  int L, R, Rp, chunk;    // rows, in adapter order, per chunk
  float alpha, beta;
};

// Where the partial sums of an adapter's chunks start whose rows start at s0, and
// of M rows, how many there are: an adapter of n > chunk rows has ceil(n / chunk)
// <= floor(2 n / chunk) of them, one of fewer none, so that the room goes with the
// rows, whatever the number of adapters.
__host__ __device__ __forceinline__ int part_slots(int s0, int chunk) { return 2 * s0 / chunk; }

constexpr int kOuterWaves = 4;
constexpr int kOuterThreads = kOuterWaves * kWave;
constexpr int kOuterCols = 128;    // columns of X a workgroup takes
constexpr int kOuterRanks = 32;    // ranks a workgroup takes

// The sums over chunk c of adapter a's rows are workgroup s = start[a] / chunk + a
// + c's (of an adapter's n rows there are no more chunks than there are s up to the
// next adapter's first), into P[part_slots(start[a]) + c].  One workgroup each, so
// that no adapter waits for another's
// sums (1000 fp32 rows of 3000 + 517 columns, five adapters: 19 us with a chunk's
// adapters in turn, 12 us so), and an adapter of one chunk goes straight to D.
//
// A lane loads 8 consecutive columns of one row (a row's 128 columns in whole
// lines); element e of the lanes is the right operand of product e, whose 16
// columns are then 8 apart, and four rows make one step.  The products are fp32,
// as V is: with the ranks as few as they are the pass over X costs more.  The
// waves take the steps in turn and their sums meet in LDS.  grid: (column
// tiles, chunks + L, jobs * rank tiles).
template <typename T>
__global__ __launch_bounds__(kOuterThreads) void lora_outer(OuterParams p) {
  __shared__ float red[kOuterWaves][16][kOuterCols + 4];
  constexpr int NR = kOuterRanks / 16;
  constexpr int VEC = El<T>::VEC;
  const int rtiles = (p.Rp + kOuterRanks - 1) / kOuterRanks;
  const OuterJob j = p.job[blockIdx.z / rtiles];
  const int r0 = blockIdx.z % rtiles * kOuterRanks;
  const int k0 = blockIdx.x * kOuterCols;
  if (k0 >= j.K) return;
  const int lane = threadIdx.x % kWave, wave = wave_id();
  const int li = lane % 16, lg = lane / 16;
  const int kc = k0 + 8 * li;
  const bool whole = k0 + kOuterCols <= j.K;
  const int slots = (p.start[p.L] + p.chunk - 1) / p.chunk + p.L;
  for (int s = blockIdx.y; s < slots; s += gridDim.y) {
    // the last adapter whose first slot is not behind s, 64 steps at once
    int a = 0;
    for (int step = p.L > kWave * kWave ? kWave * kWave : (p.L > kWave ? kWave : 1); step > 0;
         step /= kWave) {
      const int b = a + lane * step;
      const bool upto = b < p.L && p.start[b < p.L ? b : 0] / p.chunk + b <= s;
      const unsigned long long m = __ballot(upto);
      a += (m != 0 ? 63 - __builtin_clzll(m) : 0) * step;
    }
    const int s0 = p.start[a], s1 = p.start[a + 1];
    const int at = s0 + (s - s0 / p.chunk - a) * p.chunk;
    if (at >= s1) continue;
    const int stop = s1 - at < p.chunk ? s1 : at + p.chunk;
    const int rk = rank_of(p.ranks, a, p.R);
    const int nb = rk - r0 <= 0 ? 0 : (rk - r0 > 16 ? NR : 1);
    if (nb > 0) {
      f32x4 acc[NR][8];
#pragma unroll
      for (int b = 0; b < NR; ++b)
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[b][e] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      constexpr int U = 4;               // steps loaded together
      // 16 rows' numbers a lane group, those of the next turn ahead of their use
      auto rows_at = [&](int i) { return p.perm[i + li < stop ? i + li : stop - 1]; };
      int next = rows_at(at + 4 * U * wave);
      for (int i0 = at + 4 * U * wave; i0 < stop; i0 += 4 * U * kOuterWaves) {
        const int here = next;
        next = rows_at(i0 + 4 * U * kOuterWaves);
        float v[U][NR];
        float x[U][8];
        typename El<T>::Frag xf[U][8 / VEC];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const bool ok = i0 + 4 * u + lg < stop;
          const int row = __shfl(here, 4 * u + lg);
          const float *vr = j.V + (size_t)row * p.Rp + r0 + li;
#pragma unroll
          for (int b = 0; b < NR; ++b) {
            const float f = vr[b < nb ? 16 * b : 0];
            v[u][b] = ok ? f : 0.0f;
          }
          const T *xr = static_cast<const T *>(j.X) + (size_t)row * (size_t)j.ldx + kc;
#pragma unroll
          for (int h = 0; h < 8 / VEC; ++h)
            xf[u][h] = whole ? load_whole(xr + h * VEC) : load_part(xr + h * VEC, j.K - kc - h * VEC);
        }
        __builtin_amdgcn_sched_barrier(0);
        // rows behind the last enter as zeros on both sides
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int h = 0; h < 8 / VEC; ++h)
#pragma unroll
            for (int e = 0; e < VEC; ++e)
              x[u][h * VEC + e] = i0 + 4 * u + lg < stop ? (float)xf[u][h][e] : 0.0f;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int b = 0; b < NR; ++b)
            if (b < nb)
#pragma unroll
              for (int e = 0; e < 8; ++e)
                acc[b][e] =
                    __builtin_amdgcn_mfma_f32_16x16x4f32(v[u][b], x[u][e], acc[b][e], 0, 0, 0);
      }
      const bool all = at == s0 && stop == s1;
      float *out =
          j.P + (size_t)(part_slots(s0, p.chunk) + (at - s0) / p.chunk) * p.Rp * j.K;
#pragma unroll
      for (int b = 0; b < NR; ++b) {
        if (b >= nb) break;
        __syncthreads();
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int e = 0; e < 8; e += 4)
            *reinterpret_cast<f32x4 *>(&red[wave][4 * lg + q][8 * li + e]) =
                f32x4{acc[b][e][q], acc[b][e + 1][q], acc[b][e + 2][q], acc[b][e + 3][q]};
        __syncthreads();
        for (int q = threadIdx.x; q < 16 * kOuterCols; q += kOuterThreads) {
          const int r = j.tr ? q % 16 : q / kOuterCols, k = j.tr ? q / 16 : q % kOuterCols;
          if (k0 + k >= j.K) continue;
          float s = 0.0f;
#pragma unroll
          for (int w = 0; w < kOuterWaves; ++w) s += red[w][r][k];
          const int rr = r0 + 16 * b + r;
          if (!all) {
            out[j.tr ? (size_t)(k0 + k) * p.Rp + rr : (size_t)rr * j.K + k0 + k] = s;
          } else if (rr < rk) {
            float *d = j.D + (size_t)a * (size_t)j.stride +
                       (j.tr ? (size_t)(k0 + k) * (size_t)j.ldd + rr
                             : (size_t)rr * (size_t)j.ldd + k0 + k);
            const float o = p.alpha * (p.scale ? p.scale[a] : 1.0f) * s;
            *d = p.beta != 0.0f ? __builtin_fmaf(p.beta, *d, o) : o;
          }
        }
      }
    }
  }
}

// D_a from its partial sums, four adjacent elements a thread; what lora_outer
// wrote itself is left, but for the ranks beyond the adapter's.  grid: (blocks,
// L, jobs).
__global__ __launch_bounds__(256) void lora_outer_sum(OuterParams p) {
  const OuterJob j = p.job[blockIdx.z];
  const int a = blockIdx.y;
  const int rk = rank_of(p.ranks, a, p.R);
  const int b = p.start[a], n = p.start[a + 1] - b;
  const int chunks = (n + p.chunk - 1) / p.chunk;
  const bool done = chunks == 1;
  if (done && rk == p.R) return;
  const float s = p.alpha * (p.scale ? p.scale[a] : 1.0f);
  const size_t slot = (size_t)p.Rp * j.K;
  // rows of `len`: ranks of one k (tr), or k of one rank
  const int len = j.tr ? p.R : j.K, pitch = j.tr ? p.Rp : j.K;
  const long long quads = (len + 3) / 4;
  const long long total = quads * (j.tr ? j.K : p.R);
  for (long long t = (long long)blockIdx.x * 256 + threadIdx.x; t < total;
       t += (long long)gridDim.x * 256) {
    const int i = (int)(t / quads), e0 = 4 * (int)(t % quads);
    const int count = len - e0 < 4 ? len - e0 : 4;
    // of these, the ones within the rank
    const int in = n == 0 ? 0 : j.tr ? (rk - e0 < count ? rk - e0 : count) : (i < rk ? count : 0);
    if (done && in == count) continue;
    f32x4 sum = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    if (in > 0 && !done) {
      const float *q = j.P + (size_t)part_slots(b, p.chunk) * slot + (size_t)i * pitch + e0;
      for (int c = 0; c < chunks; ++c, q += slot)
        sum += count == 4 ? load_whole(q) : load_part(q, count);
    }
    float *d = j.D + (size_t)a * (size_t)j.stride + (size_t)i * (size_t)j.ldd + e0;
    const bool all = count == 4 && !(done && in > 0);
    f32x4 old = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    if (p.beta != 0.0f) old = all ? load_whole(d) : load_part(d, count);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float o = e < in ? s * sum[e] : 0.0f;
      old[e] = p.beta != 0.0f ? __builtin_fmaf(p.beta, old[e], o) : o;
    }
    if (all) {
      typedef float Any __attribute__((ext_vector_type(4), aligned(4)));
      *reinterpret_cast<Any *>(d) = old;
    } else {
      for (int e = done ? (in > 0 ? in : 0) : 0; e < count; ++e) d[e] = old[e];
    }
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

// First products of a call with many rows (`jobs`: one or two): the parts K is
// divided into and the workgroups per tile of 64 rows that share its adapters
// out (in a batch of some hundred rows every row may have its own), both so
// that all workgroups are on the CUs at once, two to each: a workgroup first
// follows its rows' numbers to their adapters, some microseconds that a second
// round would add again (4096 rows of 4096, rank 16, both products: 28 us in
// two rounds, 22 us in one).
struct TilePlan {
  int tiles, rtiles, parts, z;
};

int tile_step(const LoraCall &c) { return kStepBytes / (c.half ? 2 : 4); }

TilePlan tile_plan(const LoraCall &c, int jobs) {
  TilePlan t;
  t.tiles = (c.M + kShrinkTile - 1) / kShrinkTile;
  t.rtiles = (rank_pad(c.R) + kShrinkTile - 1) / kShrinkTile;
  const long long wgs = (long long)t.tiles * t.rtiles * jobs;
  const int longest = c.K > c.N ? c.K : c.N;
  const int most = (longest + tile_step(c) - 1) / tile_step(c);
  int parts = (int)(2 * kCUs / wgs);
  parts = parts < 8 ? parts : 8;
  parts = parts < most ? parts : most;
  t.parts = parts > 1 ? parts : 1;
  // two at least: where two requests meet in a tile the second adapter's
  // workgroup runs beside the first's, elsewhere it ends at once
  int z = (int)(2 * kCUs / (wgs * t.parts));
  z = z > 2 ? z : 2;
  z = z < c.L ? z : c.L;
  z = z < kShrinkTile ? z : kShrinkTile;
  t.z = z > 1 ? z : 1;
  return t;
}

int tile_chunk(const LoraCall &c, const TilePlan &t, int K) {
  const int step = tile_step(c);
  return ((K + t.parts - 1) / t.parts + step - 1) / step * step;
}

template <typename T>
hipError_t shrink_tiles(const LoraCall &c, const TileShrinkParams &p, const TilePlan &t,
                        int jobs) {
  hipLaunchKernelGGL((lora_shrink_tile<T>),
                     dim3((unsigned)t.tiles, (unsigned)(t.rtiles * t.parts * t.z),
                          (unsigned)jobs),
                     dim3(kTileThreads), 0, c.stream, p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(lora_shrink_sum, dim3((unsigned)((c.M + 3) / 4), (unsigned)jobs), dim3(256), 0,
                     c.stream, p);
  return hipGetLastError();
}

TileShrinkParams tile_params(const LoraCall &c, const TilePlan &t) {
  TileShrinkParams p = {};
  p.rows = c.rows;
  p.ranks = c.ranks;
  p.ascale = c.scale;
  p.M = c.M;
  p.L = c.L;
  p.R = c.R;
  p.Rp = rank_pad(c.R);
  p.parts = t.parts;
  p.z = t.z;
  return p;
}

// The shape of a skinny product: blocks of 16 rows of W a workgroup takes, and
// the parts K is divided into so that there is one workgroup per CU (the adapters
// beside them then fit in too, two to a CU: 8 parts 18.5 us, 4 parts 14.8 us at 48
// x 4096 x 4096), each wave with at least two steps.
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
  // (four blocks of each would spill at two workgroups per CU)
  for (s.NF = s.NB > 3 ? 2 : 4;; s.NF /= 2) {
    s.tiles = (c.N + br * s.NF - 1) / (br * s.NF);
    s.parts = kCUs / s.tiles > 1 ? kCUs / s.tiles : 1;
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
  else if constexpr (NF < 4) launch_skinny<T, NF, 4, 1>(p, stream);
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
  return hipGetLastError();
}

// 64 columns a wave read V least often, 16 make the most waves: 4096 x 4096, rank
// 64, 59 against 73 us; 1000 x 3000, rank 12, 9.2 against 6.9 us.
template <bool RMAJ>
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
  const unsigned y = (unsigned)(rb < 65535 ? rb : 65535);
  if ((long long)((N + 255) / 256) * rb >= 8 * kCUs)
    hipLaunchKernelGGL((lora_expand<RMAJ, 4>), dim3((unsigned)((N + 255) / 256), y), dim3(256), 0,
                       c.stream, p);
  else
    hipLaunchKernelGGL((lora_expand<RMAJ, 1>), dim3((unsigned)((N + 63) / 64), y), dim3(256), 0,
                       c.stream, p);
  return hipGetLastError();
}

unsigned flat_grid(long long total) {
  long long b = (total + 255) / 256;
  return (unsigned)(b < 1 ? 1 : (b > 8192 ? 8192 : b));
}

// Rows per chunk of the gradients' sums: as many chunks as give every CU two of
// the four workgroups it holds, but at least 64 rows each, since each leaves
// partial sums of the adapter's own size behind (2049 fp16 rows of 4096 + 2048
// columns: 45, 36 and 39 us with one, two and four).
int outer_chunk(const LoraCall &c) {
  const int cols = ((c.K + kOuterCols - 1) / kOuterCols + (c.N + kOuterCols - 1) / kOuterCols) *
                   ((rank_pad(c.R) + kOuterRanks - 1) / kOuterRanks);
  const int want = 2 * kCUs / cols > 1 ? 2 * kCUs / cols : 1;
  const int rows = (c.M + want - 1) / want;
  return rows > 64 ? rows : 64;
}

// Rows up to which the fp16 product goes to fp32 and the adapters' term is
// added in a pass of its own: batches in which every row may have another
// adapter, which the pass does not mind and the product's steps and epilogue do.
// 4096 x 4096, rank 16, 64 adapters by the pass and by the product: any to each
// row, 128 rows 43 and 65 us, 512 rows 80 and 132, 1024 rows 124 and 209; in four
// runs of rows 35 and 34, 54 and 47, 77 and 64.  Below the limit the pass loses
// little where it loses, above it batches are taken to be prompts.
constexpr int kJoinRows = 512;

// Parts of K of an fp16 product, where its smallest tiles leave CUs without one
// (in a deep K, without two): 257 x 1024 x 1024 on a term of three adapters, who
// are shared out, 24 us in one part, 15 us in four.
int product_parts(const LoraCall &c, int N, int K) {
  const long long tiles = (long long)((c.M + 63) / 64) * (((long long)N + 127) / 128);
  const int want = (int)((K >= 2048 ? 2 * kCUs : kCUs) / tiles);
  const int most = K / 256 < 8 ? K / 256 : 8;
  return want < 2 || most < 2 ? 1 : (want < most ? want : most);
}

// The shared product of a call, op(B) K x N: fp32 on top of C, fp16 on top of a
// term (`term`, whose kernel the launch takes) or, `join`, alone into fp32.
//
// Operands whose rows do not allow 16-byte loads are copied first, whatever the
// size (fp16 89 x 1216 x 1449 with odd rows, small tiles: 77 us without, 18 us
// with the copies; on a term 1643 x 3584 x 3886: 153 and 82 us, since the large
// tile has direct loads only there).  So is an fp16 B whose columns end inside a
// vector, which they do not in the copy (gradients of 1261 x 871 x 1314: 199 and
// 96 us).  Few tiles of fp32 (the gradients of 224 x 1957 x 1408: 151 us by the product's
// own choice, 79 us so) and a deep fp32 K (a gradient's, over a projection's many
// outputs; 1000 x 517 x 3000 with odd rows: 88 and 63 us) are split over four 64 x
// 64 tiles per CU.
Call product(const LoraCall &c, bool join, bool tb, int N, int K, const void *A, int lda,
             const void *B, int ldb, float beta, void *C, int ldc) {
  Call g = {};
  g.M = c.M;
  g.N = N;
  g.K = K;
  g.alpha = join ? 1.0f : c.alpha;
  g.beta = join ? 0.0f : (c.half ? beta : 1.0f);
  g.A = A;
  g.lda = lda;
  g.B = B;
  g.ldb = ldb;
  g.C = C;
  g.ldc = ldc;
  g.tb = tb;
  g.out32 = join;
  g.splits = 1;
  g.pack_mode = 2;
  g.copy_ragged_b = c.half;
  g.stream = c.stream;
  if (c.half) {
    const int parts = product_parts(c, N, K);
    if (parts > 1) g.split_mode = parts;
    return g;
  }
  const long long tiles = (long long)((c.M + 63) / 64) * ((N + 63) / 64);
  const int parts = (int)((4 * kCUs + tiles - 1) / tiles);
  if ((K >= 2 * (c.M > N ? c.M : N) || tiles < kCUs) && parts >= 2 && K / 256 >= 2) {
    g.tile_config = 7;
    g.split_mode = parts < K / 256 ? parts : K / 256;
    if (g.split_mode > 64) g.split_mode = 64;
  }
  return g;
}

// Workspace of a product (split K, copies): a part of the call's own, so that a
// captured call allocates nothing.  It is planned for operands all of whose rows
// allow the widest loads, or none of whose do, the larger of the two before they
// are known (A NULL); what a call's own plan takes beyond it it does without.
size_t product_bytes(const LoraCall &c, bool join, bool tb, int N, int K, const void *A, int lda,
                     const void *B, int ldb) {
  const int vec = c.half ? 8 : 4;
  const bool wide = lda % vec == 0 && ldb % vec == 0 && aligned_to(A, 16) && aligned_to(B, 16) &&
                    (!c.half || tb || N % vec == 0);
  void *p = reinterpret_cast<void *>((uintptr_t)256);
  size_t most = 256;
  for (int odd = 0; odd < 2; ++odd) {
    if (A != nullptr && wide == (odd != 0)) continue;
    auto ld = [&](int cols) { return odd ? cols | 1 : (cols + 7) / 8 * 8; };
    Call g = product(c, join, tb, N, K, p, ld(K), p, ld(tb ? K : N), 0.0f, p, ld(N));
    g.ws_fixed_bytes = (size_t)1 << 30;
    const size_t n = (c.half ? plan_f16(g) : plan_f32(g)).ws_bytes;
    most = n > most ? n : most;
  }
  return most;
}

struct LoraSpace {
  float *V, *S, *T, *scale;
  _Float16 *split;
  char *W;
  size_t w_bytes;
};

size_t carve(const LoraCall &c, void *base, LoraSpace *s) {
  Carve w(base);
  *s = LoraSpace{};
  const size_t rp = (size_t)rank_pad(c.R);
  if (c.M <= kSkinnyRows) {
    s->V = w.take<float>((size_t)c.M * rp);
    s->S = w.take<float>((size_t)skinny_plan(c).parts * c.M * (size_t)c.N);
    return w.used;
  }
  s->S = w.take<float>((size_t)tile_plan(c, 1).parts * c.M * rp);
  if (!c.half || c.M <= kJoinRows) {
    s->V = w.take<float>((size_t)c.M * rp);
    if (c.half) s->T = w.take<float>((size_t)c.M * (size_t)c.N);
  } else {
    s->split = w.take<_Float16>((size_t)c.M * 2 * rp);
    s->scale = w.take<float>((size_t)c.M + 256);   // read in whole tiles of rows
  }
  s->w_bytes = product_bytes(c, c.half && c.M <= kJoinRows, true, c.N, c.K, c.X, c.ldx, c.W, c.ldw);
  s->W = w.take<char>(s->w_bytes);
  return w.used;
}

struct GradSpace {
  float *V, *G, *SV, *SG, *PA, *PB, *scale;
  _Float16 *split;
  char *W;
  size_t w_bytes;
  int *start, *perm, *owner;
};

size_t carve_grad(const LoraCall &c, void *base, GradSpace *s) {
  Carve w(base);
  *s = GradSpace{};
  const size_t rp = (size_t)rank_pad(c.R);
  const size_t parts = (size_t)tile_plan(c, 2).parts;
  s->start = w.take<int>((size_t)c.L + 1);
  s->perm = w.take<int>((size_t)c.M);
  s->owner = w.take<int>((size_t)c.M);
  if (c.dX || c.dA) {
    s->G = w.take<float>((size_t)c.M * rp);
    s->SG = w.take<float>(parts * c.M * rp);
  }
  if (c.dX && c.half) {
    s->split = w.take<_Float16>((size_t)c.M * 2 * rp);
    s->scale = w.take<float>((size_t)c.M + 256);
  }
  if (c.dX) {
    s->w_bytes = product_bytes(c, false, false, c.K, c.N, c.dY, c.lddy, c.W, c.ldw);
    s->W = w.take<char>(s->w_bytes);
  }
  if (c.dB) {
    s->V = w.take<float>((size_t)c.M * rp);
    s->SV = w.take<float>(parts * c.M * rp);
  }
  const size_t slots = (size_t)part_slots(c.M, outer_chunk(c));
  if (c.dA) s->PA = w.take<float>(slots * rp * (size_t)c.K);
  if (c.dB) s->PB = w.take<float>(slots * rp * (size_t)c.N);
  return w.used;
}

hipError_t join(const LoraCall &c, const float *V, const float *S, int parts) {
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
  j.Rp = rank_pad(c.R);
  j.ldb = c.ldb;
  j.ldy = c.ldy;
  j.parts = parts;
  j.alpha = c.alpha;
  j.beta = c.beta;
  const dim3 g((unsigned)((c.N + 255) / 256), (unsigned)c.M);
  if (c.half) hipLaunchKernelGGL((lora_join<_Float16>), g, dim3(256), 0, c.stream, j);
  else hipLaunchKernelGGL((lora_join<float>), g, dim3(256), 0, c.stream, j);
  return hipGetLastError();
}

template <typename T>
hipError_t run(const LoraCall &c, const LoraSpace &s) {
  if (c.M <= kSkinnyRows) {
    const hipError_t e = skinny<T>(c, s.V, s.S);
    return e != hipSuccess ? e : join(c, s.V, s.S, skinny_plan(c).parts);
  }
  const TilePlan t = tile_plan(c, 1);
  TileShrinkParams p = tile_params(c, t);
  p.job[0] = ShrinkJob{c.X, c.A, c.stride_a, c.K, c.ldx, c.lda, 1, tile_chunk(c, t, c.K), s.S,
                       s.V, s.split, s.scale};
  hipError_t e = shrink_tiles<T>(c, p, t, 1);
  if (e != hipSuccess) return e;
  const bool joined = c.half && c.M <= kJoinRows;
  Call g = product(c, joined, true, c.N, c.K, c.X, c.ldx, c.W, c.ldw, c.beta,
                   joined ? s.T : c.Y, joined ? c.N : c.ldy);
  g.ws_fixed = s.W;
  g.ws_fixed_bytes = s.w_bytes;
  if (!c.half) {
    e = expand<true>(c, s.V, c.B, c.ldb, c.stride_b, c.N, c.alpha, c.beta,
                        static_cast<float *>(c.Y), c.ldy);
    if (e != hipSuccess) return e;
    return launch_f32(g);
  }
  if (joined) {
    e = launch_f16(g);
    return e != hipSuccess ? e : join(c, s.V, s.T, 1);
  }
  const LowRank term = {s.split, 2 * p.Rp, s.scale, c.B, c.ldb, c.stride_b, c.rows, c.ranks, c.L,
                        c.R};
  g.term = &term;
  return launch_f16_lora(g);
}

template <typename T>
hipError_t run_grad(const LoraCall &c, const GradSpace &s) {
  hipLaunchKernelGGL(lora_group, dim3((unsigned)c.L), dim3(kGroupThreads), 0, c.stream, c.rows,
                     c.M, c.L, s.start, s.perm, s.owner);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const TilePlan t = tile_plan(c, 2);
  TileShrinkParams p = tile_params(c, t);
  p.start = s.start;
  p.perm = s.perm;
  p.owner = s.owner;
  int jobs = 0;
  if (s.G)
    p.job[jobs++] = ShrinkJob{c.dY, c.B, c.stride_b, c.N, c.lddy, c.ldb, 0, tile_chunk(c, t, c.N),
                              s.SG, s.G, s.split, s.scale};
  if (s.V)
    p.job[jobs++] = ShrinkJob{c.X, c.A, c.stride_a, c.K, c.ldx, c.lda, 1, tile_chunk(c, t, c.K),
                              s.SV, s.V, nullptr, nullptr};
  e = shrink_tiles<T>(c, p, t, jobs);
  if (e != hipSuccess) return e;
  Call g = product(c, false, false, c.K, c.N, c.dY, c.lddy, c.W, c.ldw, c.beta_x, c.dX, c.lddx);
  g.ws_fixed = s.W;
  g.ws_fixed_bytes = s.w_bytes;
  if (c.dX && c.half) {
    const LowRank term = {s.split, 2 * p.Rp, s.scale, c.A, c.lda, c.stride_a, c.rows,
                          c.ranks, c.L, c.R};
    g.term = &term;
    e = launch_f16_lora(g);
    if (e != hipSuccess) return e;
  } else if (c.dX) {
    e = expand<false>(c, s.G, c.A, c.lda, c.stride_a, c.K, c.alpha, c.beta_x,
                         static_cast<float *>(c.dX), c.lddx);
    if (e != hipSuccess) return e;
    e = launch_f32(g);
    if (e != hipSuccess) return e;
  }
  if (!c.dA && !c.dB) return hipSuccess;
  OuterParams o = {};
  o.ranks = c.ranks;
  o.start = s.start;
  o.perm = s.perm;
  o.scale = c.scale;
  o.L = c.L;
  o.R = c.R;
  o.Rp = p.Rp;
  o.chunk = outer_chunk(c);
  o.alpha = c.alpha;
  o.beta = c.beta_ab;
  int n = 0, widest = 0;
  if (c.dA) {
    o.job[n++] = OuterJob{s.G, c.X, c.dA, c.stride_da, c.K, c.ldx, c.ldda, 0, s.PA};
    widest = c.K;
  }
  if (c.dB) {
    o.job[n++] = OuterJob{s.V, c.dY, c.dB, c.stride_db, c.N, c.lddy, c.lddb, 1, s.PB};
    widest = widest > c.N ? widest : c.N;
  }
  const int rtiles = (p.Rp + kOuterRanks - 1) / kOuterRanks;
  const int slots = (c.M + o.chunk - 1) / o.chunk + c.L;
  hipLaunchKernelGGL((lora_outer<T>),
                     dim3((unsigned)((widest + kOuterCols - 1) / kOuterCols),
                          (unsigned)(slots < 65535 ? slots : 65535),
                          (unsigned)(n * rtiles)),
                     dim3(kOuterThreads), 0, c.stream, o);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(lora_outer_sum,
                     dim3(flat_grid(((long long)c.R + 3) / 4 * widest), (unsigned)c.L, (unsigned)n),
                     dim3(256), 0, c.stream, o);
  return hipGetLastError();
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
