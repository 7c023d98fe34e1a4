// glu_grad.hip -- gradients of a gated block:
//
//     dG = dH * U * act'(G),  dU = dH * act(G),
//     dX = [dG dU] W,  dW = [dG dU]^T X.
//
// [dG dU] is one pass over G, U and dH where the forward pass kept G and U, else
// the forward product once more with another end (proj.hip); it is a matrix of the
// inputs' type, as a stored gradient would be: each element is rounded once (fp16:
// dX and dW are then off by 2.9e-4 of their norm in place of the 2.1e-4 that
// their own rounding leaves; two halves an element would halve both products'
// rate).
//
// The two products: large ones of rows that start at 16 bytes run as the library's
// own, one after the other; the others as one launch of both (glu_products.hip).
// fp16 operands of whole 16 bytes a row are read as they are, others from copies
// that a pass before has made, transposed so that k is contiguous in all of them.
#include "internal.hpp"
#include "proj.hpp"

namespace dgemm {

namespace {

// ---------------------------------------------------------------- [dG dU] from memory

// Z[m, f], Z[m, F + f] := dH * u * act'(g), dH * act(g), from g and u that the
// forward pass left: 16 bytes of each at a time, which may lie at any element's
// address.
template <typename T>
__device__ __forceinline__ void store_whole(T *p, const typename El<T>::Frag &v) {
  typedef T Any __attribute__((ext_vector_type(El<T>::VEC), aligned(sizeof(T))));
  *reinterpret_cast<Any *>(p) = v;
}

template <typename T>
__global__ __launch_bounds__(256) void glu_slopes(const T *Zin, int ldi, const T *dH, int lddh,
                                                  T *Z, int ldz, int M, int F, int act) {
  constexpr int VEC = El<T>::VEC;
  const unsigned pieces = (unsigned)((F + VEC - 1) / VEC);
  const long long total = (long long)M * pieces;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < total;
       i += (long long)gridDim.x * 256) {
    const int m = total < (1LL << 32) ? (int)((unsigned)i / pieces) : (int)(i / pieces);
    const int f = VEC * (int)(i - (long long)m * pieces);
    const T *z = Zin + (size_t)m * (size_t)ldi + f;
    const T *d = dH + (size_t)m * (size_t)lddh + f;
    T *o = Z + (size_t)m * (size_t)ldz + f;
    if (f + VEC <= F) {
      const typename El<T>::Frag gs = load_whole(z), us = load_whole(z + F), ds = load_whole(d);
      typename El<T>::Frag a, b;
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        float value, slope;
        act_both(act, (float)gs[e], value, slope);
        a[e] = (T)((float)ds[e] * (float)us[e] * slope);
        b[e] = (T)((float)ds[e] * value);
      }
      store_whole(o, a);
      store_whole(o + F, b);
    } else {
      for (int e = 0; f + e < F; ++e) {
        float value, slope;
        act_both(act, (float)z[e], value, slope);
        o[e] = (T)((float)d[e] * (float)z[F + e] * slope);
        o[F + e] = (T)((float)d[e] * value);
      }
    }
  }
}

template <typename T>
hipError_t slopes(const GluGradCall &c, T *Z, int ldz) {
  const long long total = (long long)c.M * ((c.F + El<T>::VEC - 1) / El<T>::VEC);
  const long long blocks = (total + 255) / 256;
  hipLaunchKernelGGL((glu_slopes<T>), dim3((unsigned)(blocks < 8192 ? blocks : 8192)), dim3(256),
                     0, c.stream, static_cast<const T *>(c.Z), c.ldz,
                     static_cast<const T *>(c.dH), c.lddh, Z, ldz, c.M, c.F, c.act);
  return hipGetLastError();
}

// ---------------------------------------------------------------- transposed copies

// dst[c, r] = src[r, c]; dst's rows are filled up with zeros to `ld` elements, a
// multiple of 16 bytes.
struct Transpose {
  const void *src;
  void *dst;            // NULL: none
  int rows, cols, lds, ld;
};

// Tiles of 64 x 64 elements through LDS: 16-byte pieces of src's rows, at any
// element's address, to 16-byte pieces of dst's.
template <typename T>
__global__ __launch_bounds__(256) void glu_transpose(Transpose a, Transpose b, Transpose c,
                                                     int na, int nb) {
  constexpr int VEC = El<T>::VEC;
  constexpr int PIECES = 64 / VEC;                     // of a tile's row
  __shared__ T tile[64][64 + VEC / 2];                 // [column][row]
  const int bid = blockIdx.x;
  const int job = bid < na ? 0 : (bid < na + nb ? 1 : 2);
  const int local = bid - (job == 0 ? 0 : (job == 1 ? na : na + nb));
  const T *src = static_cast<const T *>(job == 0 ? a.src : (job == 1 ? b.src : c.src));
  T *dst = static_cast<T *>(job == 0 ? a.dst : (job == 1 ? b.dst : c.dst));
  const int rows = job == 0 ? a.rows : (job == 1 ? b.rows : c.rows);
  const int cols = job == 0 ? a.cols : (job == 1 ? b.cols : c.cols);
  const int lds = job == 0 ? a.lds : (job == 1 ? b.lds : c.lds);
  const int ld = job == 0 ? a.ld : (job == 1 ? b.ld : c.ld);
  const int across = (cols + 63) / 64;
  const int r0 = local / across * 64, c0 = local % across * 64;
#pragma unroll
  for (int i = 0; i < 64 * PIECES / 256; ++i) {
    const int q = threadIdx.x + 256 * i;
    const int r = q / PIECES, k = q % PIECES * VEC;
    typename El<T>::Frag v = {};
    const T *p = src + (size_t)(r0 + r) * (size_t)lds + c0 + k;
    if (r0 + r < rows) {
      if (c0 + k + VEC <= cols) v = load_whole(p);
      else if (c0 + k < cols) v = load_part(p, cols - c0 - k);
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) tile[k + e][r] = v[e];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 64 * PIECES / 256; ++i) {
    const int q = threadIdx.x + 256 * i;
    const int col = q / PIECES, k = q % PIECES * VEC;
    if (c0 + col >= cols || r0 + k >= ld) continue;
    typename El<T>::Frag v;
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] = tile[col][k + e];
    *reinterpret_cast<typename El<T>::Frag *>(dst + (size_t)(c0 + col) * (size_t)ld + r0 + k) = v;
  }
}

template <typename T>
hipError_t transpose(const Transpose &a, const Transpose &b, const Transpose &c,
                     hipStream_t stream) {
  auto tiles = [](const Transpose &t) {
    return t.dst == nullptr ? 0LL : (long long)((t.rows + 63) / 64) * ((t.cols + 63) / 64);
  };
  const long long na = tiles(a), nb = tiles(b), n = na + nb + tiles(c);
  if (n == 0) return hipSuccess;
  if (n > 0x7fffffffLL) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL((glu_transpose<T>), dim3((unsigned)n), dim3(256), 0, stream, a, b, c, (int)na,
                     (int)nb);
  return hipGetLastError();
}

// The two products of the backward pass, on [dG dU] (rows of ldd elements).
Call product_x(const GluGradCall &c, const void *D, int ldd) {
  Call g = {};
  g.M = c.M;
  g.N = c.K;
  g.K = 2 * c.F;
  g.alpha = 1.0f;
  g.beta = c.beta_x;
  g.A = D;
  g.lda = ldd;
  g.B = c.W;
  g.ldb = c.ldw;
  g.C = c.dX;
  g.ldc = c.lddx;
  g.splits = 1;
  g.pack_mode = 2;
  g.copy_ragged_b = c.half;
  g.stream = c.stream;
  return g;
}

Call product_w(const GluGradCall &c, const void *D, int ldd) {
  Call g = {};
  g.M = 2 * c.F;
  g.N = c.K;
  g.K = c.M;
  g.alpha = 1.0f;
  g.beta = c.beta_w;
  g.A = D;
  g.lda = ldd;
  g.ta = true;
  g.B = c.X;
  g.ldb = c.ldx;
  g.C = c.dW;
  g.ldc = c.lddw;
  g.out32 = c.half && c.dw32;
  g.splits = 1;
  g.pack_mode = 2;
  g.copy_ragged_b = c.half;
  g.stream = c.stream;
  return g;
}

// Workspace that such a product may take: for operands whose rows all allow
// the widest loads, or do not.
size_t product_bytes(const GluGradCall &c, Call g) {
  void *p = reinterpret_cast<void *>((uintptr_t)256);
  size_t most = 0;
  for (int odd = 0; odd < (c.aligned ? 1 : 2); ++odd) {
    g.A = g.B = g.C = p;
    g.ldb = odd ? c.K | 1 : (c.K + 7) / 8 * 8;
    g.ldc = g.ldb;
    g.ws_fixed_bytes = (size_t)1 << 40;
    const size_t n = (c.half ? plan_f16(g) : plan_f32(g)).ws_bytes;
    most = n > most ? n : most;
  }
  return most;
}

// The forward pass once more, up to [dG dU].
ProjCall forward_of(const GluGradCall &c, void *D, int ldd) {
  ProjCall f = {};
  f.half = c.half;
  f.gated = true;
  f.aligned = c.aligned;
  f.M = c.M;
  f.N = c.F;
  f.K = c.K;
  f.act = c.act;
  f.X = c.X;
  f.ldx = c.ldx;
  f.W = c.W;
  f.ldw = c.ldw;
  f.Z = D;
  f.ldz = ldd;
  f.dH = c.dH;
  f.lddh = c.lddh;
  f.stream = c.stream;
  return f;
}

// ---------------------------------------------------------------- which way

int vec_ld(const GluGradCall &c, int n) {       // rows of whole 16 bytes
  const int v = c.half ? 8 : 4;
  return (n + v - 1) / v * v;
}

// The two products on k-contiguous operands, without addresses yet.
ProductJob job_x(const GluGradCall &c) {
  ProductJob j = {};
  j.M = c.M;
  j.N = c.K;
  j.K = 2 * c.F;
  j.lda = j.ldb = vec_ld(c, j.K);
  j.ldc = c.lddx;
  j.beta = c.beta_x;
  return j;
}

ProductJob job_w(const GluGradCall &c) {
  ProductJob j = {};
  j.M = 2 * c.F;
  j.N = c.K;
  j.K = c.M;
  j.lda = j.ldb = vec_ld(c, j.K);
  j.ldc = c.lddw;
  j.beta = c.beta_w;
  return j;
}

constexpr double kTogetherF16 = 1.0e10, kTogetherF32 = 2.0e8;

enum class Way { kInTurn, kCopies, kInPlace };

Way way_of(const GluGradCall &c) {
  const long long eb = c.half ? 2 : 4;
  // a tile's offsets have to fit 32 bits
  if (2LL * c.F * eb >= kTileRowBytes || c.M * eb >= kTileRowBytes) return Way::kInTurn;
  const int v = c.half ? 8 : 4;
  if (!(c.aligned && c.K % v == 0 && 2 * c.F % v == 0)) return Way::kCopies;
  if ((double)c.M * c.F * c.K >= (c.half ? kTogetherF16 : kTogetherF32)) return Way::kInTurn;
  return c.half ? Way::kInPlace : Way::kCopies;
}

struct GradSpace {
  void *D, *DT;    // [dG dU]: M rows of ldd elements; transposed
  void *XT, *WT;
  float *sx, *sw;  // parts of the products along k
  int ldd;
  char *W;         // the forward pass's and the library's products', one after the other
  size_t w_bytes;
};

size_t carve(const GluGradCall &c, void *base, GradSpace *s) {
  Carve w(base);
  *s = GradSpace{};
  const size_t eb = c.half ? 2 : 4;
  s->ldd = vec_ld(c, 2 * c.F);
  s->D = w.take<char>((size_t)c.M * (size_t)s->ldd * eb);
  s->w_bytes = c.Z != nullptr ? 0 : proj_workspace(forward_of(c, nullptr, s->ldd));
  const Way way = way_of(c);
  if (way != Way::kInTurn) {
    ProductJob x = job_x(c), d = job_w(c);
    plan_products(c.half, x, d);
    if (way == Way::kCopies) {
      s->DT = w.take<char>((size_t)d.M * (size_t)d.lda * eb);
      s->XT = w.take<char>((size_t)d.N * (size_t)d.ldb * eb);
      s->WT = w.take<char>((size_t)x.N * (size_t)x.ldb * eb);
    }
    if (x.splits > 1) s->sx = w.take<float>((size_t)x.splits * x.M * (size_t)((x.N + 3) / 4 * 4));
    if (d.splits > 1) s->sw = w.take<float>((size_t)d.splits * d.M * (size_t)((d.N + 3) / 4 * 4));
  } else {
    const size_t x = product_bytes(c, product_x(c, nullptr, s->ldd));
    const size_t d = product_bytes(c, product_w(c, nullptr, s->ldd));
    s->w_bytes = x > s->w_bytes ? x : s->w_bytes;
    s->w_bytes = d > s->w_bytes ? d : s->w_bytes;
  }
  s->W = w.take<char>(s->w_bytes);
  return w.used;
}

hipError_t sum_parts(const ProductJob &j, bool half_out, hipStream_t stream) {
  SplitReduce r = {};
  r.W = j.slab;
  r.ldw = (j.N + 3) / 4 * 4;
  r.stride = (long long)j.M * r.ldw;
  r.S = j.splits;
  r.M = j.M;
  r.N = j.N;
  r.alpha = 1.0f;
  r.beta = j.beta;
  r.C = j.C;
  r.ldc = j.ldc;
  r.half_out = half_out;
  return launch_splitk_reduce(r, stream);
}

hipError_t products_together(const GluGradCall &c, const GradSpace &s, bool inplace) {
  ProductJob x = job_x(c), d = job_w(c);
  const ProductPlan plan = plan_products(c.half, x, d);
  x.A = s.D;
  x.C = c.dX;
  x.slab = s.sx;
  d.C = c.dW;
  d.slab = s.sw;
  hipError_t e = hipSuccess;
  if (inplace) {
    x.B = c.W;
    x.ldb = c.ldw;
    d.A = s.D;
    d.lda = s.ldd;
    d.B = c.X;
    d.ldb = c.ldx;
  } else {
    x.B = s.WT;
    d.A = s.DT;
    d.B = s.XT;
    const Transpose tw = {c.W, c.dX ? s.WT : nullptr, 2 * c.F, c.K, c.ldw, x.ldb};
    const Transpose tx = {c.X, c.dW ? s.XT : nullptr, c.M, c.K, c.ldx, d.ldb};
    const Transpose td = {s.D, c.dW ? s.DT : nullptr, c.M, 2 * c.F, s.ldd, d.lda};
    e = c.half ? transpose<_Float16>(tw, tx, td, c.stream)
               : transpose<float>(tw, tx, td, c.stream);
  }
  if (e != hipSuccess) return e;
  e = launch_products(c.half, c.dw32, plan.mid, inplace, x, d, c.stream);
  if (e == hipSuccess && x.C != nullptr && x.splits > 1) e = sum_parts(x, c.half, c.stream);
  if (e == hipSuccess && d.C != nullptr && d.splits > 1)
    e = sum_parts(d, c.half && !c.dw32, c.stream);
  return e;
}

hipError_t products_in_turn(const GluGradCall &c, const GradSpace &s) {
  for (int w = 0; w < 2; ++w) {
    if ((w ? c.dW : c.dX) == nullptr) continue;
    Call g = w ? product_w(c, s.D, s.ldd) : product_x(c, s.D, s.ldd);
    g.ws_fixed = s.W;
    g.ws_fixed_bytes = s.w_bytes;
    const hipError_t e = c.half ? launch_f16(g) : launch_f32(g);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

size_t glu_grad_workspace(const GluGradCall &c) {
  GradSpace s;
  return carve(c, nullptr, &s);
}

hipError_t launch_glu_grad(const GluGradCall &c, void *ws) {
  GradSpace s;
  carve(c, ws, &s);
  hipError_t e;
  if (c.Z == nullptr) e = launch_proj(forward_of(c, s.D, s.ldd), s.W);
  else if (c.half) e = slopes(c, static_cast<_Float16 *>(s.D), s.ldd);
  else e = slopes(c, static_cast<float *>(s.D), s.ldd);
  if (e != hipSuccess) return e;
  const Way way = way_of(c);
  return way == Way::kInTurn ? products_in_turn(c, s)
                             : products_together(c, s, way == Way::kInPlace);
}

}  // namespace dgemm
