// glu_grad.hip -- gradients of a gated block:
//
//     dG = dH * U * act'(G),  dU = dH * act(G),
//     dX = [dG dU] W,  dW = [dG dU]^T X.
//
// [dG dU] is one pass over G, U and dH where the forward pass kept G and U, else
// the forward product once more with another end (proj.hip); it is a matrix of the
// inputs' type, as a stored gradient would be: each element is rounded once.  In
// fp16 dX and dW are then off by 2.9e-4 of their norm in place of the 2.1e-4 that
// their own rounding leaves, and what is below 2^-14 or beyond 65504 in [dG dU] loses
// digits or is infinite, which the caller's scale of the loss has to keep it from, as
// it does for dH; two halves an element would halve both products' rate (4096^3: 440
// of 470 us).
//
// The two products run as one launch of both (glu_products.hip), large ones as the
// library's own, one after the other.
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
// the widest loads, or do not, and for a beta of 0 or another (which of the fp32
// splits is chosen goes by whether C is read).  It must not depend on what the
// workspace's size is asked without: the betas, dW's type, the outputs' addresses
// and distances of rows.
size_t product_bytes(const GluGradCall &c, Call g) {
  void *p = reinterpret_cast<void *>((uintptr_t)256);
  size_t most = 0;
  g.A = g.B = g.C = p;
  g.out32 = false;
  g.ws_fixed_bytes = (size_t)1 << 40;
  for (int odd = 0; odd < (c.at_16 ? 1 : 2); ++odd) {
    g.ldb = odd ? c.K | 1 : (c.K + 7) / 8 * 8;
    g.ldc = g.ldb;
    for (const float beta : {0.0f, 1.0f}) {
      g.beta = beta;
      const size_t n = (c.half ? plan_f16(g) : plan_f32(g)).ws_bytes;
      most = n > most ? n : most;
    }
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

// The two products as one launch's, without addresses yet.
ProductJob job_x(const GluGradCall &c) {
  ProductJob j = {};
  j.M = c.M;
  j.N = c.K;
  j.K = 2 * c.F;
  j.lda = vec_ld(c, j.K);
  j.ldc = c.lddx;
  j.beta = c.beta_x;
  return j;
}

ProductJob job_w(const GluGradCall &c) {
  ProductJob j = {};
  j.M = 2 * c.F;
  j.N = c.K;
  j.K = c.M;
  j.lda = vec_ld(c, j.M);
  j.ldc = c.lddw;
  j.beta = c.beta_w;
  return j;
}

// Products of rows, hidden and width below which one launch is ahead of the
// library's two (us, one launch first: fp16 257 x 1024 x 1024 17, 31; 2048^3 87, 116;
// 4096 x 1024 x 4096 132, 148; 3000^3 291, 340; 4096 x 2048 x 4096 292, 236; 4096^3 600,
// 476; fp32 16 x 2000 x 1024 23, 53; 1024 x 2048 x 2048 267, 270; 2048^3 512, 510; 4096 x
// 1024 x 4096 996, 956).  In fp16 it is ahead up to kFewTogether rows at any size, the
// library's large tiles having few steps of dW's then (1024 x 8192 x 4096 302, 335;
// 1024 x 16384 x 4096 595, 671; 512 x 16384 x 4096 346, 396; but 2048 x 8192 x 4096 518,
// 465).  Rows that the library would copy or load by elements take it at any size
// (odd rows, one launch first: 3000 x 2000 x 2050 fp16 145, 387, fp32 787, 1094).  Beyond
// kTogetherF16 neither way is ahead everywhere there (fp16 with Z: 8192 x 4096 x 1024
// 370, 431; 1100 x 6800 x 4100 378, 574; 2048 x 4096 x 4096 325, 297; 2048 x 8192 x
// 4096 662, 570; 4096^3 610, 506; without Z 469, 524; 542, 771; 429, 428; 843, 836;
// 812, 749).
// All of this is measured with both gradients wanted.  One of the two alone takes the
// same way and the same parts, so that it gets the bits that it has beside the other
// (fp16 1024 x 8192 x 4096: dX 161, dW 173, both 330; 2048^3 55, 48, 85).
constexpr double kTogetherF16 = 3.0e10, kTogetherF32 = 5.0e9;
constexpr int kFewTogether = 1024;

bool together(const GluGradCall &c) {
  const long long eb = c.half ? 2 : 4;
  // a tile's offsets have to fit 32 bits
  if (2LL * c.F * eb >= kTileRowBytes || c.K * eb >= kTileRowBytes) return false;
  if (!c.half && c.K < 4) return false;        // glu_products.hip: rows of floats
  return !c.at_16 || (c.half && c.M <= kFewTogether) ||
         (double)c.M * c.F * c.K < (c.half ? kTogetherF16 : kTogetherF32);
}

struct GradSpace {
  void *D;         // [dG dU]: M rows of ldd elements
  int ldd;
  void *X, *W;     // copies with rows that start at 16 bytes
  ProductJob x, d;    // the products of one launch, as planned, with their parts' sums
  ProductPlan plan;
  char *ws;        // the forward pass's and the library's products', one after the other
  size_t ws_bytes;
};

size_t carve(const GluGradCall &c, void *base, GradSpace *s) {
  Carve w(base);
  *s = GradSpace{};
  const size_t eb = c.half ? 2 : 4;
  s->ldd = vec_ld(c, 2 * c.F);
  s->D = w.take<char>((size_t)c.M * (size_t)s->ldd * eb);
  const bool one = together(c);
  // (one launch's operands are copied ahead of the forward pass)
  if (c.Z == nullptr && !one) s->ws_bytes = proj_workspace(forward_of(c, nullptr, s->ldd));
  if (one) {
    ProductJob &x = s->x, &d = s->d;
    x = job_x(c);
    d = job_w(c);
    s->plan = plan_products(c.half, x, d);
    if (!c.aligned) {
      s->X = w.take<char>((size_t)c.M * (size_t)vec_ld(c, c.K) * eb);
      s->W = w.take<char>((size_t)c.F * 2 * (size_t)vec_ld(c, c.K) * eb);
    }
    if (x.splits > 1) x.slab = w.take<float>((size_t)x.splits * x.M * (size_t)((x.N + 3) / 4 * 4));
    if (d.splits > 1) d.slab = w.take<float>((size_t)d.splits * d.M * (size_t)((d.N + 3) / 4 * 4));
  } else {
    const size_t x = product_bytes(c, product_x(c, nullptr, s->ldd));
    const size_t d = product_bytes(c, product_w(c, nullptr, s->ldd));
    s->ws_bytes = x > s->ws_bytes ? x : s->ws_bytes;
    s->ws_bytes = d > s->ws_bytes ? d : s->ws_bytes;
  }
  s->ws = w.take<char>(s->ws_bytes);
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

hipError_t products_together(const GluGradCall &c, const GradSpace &s) {
  ProductJob x = s.x, d = s.d;
  x.A = d.A = s.D;
  x.B = c.W;
  x.ldb = c.ldw;
  x.odd = !c.half && c.dX != nullptr && !rows_at_16(c.W, c.ldw, 4);
  x.C = c.dX;
  d.B = c.X;
  d.ldb = c.ldx;
  d.odd = !c.half && c.dW != nullptr && !rows_at_16(c.X, c.ldx, 4);
  d.C = c.dW;
  hipError_t e = launch_products(c.half, c.dw32, s.plan.mid, x, d, c.stream);
  if (e == hipSuccess && x.C != nullptr && x.splits > 1) e = sum_parts(x, c.half, c.stream);
  if (e == hipSuccess && d.C != nullptr && d.splits > 1)
    e = sum_parts(d, c.half && !c.dw32, c.stream);
  return e;
}

// Copies of X and W, where the tiles need them, in place of them.
hipError_t copy_operands(GluGradCall &c, const GradSpace &s) {
  const long long eb = c.half ? 2 : 4, row = c.K * eb;
  const bool copy_w = (c.dX != nullptr || c.Z == nullptr) && !rows_for_tiles(c.W, c.ldw, (int)eb);
  const bool copy_x = (c.dW != nullptr || c.Z == nullptr) && !rows_for_tiles(c.X, c.ldx, (int)eb);
  const RowCopy w = {c.W, c.ldw * eb, row, 2 * c.F, copy_w ? s.W : nullptr};
  const RowCopy x = {c.X, c.ldx * eb, row, c.M, copy_x ? s.X : nullptr};
  if (copy_w) {
    c.W = s.W;
    c.ldw = vec_ld(c, c.K);
  }
  if (copy_x) {
    c.X = s.X;
    c.ldx = vec_ld(c, c.K);
  }
  return copy_w || copy_x ? launch_row_copies(w, x, c.stream) : hipSuccess;
}

hipError_t products_in_turn(const GluGradCall &c, const GradSpace &s) {
  for (int w = 0; w < 2; ++w) {
    if ((w ? c.dW : c.dX) == nullptr) continue;
    Call g = w ? product_w(c, s.D, s.ldd) : product_x(c, s.D, s.ldd);
    g.ws_fixed = s.ws;
    g.ws_fixed_bytes = s.ws_bytes;
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

hipError_t launch_glu_grad(const GluGradCall &call, void *ws) {
  GluGradCall c = call;
  GradSpace s;
  carve(c, ws, &s);
  const bool one = together(c);
  hipError_t e = hipSuccess;
  if (one && !c.aligned) {
    e = copy_operands(c, s);
    c.aligned = true;
  }
  if (e != hipSuccess) return e;
  if (c.Z == nullptr) e = launch_proj(forward_of(c, s.D, s.ldd), s.ws);
  else if (c.half) e = slopes(c, static_cast<_Float16 *>(s.D), s.ldd);
  else e = slopes(c, static_cast<float *>(s.D), s.ldd);
  if (e != hipSuccess) return e;
  return one ? products_together(c, s) : products_in_turn(c, s);
}

}  // namespace dgemm
