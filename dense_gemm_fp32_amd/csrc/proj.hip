// proj.hip -- products of 8-bit integers and gated blocks: which kernel runs a
// call, and the gated block's backward pass.
#include <type_traits>

#include "proj.hpp"

namespace dgemm {

namespace {

ProjParams params_of(const ProjCall &c) {
  ProjParams p = {};
  p.X = c.X;
  p.W = c.W;
  p.xs = c.xs;
  p.ws = c.ws;
  p.Y = c.Y;
  p.Z = c.Z;
  p.ldx = c.ldx;
  p.ldw = c.ldw;
  p.ldy = c.ldy;
  p.ldz = c.ldz;
  p.dH = c.dH;
  p.lddh = c.lddh;
  p.M = c.M;
  p.N = c.N;
  p.K = c.K;
  p.act = c.act;
  p.alpha = c.alpha;
  p.beta = c.beta;
  return p;
}

template <typename T, typename TO, int OUT, int NF, int NB, int P, int WAVES, int U>
hipError_t skinny(const ProjParams &p, hipStream_t stream) {
  constexpr int BR = 16 / P;
  constexpr int BC = OUT == kScaled ? BR * NF : BR * NF / 2;
  const dim3 g((unsigned)((p.N + BC - 1) / BC), (unsigned)((p.M + BR * NB - 1) / (BR * NB)));
  if (g.y > 65535) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL((proj_skinny<T, TO, OUT, NF, NB, P, WAVES, U>), g, dim3(WAVES * kWave), 0,
                     stream, p);
  return hipGetLastError();
}

// How wide a workgroup is, and how many waves divide its K.  Twice as many
// columns halve what is read of X, once that leaves a workgroup per CU (64 rows
// of 8192 8-bit integers, 8192 columns: 27.5 to 23.3 us; 4096 columns, 128
// workgroups: 10.6 to 13); with one or more per CU four waves are enough (a gated
// block of 64 x 8192 x 4096 halves: 33.7 us with four, 41.8 with eight), below it
// eight are better (64 x 1024 8-bit columns of 4096: 7.0 with eight, 8.2 with
// four).
template <typename T, typename TO, int OUT, int NB>
hipError_t skinny_wide(const ProjParams &p, hipStream_t stream) {
  constexpr int NF = OUT == kScaled ? 1 : 2;
  constexpr int U = NB == 1 ? 2 : 1;
  const long long wgs = (long long)((p.N + 15) / 16) * ((p.M + 16 * NB - 1) / (16 * NB));
  if (NB > 1 && wgs >= 2 * kCUs) return skinny<T, TO, OUT, 2 * NF, NB, 1, 4, U>(p, stream);
  if (wgs >= kCUs) return skinny<T, TO, OUT, NF, NB, 1, 4, U>(p, stream);
  return skinny<T, TO, OUT, NF, NB, 1, 8, U>(p, stream);
}

template <typename T, typename TO, int OUT>
hipError_t run_skinny(const ProjParams &p, hipStream_t stream) {
  const bool near = (long long)p.ldx * (int)sizeof(T) < kQuadRowBytes &&
                    (long long)p.ldw * (int)sizeof(T) < kQuadRowBytes;
  // up to 8 rows two stretches of k share an instruction (and rows that are
  // further apart than the other form's offsets hold)
  if (p.M <= 8 || !near) return skinny<T, TO, OUT, OUT == kScaled ? 1 : 2, 1, 2, 8, 4>(p, stream);
  if (p.M <= 16) return skinny_wide<T, TO, OUT, 1>(p, stream);
  if (p.M <= 32) return skinny_wide<T, TO, OUT, 2>(p, stream);
  if (p.M <= 48) return skinny_wide<T, TO, OUT, 3>(p, stream);
  return skinny_wide<T, TO, OUT, 4>(p, stream);
}

template <typename TO>
hipError_t run_skinny(const ProjCall &c, const ProjParams &p) {
  if (c.i8) {
    if (!c.gated) return run_skinny<int8_t, TO, kScaled>(p, c.stream);
    return run_skinny<int8_t, TO, kGated>(p, c.stream);
  }
  if (c.dH != nullptr) return run_skinny<TO, TO, kSlopes>(p, c.stream);
  return run_skinny<TO, TO, kGated>(p, c.stream);
}

int bytes_of(const ProjCall &c) { return c.i8 ? 1 : (c.half ? 2 : 4); }

// Whether a call takes the tiles.  Its rows have to be short enough that a
// tile's offsets fit 32 bits.  Up to 16 rows the streaming kernel is ahead
// everywhere, and beyond them while its 16 columns by up to 64 rows make at most
// a workgroup per CU (us, tile first: 192 x 1024 x 1024 8-bit 5.4, 4.5; 300 rows of
// it 5.4, 5.1; gated 128 x 2048 x 4096 halves 19.2, 18.1; 257 rows of it 23.2,
// 32.6).  17 to 64 rows take the 64x64 tile where there are 128 of them or more
// (gated 64 x 8192 x 4096: 8-bit 14.7, 20.7, halves 30.1, 36.7; 20 rows 14.1, 17.5
// and 30.0, 33.0; but 64 x 4096 x 4096 8-bit, 64 tiles: 11.7, 9.4).  Rows that
// have to be copied for the tiles pay for it beyond 128 rows only: a copy reads
// and writes W, which the streaming kernel reads once for every 64 rows.
bool tiled(const ProjCall &c) {
  if (!(c.i8 || c.half) || (long long)c.K * bytes_of(c) >= kTileRowBytes) return false;
  if (c.M <= 16 || (!c.aligned && c.M <= 128)) return false;
  if (c.M <= 64) return (c.gated ? c.N / 32 : c.N / 64) >= kCUs / 2;
  return (long long)((c.N + 15) / 16) * ((c.M + 63) / 64) > kCUs;
}

struct ProjSpace {
  char *X, *W;       // copies with rows of whole 16 bytes
};

size_t carve(const ProjCall &c, void *base, ProjSpace *s) {
  Carve w(base);
  *s = ProjSpace{};
  if (!tiled(c) || c.aligned) return 0;
  const size_t row = ((size_t)c.K * bytes_of(c) + 15) / 16 * 16;
  s->X = w.take<char>(row * (size_t)c.M);
  s->W = w.take<char>(row * (size_t)c.N * (c.gated ? 2 : 1));
  return w.used;
}

hipError_t run_tiles(const ProjCall &c, ProjParams p, const ProjSpace &s) {
  if (!c.aligned) {
    const int eb = bytes_of(c);
    const long long row = (long long)c.K * eb;
    RowCopy x = {c.X, (long long)c.ldx * eb, row, c.M, s.X};
    RowCopy w = {c.W, (long long)c.ldw * eb, row, c.gated ? 2 * c.N : c.N, s.W};
    if (rows_at_16(c.X, c.ldx, eb)) x.dst = nullptr;
    if (rows_at_16(c.W, c.ldw, eb)) w.dst = nullptr;
    const hipError_t e = launch_row_copies(x, w, c.stream);
    if (e != hipSuccess) return e;
    const int ld = (int)((row + 15) / 16 * 16 / eb);
    if (x.dst != nullptr) {
      p.X = s.X;
      p.ldx = ld;
    }
    if (w.dst != nullptr) {
      p.W = s.W;
      p.ldw = ld;
    }
  }
  if (!c.i8) return launch_glu_f16(p, c.dH != nullptr, c.stream);
  return c.gated ? launch_glu_i8(p, c.half, c.stream) : launch_proj_i8(p, c.half, c.stream);
}

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

struct GradSpace {
  void *D;         // [dG dU], M rows of ldd elements
  int ldd;
  char *W;         // the forward pass's and the products', one after the other
  size_t w_bytes;
};

size_t carve(const GluGradCall &c, void *base, GradSpace *s) {
  Carve w(base);
  s->ldd = (2 * c.F + 7) / 8 * 8;
  const size_t n = (size_t)c.M * (size_t)s->ldd;
  s->D = c.half ? (void *)w.take<_Float16>(n) : (void *)w.take<float>(n);
  s->w_bytes = c.Z != nullptr ? 0 : proj_workspace(forward_of(c, nullptr, s->ldd));
  if (c.dX != nullptr) {
    const size_t n = product_bytes(c, product_x(c, nullptr, s->ldd));
    s->w_bytes = n > s->w_bytes ? n : s->w_bytes;
  }
  if (c.dW != nullptr) {
    const size_t n = product_bytes(c, product_w(c, nullptr, s->ldd));
    s->w_bytes = n > s->w_bytes ? n : s->w_bytes;
  }
  s->W = w.take<char>(s->w_bytes);
  return w.used;
}

}  // namespace

size_t proj_workspace(const ProjCall &c) {
  ProjSpace s;
  return carve(c, nullptr, &s);
}

hipError_t launch_proj(const ProjCall &c, void *ws) {
  ProjSpace s;
  carve(c, ws, &s);
  const ProjParams p = params_of(c);
  if (tiled(c)) return run_tiles(c, p, s);
  return c.half ? run_skinny<_Float16>(c, p) : run_skinny<float>(c, p);
}

size_t glu_grad_workspace(const GluGradCall &c) {
  GradSpace s;
  return carve(c, nullptr, &s);
}

hipError_t launch_glu_grad(const GluGradCall &c, void *ws) {
  GradSpace s;
  carve(c, ws, &s);
  hipError_t e;
  if (c.Z != nullptr) {
    e = c.half ? slopes(c, static_cast<_Float16 *>(s.D), s.ldd)
               : slopes(c, static_cast<float *>(s.D), s.ldd);
  } else {
    e = launch_proj(forward_of(c, s.D, s.ldd), s.W);
  }
  if (e != hipSuccess) return e;
  for (int w = 0; w < 2; ++w) {
    if ((w ? c.dW : c.dX) == nullptr) continue;
    Call g = w ? product_w(c, s.D, s.ldd) : product_x(c, s.D, s.ldd);
    g.ws_fixed = s.W;
    g.ws_fixed_bytes = s.w_bytes;
    e = c.half ? launch_f16(g) : launch_f32(g);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace dgemm
