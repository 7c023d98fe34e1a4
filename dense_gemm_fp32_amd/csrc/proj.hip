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

template <typename T, typename TO, int OUT, int NF, int NB>
hipError_t skinny(const ProjParams &p, hipStream_t stream) {
  constexpr int BC = OUT == kScaled ? 16 * NF : 8 * NF;
  const dim3 g((unsigned)((p.N + BC - 1) / BC), (unsigned)((p.M + 16 * NB - 1) / (16 * NB)));
  if (g.y > 65535) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL((proj_skinny<T, TO, OUT, NF, NB, 1, 8>), g, dim3(8 * kWave), 0, stream, p);
  return hipGetLastError();
}

template <typename T, typename TO, int OUT>
hipError_t run_skinny(const ProjParams &p, hipStream_t stream) {
  constexpr int NF = OUT == kScaled ? 1 : 2;
  return p.M <= 16 ? skinny<T, TO, OUT, NF, 1>(p, stream) : skinny<T, TO, OUT, NF, 4>(p, stream);
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

constexpr int kSkinnyRows = 64;

int bytes_of(const ProjCall &c) { return c.i8 ? 1 : (c.half ? 2 : 4); }

// Whether a call takes the tiles: more rows than the other kernel is for, and rows
// short enough that a tile's offsets fit 32 bits.
bool tiled(const ProjCall &c) {
  return c.M > kSkinnyRows && (c.i8 || c.half) && (long long)c.K * bytes_of(c) < kTileRowBytes;
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
// forward pass left.
template <typename T>
__global__ __launch_bounds__(256) void glu_slopes(const T *Zin, int ldi, const T *dH, int lddh,
                                                  T *Z, int ldz, int M, int F, int act) {
  const long long total = (long long)M * F;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < total;
       i += (long long)gridDim.x * 256) {
    const int m = (int)(i / F), f = (int)(i - (long long)m * F);
    const T *z = Zin + (size_t)m * (size_t)ldi + f;
    const float g = (float)z[0], u = (float)z[F];
    const float d = (float)dH[(size_t)m * (size_t)lddh + f];
    float value, slope;
    act_both(act, g, value, slope);
    T *o = Z + (size_t)m * (size_t)ldz + f;
    o[0] = (T)(d * u * slope);
    o[F] = (T)(d * value);
  }
}

template <typename T>
hipError_t slopes(const GluGradCall &c, T *Z, int ldz) {
  const long long total = (long long)c.M * c.F;
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
