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
hipError_t skinny(const ProjCall &c) {
  constexpr int BC = OUT == kScaled ? 16 * NF : 8 * NF;
  const dim3 g((unsigned)((c.N + BC - 1) / BC), (unsigned)((c.M + 16 * NB - 1) / (16 * NB)));
  if (g.y > 65535) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL((proj_skinny<T, TO, OUT, NF, NB, 1, 8>), g, dim3(8 * kWave), 0, c.stream,
                     params_of(c));
  return hipGetLastError();
}

template <typename T, typename TO, int OUT>
hipError_t run(const ProjCall &c) {
  constexpr int NF = OUT == kScaled ? 1 : 2;
  return c.M <= 16 ? skinny<T, TO, OUT, NF, 1>(c) : skinny<T, TO, OUT, NF, 4>(c);
}

template <typename TO>
hipError_t run_out(const ProjCall &c) {
  if (c.i8) {
    if (!c.gated) return run<int8_t, TO, kScaled>(c);
    return run<int8_t, TO, kGated>(c);
  }
  if (c.dH != nullptr) return run<TO, TO, kSlopes>(c);
  return run<TO, TO, kGated>(c);
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

struct GradSpace {
  void *D;         // [dG dU], M rows of ldd elements
  int ldd;
  char *W;         // the products', one after the other
  size_t w_bytes;
};

size_t carve(const GluGradCall &c, void *base, GradSpace *s) {
  Carve w(base);
  s->ldd = (2 * c.F + 7) / 8 * 8;
  const size_t n = (size_t)c.M * (size_t)s->ldd;
  s->D = c.half ? (void *)w.take<_Float16>(n) : (void *)w.take<float>(n);
  s->w_bytes = 0;
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

size_t proj_workspace(const ProjCall &) { return 0; }

hipError_t launch_proj(const ProjCall &c, void *) {
  return c.half ? run_out<_Float16>(c) : run_out<float>(c);
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
    ProjCall f = {};
    f.half = c.half;
    f.gated = true;
    f.M = c.M;
    f.N = c.F;
    f.K = c.K;
    f.act = c.act;
    f.X = c.X;
    f.ldx = c.ldx;
    f.W = c.W;
    f.ldw = c.ldw;
    f.Z = s.D;
    f.ldz = s.ldd;
    f.dH = c.dH;
    f.lddh = c.lddh;
    f.stream = c.stream;
    e = launch_proj(f, nullptr);
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
