// proj.hip -- products of 8-bit integers and gated blocks: which kernel runs a
// call.
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

// How wide and how high a workgroup is, and how many waves divide its K.
//
// Blocks of 16 rows of X, up to four of them: what there are, if the columns alone
// make a workgroup per CU, so that each row of W is read once.  Twice as many
// columns halve what is read of X, once that leaves a workgroup per CU (64 rows of
// 8192 8-bit integers, 8192 columns: 27.5 to 23.3 us; 4096 columns, 128 workgroups:
// 10.6 to 13).  With fewer columns a workgroup takes fewer rows, W comes from the
// cache again, and what counts is what a CU reads: blocks of X and of W, a second
// workgroup on the CU at 0.4 of the first (us by blocks of X: gated 110 x 582 x 6640
// halves 1 26.4, 2 17.8, 3 19.8, 4 23.2; 64 x 2048 x 4096 1 12.2, 2 9.8, 4 14.5; 64 x
// 1024 x 4096 1 7.3, 2 9.3, 4 13.6; in 8 bits 1 4.4, 4 6.7; in fp32, gated, 1 19, 4 52).
//
// With one workgroup or more per CU four waves are enough (a gated block of 64 x
// 8192 x 4096 halves: 33.7 us with four, 41.8 with eight), below it eight are better
// (64 x 1024 8-bit columns of 4096: 7.0 with eight, 8.2 with four).
template <typename T, typename TO, int OUT, int NB>
hipError_t skinny_high(const ProjParams &p, hipStream_t stream) {
  constexpr int NF = OUT == kScaled ? 1 : 2;
  constexpr int U = NB == 1 ? 2 : 1;
  const long long wgs = (long long)((p.N + 15) / 16) * ((p.M + 16 * NB - 1) / (16 * NB));
  if constexpr (NB > 1)
    if (16 * NB >= p.M && wgs >= 2 * kCUs)
      return skinny<T, TO, OUT, 2 * NF, NB, 1, 4, U>(p, stream);
  // (fewer workgroups than CUs and four blocks of X: two make twice the workgroups at
  // most, which skinny_blocks prices lower; so does it one block before two, where
  // W's is one)
  if constexpr (NB < 4 && !(NB == 2 && NF == 1))
    if (wgs < kCUs) return skinny<T, TO, OUT, NF, NB, 1, 8, U>(p, stream);
  return skinny<T, TO, OUT, NF, NB, 1, 4, U>(p, stream);
}

int skinny_blocks(const ProjParams &p, int nf) {
  const long long cols = (p.N + 15) / 16;
  const int most = p.M >= 64 ? 4 : (p.M + 15) / 16;
  auto wgs = [&](int nb) { return cols * ((p.M + 16 * nb - 1) / (16 * nb)); };
  if (wgs(most) >= kCUs) return most;
  int best = most;
  double least = 1e300;
  for (int nb = most; nb >= 1; --nb) {
    const double rounds = (double)((wgs(nb) + kCUs - 1) / kCUs);
    const double cost = (rounds > 1.0 ? 0.7 * rounds : 1.0) * (nb + nf);
    if (cost < least) {
      least = cost;
      best = nb;
    }
  }
  return best;
}

template <typename T, typename TO, int OUT>
hipError_t run_skinny(const ProjParams &p, hipStream_t stream) {
  const bool near = (long long)p.ldx * (int)sizeof(T) < kQuadRowBytes &&
                    (long long)p.ldw * (int)sizeof(T) < kQuadRowBytes;
  // up to 8 rows two stretches of k share an instruction (and rows that are
  // further apart than the other form's offsets hold)
  if (p.M <= 8 || !near) return skinny<T, TO, OUT, OUT == kScaled ? 1 : 2, 1, 2, 8, 4>(p, stream);
  switch (skinny_blocks(p, OUT == kScaled ? 1 : 2)) {
    case 1: return skinny_high<T, TO, OUT, 1>(p, stream);
    case 2: return skinny_high<T, TO, OUT, 2>(p, stream);
    case 3: return skinny_high<T, TO, OUT, 3>(p, stream);
    default: return skinny_high<T, TO, OUT, 4>(p, stream);
  }
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
// and 30.0, 33.0; but 64 x 4096 x 4096 8-bit, 64 tiles: 11.7, 9.4), of fp32 none.
// Rows that
// have to be copied for the tiles pay a launch and their bytes: from them on three
// workgroups per CU, and beyond 128 rows, the tiles are ahead (copy and tile first:
// gated halves 512 x 1500 x 517 16.5, 11.7, 700 rows 17.4, 16.3, 1000 rows 18.1, 19.1;
// 8-bit 200 x 3000 x 700 11.0, 9.2, 342 rows 10.8, 13.6; 129 x 8000 x 3001 27.6, 31.0).
bool tiled(const ProjCall &c) {
  if ((long long)c.K * bytes_of(c) >= kTileRowBytes) return false;
  if (c.M <= 16 || (!c.aligned && c.M <= 128)) return false;
  if (c.M <= 64) return (c.i8 || c.half) && (c.gated ? c.N / 32 : c.N / 64) >= kCUs / 2;
  return (long long)((c.N + 15) / 16) * ((c.M + 63) / 64) > (c.aligned ? 1 : 3) * kCUs;
}

struct ProjSpace {
  char *X, *W;       // copies of rows that the tiles do not take as they lie
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
    if (rows_for_tiles(c.X, c.ldx, eb)) x.dst = nullptr;
    if (rows_for_tiles(c.W, c.ldw, eb)) w.dst = nullptr;
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
  if (!c.i8)
    return c.half ? launch_glu_f16(p, c.dH != nullptr, c.stream)
                  : launch_glu_f32(p, c.dH != nullptr, c.stream);
  return c.gated ? launch_glu_i8(p, c.half, c.stream) : launch_proj_i8(p, c.half, c.stream);
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

}  // namespace dgemm
