// proj_tile.hpp -- products of 8-bit integers and gated blocks of many rows, on
// the tiles, direct loads and main loop of gemm_f16_kernel.hpp.
//
// X and W are both k-contiguous, so a tile of 8-bit integers is byte for byte
// the fp16 tile of half its k: the same loads, LDS layout and fragment reads
// feed v_mfma_i32_16x16x64_i8 (32x32x32) in place of the fp16 instruction, at
// twice the products per cycle.  Sums are 32-bit integers, exact in any order.
//
// A gated block's tile covers the gate and the up rows of the same BN/2 columns
// (HLayout's PAIR), so both sums of an element meet in its wave, and activation,
// product and scales happen on the way from the accumulators to memory; nothing
// of G and U is written unless it is wanted.
//
// Rows of X and W start at 16 bytes here, those of floats anywhere (the launch
// copies others to rows that do; floats were, too: gated 1000 x 1500 x 517 with a
// copy 41 us, as they lie 33, 2048 x 2048 x 2050 263 and 247); a partial last step
// of k goes through registers with a mask.
#pragma once

#include "gemm_f16_kernel.hpp"
#include "proj.hpp"

namespace dgemm {

// Four values from / to four neighbouring elements (`count` of them inside the
// matrix) at any element's address: global accesses of 8 and 16 bytes need no more
// than the element's own alignment.
template <typename TO>
struct Four {
  typedef TO Any __attribute__((ext_vector_type(4), aligned(sizeof(TO))));
};

template <typename TO>
__device__ __forceinline__ typename Four<TO>::Any raw4(const TO *p, int count) {
  if (count >= 4) return *reinterpret_cast<const typename Four<TO>::Any *>(p);
  typename Four<TO>::Any v = {0, 0, 0, 0};
#pragma unroll
  for (int e = 0; e < 3; ++e)
    if (e < count) v[e] = p[e];
  return v;
}

template <typename TO>
__device__ __forceinline__ f32x4 load4(const TO *p, int count) {
  const typename Four<TO>::Any h = raw4(p, count);
  return f32x4{(float)h[0], (float)h[1], (float)h[2], (float)h[3]};
}

template <typename TO>
__device__ __forceinline__ void store4(TO *p, f32x4 v, int count) {
  if (count >= 4) {
    typename Four<TO>::Any h;
#pragma unroll
    for (int e = 0; e < 4; ++e) h[e] = (TO)v[e];
    *reinterpret_cast<typename Four<TO>::Any *>(p) = h;
  } else {
#pragma unroll
    for (int e = 0; e < 3; ++e)
      if (e < count) p[e] = (TO)v[e];
  }
}

__device__ __forceinline__ f32x4 act_values(int act, f32x4 g) {
  f32x4 v;
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = act_value(act, g[e]);
  return v;
}

// v[i], without an index into registers.
template <class V, int N>
__device__ __forceinline__ V pick(const V (&v)[N], int i) {
  V r = v[0];
#pragma unroll
  for (int j = 1; j < N; ++j)
    if (i == j) r = v[j];
  return r;
}

// From the accumulators, 32 rows at a time through the wave's staging area, to
// memory: a lane takes four neighbouring columns of a row.  r0, c0: first row
// and column of the wave's part of the result.  What is read on the way is on its
// way before the rows are staged (Y, dH; the rows' scales once, a row a lane):
// loaded where it is used, a pass of the loop lasts as long as a load (gated 2968 x
// 7936 x 896 8-bit, 16 passes a wave, 95 to 88 us, 4096^3 8-bit 64 to 60).
template <class T, int OUT, typename TO>
__device__ __forceinline__ void proj_epilogue(const ProjParams &p, int r0, int c0, char *lds,
                                              const typename T::Acc (&acc)[T::FM][T::FN]) {
  constexpr int COLS = OUT == kScaled ? T::WTN : T::WTN / 2;
  constexpr int LPR = COLS / 4;                   // lanes per row
  constexpr int ROWS = kWave / LPR;               // rows per pass
  constexpr int PASSES = 32 / ROWS;
  constexpr int XR = (T::WTM + kWave - 1) / kWave;
  typedef typename Four<TO>::Any Raw;
  const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
  float *stage = reinterpret_cast<float *>(lds + wave * T::EP_BYTES);
  const int cl = 4 * (lane % LPR);
  const int col = c0 + cl, count = p.N - col;
  f32x4 wa = f32x4{1.0f, 1.0f, 1.0f, 1.0f}, wb = wa;
  float xs[XR];
  if constexpr (T::EB == 1) {
    if (p.ws != nullptr && count > 0) {
      wa = load4<float>(p.ws + col, count);
      if constexpr (OUT != kScaled) wb = load4<float>(p.ws + p.N + col, count);
    }
#pragma unroll
    for (int i = 0; i < XR; ++i) {
      const int row = r0 + kWave * i + lane;
      xs[i] = p.xs != nullptr && row < p.M ? p.xs[row] : 1.0f;
    }
  }
  // what the result is formed with beside the sums: dH, or Y
  const TO *more = static_cast<const TO *>(OUT == kSlopes ? p.dH : p.Y);
  const int ldm = OUT == kSlopes ? p.lddh : p.ldy;
  const bool reads = OUT == kSlopes || (OUT == kScaled && p.beta != 0.0f);
  constexpr int AHEAD = 2;                        // passes whose values are on the way together
  auto read = [&](int g, int pass) {
    const int row = r0 + 32 * g + pass * ROWS + lane / LPR;
    return row < p.M && count > 0 ? raw4<TO>(more + (size_t)row * (size_t)ldm + col, count)
                                  : Raw{0, 0, 0, 0};
  };
  auto one = [&](int g, int pass, const Raw &m) {
    const int rl = pass * ROWS + lane / LPR;
    const int row = r0 + 32 * g + rl;
    float x = 1.0f;
    if constexpr (T::EB == 1) x = __shfl(xs[g / 2], 32 * (g & 1) + rl);
    if (row >= p.M || count <= 0) return;
    f32x4 a = *reinterpret_cast<const f32x4 *>(&stage[rl * T::EP_STRIDE + cl]);
    if constexpr (T::EB == 1) {
      if (p.xs != nullptr) a *= x;
      a *= wa;
    }
    if constexpr (OUT == kScaled) {
      a *= p.alpha;
      if (p.beta != 0.0f)
#pragma unroll
        for (int e = 0; e < 4; ++e) a[e] = __builtin_fmaf(p.beta, (float)m[e], a[e]);
      store4<TO>(static_cast<TO *>(p.Y) + (size_t)row * (size_t)p.ldy + col, a, count);
    } else {
      f32x4 b = *reinterpret_cast<const f32x4 *>(&stage[rl * T::EP_STRIDE + COLS + cl]);
      if constexpr (T::EB == 1) {
        if (p.xs != nullptr) b *= x;
        b *= wb;
      }
      TO *z = static_cast<TO *>(p.Z) + (size_t)row * (size_t)p.ldz + col;
      if constexpr (OUT == kGated) {
        store4<TO>(static_cast<TO *>(p.Y) + (size_t)row * (size_t)p.ldy + col,
                   act_values(p.act, a) * b, count);
        if (p.Z != nullptr) {
          store4<TO>(z, a, count);
          store4<TO>(z + p.N, b, count);
        }
      } else {
        f32x4 dg, du;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float value, slope;
          act_both(p.act, a[e], value, slope);
          dg[e] = (float)m[e] * b[e] * slope;
          du[e] = (float)m[e] * value;
        }
        store4<TO>(z, dg, count);
        store4<TO>(z + p.N, du, count);
      }
    }
  };
#pragma unroll
  for (int g = 0; g < T::NG; ++g) {
    if constexpr (OUT == kGated) {
      stage_rows<T>(stage, acc, g, lane);
#pragma unroll 1
      for (int pass = 0; pass < PASSES; ++pass) one(g, pass, Raw{0, 0, 0, 0});
    } else if (OUT == kScaled && !reads) {
      stage_rows<T>(stage, acc, g, lane);
#pragma unroll 2
      for (int pass = 0; pass < PASSES; ++pass) one(g, pass, Raw{0, 0, 0, 0});
    } else {
      Raw in[AHEAD];
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) in[i] = read(g, i);
      stage_rows<T>(stage, acc, g, lane);
#pragma unroll 1
      for (int first = 0; first < PASSES; first += AHEAD) {
        if (first > 0)
#pragma unroll
          for (int i = 0; i < AHEAD; ++i) in[i] = read(g, first + i);
#pragma unroll 1
        for (int i = 0; i < AHEAD; ++i) one(g, first + i, pick(in, i));
      }
    }
  }
}

template <class T, int OUT, typename TO>
__global__ __launch_bounds__(T::NT) void proj_tile(GemmParams p, ProjParams e) {
  typedef HLayout<T, false, true, OUT != kScaled> L;
  __shared__ __attribute__((aligned(1024))) char lds[T::LDS_BYTES];
  lds_poison(lds, T::LDS_BYTES);
  int tm, tn, split;
  tile_of_block(blockIdx.x, gridDim.x, p.tiles_m, p.tiles_n, p.group_m, tm, tn, split);
  const int m0 = tm * T::BM, n0 = tn * L::COLS;
  const int wave = threadIdx.x / kWave;
  const int wm0 = (wave / T::WAVES_N) * T::WTM;
  const int wn0 = (wave % T::WAVES_N) * T::WTN;
  typename T::Acc acc[T::FM][T::FN];
  zero_acc<T>(acc);
  mainloop_direct<T, L>(p, m0, n0, lds, lds_address(lds), wm0, wn0, acc);
  __builtin_amdgcn_s_waitcnt(kWaitAll);
  __syncthreads();   // every wave is done with the pipeline slots
  proj_epilogue<T, OUT, TO>(e, m0 + wm0, n0 + L::column(wn0), lds, acc);
}

template <class T, int OUT, typename TO>
hipError_t launch_tile(const ProjParams &e, hipStream_t stream) {
  constexpr int COLS = OUT == kScaled ? T::BN : T::BN / 2;
  GemmParams p = {};
  p.A = e.X;
  p.B = e.W;
  p.M = e.M;
  p.N = e.N;
  p.K = e.K;
  p.lda = e.ldx;
  p.ldb = e.ldw;
  p.tiles_m = (e.M + T::BM - 1) / T::BM;
  p.tiles_n = (e.N + COLS - 1) / COLS;
  p.group_m = T::GROUP_M;
  p.splits = 1;
  const long long blocks = (long long)p.tiles_m * p.tiles_n;
  if (blocks > 0x7fffffffLL) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL((proj_tile<T, OUT, TO>), dim3((unsigned)blocks), dim3(T::NT), 0, stream, p, e);
  return hipGetLastError();
}

template <class T, int OUT>
long long proj_tiles(const ProjParams &e) {
  constexpr int COLS = OUT == kScaled ? T::BN : T::BN / 2;
  return (long long)((e.M + T::BM - 1) / T::BM) * ((e.N + COLS - 1) / COLS);
}

// The tiles, for elements of EB bytes.  What a round of them costs, in microseconds:
// a start and an end, and so much for every 128 bytes of k (measured at 65 to 2048
// rows, 1024 to 16384 rows of W, 1024 and 4096 bytes of k):
//   256x256       12.6 + 1.45 for 256 tiles (one workgroup per CU), where at most
//                 three quarters are left 1.16
//   128x128       4.8 + 0.93 for 512 (two per CU), 0.56 where at most half are left
//   64x64         2.9 + 0.33 for 512, 0.26 where at most half are left
// with 1 and 1.8 less to start for the two smaller ones if that is all there is; they
// then take three LDS slots in place of two (64 x (2 x 8192) x 4096 halves 30 us, with
// two 35).  The least decides.  (The 128x128 and 64x128 tiles of the plain fp16
// product, four and two waves in steps of 64 bytes of k, take 27 and 26 us at 4096
// bytes of k for up to 256 tiles, against 22 and 12.)
template <int EB>
struct ProjTiles {
  typedef H16Tile<256, 256, 128 / EB, 2, 4, 2, 4, 16, EB> Large;   // 8 waves, 128 KB LDS
  typedef H16Tile<128, 128, 128 / EB, 4, 2, 2, 8, 16, EB> Mid;     // 8 waves,  68 KB
  typedef H16Tile<128, 128, 128 / EB, 4, 2, 3, 8, 16, EB> Mid3;    // 8 waves,  96 KB
  typedef H16Tile<64, 64, 256 / EB, 2, 2, 2, 8, 16, EB> Small;     // 4 waves,  64 KB
  typedef H16Tile<64, 64, 256 / EB, 2, 2, 3, 8, 16, EB> Small3;    // 4 waves,  96 KB
};

// fp32 is bound by its matrix instructions, an eighth of fp16's rate, so a tile's
// time goes with its area and the small one, which leaves less of the last round
// empty, is ahead up to some 500 of the larger (us, 64x64 first: gated 1000 x 1500 x
// 517 32.8, 40.7; 2048^3 126, 134; gated 2048^3 249, 242; 4096^3 958, 933).
template <>
struct ProjTiles<4> {
  typedef H16Tile<128, 128, 32, 4, 2, 2, 8, 16, 4> Mid;            // 8 waves,  68 KB
  typedef H16Tile<64, 64, 32, 2, 2, 2, 8, 16, 4> Small;            // 4 waves,  32 KB
};

// n tiles in rounds of `round` at `start` + `step` each; what is left, up to `few`, at
// `step_few` for a step, and `less` sooner if there is nothing before it.
inline double tile_cost(long long n, int round, int few, double start, double step,
                        double step_few, double less) {
  const long long whole = n / round, left = n % round;
  double c = (double)whole * (start + step);
  if (left > few) c += start + step;
  else if (left > 0) c += start + step_few - (whole == 0 ? less : 0.0);
  return c;
}

template <int EB, int OUT, typename TO>
hipError_t launch_tiles(const ProjParams &e, hipStream_t stream) {
  typedef ProjTiles<EB> P;
  if constexpr (EB == 4) {
    const long long mid = (proj_tiles<typename P::Mid, OUT>(e) + kCUs - 1) / kCUs;
    const long long small = (proj_tiles<typename P::Small, OUT>(e) + kCUs - 1) / kCUs;
    if (mid > 1 && 4.0 * (double)mid <= 1.03 * (double)small)
      return launch_tile<typename P::Mid, OUT, TO>(e, stream);
    return launch_tile<typename P::Small, OUT, TO>(e, stream);
  } else {
    const long long large = proj_tiles<typename P::Large, OUT>(e);
    const long long mid = proj_tiles<typename P::Mid, OUT>(e);
    const long long small = proj_tiles<typename P::Small, OUT>(e);
    const double k = (double)(((long long)e.K * EB + 127) / 128);
    const double l = tile_cost(large, kCUs, kCUs * 3 / 4, 12.6, 1.45 * k, 1.16 * k, 0.0);
    const double m = tile_cost(mid, 2 * kCUs, kCUs, 4.8, 0.93 * k, 0.56 * k, 1.0);
    const double s = tile_cost(small, 2 * kCUs, kCUs, 2.9, 0.33 * k, 0.26 * k, 1.8);
    if (l <= m && l <= s) return launch_tile<typename P::Large, OUT, TO>(e, stream);
    if (m <= s)
      return mid <= kCUs ? launch_tile<typename P::Mid3, OUT, TO>(e, stream)
                         : launch_tile<typename P::Mid, OUT, TO>(e, stream);
    return small <= kCUs ? launch_tile<typename P::Small3, OUT, TO>(e, stream)
                         : launch_tile<typename P::Small, OUT, TO>(e, stream);
  }
}

}  // namespace dgemm
