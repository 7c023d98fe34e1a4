// glu_products.hip -- the two products of a gated block's backward pass in one
// launch: dX = [dG dU] W and dW = [dG dU]^T X.
//
// Both run on the tiles of proj_tile.hpp, and the workgroups of one fill the CUs
// that the other leaves idle.  The operands are read as they lie: k runs along
// the rows of [dG dU] in the first product, along its columns in the second, and
// along W's and X's columns in both; such an operand keeps its orientation in LDS
// (HRegion) and its fragments are read across.  What a row's last 16 bytes hold
// behind it only feeds columns that are not stored.  fp16 rows start at 16 bytes
// (others are copied).  Rows of floats start anywhere: a direct load asks for no
// more than 4, and the last row of all, whose last 16 bytes may pass the end of the
// matrix, goes through registers with a mask (in rows of four or more; with fewer
// the rows before it would pass the end too).  With copies of them 1000 x 1500 x 517
// with Z took 81 us where it took 77 without (70 with the parts that are planned now),
// 257 x 1024 x 1027 44 and 37.
#include "proj_tile.hpp"

namespace dgemm {

namespace {

// b_first: the workgroups of b come first.  The first job's are rounded up to a
// multiple of the XCDs, so that both jobs' tiles keep to one XCD each.
template <class T, typename TA, typename TB>
__global__ __launch_bounds__(T::NT) void proj_products(ProductJob a, ProductJob b, int first,
                                                       bool b_first) {
  typedef HLayout<T, false, false> LA;
  typedef HLayout<T, true, false> LB;
  __shared__ __attribute__((aligned(1024))) char lds[T::LDS_BYTES];
  lds_poison(lds, T::LDS_BYTES);
  const bool early = (int)blockIdx.x < first;
  const bool second = early == b_first;     // whether this is b's
  const int local = early ? (int)blockIdx.x : (int)blockIdx.x - first;
  GemmParams p = {};
  ProjParams e = {};
  p.A = second ? b.A : a.A;
  p.B = second ? b.B : a.B;
  p.M = e.M = second ? b.M : a.M;
  p.N = e.N = second ? b.N : a.N;
  p.K = second ? b.K : a.K;
  p.lda = second ? b.lda : a.lda;
  p.ldb = second ? b.ldb : a.ldb;
  const int splits = second ? b.splits : a.splits, chunk = second ? b.chunk : a.chunk;
  e.alpha = 1.0f;
  p.tiles_m = (p.M + T::BM - 1) / T::BM;
  p.tiles_n = (p.N + T::BN - 1) / T::BN;
  const int tiles = p.tiles_m * p.tiles_n * splits;
  if (local >= tiles) return;               // (what the first job was rounded up by)
  int tm, tn, split;
  tile_of_block(local, tiles, p.tiles_m, p.tiles_n, T::GROUP_M, tm, tn, split);
  const int m0 = tm * T::BM, n0 = tn * T::BN;
  if (splits > 1) {
    const int kb = split * chunk;
    p.A = static_cast<const char *>(p.A) + (size_t)kb * T::EB * (second ? (size_t)p.lda : 1);
    p.B = static_cast<const char *>(p.B) + (size_t)kb * T::EB * (size_t)p.ldb;
    p.K = p.K - kb < chunk ? p.K - kb : chunk;
  }
  const int wave = threadIdx.x / kWave;
  const int wm0 = (wave / T::WAVES_N) * T::WTM;
  const int wn0 = (wave % T::WAVES_N) * T::WTN;
  typename T::Acc acc[T::FM][T::FN];
  zero_acc<T>(acc);
  // what the loads may read: whole 16 bytes
  if constexpr (T::EB == 2) {
    p.M = second ? (p.M + 7) / 8 * 8 : p.M;
    p.N = (p.N + 7) / 8 * 8;
  }
  const bool masked = T::EB == 4 && (second ? b.odd : a.odd) && split == splits - 1;
  if (second)
    mainloop_direct<T, LB>(p, m0, n0, lds, lds_address(lds), wm0, wn0, acc, masked);
  else
    mainloop_direct<T, LA>(p, m0, n0, lds, lds_address(lds), wm0, wn0, acc, masked);
  __builtin_amdgcn_s_waitcnt(kWaitAll);
  __syncthreads();   // every wave is done with the pipeline slots
  if (splits > 1) {
    float *slab = second ? b.slab : a.slab;
    e.ldy = (e.N + 3) / 4 * 4;
    e.Y = slab + (size_t)split * (size_t)e.M * (size_t)e.ldy;
    proj_epilogue<T, kScaled, float>(e, m0 + wm0, n0 + wn0, lds, acc);
  } else if (second) {
    e.Y = b.C;
    e.ldy = b.ldc;
    e.beta = b.beta;
    proj_epilogue<T, kScaled, TB>(e, m0 + wm0, n0 + wn0, lds, acc);
  } else {
    e.Y = a.C;
    e.ldy = a.ldc;
    e.beta = a.beta;
    proj_epilogue<T, kScaled, TA>(e, m0 + wm0, n0 + wn0, lds, acc);
  }
}

template <class T>
long long tiles_of_job(const ProductJob &j) {
  if (j.C == nullptr) return 0;
  return (long long)((j.M + T::BM - 1) / T::BM) * ((j.N + T::BN - 1) / T::BN) * j.splits;
}

template <class T, typename TA, typename TB>
hipError_t launch(const ProductJob &a, const ProductJob &b, hipStream_t stream) {
  const long long na = tiles_of_job<T>(a), nb = tiles_of_job<T>(b);
  // the longer workgroups first
  const bool b_first = b.C != nullptr && (a.C == nullptr || b.chunk > a.chunk);
  const long long first = b_first ? nb : na, other = b_first ? na : nb;
  const long long start = other > 0 ? (first + kXcds - 1) / kXcds * kXcds : first;
  if (start + other > 0x7fffffffLL) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL((proj_products<T, TA, TB>), dim3((unsigned)(start + other)), dim3(T::NT), 0,
                     stream, a, b, (int)start, b_first);
  return hipGetLastError();
}

template <int EB, typename TA, typename TB>
hipError_t run(const ProductJob &a, const ProductJob &b, bool mid, hipStream_t stream) {
  return mid ? launch<typename ProjTiles<EB>::Mid, TA, TB>(a, b, stream)
             : launch<typename ProjTiles<EB>::Small, TA, TB>(a, b, stream);
}

// A tile: its step in microseconds with the CU full, how many steps a workgroup's
// start and end take, how much of the longest is added where more workgroups than
// fit at once follow each other, and how many a CU holds.
//
// A launch whose workgroups all fit at once lasts as long as the CU that was dealt
// the most steps; parts of a sum even that out, cost a start each, and a launch that
// sums them.  (us by parts of the first product's k, [dG dU] included: fp32 1000 x
// 1500 x 517 2 77, 3 83, 4 70, 5 76, 8 75; 512 x 1408 x 512 3 46, 4 42, 5 41, 6 38, 8
// 42; fp16 in 128x128 tiles 48 x 8192 x 2048 3 63, 4 51, 8 39, in 64x64 tiles 81; 1024 x
// 1024 x 2048 1 32, 2 30, 4 35, 64x64 36.  Over 14 sizes in fp32 and 18 in fp16 the plan
// is the fastest or within 4% of it.)
struct StepCost {
  int bm, bk;
  double step, start, longest;
  int slots;
};

// Steps of the CU that is dealt the most: n1 workgroups of c1, then n2 of c2, one
// CU after another.
double most_steps(long long n1, double c1, long long n2, double c2) {
  const long long r1 = n1 % kCUs, rt = (n1 + n2) % kCUs;
  double most = 0.0;
  for (const long long i : {0LL, r1, r1 - 1, rt, rt - 1}) {   // a CU of each kind there is
    if (i < 0) continue;
    const double first = (double)(n1 / kCUs + (i < r1));
    const double all = (double)((n1 + n2) / kCUs + (i < rt));
    const double steps = first * c1 + (all - first) * c2;
    most = steps > most ? steps : most;
  }
  return most;
}

double cost(const StepCost &t, const ProductJob &a, const ProductJob &b, int sa, int sb) {
  double work = 0.0, sums = 0.0, chunk[2];
  long long wgs[2];
  for (int i = 0; i < 2; ++i) {
    const ProductJob &j = i ? b : a;
    const int s = i ? sb : sa;
    const long long tiles = (long long)((j.M + t.bm - 1) / t.bm) * ((j.N + t.bm - 1) / t.bm);
    const int steps = (j.K + t.bk - 1) / t.bk, each = (steps + s - 1) / s;
    wgs[i] = tiles * ((steps + each - 1) / each);
    chunk[i] = each + t.start;
    work += (double)wgs[i] * chunk[i];
    // what a launch adds behind another, and the parts written and read at 4 TB/s
    if (s > 1) sums += 1.5 + s * (double)j.M * (double)j.N * 8.0 / 4.0e6;
  }
  const int f = chunk[1] > chunk[0] ? 1 : 0;                  // the longer workgroups first
  const double steps = wgs[0] + wgs[1] <= t.slots * kCUs
                           ? most_steps(wgs[f], chunk[f], wgs[1 - f], chunk[1 - f])
                           : work / kCUs + t.longest * chunk[f];
  return t.step * steps + sums;
}

}  // namespace

ProductPlan plan_products(bool half, ProductJob &a, ProductJob &b) {
  const StepCost f16[2] = {{64, 128, 0.40, 2.5, 0.3, 2}, {128, 64, 0.65, 1.0, 0.3, 2}};
  const StepCost f32[2] = {{64, 32, 0.43, 2.0, 0.5, 4}, {128, 32, 1.75, 2.0, 0.5, 2}};
  ProductPlan best = {false, 1e300};
  int bsa = 1, bsb = 1;
  for (int m = 0; m < 2; ++m) {
    const StepCost &t = half ? f16[m] : f32[m];
    auto most = [&](const ProductJob &j) {      // parts of at least 8 steps
      const int s = (j.K + t.bk - 1) / t.bk / 8;
      return s < 1 ? 1 : (s > 8 ? 8 : s);
    };
    for (int sa = 1; sa <= most(a); ++sa)
      for (int sb = 1; sb <= most(b); ++sb) {
        const double c = cost(t, a, b, sa, sb);
        if (c >= best.us) continue;
        best = ProductPlan{m == 1, c};
        bsa = sa;
        bsb = sb;
      }
  }
  const StepCost &t = half ? f16[best.mid] : f32[best.mid];
  for (int i = 0; i < 2; ++i) {
    ProductJob &j = i ? b : a;
    const int steps = (j.K + t.bk - 1) / t.bk, s = i ? bsb : bsa;
    const int each = (steps + s - 1) / s;
    j.chunk = each * t.bk;
    j.splits = (steps + each - 1) / each;
  }
  return best;
}

hipError_t launch_products(bool half, bool b32, bool mid, const ProductJob &a, const ProductJob &b,
                           hipStream_t stream) {
  if (!half) return run<4, float, float>(a, b, mid, stream);
  return b32 ? run<2, _Float16, float>(a, b, mid, stream)
             : run<2, _Float16, _Float16>(a, b, mid, stream);
}

}  // namespace dgemm
