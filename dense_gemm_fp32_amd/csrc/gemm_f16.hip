// gemm_f16.hip -- the plain fp16 GEMM: plans and launches of the kernel in
// gemm_f16_kernel.hpp.
#include "gemm_f16_kernel.hpp"

namespace dgemm {

template <class T>
static Plan plan_cfg(const Call &c, const char *name, int want) {
  Plan pl = make_plan<T>(c, name);
  int kc = 0;
  pl.splits = clamp_splits(c, want, T::BK, pl.blocks, &kc);
  pl.ws_bytes = pl.splits > 1 ? split_ws_bytes(pl.splits, c.M, c.N) : 0;
  return pl;
}

static Plan plan_f16_as_is(const Call &c) {
  const F16Choice ch = choose_f16(c);
  switch (ch.cfg) {
    case F16Cfg::kBig:
      if (c.ta && c.tb)   // both operands transposed: 32x32x16 blocks (see dispatch_out)
        return plan_cfg<F16Big>(c, c.out32 ? "f16 mfma32x32x16 tile 256x256x64 8 waves 2 slots out f32"
                                           : "f16 mfma32x32x16 tile 256x256x64 8 waves 2 slots",
                                ch.splits);
      return plan_cfg<F16Big>(c, c.out32 ? "f16 mfma16x16x32 tile 256x256x64 8 waves 2 slots out f32"
                                         : "f16 mfma16x16x32 tile 256x256x64 8 waves 2 slots", ch.splits);
    case F16Cfg::kBig32:
      return plan_cfg<F16Big32>(c, c.out32 ? "f16 mfma32x32x16 tile 256x256x64 8 waves 2 slots out f32"
                                           : "f16 mfma32x32x16 tile 256x256x64 8 waves 2 slots",
                                ch.splits);
    case F16Cfg::kMid:
      return plan_cfg<F16Mid>(c, c.out32 ? "f16 mfma32x32x16 tile 128x128x32 4 waves 4 slots out f32"
                                         : "f16 mfma32x32x16 tile 128x128x32 4 waves 4 slots", ch.splits);
    default:
      return plan_cfg<F16Small>(c, c.out32 ? "f16 mfma32x32x16 tile 64x128x32 2 waves 4 slots out f32"
                                           : "f16 mfma32x32x16 tile 64x128x32 2 waves 4 slots", ch.splits);
  }
}

// Operands whose rows do not allow 16-byte loads may first be copied to ones
// that do (pack.hip); the tile and split are then chosen for the copies.
Plan plan_f16(const Call &c) { return plan_packed(c, 2, plan_f16_as_is); }

hipError_t launch_f16(const Call &c) { return run_packed(c, 2, plan_f16_as_is, launch_f16_as_is<false>); }

}  // namespace dgemm
