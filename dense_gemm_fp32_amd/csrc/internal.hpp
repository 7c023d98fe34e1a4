// internal.hpp -- host-side interface between the C ABI (api.hip) and the
// kernel translation units.  Not installed; not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dgemm {

// A low-rank term that a product's accumulators start from (fp16 products):
// scale[i] * sum_r V[i, r] U_a[n, r] in row i, column n, a = rows[i].  V: rows
// of ldv halves, for every 16 ranks 16 high parts, then 16 low parts; U:
// adapter a's matrix at U + a*stride, column n of C its row n (a product with B
// stored transposed) or its column n (with B as stored); ranks NULL: R.
struct LowRank {
  const void *V;
  int ldv;
  const float *scale;
  const void *U;
  int ldu;
  long long stride;
  const int *rows, *ranks;
  int L, R;
  int columns;           // of B that the direct loads may read (set by the launch)
};

// One validated GEMM call, after quick returns have been taken: M, N, K > 0
// and alpha != 0.
struct Call {
  int M, N, K;
  float alpha, beta;
  const void *A;
  int lda;
  const void *B;
  int ldb;
  void *C;
  int ldc;
  bool out32;            // fp16 inputs: C and the result are fp32 (else fp16)
  bool ta, tb;           // A stored transposed (K x M, lda >= M) / B (N x K, ldb >= K)
  bool force_scalar;     // diagnostic: element-wise loads/stores everywhere
  int split_mode;        // 0 = split K by size, 1 = never, >= 2 = that many splits (diagnostic)
  // Set by the launcher for the partial pass of a split-K call (else 1, 0, 0).
  int splits;
  int k_chunk;
  long long split_stride;
  // Set by the launcher for a launch over part of the tile order (else 0, 0,
  // false): tiles [tile_base, tile_base + tile_count) of the grouped order;
  // c_tiles: the split-K pass writes dense per-(split, tile) blocks.
  int tile_base, tile_count;
  bool c_tiles;
  int tail_mode;         // 0 = split the last round's tiles by size, 1 = never, >= 2 = that many (diagnostic)
  int tile_config;       // diagnostic: 0 = by size, 1/2/3/4 = large/medium/small/tiny,
                         // 5 = medium with the loads of a step issued together,
                         // 6 = fp32 256x256 (fp16: its large tile),
                         // 7 = fp32 64x64 with four waves (fp16: its small tile),
                         // 8 = fp32 128x64 with four waves (fp16: its medium tile),
                         // 9 = fp32 64x64 four waves, 64-k steps (fp16: its small tile),
                         // 10 = fp32 32x32 one wave, 64-k steps (fp16: its small tile)
  // Split-K workspace source: the library's per-device pool (ws_fixed ==
  // nullptr), requests above ws_limit bytes failing (-1: no limit), or a
  // fixed device region of ws_fixed_bytes bytes that is never allocated or
  // freed (the entry point that allocates nothing).
  long long ws_limit;
  void *ws_fixed;
  size_t ws_fixed_bytes;
  // Copies of A and B with 16-byte rows (pack.hip): 0 = when an operand's rows
  // do not allow 16-byte loads and the call is large enough, 1 = never,
  // 2 = whenever an operand's rows do not allow them (diagnostic).
  int pack_mode;
  // Stream-K (fp32): 0 = by size, 1 = never, 2..6 = in that mode (see
  // streamk_geometry) whenever the four-wave 64x64 tile or a forced tile
  // configuration (1, 5, 6, 7) is taken.
  int streamk_mode;
  const LowRank *term;   // launch_f16_lora only
  bool copy_ragged_b;    // copy B (as stored) also where only its columns do not end with 16 bytes
  bool b_padded;         // B is a copy whose rows end with whole 16 bytes
  hipStream_t stream;
};

// Chosen kernel variant (for launching and for gemm_describe).
struct Plan {
  const char *name;      // tile configuration, e.g. "f32 mfma32x32x2 128x128x32 w2x2"
  int bm, bn, bk;
  int threads;
  int vec_a, vec_b, vec_c;   // elements per global access (1 = scalar)
  long long blocks;          // tiles
  int splits;                // K chunks (1 = no split)
  int tail;                  // K chunks of the last round's tiles (1 = none)
  size_t ws_bytes;           // workspace the call takes: copies of A and B, split K (0 = none)
  bool packed_a = false;     // the GEMM runs on a 16-byte-row copy of A ...
  bool packed_b = false;     // ... of B
  bool streamk = false;      // Stream-K over `blocks` workgroups, then a fix-up pass ...
  long long sk_whole = 0;    // ... the first sk_whole of them computing whole tiles
};

// The reduction pass of a split-K run of tiles: for each of `tiles` tiles
// (positions tile_base.. of the grouped order over a tiles_m x tiles_n grid
// of BM x BN tiles), C := alpha * sum_s W[s][tile] + beta * C on the part of
// the tile inside the M x N matrix; W[s][tile] is a dense BM x BN fp32 block
// at W + (s*tiles + tile)*BM*BN.  fp32 C.
struct TileReduce {
  const float *W;
  int S, tiles, tile_base;
  int BM, BN, tiles_m, tiles_n, group_m;
  int M, N;
  float alpha, beta;
  float *C;
  int ldc;
  bool force_scalar;
};
hipError_t launch_tile_reduce(const TileReduce &r, hipStream_t s);

// The fix-up pass of a Stream-K launch: tiles tile_base .. tiles-1 of
// `steps` K steps each, dealt out in runs of `iters` steps per Stream-K
// workgroup; for every tile that more than one workgroup covered, C :=
// alpha * (sum of its workgroups' partial blocks, in workgroup order) +
// beta * C on the part of the tile inside the matrix.  Stream-K workgroup
// g's partial blocks are W[2g] (its first segment) and W[2g + 1] (its last),
// dense BM x BN fp32 each.  fp32 C.
struct StreamKFixup {
  const float *W;
  int tiles, tile_base, steps;
  long long iters;
  int BM, BN, tiles_m, tiles_n, group_m;
  int M, N;
  float alpha, beta;
  float *C;
  int ldc;
  bool force_scalar;
};
hipError_t launch_streamk_fixup(const StreamKFixup &f, hipStream_t s);

// The reduction pass of a split-K call: C := alpha * sum_s W_s + beta * C over
// an M x N matrix, the S slabs of W (fp32, row pitch ldw, `stride` floats
// apart) summed in order s = 0..S-1.
struct SplitReduce {
  const float *W;
  long long stride;
  int ldw, S, M, N;
  float alpha, beta;
  void *C;
  int ldc;
  bool half_out;       // C is fp16 (else fp32)
  bool force_scalar;
};

// Split-K workspace of `bytes` bytes for call c, ordered on c.stream: from
// c's fixed region when it has one (no allocation; fails if too small), else
// from the library's per-device memory pool (fails above c.ws_limit).  A
// launcher that cannot get its workspace runs the call unsplit.
hipError_t workspace_alloc(const Call &c, size_t bytes, void **ptr);
hipError_t workspace_free(const Call &c, void *ptr);
// Whether work on `s` is being captured into a graph.
bool capturing(hipStream_t s);

// Bytes of a whole split-K workspace (S slabs of M x ceil(N/4)*4 floats) and
// of a last-round split (S dense BM x BN fp32 blocks per leftover tile).
inline size_t split_ws_bytes(int S, int M, int N) {
  return (size_t)S * (size_t)M * (size_t)((N + 3) / 4 * 4) * sizeof(float);
}
inline size_t tail_ws_bytes(int S, int tiles, int BM, int BN) {
  return (size_t)S * (size_t)tiles * (size_t)BM * (size_t)BN * sizeof(float);
}

// The fixed scratch region of the entry point that allocates nothing: a
// file-scope device array of kScratchBytes bytes, its address on device
// `dev` looked up once per device and kept.
constexpr size_t kScratchBytes = (size_t)64 << 20;
hipError_t scratch_region(int dev, void **ptr);
// Device a stream belongs to (NULL stream: the current device); -1 on error.
int stream_device(hipStream_t s);
hipError_t launch_splitk_reduce(const SplitReduce &r, hipStream_t s);

// Split count for a problem with `tiles` tiles of K step `bk`, given the
// call's split mode and the heuristic's choice `want` (1 = no split): clamped
// so every split has at least one K step, the grid stays within range and the
// workspace under its cap (ws_elems_per_split floats per split; 0: an M x N
// slab).  Also returns the chunk length.
int clamp_splits(const Call &c, int want, int bk, long long tiles, int *k_chunk,
                 long long ws_elems_per_split = 0);

// Copies of A and B whose rows allow 16-byte loads (pack.hip).  pack_choice:
// which operands of call c (elements of eb bytes: 4 or 2) are copied and the
// workspace that takes, including the split-K workspace of the GEMM on the
// copies (planned by `plan`); nothing is copied when both operands already
// allow 16-byte loads, under the test switches, for small calls, or when the
// total exceeds the workspace the call may take.  plan_packed / run_packed:
// the plan and the launch of call c with those copies (the copy kernel, then
// `launch` on the copies, on c's stream, from one workspace allocation; the
// call runs on the original operands when that allocation fails).
struct PackChoice {
  bool a = false, b = false;
  int lda = 0, ldb = 0;            // leading dimensions of the copies
  size_t a_bytes = 0, b_bytes = 0;
  size_t inner_ws = 0;             // split-K workspace of the GEMM on the copies
  size_t bytes = 0;                // the whole workspace
};
PackChoice pack_choice(const Call &c, int eb, Plan (*plan)(const Call &));

// Copies of one or two matrices, byte for byte, to rows of whole 16 bytes, the
// last filled up with zeros (dst NULL: none).
struct RowCopy {
  const void *src;
  long long pitch, row_bytes;   // bytes between src's rows, and of a row
  int rows;
  void *dst;
};
hipError_t launch_row_copies(const RowCopy &a, const RowCopy &b, hipStream_t stream);

// Workspace a call may take: its fixed region, else its limit, else the
// pool's per-call cap.
long long ws_available(const Call &c);
Plan plan_packed(const Call &c, int eb, Plan (*plan)(const Call &));
hipError_t run_packed(const Call &c, int eb, Plan (*plan)(const Call &),
                      hipError_t (*launch)(const Call &));

Plan plan_f32(const Call &c);
Plan plan_f16(const Call &c);
hipError_t launch_f32(const Call &c);
// fp32 on the vector ALUs (the SIMT register-blocked design; ablation).
hipError_t launch_f32_valu(const Call &c);

// Matrix-core ceiling probe (probe.hip): buffer sizes it needs, its flop
// count per launch, and the launch (dtype 0 = fp32, 1 = fp16).
size_t probe_operand_bytes();
size_t probe_out_bytes();
double probe_flops(int dtype, int iters);
hipError_t launch_probe(int dtype, int iters, const void *operands, float *out, hipStream_t s);
hipError_t launch_f16(const Call &c);
hipError_t launch_f16_lora(const Call &c);   // on top of *c.term

// C := beta * C over an M x N matrix (beta == 0 writes zeros without reading).
hipError_t launch_scale_f32(int M, int N, float beta, float *C, int ldc, hipStream_t s);
hipError_t launch_scale_f16(int M, int N, float beta, uint16_t *C, int ldc, hipStream_t s);

// Low-rank adapters beside a shared projection, and their gradients
// (lora.hip).  One validated call, M, N, K > 0 and alpha != 0 (lora: L and R
// > 0 too).  half: fp16 matrices, else fp32; dA and dB are always fp32.
struct LoraCall {
  bool half;
  int M, N, K;
  float alpha;
  const void *X;
  int ldx;
  const void *W;
  int ldw;
  float beta;              // lora: of Y
  void *Y;
  int ldy;
  int L, R;
  const void *A;
  int lda;
  long long stride_a;
  const void *B;
  int ldb;
  long long stride_b;
  const float *scale;
  const int *ranks, *rows;
  const void *dY;          // gradients only, from here
  int lddy;
  float beta_x;
  void *dX;
  int lddx;
  float beta_ab;
  float *dA;
  int ldda;
  long long stride_da;
  float *dB;
  int lddb;
  long long stride_db;
  hipStream_t stream;
};
size_t lora_workspace(const LoraCall &c);
hipError_t launch_lora(const LoraCall &c, void *ws);
size_t lora_grad_workspace(const LoraCall &c);
hipError_t launch_lora_grad(const LoraCall &c, void *ws);
// Gradients of a call without a product term (alpha == 0): D_a := beta * D_a
// for the L adapters' rows x cols matrices.
hipError_t launch_scale_batch_f32(int L, int rows, int cols, float beta, float *D, int ldd,
                                  long long stride, hipStream_t s);

// Parts of a workspace, in order, each 256-byte aligned; a null base only
// counts.
struct Carve {
  char *base;
  size_t used = 0;
  explicit Carve(void *b) : base(static_cast<char *>(b)) {}
  template <typename T>
  T *take(size_t count) {
    char *p = base ? base + used : nullptr;
    used += (count * sizeof(T) + 255) / 256 * 256;
    return reinterpret_cast<T *>(p);
  }
};

// A mixture-of-experts layer for a few tokens (moe.hip); validated, M, D > 0.
struct MoeCall {
  bool half;
  int M, D, F, E, k;
  bool renorm;
  float alpha;
  const void *X;
  int ldx;
  const void *Wr;
  int ldr;
  const void *W1;
  int ld1;
  long long stride1;
  const void *W2;
  int ld2;
  long long stride2;
  float beta;
  void *Y;
  int ldy;
  int *ids;
  float *weights;
  hipStream_t stream;
};
constexpr int kMoeMaxTokens = 256;
constexpr int kMoeMaxExperts = 1024;
size_t moe_workspace(const MoeCall &c);
hipError_t launch_moe(const MoeCall &c, void *ws);

// Rows to 8-bit integers with a scale each (quant.hip); M > 0.
hipError_t launch_quant(bool half, int M, int K, const void *X, int ldx, int8_t *Q, int ldq,
                        float *scale, hipStream_t stream);

// A projection X W^T with what follows it (proj.hip): a product of 8-bit
// integers, or a gated block (gated: W has 2N rows), with dH its [dG dU].
// Validated; M, N, K > 0.
struct ProjCall {
  bool i8;                 // X and W hold 8-bit integers, else Y's type
  bool half;               // Y (Z, dH) holds fp16, else fp32
  bool gated;
  bool aligned;            // X and W are rows_for_tiles
  int M, N, K;
  int act;
  float alpha, beta;       // of a product
  const void *X;
  int ldx;
  const float *xs;
  const void *W;
  int ldw;
  const float *ws;
  void *Y;
  int ldy;
  void *Z;
  int ldz;
  const void *dH;
  int lddh;
  hipStream_t stream;
};
// Whether every row of a matrix with elements of eb bytes starts at 16 bytes, and
// its rows are near enough for a tile's 32-bit offsets.
inline bool rows_at(uintptr_t bytes, const void *p, int ld, int eb) {
  return reinterpret_cast<uintptr_t>(p) % bytes == 0 &&
         (long long)ld * eb % (long long)bytes == 0 && (long long)ld * eb < (1LL << 23);
}
inline bool rows_at_16(const void *p, int ld, int eb) { return rows_at(16, p, ld, eb); }
// Whether the tiles' loads take it as it lies: a direct load of 16 bytes asks for an
// address of 4, which every float has, and the last ones of a row of fewer bytes
// for one of 16.
inline bool rows_for_tiles(const void *p, int ld, int eb) {
  return rows_at(eb == 4 ? 4 : 16, p, ld, eb);
}
size_t proj_workspace(const ProjCall &c);
hipError_t launch_proj(const ProjCall &c, void *ws);

// Gradients of a gated block; validated; M, F, K > 0.
struct GluGradCall {
  bool half, dw32;         // dw32: dW holds fp32 whatever the others hold
  bool aligned;            // X and W are rows_for_tiles
  bool at_16;              // X and W are rows_at_16
  int M, F, K;
  int act;
  const void *dH;
  int lddh;
  const void *X;
  int ldx;
  const void *W;
  int ldw;
  const void *Z;           // NULL: G and U are computed again
  int ldz;
  float beta_x;
  void *dX;
  int lddx;
  float beta_w;
  void *dW;
  int lddw;
  hipStream_t stream;
};
size_t glu_grad_workspace(const GluGradCall &c);
hipError_t launch_glu_grad(const GluGradCall &c, void *ws);

// The process-wide switch the calls above go by (api.hip).
long long workspace_limit();

inline bool aligned_to(const void *p, uintptr_t bytes) {
  return (reinterpret_cast<uintptr_t>(p) % bytes) == 0;
}

}  // namespace dgemm
