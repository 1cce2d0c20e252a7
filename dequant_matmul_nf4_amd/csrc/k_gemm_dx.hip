// Input gradient through the frozen 4-bit base, for QLoRA training (tutorial
// page "bitsandbytes quantization tutorial: 4-bit and 8-bit models", section
// "QLoRA: Fine-Tuning a 4-bit Model": the base stays frozen while gradients
// pass through it to the adapters):
//
//   dX = dY . deq(W) + s . (dY . B) . A          dY [m][rows], dX [m][cols]
//
// The reduction runs over the weight's rows, so W enters in the other
// orientation than in the forward GEMM and has to be transposed on chip.
//
// Tiling: a workgroup of 8 waves (two per SIMD) computes a 256 (m) x 256
// (col) tile of dX.  Wave (h, w) = (wave / 4, wave % 4) owns columns
// [64 w, 64 w + 64) for rows [128 h, 128 h + 128): 4 x 2 tiles of
// v_mfma_f32_32x32x16_bf16, transposed so that a lane holds 4 consecutive
// output columns.  A step covers 64 weight rows:
//  - dY: the 256 x 64 tile goes to LDS by direct global-to-LDS loads (two
//    stages, swizzled rows), issued one step ahead;
//  - W: column quarter w is expanded into a Wt tile in LDS, Wt[col][row] (two
//    buffers per quarter), shared by the two waves (0, w) and (1, w): wave
//    (h, w) expands weight rows 32 h .. 32 h + 31 of the step.  Lane
//    (g, q) = (lane % 4, lane / 4) holds the codes of rows 32 h + 8 g .. + 7 at
//    columns 4 q .. 4 q + 3 (one 2-byte load per row), looks up the level
//    pair of each code byte (a 256-entry table in LDS, read half a step ahead
//    of use), multiplies by the row's block scale and rounds once to bf16 --
//    the value nf4_dequantize writes -- and stores each column's 8 values as
//    one 16-byte run.  Runs of a Wt row are swizzled (run c of column k at
//    slot c ^ ((k / 16) % 8), rows padded to 144 bytes), which keeps both
//    these stores and the fragment reads free of bank conflicts.
//  - Software pipeline: while the MFMAs of step s run, the wave expands its
//    half of step s + 1 (codes loaded during step s - 1) and loads the codes
//    of step s + 2; the one barrier per step guards the dY stages and the
//    shared Wt buffers.  The step's body is kept free of branches so that
//    the expansion can be interleaved with the MFMAs, and the second wave on
//    each SIMD fills the gaps of the first.
// A last partial step (rows % 64 != 0) loads its dY tile through registers,
// zero past the end.
//
// The LoRA term is folded in as extra reduction indices,
//   [dY | U_hi | U_lo] . [deq(W) ; A ; A]  with U = s . dY . B,
// U split into two bf16 parts (hi = bf16(U), lo = bf16(U - hi)) by the LoRA
// prep kernel (run on dY and B transposed), so the adapter product keeps
// about 16 significant bits.
#include "gemm_dx_tile.h"

namespace nf4i {
namespace {

using gt::DxArgs;

constexpr int kMI = 4;  // 32 x 32 tiles per wave along m (128 rows)
constexpr int kTm = 64 * kMI, kTk = gt::kTk;

template <bool kDQ, bool kF8>
__global__ __launch_bounds__(gt::kDxThreads) void k_gemm_dx(DxArgs a, Codebook cb) {
  __shared__ __align__(16) char stage0[gt::act_stage_bytes<kTm>()], stage1[gt::act_stage_bytes<kTm>()];
  __shared__ __align__(16) char wts[4][2][gt::kWtBytes];
  __shared__ __align__(16) float scl[8][32];  // per wave: a_hat of its 32 rows of the step
  __shared__ __align__(16) float2 pairs[256 * gt::kPairCopies];  // 16 KB
  const int64_t tiles_k = (a.cols + kTk - 1) / kTk;
  const int64_t tiles = tiles_k * ((a.m + kTm - 1) / kTm);
  int64_t tid = blockIdx.x;
  // consecutive tiles (one dY row strip) on one XCD: dispatch deals workgroups round-robin over 8
  if (tiles % 8 == 0) tid = (tid % 8) * (tiles / 8) + tid / 8;
  gt::dx_tile<kMI, kDQ, kF8>(a, cb, (tid / tiles_k) * kTm, (tid % tiles_k) * kTk, stage0, stage1, wts, scl, pairs);
}

// Elements of u before Bt in the workspace, rounded up to 256 bytes.
int64_t u_elems(int64_t m, int r) {
  return (m * static_cast<int64_t>(gemm_lora_cols(r)) + 127) / 128 * 128;
}

}  // namespace

// Bt[j][n] = B[n][j], so that the prep reads both of its operands along n.
static __global__ __launch_bounds__(256) void k_transpose_b(const uint16_t* __restrict__ lb, int64_t rows, int r,
                                                            uint16_t* __restrict__ bt) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i >= rows * r) return;
  const int64_t n = i / r, j = i - n * r;
  bt[j * rows + n] = lb[i];
}

hipError_t launch_transpose_b(const uint16_t* b, int64_t rows, int r, uint16_t* bt, hipStream_t s) {
  const int64_t nt = rows * r;
  if ((nt + 255) / 256 > 0x7FFFFFFF) return hipErrorInvalidValue;
  hipLaunchKernelGGL(k_transpose_b, dim3(static_cast<unsigned>((nt + 255) / 256)), dim3(256), 0, s, b, rows, r, bt);
  return hipSuccess;
}

size_t gemm_dx_workspace(int64_t m, int64_t rows, int r) {
  if (r <= 0) return 0;
  return static_cast<size_t>(u_elems(m, r) + rows * r) * sizeof(uint16_t);
}

hipError_t launch_gemm_dx(const uint8_t* packed, int64_t rows, int64_t cols, Scales sc, const uint16_t* dy,
                          int64_t m, uint16_t* dx, const uint16_t* lora_a, const uint16_t* lora_b, int r,
                          float lora_scale, uint16_t* ws, hipStream_t s) {
  DxArgs a{};
  a.packed = packed; a.rows = rows; a.cols = cols; a.sc = sc; a.dy = dy; a.m = m; a.dx = dx;
  const int64_t tiles = ((m + kTm - 1) / kTm) * ((cols + kTk - 1) / kTk);
  if (tiles > 0x7FFFFFFF) return hipErrorInvalidValue;
  if (r > 0) {
    a.r = r;
    a.r_pad = (r + 15) / 16 * 16;
    a.kl = static_cast<int>(gemm_lora_cols(r));
    a.la = lora_a;
    a.u = ws;
    uint16_t* bt = ws + u_elems(m, r);
    if (hipError_t e = launch_transpose_b(lora_b, rows, r, bt, s)) return e;
    if (hipError_t e = launch_lora_u(dy, bt, m, rows, r, lora_scale, ws, s)) return e;
  }
  const Codebook& cb = codebook(sc.fp4);
  const dim3 gd(static_cast<unsigned>(tiles)), bd(gt::kDxThreads);
  if (sc.absmax) hipLaunchKernelGGL((k_gemm_dx<false, false>), gd, bd, 0, s, a, cb);
  else if (sc.f8) hipLaunchKernelGGL((k_gemm_dx<true, true>), gd, bd, 0, s, a, cb);
  else hipLaunchKernelGGL((k_gemm_dx<true, false>), gd, bd, 0, s, a, cb);
  return hipGetLastError();
}

}  // namespace nf4i
