// The input gradient of the product grouped by expert:
//
//   dx[p] = dy[p] . deq(W_e)     for offsets[e] <= p < offsets[e + 1]
//
// The tile is the dense input gradient's (gemm_dx_tile.h): (64 MI) rows of one
// expert x 256 columns, the expert's codes expanded and turned on chip, the
// weight rounded once to bfloat16 after scaling.  Row counts are device data:
// the grid covers the most tiles that m rows of that many experts can make,
// and workgroups past the last tile leave at once.
#include "expert_tiles.h"
#include "gemm_dx_tile.h"

namespace nf4i {
namespace {

struct ExpertDxArgs {
  gt::DxArgs d;  // rows, cols: one expert's; packed, dy, dx, m: of the whole product
  ExpertRows er;
  Codebook cb;
};

template <int MI, bool kDQ, bool kF8>
__global__ __launch_bounds__(gt::kDxThreads) void k_expert_gemm_dx(ExpertDxArgs a) {
  constexpr int kTm = 64 * MI;
  __shared__ __align__(16) char stage0[gt::act_stage_bytes<kTm>()], stage1[gt::act_stage_bytes<kTm>()];
  __shared__ __align__(16) char wts[4][2][gt::kWtBytes];
  __shared__ __align__(16) float scl[8][32];
  __shared__ __align__(16) float2 pairs[256 * gt::kPairCopies];
  const int lane = threadIdx.x & 63;
  const int64_t tiles_k = (a.d.cols + gt::kTk - 1) / gt::kTk;
  const ExpertScan scan = scan_experts(a.er, kTm, lane);
  const int64_t tiles = tiles_k * scan.tiles;
  if (static_cast<int64_t>(blockIdx.x) >= tiles) return;
  const int64_t id = xcd_run(blockIdx.x, tiles);
  const ExpertTile t = find_expert_tile(a.er, scan, kTm, static_cast<int>(id / tiles_k), lane);
  gt::DxArgs d = a.d;
  const int64_t w0 = t.e * d.rows * d.cols;  // the expert's first weight
  d.packed += w0 / 2;
  d.blk0 = w0 / 64;
  d.dy += t.lo * d.rows;
  d.dx += t.lo * d.cols;
  d.m = t.hi - t.lo;
  gt::dx_tile<MI, kDQ, kF8>(d, a.cb, t.row0 - t.lo, id % tiles_k * gt::kTk, stage0, stage1, wts, scl, pairs);
}

template <int MI>
hipError_t launch(const ExpertDxArgs& a, hipStream_t s) {
  const int64_t most = ((a.er.m + 64 * MI - 1) / (64 * MI) + a.er.experts) * ((a.d.cols + gt::kTk - 1) / gt::kTk);
  if (most > 0x7FFFFFFF) return hipErrorInvalidValue;
  const dim3 gd(static_cast<unsigned>(most)), bd(gt::kDxThreads);
  if (a.d.sc.absmax) hipLaunchKernelGGL((k_expert_gemm_dx<MI, false, false>), gd, bd, 0, s, a);
  else if (a.d.sc.f8) hipLaunchKernelGGL((k_expert_gemm_dx<MI, true, true>), gd, bd, 0, s, a);
  else hipLaunchKernelGGL((k_expert_gemm_dx<MI, true, false>), gd, bd, 0, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_expert_gemm_dx(const uint8_t* packed, int64_t rows, int64_t cols, Scales sc, const ExpertRows& er,
                                 const uint16_t* dy, uint16_t* dx, hipStream_t s) {
  // Fewer rows on the mean than a tile go without turning weights on chip: at 256
  // rows it takes 161 against 134 us here (64 experts of 1024x2048), and 464
  // against 468 us (8 experts of 14336x4096).
  if (er.m < 256 * static_cast<int64_t>(er.experts)) return launch_expert_skinny_dx(packed, rows, cols, sc, er, dy, dx, s);
  ExpertDxArgs a{};
  a.d.packed = packed; a.d.rows = rows; a.d.cols = cols; a.d.sc = sc; a.d.dy = dy; a.d.m = er.m; a.d.dx = dx;
  a.cb = codebook(sc.fp4);
  a.er = er;
  return launch<4>(a, s);
}

}  // namespace nf4i
