// The input gradient of the product grouped by expert:
//
//   dx[p] = dy[p] . deq(W_e)     for offsets[e] <= p < offsets[e + 1]
//
// The tile is the dense input gradient's (gemm_dx_tile.h): (64 MI) rows of one
// expert x 256 columns, the expert's codes expanded and turned on chip, the
// weight rounded once to bfloat16 after scaling.
//
// Such a tile keeps a compute unit for long (0.46 ms at 14336 weight rows), so a
// last round that fills a few of them and the experts' partial tiles would cost
// as much as full ones.  It is taken for full rounds alone, of tiles that are whole or
// more than half full; the kernel that turns no weights (k_expert_skinny_dx.hip) does the rest, in
// tiles of 128 rows.  Row counts are device data: both kernels count the tiles
// from the offsets, and workgroups past the last tile leave at once.
//
// 8192 rows over 8 experts of 14336x4096: 1240 us, 780 TFLOP/s (1430 us with tall
// tiles alone, 1420 us without any).
#include "expert_tiles.h"
#include "gemm_dx_tile.h"

namespace nf4i {
namespace {

struct ExpertDxArgs {
  gt::DxArgs d;  // rows, cols: one expert's; packed, dy, dx, m: of the whole product
  ExpertRows er;
  Codebook cb;
};

constexpr int kTm = kCoverRows, kMI = kTm / 64;

template <bool kDQ, bool kF8>
__global__ __launch_bounds__(gt::kDxThreads) void k_expert_gemm_dx(ExpertDxArgs a) {
  __shared__ __align__(16) char stage0[gt::act_stage_bytes<kTm>()], stage1[gt::act_stage_bytes<kTm>()];
  __shared__ __align__(16) char wts[4][2][gt::kWtBytes];
  __shared__ __align__(16) float scl[8][32];
  __shared__ __align__(16) float2 pairs[256 * gt::kPairCopies];
  const int lane = threadIdx.x & 63;
  const int64_t tiles_k = (a.d.cols + gt::kTk - 1) / gt::kTk;
  const int64_t units = tiles_k * covered_tiles(a.er, lane);
  if (static_cast<int64_t>(blockIdx.x) >= units) return;
  const int64_t id = xcd_run(blockIdx.x, units);
  const ExpertTile t = find_cover_tile(a.er, id / tiles_k, lane);
  gt::DxArgs d = a.d;
  const int64_t w0 = t.e * d.rows * d.cols;  // the expert's first weight
  d.packed += w0 / 2;
  d.blk0 = w0 / 64;
  d.dy += t.lo * d.rows;
  d.dx += t.lo * d.cols;
  d.m = t.hi - t.lo;
  gt::dx_tile<kMI, kDQ, kF8>(d, a.cb, t.row0 - t.lo, id % tiles_k * gt::kTk, stage0, stage1, wts, scl, pairs);
}

}  // namespace

hipError_t launch_expert_gemm_dx(const uint8_t* packed, int64_t rows, int64_t cols, Scales sc, const ExpertRows& er,
                                 const uint16_t* dy, uint16_t* dx, hipStream_t s) {
  // Fewer rows on the mean than a tile: all of it goes without turning weights.
  if (er.m < kTm * static_cast<int64_t>(er.experts)) return launch_expert_skinny_dx(packed, rows, cols, sc, er, dy, dx, s);
  const int64_t tiles_k = (cols + gt::kTk - 1) / gt::kTk, most = (er.m / kTm + er.experts) * tiles_k;
  if (most * gt::kDxThreads > 0xFFFFFFFF) return hipErrorInvalidValue;  // a grid's threads are counted in 32 bits
  ExpertDxArgs a{};
  a.d.packed = packed; a.d.rows = rows; a.d.cols = cols; a.d.sc = sc; a.d.dy = dy; a.d.m = er.m; a.d.dx = dx;
  a.cb = codebook(sc.fp4);
  a.er = er;
  a.er.cover_slots = device_cus();
  a.er.cover_units = static_cast<int>(tiles_k);
  const dim3 gd(static_cast<unsigned>(most)), bd(gt::kDxThreads);
  if (sc.absmax) hipLaunchKernelGGL((k_expert_gemm_dx<false, false>), gd, bd, 0, s, a);
  else if (sc.f8) hipLaunchKernelGGL((k_expert_gemm_dx<true, true>), gd, bd, 0, s, a);
  else hipLaunchKernelGGL((k_expert_gemm_dx<true, false>), gd, bd, 0, s, a);
  if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  return launch_expert_skinny_dx(packed, rows, cols, sc, a.er, dy, dx, s);
}

}  // namespace nf4i
