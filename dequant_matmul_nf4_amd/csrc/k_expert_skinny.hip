// The product grouped by expert for few rows per expert (decode):
//
//   y[p] = x[row(p)] . deq(W_e)^T     for offsets[e] <= p < offsets[e + 1]
//
// Reading the codes of the experts that have rows is what bounds it; see
// skinny_tile.h for how a wave walks them.  An expert's rows are cut into tiles
// of up to 16, the tiles' weight rows into groups of 16, and all groups are
// dealt out evenly, one contiguous run to each workgroup (the row counts are
// device data, so a workgroup finds its run from the offsets).
//
// A byte of codes indexes a table of level pairs in LDS, rounded to float16 (11
// significant bits: off by less than 2^-11 of a level), and the sums of a
// 64-block are scaled in float32, so no scaled weight is rounded to 16 bits.
// x becomes float16 exactly: a wave scales its columns of a row by the power
// of two that brings their largest value to [2^14, 2^15) and scales the sums
// back (values 2^-29 of the largest and below lose bits; a block scale of 2^104
// could overflow the sum of a segment, 8 blocks of 64 products below 2^15).  Two
// bfloat16 parts per level instead were exact to 2^-17 but moved two registers per
// lookup to line up the operands: 66 against 57 us (16 rows over 8 experts of
// 14336x4096).
//
// That product takes 49 us now where 7 of the 8 experts have rows (4.4 TB/s; the
// codes and scales of 7 take 42 us at the rate of a large copy), 56 us where all
// have (47 us).  One row alone takes 15 us (6 us), where launch, offsets, index and
// x follow each other.  Measured without gain: 16 waves with steps of 256 columns,
// three or four steps on their way, codes kept in the caches, groups taken in
// rotated order.  Rows of more than 4096 columns re-read x for every batch of groups
// (8 experts of 4096x14336, 16 rows: 72 us).
#include "expert_tiles.h"
#include "skinny_walk.h"

namespace nf4i {
namespace {

struct SkinnyArgs {
  sk::WalkArgs walk;
  ExpertRows er;
  ExpertX ex;
  uint16_t* y;         // [m][rows]
};

struct ExpertJob {
  const SkinnyArgs& a;
  const ExpertScan& scan;
  int lane;
  struct Tile {
    int64_t e, row0;
    int cnt;
  };
  __device__ __forceinline__ int64_t tiles() const { return scan.tiles; }
  __device__ __forceinline__ Tile tile(int64_t tid) const {
    const ExpertTile t = find_expert_tile(a.er, scan, sk::kRows, tid, lane);
    return Tile{t.e, t.row0, static_cast<int>(t.hi - t.row0 < sk::kRows ? t.hi - t.row0 : sk::kRows)};
  }
  __device__ __forceinline__ const uint16_t* x_row(int64_t p) const {
    int64_t r = p;
    if (a.ex.index) {
      r = a.ex.index[p] / a.ex.slots;
      r = r < 0 ? 0 : r < a.ex.rows ? r : a.ex.rows - 1;
    }
    return a.ex.x + r * a.walk.cols;
  }
  __device__ __forceinline__ void store(int64_t p, int64_t row, float v) const {
    a.y[p * a.walk.rows + row] = static_cast<uint16_t>(f32_to_bf16(v));
  }
};

template <bool kDQ, bool kF8, int kG, bool kOnce>
__global__ __launch_bounds__(sk::kThreads, 2) void k_expert_skinny(SkinnyArgs a) {
  __shared__ sk::WalkLds<kG, kF8> lds;
  const int lane = threadIdx.x & 63;
  // the workgroup's run of the groups of all tiles
  const ExpertScan scan = scan_experts(a.er, sk::kRows, lane);
  sk::walk<kDQ, kF8, kG, kOnce>(a.walk, lds, ExpertJob{a, scan, lane});
}

template <bool kDQ, bool kF8>
void launch(const SkinnyArgs& a, hipStream_t s) {
  const int64_t ngr = (a.walk.rows + 15) / 16;
  const int64_t tiles = a.er.m < a.er.experts ? a.er.m : a.er.experts;  // about; the offsets are device data
  const int64_t want = (ngr * tiles + a.walk.pl.rs - 1) / a.walk.pl.rs;
  int64_t grid = want < device_cus() ? want : device_cus();
  while (ngr / grid >= (int64_t{1} << 26)) grid *= 2;
  const dim3 gd(static_cast<unsigned>(grid)), bd(sk::kThreads);
  if (a.walk.pl.per <= sk::kSeg) hipLaunchKernelGGL((k_expert_skinny<kDQ, kF8, 4, true>), gd, bd, 0, s, a);
  else hipLaunchKernelGGL((k_expert_skinny<kDQ, kF8, 4, false>), gd, bd, 0, s, a);
}

}  // namespace

hipError_t launch_expert_skinny(const uint8_t* packed, int64_t rows, int64_t cols, Scales sc, const ExpertRows& er,
                                const ExpertX& ex, uint16_t* y, hipStream_t s) {
  SkinnyArgs a{};
  a.walk = sk::WalkArgs{packed, rows, cols, sc, codebook(sc.fp4), sk::make_plan(cols)};
  a.er = er; a.ex = ex; a.y = y;
  if (sc.absmax) launch<false, false>(a, s);
  else if (sc.f8) launch<true, true>(a, s);
  else launch<true, false>(a, s);
  return hipGetLastError();
}

}  // namespace nf4i
