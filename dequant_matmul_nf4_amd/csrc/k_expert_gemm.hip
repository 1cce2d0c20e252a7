// The forward product grouped by expert, for prompts and training:
//
//   y[p] = x[row(p)] . deq(W_e)^T     for offsets[e] <= p < offsets[e + 1]
//
// with row(p) = index[p] / slots (or p), and W the experts' weights stacked
// along the rows.  The tile is the forward GEMM's (gemm_fwd.h): (32 MI) rows
// of one expert x 256 columns, the weights expanded straight into the matrix
// cores' operands, rounded once to bfloat16 after scaling as there (an operand
// of the matrix cores has 16 bits; the sums are float32).
//
// The row counts are device data, so the grid does not depend on them:
// persistent workgroups count the tiles from the offsets and take theirs,
// those of one expert's row band next to each other.  Of many rows, full rounds
// of 256-row tiles (whole, or more than half full) go first and a second launch
// takes what is left in tiles of 64 rows, so that no round runs nearly empty.
//
// Bound: the matrix cores and what feeds them (as the forward GEMM).  8192 rows
// over 8 experts of 14336x4096: 1040 us, 925 TFLOP/s; 1075 us with 256-row tiles alone.  The rows of x are
// gathered by the loads that bring them into LDS, so no sorted copy of x is
// made.
#include "expert_tiles.h"
#include "gemm_fwd.h"

namespace nf4i {
namespace {

using gt::floatx16;
using gt::kCopies;
using gt::kThreads;

struct ExpertGemmArgs {
  const uint8_t* packed;
  int64_t rows, cols;  // of one expert
  Scales sc;
  ExpertRows er;
  ExpertX ex;
  uint16_t* y;         // [m][rows]
  Codebook cb;
};

template <int MI, bool kDQ, bool kF8>
__global__ __launch_bounds__(kThreads, MI == 2 ? 2 : 1) void k_expert_gemm(ExpertGemmArgs a) {
  constexpr int kBM = 32 * MI, kBN = gt::kTileN;
  __shared__ __align__(16) char xs0[gt::act_stage_bytes<kBM>()], xs1[gt::act_stage_bytes<kBM>()];
  __shared__ __align__(16) float2 tab[256 * kCopies];
  const char* tabc = reinterpret_cast<const char*>(tab);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t slot = static_cast<uint32_t>(lane & (kCopies - 1)) << 3;
  const int64_t tiles_n = (a.rows + kBN - 1) / kBN;
  // MI = 8: the cover tiles of full rounds; else every tile, or what those leave
  const int64_t covered = a.er.cover_slots ? covered_tiles(a.er, lane) : 0;
  ExpertScan scan;
  if constexpr (MI < 8) scan = scan_experts(a.er, kBM, lane, covered);
  const int64_t units = tiles_n * (MI == 8 ? covered : scan.tiles);
  if (static_cast<int64_t>(blockIdx.x) >= units) return;
  gt::fill_level_pairs<kCopies>(tab, a.cb);  // ends with a barrier
  const float mean = kDQ ? *a.sc.mean : 0.0f;
  const int64_t nk = a.cols / gt::kStep;

  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int64_t id = xcd_run(u, units);
    ExpertTile tile;
    if constexpr (MI == 8) tile = find_cover_tile(a.er, id / tiles_n, lane);
    else tile = find_expert_tile(a.er, scan, kBM, id / tiles_n, lane);
    const int64_t n0 = id % tiles_n * kBN;

    // the lane's pieces of the x tile: rows past the expert's last repeat it (never stored)
    const uint8_t* xp[MI];
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      int64_t p = tile.row0 + 8 * (MI * wave + i) + (lane >> 3);
      p = p < tile.hi ? p : tile.hi - 1;
      int64_t r = p;
      if (a.ex.index) {
        r = a.ex.index[p] / a.ex.slots;
        r = r < 0 ? 0 : r < a.ex.rows ? r : a.ex.rows - 1;
      }
      xp[i] = reinterpret_cast<const uint8_t*>(a.ex.x + r * a.cols) + (gt::act_piece(MI * wave + i, lane) << 4);
    }
    gt::WPtrs wp;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int64_t n = n0 + wave * 64 + j * 32 + (lane & 31);
      const int64_t row = tile.e * a.rows + (n < a.rows ? n : a.rows - 1);  // past the end: never stored
      wp.c[j] = a.packed + row * (a.cols / 2) + (lane >> 5) * 16;
      wp.blk[j] = row * (a.cols / 64);
    }
    floatx16 acc[MI][2];
    gt::zero_acc(acc);
    gt::fwd_steps<MI, kDQ, kF8>(
        a.sc, nk,
        [&](int64_t ks, char* stage) {
#pragma unroll
          for (int i = 0; i < MI; ++i) gt::dma16(xp[i] + ks * (gt::kStep * 2), stage + (MI * wave + i) * 1024);
        },
        wp, xs0, xs1, tabc, slot, mean, lane, acc);
    gt::store_acc(acc, a.y, tile.hi, a.rows, tile.row0, n0, wave, lane);
  }
}

template <int MI>
hipError_t launch(const ExpertGemmArgs& a, hipStream_t s) {
  // at most this many units: every expert may end in a partial tile
  const int64_t most = ((a.er.m + 32 * MI - 1) / (32 * MI) + a.er.experts) * ((a.rows + gt::kTileN - 1) / gt::kTileN);
  const int64_t slots = static_cast<int64_t>(device_cus()) * (MI == 2 ? 2 : 1);
  const dim3 gd(static_cast<unsigned>(most < slots ? most : slots)), bd(kThreads);
  if (a.sc.absmax) hipLaunchKernelGGL((k_expert_gemm<MI, false, false>), gd, bd, 0, s, a);
  else if (a.sc.f8) hipLaunchKernelGGL((k_expert_gemm<MI, true, true>), gd, bd, 0, s, a);
  else hipLaunchKernelGGL((k_expert_gemm<MI, true, false>), gd, bd, 0, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_expert_gemm(const uint8_t* packed, int64_t rows, int64_t cols, Scales sc, const ExpertRows& er,
                              const ExpertX& ex, uint16_t* y, hipStream_t s) {
  // By the mean number of rows of an expert (the only one known here).  Measured in
  // us: streaming tiles of 16 rows, then tiles of 64, 128 and 256 rows here:
  //   8 experts of 14336x4096, mean  10:   67  106  169  223
  //                                  32:  136  181  175  227
  //                                  64:  241  189  250  236
  //                                 150:  507  316  260  351
  //                                 256:  854  441  424  371
  //   64 experts of 1024x2048, mean  32:   49   55   53   67
  //                                  64:   81   55   93   71
  //                                 128:  138   96   95  128
  //                                 256:  258  149  137  135
  const int64_t experts = er.experts;
  if (er.m <= 40 * experts) return launch_expert_skinny(packed, rows, cols, sc, er, ex, y, s);
  ExpertGemmArgs a{};
  a.packed = packed; a.rows = rows; a.cols = cols; a.sc = sc; a.er = er; a.ex = ex; a.y = y;
  a.cb = codebook(sc.fp4);
  if (er.m <= 112 * experts) return launch<2>(a, s);
  if (er.m <= 224 * experts) return launch<4>(a, s);
  a.er.cover_slots = device_cus();
  a.er.cover_units = static_cast<int>((rows + gt::kTileN - 1) / gt::kTileN);
  if (hipError_t e = launch<8>(a, s); e != hipSuccess) return e;
  return launch<2>(a, s);
}

}  // namespace nf4i
