// The forward product grouped by expert, for prompts and training:
//
//   y[p] = x[row(p)] . deq(W_e)^T     for offsets[e] <= p < offsets[e + 1]
//
// with row(p) = index[p] / slots (or p), and W the experts' weights stacked
// along the rows.  The tile is the forward GEMM's (gemm_tiles.h): (32 MI) rows
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
// The rows of x are gathered by the loads that bring them into LDS, so no sorted
// copy of x is made.  In tiles of 128 and 256 rows a wave is alone on its SIMD: its
// codes and scales come through LDS three steps ahead, and what it does besides the
// products is spelled out between them (expert_phases.h).  In 64-row tiles, two
// workgroups per compute unit, the forward GEMM's loop is faster (4096 rows over
// 64 experts of 1024x2048: 55 against 59 us).
//
// Bound: the matrix cores.  8192 rows over 8 experts of 14336x4096: 981 us, 980
// TFLOP/s (1040 us with the forward GEMM's loop).
#include "expert_phases.h"
#include "expert_tiles.h"

namespace nf4i {
namespace {

using gt::floatx16;
using gt::kStep;
using gt::kThreads;
using gt::u32x4;

struct ExpertGemmArgs {
  const uint8_t* packed;
  int64_t rows, cols;  // of one expert
  Scales sc;
  ExpertRows er;
  ExpertX ex;
  uint16_t* y;         // [m][rows]
  Codebook cb;
};


constexpr int kCodeStage = gt::kTileN * kStep / 2;

// The lane's pieces of a tile's rows of x; rows past the expert's last repeat it
// (never stored).
template <int MI>
__device__ __forceinline__ void gather_rows(const uint8_t* (&xp)[MI], const ExpertX& ex, const ExpertTile& tile, int64_t cols,
                                            int wave, int lane) {
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    int64_t p = tile.row0 + 8 * (MI * wave + i) + (lane >> 3);
    p = p < tile.hi ? p : tile.hi - 1;
    int64_t r = p;
    if (ex.index) {
      r = ex.index[p] / ex.slots;
      r = r < 0 ? 0 : r < ex.rows ? r : ex.rows - 1;
    }
    xp[i] = reinterpret_cast<const uint8_t*>(ex.x + r * cols) + (gt::act_piece(MI * wave + i, lane) << 4);
  }
}

// 64-row tiles, two workgroups per compute unit: the codes straight into registers.
template <bool kDQ, bool kF8>
__global__ __launch_bounds__(kThreads, 2) void k_expert_gemm_64(ExpertGemmArgs a) {
  constexpr int MI = 2, kBM = 32 * MI, kBN = gt::kTileN, kCopies = gt::kCopies;
  __shared__ __align__(16) char xs0[gt::act_stage_bytes<kBM>()], xs1[gt::act_stage_bytes<kBM>()];
  __shared__ __align__(16) float2 tab[256 * kCopies];
  const char* tabc = reinterpret_cast<const char*>(tab);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t slot = static_cast<uint32_t>(lane & (kCopies - 1)) << 3;
  const int64_t tiles_n = (a.rows + kBN - 1) / kBN;
  // every tile, or what 256-row tiles leave
  const ExpertScan scan = scan_experts(a.er, kBM, lane, a.er.cover_slots ? covered_tiles(a.er, lane) : 0);
  const int64_t units = tiles_n * scan.tiles;
  if (static_cast<int64_t>(blockIdx.x) >= units) return;
  gt::fill_level_pairs<kCopies>(tab, a.cb);  // ends with a barrier
  const float mean = kDQ ? *a.sc.mean : 0.0f;
  const int64_t nk = a.cols / gt::kStep;

  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int64_t id = xcd_run(u, units);
    const ExpertTile tile = find_expert_tile(a.er, scan, kBM, id / tiles_n, lane);
    const int64_t n0 = id % tiles_n * kBN;

    const uint8_t* xp[MI];
    gather_rows<MI>(xp, a.ex, tile, a.cols, wave, lane);
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

// The same in every lane, said so.
__device__ __forceinline__ int64_t uniform(int64_t x) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<int>(x)), hi = __builtin_amdgcn_readfirstlane(static_cast<int>(x >> 32));
  return static_cast<int64_t>(static_cast<uint64_t>(hi) << 32 | lo);
}

// Taller tiles, one workgroup per compute unit: the codes through LDS.
template <int MI, bool kDQ, bool kF8>
__global__ __launch_bounds__(kThreads) void k_expert_gemm(ExpertGemmArgs a) {
  constexpr int kBM = 32 * MI, kBN = gt::kTileN, kC = gt::kCopies;
  __shared__ __align__(16) char xs0[gt::act_stage_bytes<kBM>()], xs1[gt::act_stage_bytes<kBM>()];
  __shared__ __align__(16) char cs_all[3][kCodeStage];  // a wave's 2 KB: the first 16 bytes of its 64 rows, the second
  __shared__ __align__(16) float2 tab[256 * kC];
  __shared__ __align__(16) float raw_all[4][2][kDQ ? 2 : 1][64];  // a block scale's inputs as they are
  __shared__ float rtab[kF8 ? 256 : 1];
  const char* tabc = reinterpret_cast<const char*>(tab);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t slot = static_cast<uint32_t>(lane & (kC - 1)) << 3;
  const int64_t tiles_n = (a.rows + kBN - 1) / kBN;
  // MI = 8: the cover tiles of full rounds
  ExpertScan scan;
  if constexpr (MI < 8) scan = scan_experts(a.er, kBM, lane);
  const int64_t units = tiles_n * (MI == 8 ? covered_tiles(a.er, lane) : scan.tiles);
  if (static_cast<int64_t>(blockIdx.x) >= units) return;
  if constexpr (kF8) rtab[threadIdx.x] = kE4m3Ratio.v[threadIdx.x];
  gt::fill_level_pairs<kC>(tab, a.cb);  // ends with a barrier
  const float mean = kDQ ? *a.sc.mean : 0.0f;
  const int nk = static_cast<int>(a.cols / kStep);
  const uint32_t row_bytes = static_cast<uint32_t>(a.cols / 2), nblk = static_cast<uint32_t>(nk);
  const float* raw = &raw_all[wave][0][0][0];
  // where the wave's requests go
  const uint32_t raw0 = gt::lds_address(raw), codes0 = gt::lds_address(cs_all[0]) + 2 * wave * 1024;
  const uint32_t dst0 = gt::lds_address(xs0) + MI * wave * 1024, dst1 = gt::lds_address(xs1) + MI * wave * 1024;
  const uint32_t sw = ((lane & 31) >> 1) & 7, h4 = (lane >> 5) * 4;

  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int64_t id = xcd_run(u, units);
    ExpertTile tile;
    if constexpr (MI == 8) tile = find_cover_tile(a.er, id / tiles_n, lane);
    else tile = find_expert_tile(a.er, scan, kBM, id / tiles_n, lane);
    const int64_t n0 = id % tiles_n * kBN;

    const uint8_t* xp[MI];
    gather_rows<MI>(xp, a.ex, tile, a.cols, wave, lane);
    // The wave's 64 weight rows, one per lane: codes and scales (rows past the
    // expert's end repeat its last: never stored).  Offsets from the wave's first.
    const int64_t first = n0 + wave * 64 < a.rows ? n0 + wave * 64 : a.rows - 1;
    const uint32_t wr = static_cast<uint32_t>(first + lane < a.rows ? lane : a.rows - 1 - first);
    const int64_t row0 = uniform(tile.e * a.rows + first);
    const uint8_t* cop = a.packed + row0 * row_bytes;
    const int64_t blk = row0 * nblk;
    const uint32_t coff = wr * row_bytes, soff = wr * nblk;
    auto clamp = [&](int k) { return k < nk ? k : nk - 1; };  // past the last step: the last again
    auto dma_x = [&](int i, int k, uint32_t stage) { gt::request16(xp[i] + k * (kStep * 2), stage + i * 1024); };
    auto dma_codes = [&](int i, int k, int stage) {
      gt::request16(cop + k * (kStep / 2) + 16 * i, coff, codes0 + stage * kCodeStage + i * 1024);
    };
    auto dma_scale = [&](int k, int to) {
      const uint32_t at = raw0 + (to & 1) * sizeof(raw_all[0][0]);
      const int64_t b = blk + k;
      if constexpr (kDQ) {
        gt::request1(a.sc.q + b, soff, at);
        gt::request4(a.sc.absmax2 + (b >> 8), (static_cast<uint32_t>(b & 255) + soff) >> 8 << 2, at + 4 * 64);
      } else {
        gt::request4(a.sc.absmax + b, soff << 2, at);
      }
    };
    // the scales of the lane's rows j * 32 + lane % 32
    auto read_scales = [&](float (&s)[2], int k) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float* r = raw + (k & 1) * (sizeof(raw_all[0][0]) / 4) + j * 32 + (lane & 31);
        if constexpr (kDQ) {
          const int q = *reinterpret_cast<const int8_t*>(r);
          s[j] = (kF8 ? rtab[q & 0xFF] : div127(q)) * r[64] + mean;  // a_hat, three roundings
        } else {
          s[j] = *r;
        }
      }
    };
    auto read_codes = [&](u32x4 (&w)[2], int stage) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
        w[j] = *reinterpret_cast<const u32x4*>(cs_all[stage] + 2 * wave * 1024 + (lane >> 5) * 1024 + (j * 32 + (lane & 31)) * 16);
    };

    floatx16 acc[MI][2];
    gt::zero_acc(acc);
    // The barrier of a step is between s = 2 and 3: by then all of its x and the
    // next step's codes have been read.  x is requested one to two steps ahead,
    // codes and scales three (the wave's own: they need no barrier).
    u32x4 w[2], wn[2];
    float sa[2], sn[2];
    gt::Operands<MI> o;
    const auto now = [&](int j, int, const float2& l) { return gt::bf16_pair(l.x * sa[j], l.y * sa[j]); };
    const auto next = [&](int j, int, const float2& l) { return gt::bf16_pair(l.x * sn[j], l.y * sn[j]); };
    const auto none = [](int) {};
#pragma unroll
    for (int i = 0; i < MI; ++i) dma_x(i, 0, dst0);
    dma_scale(0, 0);
    dma_scale(clamp(1), 1);
#pragma unroll
    for (int i = 0; i < 4; ++i) dma_codes(i & 1, clamp(i >> 1), i >> 1);
    gt::wait_requests<0>();
    sk::lds_barrier();
    read_codes(w, 0);
    read_scales(sa, 0);
    sk::lds_barrier();  // (waits for these reads)
#pragma unroll
    for (int i = 0; i < MI; ++i) dma_x(i, clamp(1), dst1);
    dma_scale(clamp(2), 2);
#pragma unroll
    for (int i = 0; i < 4; ++i) dma_codes(i & 1, clamp(2 + (i >> 1)), i < 2 ? 2 : 0);
    const char* xa = xs0 + (lane & 31) * gt::kActRowBytes;
    gt::first_operands<MI, kC>(o, w, xa, sw, h4, tabc, slot, now);
    int stage = 1;  // of the next step's codes
    for (int ks = 0; ks < nk; ++ks) {
      gt::mfma_phase<MI, kC>(0, o, acc, w, 2, xa, 1, sw, h4, tabc, slot, now, none);
      gt::mfma_phase<MI, kC>(1, o, acc, w, 3, xa, 2, sw, h4, tabc, slot, now, [&](int q) {
        if (q == 0) read_codes(wn, stage);
        if (q == 2) read_scales(sn, ks + 1);
      });
      w[0] = wn[0];
      w[1] = wn[1];
      gt::mfma_phase<MI, kC>(2, o, acc, w, 0, xa, 3, sw, h4, tabc, slot, now, none);
      // the next step's x is here, and the codes and scales of the one after
      gt::wait_requests<2>();
      sk::lds_barrier();
      const uint32_t freed = (ks & 1) ? dst1 : dst0;
      xa = ((ks & 1) ? xs0 : xs1) + (lane & 31) * gt::kActRowBytes;
      gt::mfma_phase<MI, kC>(3, o, acc, w, 1, xa, 0, sw, h4, tabc, slot, next, [&](int q) {
        if (q < MI) dma_x(q, clamp(ks + 2), freed);
        if (q == MI) dma_scale(clamp(ks + 3), ks + 3);
        if (q == MI + 1) {
          dma_codes(0, clamp(ks + 4), stage);
          dma_codes(1, clamp(ks + 4), stage);
        }
      });
      sa[0] = sn[0];
      sa[1] = sn[1];
      stage = stage == 2 ? 0 : stage + 1;
    }
    gt::wait_requests<0>();
    sk::lds_barrier();  // the last reads of x, before the next tile's is requested
    gt::store_acc(acc, a.y, tile.hi, a.rows, tile.row0, n0, wave, lane);
  }
}

template <int MI>
hipError_t launch(const ExpertGemmArgs& a, hipStream_t s) {
  // at most this many units: every expert may end in a partial tile
  const int64_t most = ((a.er.m + 32 * MI - 1) / (32 * MI) + a.er.experts) * ((a.rows + gt::kTileN - 1) / gt::kTileN);
  const int64_t slots = static_cast<int64_t>(device_cus()) * (MI == 2 ? 2 : 1);
  const dim3 gd(static_cast<unsigned>(most < slots ? most : slots)), bd(kThreads);
  if constexpr (MI == 2) {
    if (a.sc.absmax) hipLaunchKernelGGL((k_expert_gemm_64<false, false>), gd, bd, 0, s, a);
    else if (a.sc.f8) hipLaunchKernelGGL((k_expert_gemm_64<true, true>), gd, bd, 0, s, a);
    else hipLaunchKernelGGL((k_expert_gemm_64<true, false>), gd, bd, 0, s, a);
  } else {
    if (a.sc.absmax) hipLaunchKernelGGL((k_expert_gemm<MI, false, false>), gd, bd, 0, s, a);
    else if (a.sc.f8) hipLaunchKernelGGL((k_expert_gemm<MI, true, true>), gd, bd, 0, s, a);
    else hipLaunchKernelGGL((k_expert_gemm<MI, true, false>), gd, bd, 0, s, a);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_expert_gemm(const uint8_t* packed, int64_t rows, int64_t cols, Scales sc, const ExpertRows& er,
                              const ExpertX& ex, uint16_t* y, hipStream_t s) {
  // By the mean number of rows of an expert (the only one known here).  Measured in
  // us, rows unevenly spread, stacks changing from call to call: streaming tiles of
  // 16 rows, then tiles of 64, of 128, and of 256 rows with 64-row tiles for the rest:
  //   8 experts of 14336x4096, mean  10:   68  106  146  108
  //                                  40:  153  173  152  176
  //                                  64:  239  179  218  183
  //                                 112:  386  219  225  219
  //                                 150:  508  291  242  296
  //                                 224:  735  403  380  338
  //                                 512: 1624  788  659  589
  //   64 experts of 1024x2048, mean  32:   50   55   48   58
  //                                  64:   80   55   82   58
  //                                 128:  143   92   86   94
  //                                 256:  265  137  128  124
  // The last bound lies between the two shapes' crossings, of which the first is
  // below 224 and the second above 128: at 224 it costs the first 12%.  What the
  // spread does to full rounds is not known here either: 8 of 14336x4096 at a mean
  // of 64 take 117 us where the rows are evenly spread.
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
