// The input gradient grouped by expert:
//
//   dx[p] = dy[p] . deq(W_e)     for offsets[e] <= p < offsets[e + 1]
//
// The reduction runs over the weight's rows n, along which the codes are not
// contiguous.  A workgroup of 4 waves computes (32 MI) rows of one expert x 256
// columns.  Per step of 64 weight rows, dy goes to LDS as x does in the forward
// product (gemm_fwd.h), and so do the step's codes as they are (8 KB).  A wave turns
// the codes of its 64 columns with ds_read_b64_tr_b4: of 16 rows x 16 columns of
// 4 bits it hands lane i the 16 codes of column i, operands of two products.
// Expanding them then costs what it does in the forward product: a byte looks up
// the levels of two weight rows, each is multiplied by its row's scale, the pair
// is rounded once to bfloat16 (a scale per row of the reduction cannot wait for
// the sums).  A wave's 64 columns are one block of a weight row, so a step has 64
// scales, one made by each lane and read back from LDS.
//
// A wave is alone on its SIMD (two waves at 64 rows), so what it does besides the
// products is spelled out between them (expert_phases.h); left to the compiler it
// collects behind them (8192 rows over 8 experts of 14336x4096: 1110 us; in place
// 962 us).  The codes come from HBM and
// are requested three steps ahead, dy one to two.  As in the forward product,
// tiles are counted from the offsets, and of many rows full rounds of 256-row
// tiles go first and 64-row tiles take the rest.
//
// Bound: the matrix cores.  8192 rows over 8 experts of 14336x4096: 962 us, 1000
// TFLOP/s; 4096 over 64 of 1024x2048: 46 us.  Expanding to bfloat16 first and
// turning that in LDS, 8 waves a tile, took 1240 and 85.
#include "expert_phases.h"
#include "expert_tiles.h"

namespace nf4i {
namespace {

using gt::bf16x8;
using gt::floatx16;
using gt::kStep;
using gt::u32x4;

typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef int intx2 __attribute__((ext_vector_type(2)));

struct ExpertDxArgs {
  const uint8_t* packed;
  int64_t rows, cols;  // of one expert
  Scales sc;
  ExpertRows er;
  const uint16_t* dy;  // [m][rows]
  uint16_t* dx;        // [m][cols]
  Codebook cb;
};

constexpr int kCodeRow = gt::kTileN / 2;  // bytes of a tile's weight row
constexpr int kCodeStage = kStep * kCodeRow;

template <int MI>
constexpr int pair_copies() { return MI == 2 ? 16 : 32; }

// 16 codes of one column: 16 lanes point at 8 bytes of 16 rows each.
__device__ __forceinline__ uint2 turn_codes(const char* p) {
  const intx2 v = __builtin_amdgcn_ds_read_tr4_b64_v2i32((__attribute__((address_space(3))) intx2*)(char*)p);
  return make_uint2(static_cast<uint32_t>(v[0]), static_cast<uint32_t>(v[1]));
}

template <int MI, bool kDQ, bool kF8>
__global__ __launch_bounds__(gt::kThreads, MI == 2 ? 2 : 1) void k_expert_gemm_dx(ExpertDxArgs a) {
  constexpr int kBM = 32 * MI, kBN = gt::kTileN, kC = pair_copies<MI>();
  __shared__ __align__(16) char xs0[gt::act_stage_bytes<kBM>()], xs1[gt::act_stage_bytes<kBM>()];
  __shared__ __align__(16) char cs_all[3][kCodeStage];
  __shared__ __align__(16) float scl_all[4][2][kStep];
  __shared__ __align__(16) float2 tab[256 * kC];
  __shared__ __align__(16) float raw_all[4][2][kDQ ? 2 : 1][kStep];  // a block scale's inputs as they are
  __shared__ float rtab[kF8 ? 256 : 1];
  const char* tabc = reinterpret_cast<const char*>(tab);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t slot = static_cast<uint32_t>(lane & (kC - 1)) << (kC == 32 ? 3 : 4);
  const int64_t tiles_k = (a.cols + kBN - 1) / kBN;
  const int64_t covered = a.er.cover_slots ? covered_tiles(a.er, lane) : 0;
  ExpertScan scan;
  if constexpr (MI < 8) scan = scan_experts(a.er, kBM, lane, covered);
  const int64_t units = tiles_k * (MI == 8 ? covered : scan.tiles);
  if (static_cast<int64_t>(blockIdx.x) >= units) return;
  {
    // entry e: the levels of its low half (the even weight row) and its high half
    const int e = threadIdx.x;
    const float2 v = make_float2(a.cb.level[e & 15], a.cb.level[e >> 4]);
#pragma unroll
    for (int c = 0; c < kC; ++c) tab[e * kC + c] = v;
    if constexpr (kF8) rtab[e] = kE4m3Ratio.v[e];
  }
  __syncthreads();
  const float mean = kDQ ? *a.sc.mean : 0.0f;
  const int rows = static_cast<int>(a.rows), nk = (rows + kStep - 1) / kStep;
  const uint32_t row_bytes = static_cast<uint32_t>(a.cols / 2), nblk = static_cast<uint32_t>(a.cols / 64);
  const uint32_t ld = static_cast<uint32_t>(a.rows * 2);
  float* scl = &scl_all[wave][0][0];
  const float* raw = &raw_all[wave][0][0][0];
  // where the wave's requests go
  const uint32_t raw0 = gt::lds_address(raw), codes0 = gt::lds_address(cs_all[0]) + 2 * wave * 1024;
  const uint32_t dst0 = gt::lds_address(xs0) + MI * wave * 1024, dst1 = gt::lds_address(xs1) + MI * wave * 1024;
  const uint32_t sw = ((lane & 31) >> 1) & 7, h4 = (lane >> 5) * 4;
  // where the lane reads the codes it turns: row 32 h + 16 t + lane % 16, 16-byte
  // piece 2 wave + j of the row at slot piece ^ (row % 8)
  const uint32_t turn = (32 * (lane >> 5) + (lane & 15)) * kCodeRow + (((2 * wave) ^ (lane & 7)) << 4) + ((lane >> 4) & 1) * 8;

  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int64_t id = xcd_run(u, units);
    ExpertTile tile;
    if constexpr (MI == 8) tile = find_cover_tile(a.er, id / tiles_k, lane);
    else tile = find_expert_tile(a.er, scan, kBM, id / tiles_k, lane);
    const int64_t k0 = id % tiles_k * kBN;
    const int cnt = static_cast<int>(tile.hi - tile.row0 < kBM ? tile.hi - tile.row0 : kBM);

    // what is requested next, and the weight rows left from there
    const uint8_t* dyp = reinterpret_cast<const uint8_t*>(a.dy + tile.row0 * a.rows);
    const uint8_t* cop = a.packed + tile.e * a.rows * row_bytes;
    int64_t blk = tile.e * a.rows * nblk + (k0 / 64 + wave < nblk ? k0 / 64 + wave : nblk - 1);
    int dy_left = static_cast<int>(a.rows), co_left = dy_left, sc_left = dy_left;
    // Offsets of the lane's requests.  Those past the weight's rows repeat the last
    // ones (of dy the last 8 of the same row); their scales are 0.  Pieces past the
    // end of a row of codes repeat its last: such columns are not stored.
    const uint32_t cp = static_cast<uint32_t>(k0 / 32) + ((lane & 7) ^ (lane >> 3));
    const uint32_t cpiece = (cp < row_bytes / 16 ? cp : row_bytes / 16 - 1) * 16, crow = (16 * wave + (lane >> 3)) * row_bytes;
    const uint32_t piece[2] = {static_cast<uint32_t>(gt::act_piece(0, lane)) << 4, static_cast<uint32_t>(gt::act_piece(1, lane)) << 4};
    uint32_t drow[MI];
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const int r = 8 * (MI * wave + i) + (lane >> 3);
      drow[i] = static_cast<uint32_t>(r < cnt ? r : cnt - 1) * ld;
    }
    auto least = [](uint32_t x, uint32_t y) { return x < y ? x : y; };
    // Each of these requests a part of the next step's data, the last one moves on
    // (past the last step: it stays).
    uint32_t dy_last = 0, co_last = 0;  // of the step that is requested: the last piece of a row, the last row
    auto dma_dy = [&](int i, uint32_t stage) {
      if (i == 0) dy_last = (static_cast<uint32_t>(dy_left < kStep ? dy_left : kStep) - 8) * 2;
      gt::request16(dyp, drow[i] + least(piece[i & 1], dy_last), stage + i * 1024);
      if (i == MI - 1) {
        const int by = dy_left > kStep ? kStep : 0;
        dyp += by * 2;
        dy_left -= by;
      }
    };
    auto dma_codes = [&](int i, int stage) {
      if (i == 0) co_last = static_cast<uint32_t>((co_left < kStep ? co_left : kStep) - 1) * row_bytes;
      gt::request16(cop, cpiece + least(crow + i * 8 * row_bytes, co_last), codes0 + stage * kCodeStage + i * 1024);
      if (i == 1) {
        const int by = co_left > kStep ? kStep : 0;
        cop += by * static_cast<int64_t>(row_bytes);
        co_left -= by;
      }
    };
    // lane n: the scale of the step's weight row n in the wave's block
    const uint32_t srow = lane * nblk;
    auto dma_scale = [&](int ks) {
      const uint32_t to = raw0 + (ks & 1) * sizeof(raw_all[0][0]);
      const uint32_t o = least(srow, static_cast<uint32_t>((sc_left < kStep ? sc_left : kStep) - 1) * nblk);
      if constexpr (kDQ) {
        gt::request1(a.sc.q + blk, o, to);
        gt::request4(a.sc.absmax2 + (blk >> 8), (static_cast<uint32_t>(blk & 255) + o) >> 8 << 2, to + 4 * kStep);
      } else {
        gt::request4(a.sc.absmax + blk, o << 2, to);
      }
      const int by = sc_left > kStep ? kStep : 0;
      blk += by * static_cast<int64_t>(nblk);
      sc_left -= by;
    };
    auto put_scale = [&](int ks) {
      const float* r = raw + (ks & 1) * (sizeof(raw_all[0][0]) / 4) + lane;
      float s;
      if constexpr (kDQ) {
        const int q = *reinterpret_cast<const int8_t*>(r);
        s = (kF8 ? rtab[q & 0xFF] : div127(q)) * r[kStep] + mean;  // a_hat, three roundings
      } else {
        s = *r;
      }
      scl[(ks & 1) * kStep + lane] = ks * kStep + lane < rows ? s : 0.0f;
    };
    auto read_scales = [&](floatx4 (&s)[2], int ks, int step) {
      const float* p = scl + (ks & 1) * kStep + 32 * (lane >> 5) + 8 * step;
      s[0] = *reinterpret_cast<const floatx4*>(p);
      s[1] = *reinterpret_cast<const floatx4*>(p + 4);
    };
    // words 2 t, 2 t + 1 of both columns: reduction steps 2 t, 2 t + 1
    u32x4 w[2];
    auto turn_half = [&](int t, const char* stage) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint2 v = turn_codes(stage + (turn ^ (16 * j)) + 16 * kCodeRow * t);
        w[j][2 * t] = v.x;
        w[j][2 * t + 1] = v.y;
      }
    };

    floatx16 acc[MI][2];
    gt::zero_acc(acc);
    // A step's four phases as in the forward product, the barrier between s = 2 and
    // 3: by then all of this step's dy and the next step's codes have been read.
    floatx4 sb[2][2];  // the scales of s in sb[s % 2]
    gt::Operands<MI> o;
    const auto expand = [&](const floatx4 (&f)[2], int t, const float2& l) {
      return gt::bf16_pair(l.x * f[t >> 1][2 * (t & 1)], l.y * f[t >> 1][2 * (t & 1) + 1]);
    };
    const auto even = [&](int, int t, const float2& l) { return expand(sb[0], t, l); };
    const auto odd = [&](int, int t, const float2& l) { return expand(sb[1], t, l); };
#pragma unroll
    for (int i = 0; i < MI; ++i) dma_dy(i, dst0);
    dma_scale(0);
    dma_scale(1);
#pragma unroll
    for (int i = 0; i < 4; ++i) dma_codes(i & 1, i >> 1);
    gt::wait_requests<0>();
    sk::wave_lds_order();
    put_scale(0);
    sk::lds_barrier();
    turn_half(0, cs_all[0]);
    turn_half(1, cs_all[0]);
    sk::lds_barrier();  // before the first codes are overwritten
#pragma unroll
    for (int i = 0; i < MI; ++i) dma_dy(i, dst1);
    dma_scale(2);
#pragma unroll
    for (int i = 0; i < 4; ++i) dma_codes(i & 1, i < 2 ? 2 : 0);
    const char* xa = xs0 + (lane & 31) * gt::kActRowBytes;
    read_scales(sb[0], 0, 0);
    read_scales(sb[1], 0, 1);
    gt::first_operands<MI, kC>(o, w, xa, sw, h4, tabc, slot, even);
    int next = 1;  // the stage of the next step's codes
    for (int ks = 0; ks < nk; ++ks) {
      gt::mfma_phase<MI, kC>(0, o, acc, w, 2, xa, 1, sw, h4, tabc, slot, odd, [&](int q) {
        if (q == 0) read_scales(sb[0], ks, 2);
      });
      gt::mfma_phase<MI, kC>(1, o, acc, w, 3, xa, 2, sw, h4, tabc, slot, even, [&](int q) {
        if (q == 0) read_scales(sb[1], ks, 3);
        if (q == 1) turn_half(0, cs_all[next]);
        if (q == 2) put_scale(ks + 1);
      });
      sk::wave_lds_order();
      gt::mfma_phase<MI, kC>(2, o, acc, w, 0, xa, 3, sw, h4, tabc, slot, odd, [&](int q) {
        if (q == 0) read_scales(sb[0], ks + 1, 0);
        if (q == 1) turn_half(1, cs_all[next]);
      });
      // the next step's dy is here, and the codes of the one after
      gt::wait_requests<2>();
      sk::lds_barrier();
      const uint32_t freed = (ks & 1) ? dst1 : dst0;
      xa = ((ks & 1) ? xs0 : xs1) + (lane & 31) * gt::kActRowBytes;
      gt::mfma_phase<MI, kC>(3, o, acc, w, 1, xa, 0, sw, h4, tabc, slot, even, [&](int q) {
        if (q == 0) read_scales(sb[1], ks + 1, 1);
        if (q < MI) dma_dy(q, freed);
        if (q == MI) dma_scale(ks + 3);
        if (q == MI + 1) {
          dma_codes(0, next);
          dma_codes(1, next);
        }
      });
      next = next == 2 ? 0 : next + 1;
    }
    gt::wait_requests<0>();
    sk::lds_barrier();  // the last reads of dy, before the next tile's is requested
    gt::store_acc<MI, true>(acc, a.dx, tile.hi, a.cols, tile.row0, k0, wave, lane);
  }
}

template <int MI>
hipError_t launch(const ExpertDxArgs& a, hipStream_t s) {
  const int64_t most = ((a.er.m + 32 * MI - 1) / (32 * MI) + a.er.experts) * ((a.cols + gt::kTileN - 1) / gt::kTileN);
  const int64_t slots = static_cast<int64_t>(device_cus()) * (MI == 2 ? 2 : 1);
  const dim3 gd(static_cast<unsigned>(most < slots ? most : slots)), bd(gt::kThreads);
  if (a.sc.absmax) hipLaunchKernelGGL((k_expert_gemm_dx<MI, false, false>), gd, bd, 0, s, a);
  else if (a.sc.f8) hipLaunchKernelGGL((k_expert_gemm_dx<MI, true, true>), gd, bd, 0, s, a);
  else hipLaunchKernelGGL((k_expert_gemm_dx<MI, true, false>), gd, bd, 0, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_expert_gemm_dx(const uint8_t* packed, int64_t rows, int64_t cols, Scales sc, const ExpertRows& er,
                                 const uint16_t* dy, uint16_t* dx, hipStream_t s) {
  // By the mean number of rows of an expert (the only one known here) and whether
  // about this many tiles of 64 rows occupy most compute units; if not, the kernel
  // that splits the reduction.  Measured in us, rows unevenly spread, stacks changing
  // from call to call: that kernel (k_expert_skinny_dx.hip), then tiles of 64 and of
  // 128 rows, and full rounds of 256 rows here:
  //   64 experts of 1024x2048,  mean  12:   48   31   42   34
  //                                   48:   61   44   66   47
  //                                  160:  126   89   90   93
  //                                  300:  188  148  134  136
  //   16 of 4096x4096,          mean   4:   57   65   67   68
  //                                   24:   93   83   74   87
  //                                  160:  193  179  144  182
  //                                  300:  282  277  225  219
  //   4 of 2048x8192,           mean  24:   28   37   38   40
  //                                   48:   44   36   40   40
  //   8 of 14336x4096,          mean  32:  186  208  209  212
  //                                  150:  307  281  218  285
  //                                  512:  874  704  678  589
  // (Where 64-row tiles fill one round and a little of the next, 128-row tiles are
  // faster from a lower mean on: 16 of 4096x4096 at 24, 12%.)
  const int64_t experts = er.experts, tiles_k = (cols + gt::kTileN - 1) / gt::kTileN;
  const int64_t about = ((er.m < experts ? er.m : experts) / 2 + er.m / 64) * tiles_k;
  if (8 * about < 5 * device_cus()) return launch_expert_skinny_dx(packed, rows, cols, sc, er, dy, dx, s);
  ExpertDxArgs a{};
  a.packed = packed; a.rows = rows; a.cols = cols; a.sc = sc; a.er = er; a.dy = dy; a.dx = dx;
  a.cb = codebook(sc.fp4);
  if (er.m <= 112 * experts) return launch<2>(a, s);
  if (er.m <= 224 * experts) return launch<4>(a, s);
  a.er.cover_slots = device_cus();
  a.er.cover_units = static_cast<int>(tiles_k);
  if (hipError_t e = launch<8>(a, s); e != hipSuccess) return e;
  return launch<2>(a, s);
}

}  // namespace nf4i
