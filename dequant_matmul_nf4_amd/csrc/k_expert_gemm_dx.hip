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
// The codes come from HBM and are requested three steps ahead, dy one.  As in the
// forward product, tiles are counted from the offsets, and of many rows full
// rounds of 256-row tiles go first and 64-row tiles take the rest.
//
// Bound: the matrix cores are busy 47% of the cycles, like the forward product's;
// a wave's waits for LDS and at barriers are 22%, its own instructions between
// the products the rest.  8192 rows over 8 experts of 14336x4096: 1140 us, 845
// TFLOP/s; 4096 over 64 of 1024x2048: 50 us.  Expanding to bfloat16 and turning
// that in LDS, 8 waves a tile, took 1240 and 85.
#include "expert_tiles.h"
#include "gemm_fwd.h"
#include "skinny_tile.h"

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

// Direct global-to-LDS loads of a wave: lane l's 16 (4, 1) bytes at base + off
// to lds + 16 l (4 l, 4 l).  Inline assembly, since the compiler lets every
// turn_codes wait for all loads to LDS that it knows of; the waits are counted
// by hand (wait_loads).
__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const char*)(const char*)p));
}
__device__ __forceinline__ void dma16(const void* base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base), "s"(lds) : "memory", "m0");
}
__device__ __forceinline__ void dma4(const void* base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dword %0, %1" ::"v"(off), "s"(base), "s"(lds) : "memory", "m0");
}
__device__ __forceinline__ void dma1(const void* base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_ubyte %0, %1" ::"v"(off), "s"(base), "s"(lds) : "memory", "m0");
}
// Until at most N of the wave's loads are on their way.
template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

__device__ __forceinline__ bf16x8 expand_rows(const float2 (&l)[4], const floatx4 (&s)[2]) {
  const u32x4 v = {gt::bf16_pair(l[0].x * s[0][0], l[0].y * s[0][1]), gt::bf16_pair(l[1].x * s[0][2], l[1].y * s[0][3]),
                   gt::bf16_pair(l[2].x * s[1][0], l[2].y * s[1][1]), gt::bf16_pair(l[3].x * s[1][2], l[3].y * s[1][3])};
  return __builtin_bit_cast(bf16x8, v);
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
  const uint32_t raw0 = lds_address(raw);
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
    // the lane's piece of a row of codes (pieces past the row's end repeat its
    // last: such columns are not stored)
    const uint32_t cp = static_cast<uint32_t>(k0 / 32) + ((lane & 7) ^ (lane >> 3));
    const uint32_t coff = (cp < row_bytes / 16 ? cp : row_bytes / 16 - 1) * 16 + (16 * wave + (lane >> 3)) * row_bytes;
    uint32_t off[MI];
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const int r = 8 * (MI * wave + i) + (lane >> 3);
      off[i] = static_cast<uint32_t>(r < cnt ? r : cnt - 1) * ld + (gt::act_piece(MI * wave + i, lane) << 4);
    }
    // Requests past the weight's rows repeat the last ones (of dy the last 8 of
    // the same row); their scales are 0.  Past the last step they repeat it.
    auto dma_dy = [&](char* stage) {
      const uint32_t to = lds_address(stage) + MI * wave * 1024;
      if (dy_left >= kStep) {
#pragma unroll
        for (int i = 0; i < MI; ++i) dma16(dyp, off[i], to + i * 1024);
      } else {
        const int l2 = opaque(lane);
#pragma unroll
        for (int i = 0; i < MI; ++i) {
          const int r = 8 * (MI * wave + i) + (l2 >> 3), piece = gt::act_piece(MI * wave + i, l2), last = dy_left / 8 - 1;
          dma16(dyp, static_cast<uint32_t>(r < cnt ? r : cnt - 1) * ld + ((piece < last ? piece : last) << 4), to + i * 1024);
        }
      }
      if (dy_left > kStep) {
        dyp += kStep * 2;
        dy_left -= kStep;
      }
    };
    auto dma_codes = [&](int stage) {
      const uint32_t to = lds_address(cs_all[0]) + stage * kCodeStage + 2 * wave * 1024;
      if (co_left >= kStep) {
#pragma unroll
        for (int i = 0; i < 2; ++i) dma16(cop, coff + i * 8 * row_bytes, to + i * 1024);
      } else {
        const int l2 = opaque(lane);
        const uint32_t at = coff - (16 * wave + (lane >> 3)) * row_bytes;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = 16 * wave + 8 * i + (l2 >> 3);
          dma16(cop, at + static_cast<uint32_t>(r < co_left ? r : co_left - 1) * row_bytes, to + i * 1024);
        }
      }
      if (co_left > kStep) {
        cop += kStep * static_cast<int64_t>(row_bytes);
        co_left -= kStep;
      }
    };
    // lane n: the scale of the step's weight row n in the wave's block
    auto dma_scale = [&](int ks) {
      const uint32_t to = raw0 + (ks & 1) * sizeof(raw_all[0][0]);
      const uint32_t o = static_cast<uint32_t>(lane < sc_left ? lane : sc_left - 1) * nblk;
      if constexpr (kDQ) {
        dma1(a.sc.q + blk, o, to);
        dma4(a.sc.absmax2 + (blk >> 8), (static_cast<uint32_t>(blk & 255) + o) >> 8 << 2, to + 4 * kStep);
      } else {
        dma4(a.sc.absmax + blk, o << 2, to);
      }
      if (sc_left > kStep) {
        blk += kStep * static_cast<int64_t>(nblk);
        sc_left -= kStep;
      }
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
    auto turn_step = [&](u32x4 (&w)[2], const char* stage) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint2 lo = turn_codes(stage + (turn ^ (16 * j))), hi = turn_codes(stage + (turn ^ (16 * j)) + 16 * kCodeRow);
        w[j] = u32x4{lo.x, lo.y, hi.x, hi.y};
      }
    };

    floatx16 acc[MI][2];
    gt::zero_acc(acc);
    constexpr int kV = 24 / MI, kL = MI == 8 ? 2 : 8 / MI + 1;
    // As the forward product's loop, and the codes come three steps ahead: while
    // step k is multiplied, those of k + 1 are turned, those of k + 2 and k + 3 and
    // dy of k + 1 are on their way.  The wait at its end leaves the youngest.
    constexpr int kYoungest = 2 + (kDQ ? 2 : 1);
    u32x4 wc[2], wn[2];
    dma_dy(xs0);
    dma_codes(0);
    dma_codes(1);
    dma_scale(0);
    dma_scale(1);
    wait_loads<0>();
    sk::wave_lds_order();
    put_scale(0);
    sk::wave_lds_order();
    dma_codes(2);
    dma_scale(2);
    floatx4 sb[2][2];
    bf16x8 bf[2][2];
    gt::Lookups lk[3];
    bf16x8 af[3][MI];
    sk::lds_barrier();
    turn_step(wc, cs_all[0]);
    read_scales(sb[0], 0, 0);
    read_scales(sb[1], 0, 1);
    gt::lookup_step<kC>(lk[0], wc, 0, tabc, slot);
    bf[0][0] = expand_rows(lk[0].l[0], sb[0]);
    bf[0][1] = expand_rows(lk[0].l[1], sb[0]);
    sk::lds_barrier();  // before the first codes are overwritten
    int free = 0;   // the codes' stage of step ks, ks % 3
    for (int ks = 0; ks < nk; ++ks) {
      dma_dy((ks & 1) ? xs0 : xs1);
      dma_codes(free);
      free = free == 2 ? 0 : free + 1;
      __builtin_amdgcn_sched_barrier(0);
      const char* xa = ((ks & 1) ? xs1 : xs0) + (lane & 31) * gt::kActRowBytes;
      gt::read_act(xa, 0, sw, h4, af[0]);
      gt::read_act(xa, 1, sw, h4, af[1]);
      gt::lookup_step<kC>(lk[1], wc, 1, tabc, slot);
      __builtin_amdgcn_sched_barrier(0);
      // s = 0
      gt::mfma16(af[0], bf[0], acc);
      bf[1][0] = expand_rows(lk[1].l[0], sb[1]);
      bf[1][1] = expand_rows(lk[1].l[1], sb[1]);
      gt::read_act(xa, 2, sw, h4, af[2]);
      gt::lookup_step<kC>(lk[2], wc, 2, tabc, slot);
      read_scales(sb[0], ks, 2);
      gt::mfma_interleave<2 * MI, kV, kL>();
      __builtin_amdgcn_sched_barrier(0);
      sk::wave_lds_order();
      put_scale(ks + 1);
      sk::wave_lds_order();
      dma_scale(ks + 3);
      // s = 1
      gt::mfma16(af[1], bf[1], acc);
      bf[0][0] = expand_rows(lk[2].l[0], sb[0]);
      bf[0][1] = expand_rows(lk[2].l[1], sb[0]);
      gt::read_act(xa, 3, sw, h4, af[0]);
      gt::lookup_step<kC>(lk[0], wc, 3, tabc, slot);
      read_scales(sb[1], ks, 3);
      gt::mfma_interleave<2 * MI, kV, kL>();
      __builtin_amdgcn_sched_barrier(0);
      // s = 2, with the next step's codes
      gt::mfma16(af[2], bf[0], acc);
      bf[1][0] = expand_rows(lk[0].l[0], sb[1]);
      bf[1][1] = expand_rows(lk[0].l[1], sb[1]);
      turn_step(wn, cs_all[free]);
      read_scales(sb[0], ks + 1, 0);
      gt::mfma_interleave<2 * MI, kV, kL>();
      __builtin_amdgcn_sched_barrier(0);
      // s = 3, with the next step's s = 0 expansion
      gt::mfma16(af[0], bf[1], acc);
      gt::lookup_step<kC>(lk[1], wn, 0, tabc, slot);
      bf[0][0] = expand_rows(lk[1].l[0], sb[0]);
      bf[0][1] = expand_rows(lk[1].l[1], sb[0]);
      read_scales(sb[1], ks + 1, 1);
      gt::mfma_interleave<2 * MI, kV, kL>();
      __builtin_amdgcn_sched_barrier(0);
      wait_loads<kYoungest>();
      sk::lds_barrier();
      wc[0] = wn[0];
      wc[1] = wn[1];
    }
    wait_loads<0>();
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
  // about this many tiles of 64 rows give every compute unit one; where the
  // reduction is long, an emptier last round costs more than what the kernel that
  // splits it (k_expert_skinny_dx.hip) loses.  Measured in us: that kernel, then
  // tiles of 64 and of 128 rows, and full rounds of 256 rows here:
  //   64 experts of 1024x2048,  mean  12:   48   33   52   35
  //                                   48:   61   50   79   53
  //                                  160:  126   98  107  102
  //                                  300:  188  160  159  146
  //   16 of 4096x4096,          mean  24:   93   97   90  100
  //                                  160:  193  197  176  200
  //                                  300:  282  301  265  241
  //   4 of 2048x8192,           mean  24:   28   43   49   46
  //                                   96:   63   43   51   46
  //   8 of 14336x4096,          mean  64:  210  253  289  257
  //                                  256:  470  536  571  540
  //                                 1024: 1437 1541 1454 1138
  const int64_t experts = er.experts, tiles_k = (cols + gt::kTileN - 1) / gt::kTileN;
  const int64_t about = ((er.m < experts ? er.m : experts) / 2 + er.m / 64) * tiles_k;
  if (about < device_cus() * (rows > 8192 ? 3 : 1)) return launch_expert_skinny_dx(packed, rows, cols, sc, er, dy, dx, s);
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
