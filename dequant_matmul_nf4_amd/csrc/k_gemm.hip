// Dequantize-and-multiply bf16 matrix-core GEMM with an optional fused LoRA
// term:
//   y = x . deq(W)^T + s . (x . A^T) . B^T
// (bitsandbytes tool page, "How it works", Step 5: matrix hardware works best
// on 16-bit numbers, so each block is expanded to 16-bit and multiplied; the
// tutorial page, "QLoRA: Fine-Tuning a 4-bit Model": low-rank adapters on the
// frozen 4-bit base, their output multiplied by a scale factor.)
//
// Tiling: a workgroup of 4 waves computes a (32 MI) x 256 tile of y.  Wave w
// owns the 64 output columns [64 w, 64 w + 64) for all 32 MI rows: MI x 2
// tiles of v_mfma_f32_32x32x16_bf16 per 16-wide k step (MI = 8: 256 fp32
// accumulators per lane).  A K step covers 64 columns, exactly one NF4 block
// of every weight row.  Within a step the LDS reads of 16-wide k step s + 1 (x
// fragments and level lookups) are issued before the MFMAs of k step s, so
// their latency is spent while the matrix cores run.
//
// Work units: the persistent workgroups take 256-row tiles round by round.
// When the last round would leave compute units idle (its tiles number at
// most half the workgroups), each of its tiles is cut into two 128-row halves
// (MI = 4) taken by two workgroups: a half costs more than half a tile (its
// weight tile is expanded for half as many rows) but the round ends sooner.
//
// Operands:
//  - x: the (32 MI) x 64 tile is staged in LDS (two stages of 128-byte rows) by
//    direct global-to-LDS loads (global_load_lds_dwordx4: each wave
//    instruction fills 1 KB, lane l at byte 16 l), issued at the top of the
//    previous step.  16-byte piece p of row r sits at slot p ^ ((r / 2) % 8),
//    so the fragment reads of 16 consecutive rows hit distinct banks.
//  - W: never staged.  Each lane loads the 16 bytes of codes it needs
//    (32 consecutive k of one row) and expands them straight into its MFMA
//    B fragments: a byte (two codes) indexes a 256-entry table of float32
//    level pairs in LDS (kCopies interleaved copies, lane slot
//    lane % kCopies, so the lanes served together hit distinct banks), each
//    level is multiplied by the block scale and the pair rounded once to bf16
//    -- the same value nf4_dequantize writes.  The next step's codes are
//    loaded one step ahead.
//  - The k index of a lane's fragment is a permutation of the step's 64
//    columns (lane half h takes columns 32 h .. 32 h + 31, eight per 16-wide
//    k step); A and B fragments use the same one, so the sum is unchanged.
//
// LoRA: the low-rank term is folded in as extra K columns,
//   [x | s T_hi | s T_lo] . [deq(W) | B | B]^T  with T = x . A^T,
// where s T is split into two bf16 parts (hi = bf16(sT), lo = bf16(sT - hi))
// by the LoRA prep kernel, so the adapter product keeps about 16 significant
// bits.  Those columns (2 r rounded up to a multiple of 64) run as one or two
// more K steps: the x side through the same staged tile, the W side
// [B | B | 0] (laid out row by row in the workspace by k_lora_bx) loaded
// straight into fragments.
#include "gemm_fwd.h"

namespace nf4i {
namespace {

using gt::bf16x8;
using gt::floatx16;
using gt::kCopies;
using gt::kThreads;

constexpr int kBN = gt::kTileN, kBK = gt::kStep;
// The configuration the launcher uses: 256-row tiles and 32 copies of the
// pair table (x stages 64 KB + table 64 KB), one workgroup per compute unit.
// (128-row tiles with two workgroups per compute unit measured slower: each
// weight tile is then expanded for half as many rows.)
constexpr int kMI = 8;
constexpr int kWgPerCu = 1;
constexpr int kBM = 32 * kMI;
constexpr int kStageBytes = gt::act_stage_bytes<kBM>();

struct GemmArgs {
  const uint8_t* packed;
  int64_t rows, cols;    // W [rows][cols]; y has `rows` columns
  Scales sc;
  const uint16_t* x;     // [m][cols]
  int64_t m;
  uint16_t* y;           // [m][rows]
  const uint16_t* u;     // LoRA columns of x: [m][kl] (s T hi | s T lo | 0), or null
  const uint16_t* bx;    // LoRA columns of W: [rows][kl] (B | B | 0)
  int kl;                // extra K (multiple of 64), 0 without LoRA
  int64_t whole;         // work units 0 .. whole - 1: tile u, all 256 rows
  int64_t units;         // units whole .. units - 1: tile whole + (u - whole) / 2, half (u - whole) % 2
  Codebook cb;
};

// One work unit: the (32 MI) x 256 tile of y at rows m0.., columns n0..
// (MI = 8: a whole tile; MI = 4: half of one).  Every LDS stage read here is
// read before a barrier that all waves pass before the unit returns.
template <int MI, bool kDQ, bool kF8>
__device__ __forceinline__ void gemm_unit(const GemmArgs& a, int64_t m0, int64_t n0, char* xs0, char* xs1,
                                          const char* tabc, uint32_t slot, float mean, int wave, int lane) {
  const int64_t nk = a.cols / kBK;
  const gt::ActPtrs<MI> xp = gt::make_act_ptrs<MI, 32 * MI>(a.x, a.cols, a.m, m0, wave, lane);
  gt::WPtrs wp;
  int64_t nrow[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int64_t n = n0 + wave * 64 + j * 32 + (lane & 31);
    nrow[j] = n < a.rows ? n : a.rows - 1;  // rows past the end: never stored
    wp.c[j] = a.packed + nrow[j] * (a.cols / 2) + (lane >> 5) * 16;
    wp.blk[j] = nrow[j] * (a.cols / 64);
  }

  floatx16 acc[MI][2];
  gt::zero_acc(acc);

  gt::fwd_steps<MI, kDQ, kF8>(
      a.sc, nk, [&](int64_t ks, char* stage) { gt::dma_act(xp, ks, stage, wave); }, wp, xs0, xs1, tabc, slot, mean, lane, acc);
  if (a.kl > 0) {
    // LoRA K steps: u through the x stage, [B | B | 0] rows straight into fragments
    const gt::ActPtrs<MI> up = gt::make_act_ptrs<MI, 32 * MI>(a.u, a.kl, a.m, m0, wave, lane);
    const uint32_t sw = ((lane & 31) >> 1) & 7, h4 = (lane >> 5) * 4;
    for (int64_t k0 = 0; k0 < a.kl; k0 += kBK) {
      gt::dma_act(up, k0 / kBK, xs0, wave);  // xs0 was last read before the previous barrier
      bf16x8 bl[4][2];
#pragma unroll
      for (int s4 = 0; s4 < 4; ++s4)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          bl[s4][j] = *reinterpret_cast<const bf16x8*>(a.bx + nrow[j] * a.kl + k0 + h4 * 8 + 8 * s4);
      gt::wait_vmem();
      __syncthreads();
      const char* xa = xs0 + (lane & 31) * gt::kActRowBytes;
#pragma unroll
      for (int s4 = 0; s4 < 4; ++s4) {
        bf16x8 af[MI];
        gt::read_act(xa, s4, sw, h4, af);
        gt::mfma16(af, bl[s4], acc);
      }
      __syncthreads();
    }
  }

  gt::store_acc(acc, a.y, a.m, a.rows, m0, n0, wave, lane);
}

template <bool kDQ, bool kF8>
__global__ __launch_bounds__(kThreads, kWgPerCu) void k_gemm(GemmArgs a) {
  __shared__ __align__(16) char xs0[kStageBytes], xs1[kStageBytes];
  __shared__ __align__(16) float2 tab[256 * kCopies];
  const char* tabc = reinterpret_cast<const char*>(tab);
  const int t = threadIdx.x;
  const int lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  constexpr int kShift = kCopies == 32 ? 0 : kCopies == 16 ? 1 : 2;
  const uint32_t slot = static_cast<uint32_t>(lane & (kCopies - 1)) << (3 + kShift);

  gt::fill_level_pairs<kCopies>(tab, a.cb);  // once per workgroup; ends with a barrier
  const float mean = kDQ ? *a.sc.mean : 0.0f;
  const int64_t tiles_n = (a.rows + kBN - 1) / kBN;
  const int64_t tiles = tiles_n * ((a.m + kBM - 1) / kBM);

  // Persistent: the grid holds the resident workgroups and each takes units
  // blockIdx.x, blockIdx.x + gridDim.x, ...  Tile order: dispatch deals
  // workgroups round-robin over the 8 XCDs, so the workgroups of one XCD
  // that run at the same time get neighbouring tiles along N and share x rows.
  for (int64_t u = blockIdx.x; u < a.units; u += gridDim.x) {
    const bool half = u >= a.whole;
    const int64_t tile = half ? a.whole + (u - a.whole) / 2 : u;
    int64_t tid = tile;
    if (tiles % 8 == 0) tid = (tile % 8) * (tiles / 8) + tile / 8;
    const int64_t m0 = (tid / tiles_n) * kBM;
    const int64_t n0 = (tid % tiles_n) * kBN;
    if (!half) {
      gemm_unit<kMI, kDQ, kF8>(a, m0, n0, xs0, xs1, tabc, slot, mean, wave, lane);
    } else {
      const int64_t mh = m0 + ((u - a.whole) & 1) * (kBM / 2);
      if (mh < a.m) gemm_unit<kMI / 2, kDQ, kF8>(a, mh, n0, xs0, xs1, tabc, slot, mean, wave, lane);
    }
  }
}

// bx[n][c] = (B | B | 0)[n][c] for c < kl: B[n][c] for c < r, B[n][c - r_pad]
// for r_pad <= c < r_pad + r, zero elsewhere.
__global__ __launch_bounds__(256) void k_lora_bx(const uint16_t* __restrict__ lb, int64_t rows, int r, int r_pad,
                                                 int kl, uint16_t* __restrict__ bx) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i >= rows * kl) return;
  const int64_t n = i / kl;
  const int c = static_cast<int>(i - n * kl);
  const int j = c < r_pad ? c : c - r_pad;
  const bool live = c < 2 * r_pad && j < r;
  bx[i] = live ? lb[n * r + j] : static_cast<uint16_t>(0);
}

}  // namespace

size_t gemm_lora_cols(int r) {
  if (r <= 0) return 0;
  const int r_pad = (r + 15) / 16 * 16;
  return static_cast<size_t>((2 * r_pad + kBK - 1) / kBK * kBK);
}

size_t gemm_workspace(int64_t m, int64_t rows, int r) {
  if (r <= 0) return 0;
  const size_t kl = gemm_lora_cols(r);
  const size_t ub = (static_cast<size_t>(m) * kl * sizeof(uint16_t) + 255) & ~size_t(255);
  return ub + static_cast<size_t>(rows) * kl * sizeof(uint16_t);
}

hipError_t launch_gemm(const uint8_t* packed, int64_t rows, int64_t cols, Scales sc, const uint16_t* x,
                       int64_t m, uint16_t* y, const uint16_t* lora_a, const uint16_t* lora_b, int r,
                       float lora_scale, uint16_t* u_ws, hipStream_t s) {
  GemmArgs a{};
  a.packed = packed; a.rows = rows; a.cols = cols; a.sc = sc; a.x = x; a.m = m; a.y = y;
  a.cb = codebook(sc.fp4);
  if (r > 0) {
    const int r_pad = (r + 15) / 16 * 16;
    a.kl = static_cast<int>(gemm_lora_cols(r));
    a.u = u_ws;
    uint16_t* bx = u_ws + ((static_cast<size_t>(m) * a.kl * sizeof(uint16_t) + 255) & ~size_t(255)) / sizeof(uint16_t);
    a.bx = bx;
    const int64_t nb = rows * a.kl;
    if ((nb + 255) / 256 > 0x7FFFFFFF) return hipErrorInvalidValue;
    hipLaunchKernelGGL(k_lora_bx, dim3(static_cast<unsigned>((nb + 255) / 256)), dim3(256), 0, s, lora_b, rows, r,
                       r_pad, a.kl, bx);
    if (hipError_t e = launch_lora_u(x, lora_a, m, cols, r, lora_scale, u_ws, s)) return e;
  }
  const int64_t tiles = ((rows + kBN - 1) / kBN) * ((m + kBM - 1) / kBM);
  const int64_t slots = kWgPerCu * device_cus();  // resident workgroups
  // Tiles of the last round (all of them when they fill less than one): cut
  // into halves when those fit in one round and the tiles have more than 128 rows.
  const int64_t last = tiles - tiles / slots * slots;
  const bool halve = last > 0 && 2 * last <= slots && m > kBM / 2;
  a.whole = halve ? tiles - last : tiles;
  a.units = halve ? tiles + last : tiles;
  const unsigned grid = static_cast<unsigned>(a.units < slots ? a.units : slots);
  if (sc.absmax) hipLaunchKernelGGL((k_gemm<false, false>), dim3(grid), dim3(kThreads), 0, s, a);
  else if (sc.f8) hipLaunchKernelGGL((k_gemm<true, true>), dim3(grid), dim3(kThreads), 0, s, a);
  else hipLaunchKernelGGL((k_gemm<true, false>), dim3(grid), dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace nf4i
