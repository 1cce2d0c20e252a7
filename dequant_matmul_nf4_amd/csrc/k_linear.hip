// A layer's product with its epilogue for many rows of x (prompts, training):
//
//   z = x . deq(W)^T + s (x . A^T) . B^T + bias;   y = act(z) + residual
//
// Operands are float16: a weight is the product of its level, rounded to
// float16, and its block scale times a power of two of its row's own, rounded to
// float16 -- one packed multiplication for two weights, whose three roundings (at
// most 3 2^-11) are well below the one to bf16 of the dense GEMM (2^-8 at most),
// whose expansion costs twice the instructions.  x becomes float16 exactly in a
// small kernel before this one, scaled by a power of two per row.  Both powers
// are taken back on the finished sums.  Blocks whose scale is 2^-24 of the
// row's largest and below lose bits, and so do values of x 2^-29 of their row's
// largest and below.
//
// The K loop's schedule, work units and stages are those of the forward GEMM
// (k_gemm.hip).  The adapters are extra K columns in bf16 (s T in two parts), as
// there; their operands come straight from memory, B from its own rows, and are
// brought to the sums' powers of two.
//
// The epilogue: the matrix cores leave a lane with 4 consecutive columns of 32
// rows, 8 bytes of bf16 each, which as they are would touch a line of memory per
// row with every store.  A wave turns its 64 columns in LDS instead, 64 rows at a
// time in a quarter of the stages that is its own (free after the last step), and
// takes them back as 8 columns of 8 rows, so that residual, pre and y move in
// whole lines and the lane's bias stays in registers.  16-byte piece p of row r
// sits at slot p ^ (r % 16): no two rows of a store meet in a bank.
//
// Measured: 4096 rows of 14336x4096 with adapters, bias, pre and gelu_tanh 559 us (860
// TFLOP/s; weights rounded to bf16 instead 10 us more), 504 for the whole call without
// any of them.  The dense GEMM takes 485 with the same adapters and 467 without, and a
// pass over y and pre 56 to 71: the fusion saves no time here, it keeps the precision.
// Issue bounds it: the matrix cores are busy 40% of the cycles, at 2.05 GHz,
// beside 3.3 vector and 1.1 LDS instructions a product.  Eight waves in place of four,
// and that work pinned between the products as k_linear_mid.hip has it, were slower.
#include "gemm_tiles.h"
#include "linear_epilogue.h"
#include "linear_f16.h"

namespace nf4i {
namespace {

using gt::bf16x8;
using gt::floatx16;
using gt::kThreads;

constexpr int kBN = gt::kTileN, kBK = gt::kStep;
constexpr int kMI = 8;
// Which kernels take m rows of x.  A decode batch, and as many more as leave little work for a
// workgroup (in tiles of 16 x 16 outputs, each with about 512 columns' worth of its own): the codes
// streamed past x as it is, in one launch instead of two or three.  Measured against the best of the
// others, us: 4096x4096 with 128 rows 24 and 30, with 192 43 and 34; 28672x8192 with 16 rows 42 and 61,
// with 32 69 and 60; 1024x4096 with 512 rows 27 and 35, with 768 44 and 36; 4096x64 with 512 rows 14 and
// 19, with 1024 23 and 19; 512x512 with 64 rows 5 and 20.
// For a full chip, whatever the device: what a call needs of its workspace and how it rounds the
// weight follow from the sizes alone.
constexpr int64_t kChip = 256;
bool few(int64_t m, int64_t rows, int64_t cols) {
  const int64_t groups = (rows + 15) / 16, tiles = (m + 15) / 16;
  if (tiles == 1) return true;
  if (tiles > kChip) return false;
  const int64_t each = (groups + kChip / tiles - 1) / (kChip / tiles);
  return each * (cols + 512) <= 40960;
}
// Up to about 96 of this file's tiles, fewer of short rows: the kernel that cuts the reduction
// (k_linear_mid.hip).  There and here, us: 14336x4096 with 384 rows (84 tiles) 79 and 97, with 512 (112)
// 115 and 100; 28672x8192 with 192 rows (84) 131 and 185, with 256 (112) 188 and 185; 4096x14336 with 1024
// (64) 190 and 292; 4096x1024 with 768 (48) 28 and 35, with 1024 (64) 46 and 35; 14336x256 with 192 (42)
// 21 and 22, with 256 (56) 34 and 23.
bool mid(int64_t m, int64_t rows, int64_t cols) {
  const int64_t most = cols >= 3584 ? 96 : 40 + cols / 64;
  return cols >= 256 && m <= 65536 && m <= (most * 65536 + rows - 1) / rows;
}
constexpr int kBM = 32 * kMI;
constexpr int kStageBytes = gt::act_stage_bytes<kBM>();
constexpr int kTurnRows = 64;
static_assert(kTurnRows * 64 * 4 * 4 == 2 * kStageBytes, "four waves' quarters fill both stages");

struct LinearArgs {
  const uint8_t* packed;
  int64_t rows, cols;
  Scales sc;
  const uint16_t* x;   // x in float16 blocks (launch_linear_prep), row t scaled by 2^-xe[t]
  const int32_t *xe, *we;
  int64_t m;
  uint16_t* y;
  Epilogue ep;
  const uint16_t* u;   // adapter columns of x: [m][kl] (s T hi | s T lo | 0)
  const uint16_t* lb;  // B [rows][r]
  int r, r_pad, kl;    // 0 without adapters
  int64_t whole, units;  // as in the forward GEMM
  Codebook cb;
};

// The adapters' share of the sums, brought to their powers of two.  Lane half h
// takes columns c + 8 h .. + 7 of each 16.
template <int MI>
__device__ __forceinline__ void adapters(floatx16 (&acc)[MI][2], const LinearArgs& a, int64_t m0, const int64_t (&nrow)[2],
                                         const int (&we)[2], int lane) {
  if (a.r == 0) return;
  int64_t tc[MI];
  float by[MI];
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    const int64_t t = m0 + 32 * i + (lane & 31);
    tc[i] = t < a.m ? t : a.m - 1;
    by[i] = f16::power(-a.xe[tc[i]]);
  }
  for (int c = 0; c < 2 * a.r_pad; c += 16) {
    const int ch = c + 8 * (lane >> 5);
    gt::u32x4 v[MI];
#pragma unroll
    for (int i = 0; i < MI; ++i) v[i] = *reinterpret_cast<const gt::u32x4*>(a.u + tc[i] * a.kl + ch);
    bf16x8 bl[2], uf[MI];
#pragma unroll
    for (int j = 0; j < 2; ++j) bl[j] = lin::adapter_w(a.lb, a.r, a.r_pad, nrow[j], ch, f16::power(-we[j]));
#pragma unroll
    for (int i = 0; i < MI; ++i) uf[i] = lin::times(v[i], by[i]);
    gt::mfma16(uf, bl, acc);
  }
}

template <int MI>
__device__ __forceinline__ void epilogue(const floatx16 (&acc)[MI][2], const LinearArgs& a, int64_t m0, int64_t n0,
                                         const int (&we)[2], char* turn, int wave, int lane) {
  const int64_t col = n0 + wave * 64 + 8 * (lane & 7);
  const bool vec = (a.rows & 7) == 0;  // every row of the outputs 16-byte aligned
  const int left = static_cast<int>(a.rows - col < 8 ? a.rows - col : 8);
  float bias[8];
  lin::load_bias(bias, a.ep, col, left);
  // exponents of the weight rows that a lane's sums belong to: 4 consecutive ones per group
#pragma unroll
  for (int j = 0; j < 2; ++j) reinterpret_cast<int*>(turn)[32 * j + (lane & 31)] = we[j];
  f16::wave_lds_order();
  int4 wex[2][4];
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int g = 0; g < 4; ++g) wex[j][g] = *reinterpret_cast<const int4*>(turn + 4 * (32 * j + 8 * g + 4 * (lane >> 5)));
  f16::wave_lds_order();
#pragma unroll
  for (int rd = 0; rd < MI / 2; ++rd) {
    int xe[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t t = m0 + 64 * rd + 32 * i + (lane & 31);
      xe[i] = a.xe[t < a.m ? t : a.m - 1];
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int row = 32 * i + (lane & 31), p = 8 * j + 2 * g + (lane >> 5);
          const floatx16& s = acc[2 * rd + i][j];
          // the powers of two taken back
          *reinterpret_cast<float4*>(turn + row * 256 + ((p ^ (row & 15)) << 4)) =
              make_float4(__builtin_amdgcn_ldexpf(s[4 * g], xe[i] + wex[j][g].x), __builtin_amdgcn_ldexpf(s[4 * g + 1], xe[i] + wex[j][g].y),
                          __builtin_amdgcn_ldexpf(s[4 * g + 2], xe[i] + wex[j][g].z), __builtin_amdgcn_ldexpf(s[4 * g + 3], xe[i] + wex[j][g].w));
        }
    f16::wave_lds_order();
#pragma unroll 1
    for (int it = 0; it < 8; ++it) {
      const int row = 8 * it + (lane >> 3), p = 2 * (lane & 7);
      const int64_t t = m0 + 64 * rd + row;
      const float4 lo = *reinterpret_cast<const float4*>(turn + row * 256 + ((p ^ (row & 15)) << 4));
      const float4 hi = *reinterpret_cast<const float4*>(turn + row * 256 + (((p + 1) ^ (row & 15)) << 4));
      if (t >= a.m || left <= 0) continue;
      float v[8] = {lo.x + bias[0], lo.y + bias[1], lo.z + bias[2], lo.w + bias[3],
                    hi.x + bias[4], hi.y + bias[5], hi.z + bias[6], hi.w + bias[7]};
      lin::finish8(a.ep, a.y, t * a.rows + col, v, left, vec && left == 8);
    }
    f16::wave_lds_order();
  }
}

// The codes a lane expands in one K step: for its two weight rows (j = 0, 1) the
// 16 bytes of columns 32 h .. 32 h + 31, and the rows' block scale inputs.
struct WRegs {
  gt::u32x4 w[2];
  float am[2];
  int q[2];
  float s2[2];
};

struct WPtrs {
  const uint8_t* c[2];
  int64_t blk[2];
};

template <bool kDQ>
__device__ __forceinline__ void load_w(WRegs& r, const WPtrs& p, const Scales& sc, int64_t ks) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    r.w[j] = *reinterpret_cast<const gt::u32x4*>(p.c[j] + ks * (kBK / 2));
    const int64_t blk = p.blk[j] + ks;
    if constexpr (kDQ) {
      r.q[j] = sc.q[blk];
      r.s2[j] = sc.absmax2[blk >> 8];
    } else {
      r.am[j] = sc.absmax[blk];
    }
  }
}

// The float16 scales of the lane's two blocks, twice each.
template <bool kDQ, bool kF8>
__device__ __forceinline__ void block_scales(const WRegs& r, float mean, const float (&up)[2], f16::half2 (&sa)[2]) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    float s;
    if constexpr (kDQ) s = (code_ratio(r.q[j], kF8 ? 1 : 0) * r.s2[j]) + mean;  // a_hat, three roundings
    else s = r.am[j];
    sa[j] = f16::twice(s * up[j]);
  }
}

// Level pairs of code bytes 4 s .. 4 s + 3 of the lane's 16 bytes of both rows.
struct Lookups {
  uint32_t l[2][4];
};
__device__ __forceinline__ void lookup_step(Lookups& lk, const gt::u32x4 (&w)[2], int s, const char* tab, uint32_t slot) {
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int b = 0; b < 4; ++b) lk.l[j][b] = f16::look_up(w[j][s], b, tab, slot);
}

template <int MI>
__device__ __forceinline__ void mfma16(const f16::halfx8 (&af)[MI], const f16::halfx8 (&bf)[2], floatx16 (&acc)[MI][2]) {
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    acc[i][0] = __builtin_amdgcn_mfma_f32_32x32x16_f16(bf[0], af[i], acc[i][0], 0, 0, 0);
    acc[i][1] = __builtin_amdgcn_mfma_f32_32x32x16_f16(bf[1], af[i], acc[i][1], 0, 0, 0);
  }
}

// Stage layout: as x16's, 4 KB for each 32 rows, of 4 blocks of 1 KB.
template <int MI>
__device__ __forceinline__ void read_act(const char* xa, int s, f16::halfx8 (&f)[MI]) {
#pragma unroll
  for (int i = 0; i < MI; ++i) f[i] = *reinterpret_cast<const f16::halfx8*>(xa + (4 * i + s) * 1024);
}

// The tile's x of one step: wave w moves 32-row blocks w MI / 4 .. (MI of 1 KB each
// instruction); rows past the last 32 of x16 repeat them (never stored).
template <int MI>
struct XTile {
  const char* base;
  int64_t band;    // bytes of a 32-row band
  int64_t first, last;
};
template <int MI>
__device__ __forceinline__ void dma_x(const XTile<MI>& x, int64_t ks, char* stage, int wave, int lane) {
#pragma unroll
  for (int q = 0; q < MI; ++q) {
    const int b = MI * wave + q;  // block of the stage
    const int64_t band = x.first + b / 4 < x.last ? x.first + b / 4 : x.last;
    gt::dma16(reinterpret_cast<const uint8_t*>(x.base + band * x.band + ks * 4096 + (b & 3) * 1024 + lane * 16), stage + b * 1024);
  }
}

// Per MFMA of a 16-wide k step: V VALU operations and L LDS reads of the next.
template <int N, int V, int L>
__device__ __forceinline__ void interleave() {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    __builtin_amdgcn_sched_group_barrier(0x002, V, 0);
    __builtin_amdgcn_sched_group_barrier(0x080, L, 0);
  }
}

// acc += x16 . w16^T over nk steps, two LDS stages, software-pipelined as in the
// forward GEMM: while the products of 16-wide step s run, the weights of s + 1
// are multiplied out and those of s + 2 looked up.
template <int MI, bool kDQ, bool kF8>
__device__ __forceinline__ void steps(const LinearArgs& a, const XTile<MI>& xp, const WPtrs& wp, const float (&up)[2], char* xs0,
                                      char* xs1, const char* tabc, uint32_t slot, float mean, int wave, int lane,
                                      floatx16 (&acc)[MI][2]) {
  constexpr int kV = 16 / MI > 1 ? 16 / MI : 1, kL = 8 / MI;
  const int64_t nk = a.cols / kBK;
  WRegs wc, wnx;
  dma_x(xp, 0, xs0, wave, lane);
  load_w<kDQ>(wc, wp, a.sc, 0);
  f16::half2 sa[2];
  f16::halfx8 bf[2][2];
  Lookups lk[3];
  f16::halfx8 af[3][MI];
  block_scales<kDQ, kF8>(wc, mean, up, sa);
  lookup_step(lk[0], wc.w, 0, tabc, slot);
  bf[0][0] = f16::expand(lk[0].l[0], sa[0]);
  bf[0][1] = f16::expand(lk[0].l[1], sa[1]);
  gt::wait_vmem();
  __syncthreads();
  for (int64_t ks = 0; ks < nk; ++ks) {
    const int64_t kn = ks + 1 < nk ? ks + 1 : ks;
    dma_x(xp, kn, (ks & 1) ? xs0 : xs1, wave, lane);  // the other stage was last read before the previous barrier
    load_w<kDQ>(wnx, wp, a.sc, kn);
    __builtin_amdgcn_sched_barrier(0);
    const char* xa = ((ks & 1) ? xs1 : xs0) + 16 * lane;
    read_act(xa, 0, af[0]);
    read_act(xa, 1, af[1]);
    lookup_step(lk[1], wc.w, 1, tabc, slot);
    __builtin_amdgcn_sched_barrier(0);
    mfma16(af[0], bf[0], acc);
    bf[1][0] = f16::expand(lk[1].l[0], sa[0]);
    bf[1][1] = f16::expand(lk[1].l[1], sa[1]);
    read_act(xa, 2, af[2]);
    lookup_step(lk[2], wc.w, 2, tabc, slot);
    interleave<2 * MI, kV, kL>();
    __builtin_amdgcn_sched_barrier(0);
    mfma16(af[1], bf[1], acc);
    bf[0][0] = f16::expand(lk[2].l[0], sa[0]);
    bf[0][1] = f16::expand(lk[2].l[1], sa[1]);
    read_act(xa, 3, af[0]);
    lookup_step(lk[0], wc.w, 3, tabc, slot);
    interleave<2 * MI, kV, kL>();
    __builtin_amdgcn_sched_barrier(0);
    mfma16(af[2], bf[0], acc);
    bf[1][0] = f16::expand(lk[0].l[0], sa[0]);
    bf[1][1] = f16::expand(lk[0].l[1], sa[1]);
    interleave<2 * MI, kV, kL>();
    __builtin_amdgcn_sched_barrier(0);
    mfma16(af[0], bf[1], acc);
    block_scales<kDQ, kF8>(wnx, mean, up, sa);
    lookup_step(lk[1], wnx.w, 0, tabc, slot);
    bf[0][0] = f16::expand(lk[1].l[0], sa[0]);
    bf[0][1] = f16::expand(lk[1].l[1], sa[1]);
    interleave<2 * MI, kV, kL>();
    __builtin_amdgcn_sched_barrier(0);
    gt::wait_vmem();
    __syncthreads();
    wc = wnx;
  }
}

// One work unit: the (32 MI) x 256 tile of y at rows m0.., columns n0..
template <int MI, bool kDQ, bool kF8>
__device__ __forceinline__ void linear_unit(const LinearArgs& a, int64_t m0, int64_t n0, char* xs, const char* tabc,
                                            uint32_t slot, float mean, int wave, int lane) {
  char *xs0 = xs, *xs1 = xs + kStageBytes;
  char* turn = xs + wave * (2 * kStageBytes / 4);  // the wave's own quarter, once the steps are through
  const XTile<MI> xp{reinterpret_cast<const char*>(a.x), a.cols / kBK * 4096, m0 / 32, (a.m - 1) / 32};
  WPtrs wp;
  int64_t nrow[2];
  int we[2];
  float up[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int64_t n = n0 + wave * 64 + j * 32 + (lane & 31);
    nrow[j] = n < a.rows ? n : a.rows - 1;  // rows past the end: never stored
    wp.c[j] = a.packed + nrow[j] * (a.cols / 2) + (lane >> 5) * 16;
    wp.blk[j] = nrow[j] * (a.cols / 64);
    we[j] = a.we[nrow[j]];
    up[j] = f16::power(-we[j]);
  }
  floatx16 acc[MI][2];
  gt::zero_acc(acc);
  steps<MI, kDQ, kF8>(a, xp, wp, up, xs0, xs1, tabc, slot, mean, wave, lane, acc);
  adapters<MI>(acc, a, m0, nrow, we, lane);
  epilogue<MI>(acc, a, m0, n0, we, turn, wave, lane);
  __syncthreads();  // the next unit's first stage may lie in another wave's quarter
}

template <bool kDQ, bool kF8>
__global__ __launch_bounds__(kThreads, 1) void k_linear(LinearArgs a) {
  // the table at LDS address 0: a lookup's address is then its one permute
  __shared__ __align__(16) char lds[4 * f16::kTabWords + 2 * kStageBytes];
  uint32_t* tab = reinterpret_cast<uint32_t*>(lds);
  char* xs = lds + 4 * f16::kTabWords;
  const char* tabc = lds;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t slot = f16::table_slot(lane);
  f16::fill_table<kThreads>(tab, a.cb);
  __syncthreads();
  const float mean = kDQ ? *a.sc.mean : 0.0f;
  const int64_t tiles_n = (a.rows + kBN - 1) / kBN;
  const int64_t tiles = tiles_n * ((a.m + kBM - 1) / kBM);
  for (int64_t u = blockIdx.x; u < a.units; u += gridDim.x) {
    const bool half = u >= a.whole;
    const int64_t tile = half ? a.whole + (u - a.whole) / 2 : u;
    int64_t tid = tile;
    if (tiles % 8 == 0) tid = (tile % 8) * (tiles / 8) + tile / 8;
    const int64_t m0 = (tid / tiles_n) * kBM;
    const int64_t n0 = (tid % tiles_n) * kBN;
    if (!half) {
      linear_unit<kMI, kDQ, kF8>(a, m0, n0, xs, tabc, slot, mean, wave, lane);
    } else {
      const int64_t mh = m0 + ((u - a.whole) & 1) * (kBM / 2);
      if (mh < a.m) linear_unit<kMI / 2, kDQ, kF8>(a, mh, n0, xs, tabc, slot, mean, wave, lane);
    }
  }
}

// x in float16, its rows' exponents and the weight's, the adapter columns, the splits' sums: each at a multiple of 256 bytes.
struct Workspace {
  size_t xe, we, u, part, bytes;
};
Workspace workspace_of(int64_t m, int64_t rows, int64_t cols, int r) {
  const auto round = [](size_t n) { return (n + 255) & ~size_t(255); };
  Workspace w{};
  if (few(m, rows, cols)) {
    w.bytes = r > 0 ? round(static_cast<size_t>(m) * gemm_lora_cols(r) * sizeof(uint16_t)) : 0;
    return w;
  }
  w.xe = round(static_cast<size_t>(x16_rows(m)) * static_cast<size_t>(cols) * sizeof(uint16_t));
  w.we = w.xe + round(static_cast<size_t>(m) * sizeof(int32_t));
  w.u = w.we + round(static_cast<size_t>(rows) * sizeof(int32_t));
  w.part = w.u + (r > 0 ? round(static_cast<size_t>(m) * gemm_lora_cols(r) * sizeof(uint16_t)) : 0);
  w.bytes = w.part;
  if (mid(m, rows, cols)) {
    const MidPlan p = mid_plan(m, rows, cols);
    if (p.splits > 1) w.bytes += round(static_cast<size_t>(p.splits) * m * rows * sizeof(float));
  }
  return w;
}

}  // namespace

size_t linear_workspace(int64_t m, int64_t rows, int64_t cols, int r) {
  return workspace_of(m, rows, cols, r).bytes;
}

hipError_t launch_linear(const uint8_t* packed, int64_t rows, int64_t cols, Scales sc, const uint16_t* x, int64_t m,
                         uint16_t* y, const Epilogue& ep, const uint16_t* lora_a, const uint16_t* lora_b, int r,
                         float lora_scale, void* ws, hipStream_t s) {
  const Workspace at = workspace_of(m, rows, cols, r);
  char* const w8 = static_cast<char*>(ws);
  uint16_t* const u = reinterpret_cast<uint16_t*>(w8 + at.u);
  const AdapterU ad{lora_a, r, (r + 15) / 16 * 16, static_cast<int>(gemm_lora_cols(r)), lora_scale, u};
  const bool row = linear_row_fits(m, rows, cols);
  if (row || few(m, rows, cols)) {
    if (r > 0)
      if (hipError_t e = launch_adapter_u(x, m, cols, ad, s)) return e;
    return row ? launch_linear_row(packed, rows, cols, sc, x, m, y, ep, u, lora_b, r, s)
               : launch_linear_few(packed, rows, cols, sc, x, m, y, ep, u, lora_b, r, s);
  }
  LinearArgs a{};
  a.packed = packed; a.rows = rows; a.cols = cols; a.sc = sc; a.m = m; a.y = y; a.ep = ep;
  a.x = reinterpret_cast<const uint16_t*>(w8);
  a.xe = reinterpret_cast<const int32_t*>(w8 + at.xe);
  a.we = reinterpret_cast<const int32_t*>(w8 + at.we);
  if (hipError_t e = launch_linear_prep(x, m, cols, reinterpret_cast<uint16_t*>(w8), reinterpret_cast<int32_t*>(w8 + at.xe), sc, rows,
                                        reinterpret_cast<int32_t*>(w8 + at.we), ad, s))
    return e;
  a.cb = codebook(sc.fp4);
  a.u = u;
  a.lb = lora_b;
  a.r = r;
  a.r_pad = ad.r_pad;
  a.kl = ad.kl;
  if (mid(m, rows, cols))
    return launch_linear_mid(mid_plan(m, rows, cols), packed, rows, cols, sc, a.x, a.xe, a.we, m, y, ep, a.u, lora_b, r,
                             reinterpret_cast<float*>(w8 + at.part), s);
  const int64_t tiles = ((rows + kBN - 1) / kBN) * ((m + kBM - 1) / kBM);
  const int64_t slots = device_cus();
  const int64_t last = tiles - tiles / slots * slots;
  const bool halve = last > 0 && 2 * last <= slots && m > kBM / 2;
  a.whole = halve ? tiles - last : tiles;
  a.units = halve ? tiles + last : tiles;
  const unsigned grid = static_cast<unsigned>(a.units < slots ? a.units : slots);
  if (sc.absmax) hipLaunchKernelGGL((k_linear<false, false>), dim3(grid), dim3(kThreads), 0, s, a);
  else if (sc.f8) hipLaunchKernelGGL((k_linear<true, true>), dim3(grid), dim3(kThreads), 0, s, a);
  else hipLaunchKernelGGL((k_linear<true, false>), dim3(grid), dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace nf4i
