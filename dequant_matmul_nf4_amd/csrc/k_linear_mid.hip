// A layer's product with its epilogue for some tens to some hundreds of rows of x
// (large decode batches, chunks of prompts): what bounds it is reading the codes once.
//
// Operands as in k_linear.hip: weights as level times scale in float16, x in
// float16 blocks.  A workgroup of 4 waves takes 128 columns of y for up to 32 MI
// rows, and each wave a fourth of its reduction, so that no x is shared and
// nothing waits for another wave: codes and x come straight from memory into
// operands, and a wave multiplies 4 x MI tiles of 32 x 32 (weights x rows of x).
// The reduction goes in groups of four 64-column steps: a row's codes of a group are
// one line of memory, loaded together a group ahead; x comes a step ahead, from
// whole blocks.  The waves' sums meet in LDS.
//
// Where the columns alone give too few workgroups the reduction is cut over
// workgroups too: their sums go to the workspace in float32, and a second kernel
// adds them in order and has the epilogue.
//
// Measured, us in all: 4096x14336 with 96 rows 39.5 (x's preparation 6, this kernel
// 28, the joining 5.5), 14336x4096 with 96 rows 37, with 384 79 (570 TFLOP/s),
// 28672x8192 with 64 rows 67.  The first loads and the level table are 10 us of
// each, a step of 64 columns 0.95 us per 32 rows; what a product waits for is spelled
// out between the products before it (left to the compiler, loads sank to their
// use: 70 us instead of 41).
#include "gemm_tiles.h"
#include "linear_epilogue.h"
#include "linear_f16.h"

namespace nf4i {
namespace {

using gt::bf16x8;
using gt::floatx16;
using gt::u32x4;

constexpr int kWaves = 4, kThreads = 64 * kWaves;
constexpr int kJ = 4;                  // 32-column tiles of a wave
constexpr int kCols = 32 * kJ;
constexpr int kGroup = 4;              // steps loaded together
constexpr int kBK = 64;

struct MidArgs {
  const uint8_t* packed;
  int64_t rows, cols;
  Scales sc;
  const uint16_t* x;   // x in float16 blocks (launch_linear_prep)
  const int32_t *xe, *we;
  int64_t m;
  uint16_t* y;
  Epilogue ep;
  const uint16_t* u;   // adapter columns of x: [m][kl] (s T hi | s T lo | 0)
  const uint16_t* lb;  // B [rows][r]
  int r, r_pad, kl;    // 0 without adapters
  int splits;          // of the reduction over workgroups
  int per;             // steps of a wave
  float* part;         // [splits][m][rows] where splits > 1
  Codebook cb;
};

// The scale inputs of a row's four blocks of a group, from block `at` on (as many as
// the row has): int8 codes and the two group scales that can occur, or the absmax.
typedef uint32_t u32_any __attribute__((aligned(1)));
typedef float floatx4_any __attribute__((ext_vector_type(4), aligned(4)));
typedef float floatx4 __attribute__((ext_vector_type(4)));
template <bool kDQ>
struct ScaleInputs {
  uint32_t q[kJ];
  float lo[kJ], hi[kJ];
};
template <>
struct ScaleInputs<false> {
  floatx4 v[kJ];
};

// The adapters' share, brought to the sums' powers of two: as in k_linear.hip.
template <int MI>
__device__ __forceinline__ void adapters(floatx16 (&acc)[MI][kJ], const MidArgs& a, int64_t m0, const int64_t (&nrow)[kJ],
                                         const int (&we)[kJ], int lane) {
  for (int c = 0; c < 2 * a.r_pad; c += 16) {
    const int ch = c + 8 * (lane >> 5);
    bf16x8 bl[kJ], uf[MI];
#pragma unroll
    for (int j = 0; j < kJ; ++j) bl[j] = lin::adapter_w(a.lb, a.r, a.r_pad, nrow[j], ch, f16::power(-we[j]));
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const int64_t t = m0 + 32 * i + (lane & 31), tc = t < a.m ? t : a.m - 1;
      uf[i] = lin::adapter_x(a.u + tc * a.kl + ch, f16::power(-a.xe[tc]));
    }
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < kJ; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(bl[j], uf[i], acc[i][j], 0, 0, 0);
  }
}

__device__ uint4 kZeros[256];  // a step of 32 rows of x, never written

template <int MI, bool kDQ, bool kF8>
__global__ __launch_bounds__(kThreads, 1) void k_linear_mid(MidArgs a) {
  constexpr int kX = MI < 2 ? 4 : 2;              // steps of x in registers
  constexpr int kC = MI < 3 ? 2 * kGroup : kGroup;  // steps of codes
  constexpr int kMeet = kWaves * MI * 4096;  // a 32-column tile of all waves
  constexpr int kTab = 4 * f16::kTabWords;
  constexpr int kLds = kTab > kMeet ? kTab : kMeet;
  __shared__ __align__(16) char lds[kLds];   // the table, then the waves' sums
  __shared__ int wex[kCols];
  __shared__ float rtab[kF8 ? 256 : 1];
  const char* tabc = lds;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t slot = f16::table_slot(lane);
  const int64_t m0 = static_cast<int64_t>(blockIdx.y) * 32 * MI, n0 = static_cast<int64_t>(blockIdx.x) * kCols;
  const int nk = static_cast<int>(a.cols / kBK);
  const uint32_t row_bytes = static_cast<uint32_t>(a.cols / 2), nblk = static_cast<uint32_t>(nk);
  const int kb = (static_cast<int>(blockIdx.z) * kWaves + wave) * a.per, ke = kb + a.per < nk ? kb + a.per : nk;
  const float mean = kDQ ? *a.sc.mean : 0.0f;

  // the lane's weight rows (past the end the last one: never stored), as offsets from the first
  const uint8_t* cop = a.packed + n0 * row_bytes;
  const int64_t blk = n0 * nblk;
  int64_t nrow[kJ];
  uint32_t coff[kJ], soff[kJ];
#pragma unroll
  for (int j = 0; j < kJ; ++j) {
    const int64_t n = n0 + j * 32 + (lane & 31);
    nrow[j] = n < a.rows ? n : a.rows - 1;
    const uint32_t wr = static_cast<uint32_t>(nrow[j] - n0);
    coff[j] = wr * row_bytes + 16 * (lane >> 5);
    soff[j] = wr * nblk;
  }
  auto clamp = [&](int k) { return k < nk ? k : nk - 1; };  // past the end: the last again, its scale zero
  auto load_scales = [&](ScaleInputs<kDQ>& g, int k0) {
    const int64_t b = blk + (k0 < nk - kGroup ? k0 : nk - kGroup);
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
      if constexpr (kDQ) {
        g.q[j] = *reinterpret_cast<const u32_any*>(a.sc.q + b + soff[j]);
        const float* s2 = a.sc.absmax2 + (b >> 8);
        const uint32_t at = static_cast<uint32_t>(b & 255) + soff[j];
        g.lo[j] = s2[at >> 8];
        g.hi[j] = s2[(at + 3) >> 8];
      } else {
        g.v[j] = *reinterpret_cast<const floatx4_any*>(a.sc.absmax + b + soff[j]);
      }
    }
  };
  auto load_codes = [&](u32x4 (&c)[kJ], int k) {
    const uint8_t* p = cop + static_cast<int64_t>(clamp(k)) * (kBK / 2);
#pragma unroll
    for (int j = 0; j < kJ; ++j) c[j] = *reinterpret_cast<const u32x4*>(p + coff[j]);
  };
  // x of a step: blocks of the 32-row bands (past the last band: the last)
  const int64_t band = static_cast<int64_t>(nk) * 4096, last = (a.m - 1) / 32;
  const char* xb[MI];
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    const int64_t b = m0 / 32 + i;
    xb[i] = reinterpret_cast<const char*>(a.x) + (b < last ? b : last) * band;
  }
  // (steps past the wave's last take zeros: times their scale of zero, an infinity in x would be NaN)
  auto load_x = [&](f16::halfx8 (&x)[MI][4], int k) {
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const char* p = k < ke ? xb[i] + static_cast<int64_t>(k) * 4096 : reinterpret_cast<const char*>(kZeros);
#pragma unroll
      for (int s = 0; s < 4; ++s) x[i][s] = *reinterpret_cast<const f16::halfx8*>(p + s * 1024 + 16 * lane);
    }
  };

  // rings of registers
  u32x4 c[kC][kJ];
  ScaleInputs<kDQ> in[kC / kGroup];
  f16::halfx8 xv[kX][MI][4];
  int we[kJ];
#pragma unroll
  for (int j = 0; j < kJ; ++j) we[j] = a.we[nrow[j]];
  load_scales(in[0], kb);
#pragma unroll
  for (int s = 0; s < kGroup; ++s) load_codes(c[s], kb + s);
#pragma unroll
  for (int s = 0; s < kX - 1; ++s) load_x(xv[s], kb + s);
  if constexpr (kC > kGroup) {
    load_scales(in[1], kb + kGroup);
#pragma unroll
    for (int s = kGroup; s < kC; ++s) load_codes(c[s], kb + s);
  }
  if constexpr (kF8) rtab[threadIdx.x] = kE4m3Ratio.v[threadIdx.x];
  f16::fill_table<kThreads>(reinterpret_cast<uint32_t*>(lds), a.cb);
  float up[kJ];
#pragma unroll
  for (int j = 0; j < kJ; ++j) up[j] = f16::power(-we[j]);
  if (wave == 0 && lane < 32)
#pragma unroll
    for (int j = 0; j < kJ; ++j) wex[32 * j + lane] = we[j];
  f16::lds_barrier();

  // the float16 scales of a group's steps, zero past the wave's last
  f16::half2 sa[kGroup][kJ];
  auto scales = [&](const ScaleInputs<kDQ>& g, int k0) {
    const int off = k0 < nk - kGroup ? 0 : k0 - (nk - kGroup);  // of the loaded blocks the group begins here
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
      float v[kGroup];
      if constexpr (kDQ) {
        const int64_t b = blk + k0 - off;
        const int cross = 256 - static_cast<int>((static_cast<uint32_t>(b & 255) + soff[j]) & 255);  // the first block under hi
#pragma unroll
        for (int s = 0; s < kGroup; ++s) {
          const int q = static_cast<int>(g.q[j] << (24 - 8 * s)) >> 24;
          v[s] = (kF8 ? rtab[q & 0xFF] : div127(q)) * (s >= cross ? g.hi[j] : g.lo[j]) + mean;  // a_hat, three roundings
        }
      } else {
#pragma unroll
        for (int s = 0; s < kGroup; ++s) v[s] = g.v[j][s];
      }
      if (off > 0) {  // the row's last blocks, loaded from before the group's first
#pragma unroll
        for (int s = 0; s < kGroup; ++s) v[s] = off + s == 1 ? v[1] : off + s == 2 ? v[2] : v[3];
      }
#pragma unroll
      for (int s = 0; s < kGroup; ++s) sa[s][j] = f16::twice(k0 + s < ke ? v[s] * up[j] : 0.0f);
    }
  };
  floatx16 acc[MI][kJ];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < kJ; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

  // The products of a 16-wide step q, and pinned between them (left to the compiler it
  // all collects behind or before them) what comes next: the weights of q + 1
  // multiplied out, the levels of q + 2 looked up (its code words w), and more(i).
  uint32_t lk[2][kJ][4];
  u32x4 bf[2][kJ];
  constexpr int kN = MI * kJ;
  auto products = [&](int q, const f16::halfx8 (&x)[MI][4], int xq, const u32x4 (&w)[kJ], int word, const f16::half2 (&sc)[kJ], const auto& more) {
    const int cur = q & 1, nxt = cur ^ 1;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      acc[i / kJ][i % kJ] = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16::halfx8, bf[cur][i % kJ]), x[i / kJ][xq], acc[i / kJ][i % kJ], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
      more(i);
#pragma unroll
      for (int e = 4 * kJ * i / kN; e < 4 * kJ * (i + 1) / kN; ++e) bf[nxt][e >> 2][e & 3] = opaque(f16::times(lk[nxt][e >> 2][e & 3], sc[e >> 2]));
#pragma unroll
      for (int e = 4 * kJ * i / kN; e < 4 * kJ * (i + 1) / kN; ++e) lk[cur][e >> 2][e & 3] = f16::look_up(w[e >> 2][word], e & 3, tabc, slot);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  if (kb < ke) {
    scales(in[0], kb);
#pragma unroll
    for (int j = 0; j < kJ; ++j)
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        bf[0][j][b] = f16::times(f16::look_up(c[0][j][0], b, tabc, slot), sa[0][j]);
        lk[1][j][b] = f16::look_up(c[0][j][1], b, tabc, slot);
      }
  }
  for (int k0 = kb; k0 < ke; k0 += kC) {
#pragma unroll
    for (int s = 0; s < kC; ++s) {
      const int sn = (s + 1) % kC;
      // x of kX - 1 steps ahead; and two steps' codes at a time, half a line of each
      // row, kC steps ahead into the places of what is done
      products(0, xv[s % kX], 0, c[s], 2, sa[s % kGroup], [&](int i) {
        if (i == 0) load_x(xv[(s + kX - 1) % kX], k0 + s + kX - 1);
      });
      products(1, xv[s % kX], 1, c[s], 3, sa[s % kGroup], [](int) {});
      products(2, xv[s % kX], 2, c[sn], 0, sa[s % kGroup], [&](int i) {
        if (s % 2 == 1 && i == 0) {
          load_codes(c[s - 1], k0 + s - 1 + kC);
          if (s % kGroup == 1) load_scales(in[s / kGroup], k0 + s - 1 + kC);
        }
        if (s % 2 == 1 && i == kN / 2) load_codes(c[s], k0 + s + kC);
      });
      products(3, xv[s % kX], 3, c[sn], 1, sa[sn % kGroup], [&](int i) {
        if (sn % kGroup == 0 && i == 0) scales(in[sn / kGroup], k0 + s + 1);
      });
    }
  }
  if (a.r > 0 && blockIdx.z == 0 && wave == 0) adapters<MI>(acc, a, m0, nrow, we, lane);

  // the waves' sums of 32 columns at a time: 16 bytes of lane l for tile i, group g of 4 columns at ((w MI + i) 4 + g) 64 + l
  float4* meet = reinterpret_cast<float4*>(lds);
#pragma unroll
  for (int j = 0; j < kJ; ++j) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int g = 0; g < 4; ++g)
        meet[((wave * MI + i) * 4 + g) * 64 + lane] =
            make_float4(acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]);
    __syncthreads();
    // a thread takes 8 columns of a row: both lane halves' groups of 4
    for (int v = threadIdx.x; v < MI * 128; v += kThreads) {
      const int t32 = v & 31, g = (v >> 5) & 3, i = v >> 7;
      const int64_t t = m0 + 32 * i + t32, col = n0 + 32 * j + 8 * g;
      if (t >= a.m || col >= a.rows) continue;
      float z[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
      for (int w = 0; w < kWaves; ++w)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float4 p = meet[((w * MI + i) * 4 + g) * 64 + 32 * h + t32];
          z[4 * h] += p.x;
          z[4 * h + 1] += p.y;
          z[4 * h + 2] += p.z;
          z[4 * h + 3] += p.w;
        }
      const int xe = a.xe[t];
#pragma unroll
      for (int c = 0; c < 8; ++c) z[c] = __builtin_amdgcn_ldexpf(z[c], xe + wex[32 * j + 8 * g + c]);
      const int left = static_cast<int>(a.rows - col < 8 ? a.rows - col : 8);
      const bool whole = left == 8 && (a.rows & 7) == 0;
      if (a.splits == 1) {
        float bias[8];
        lin::load_bias(bias, a.ep, col, left);
#pragma unroll
        for (int c = 0; c < 8; ++c) z[c] += bias[c];
        lin::finish8(a.ep, a.y, t * a.rows + col, z, left, whole);
      } else {
        float* p = a.part + (static_cast<int64_t>(blockIdx.z) * a.m + t) * a.rows + col;
        if (whole) {
          reinterpret_cast<float4*>(p)[0] = make_float4(z[0], z[1], z[2], z[3]);
          reinterpret_cast<float4*>(p)[1] = make_float4(z[4], z[5], z[6], z[7]);
        } else {
#pragma unroll
          for (int c = 0; c < 8; ++c)
            if (c < left) p[c] = z[c];
        }
      }
    }
  }
}

// The splits' sums in order, and the epilogue: 8 columns of a row per thread.
__global__ __launch_bounds__(256) void k_linear_join(const float* part, int splits, int64_t m, int64_t rows, uint16_t* y, Epilogue ep) {
  const int64_t vec = (rows + 7) / 8;
  const int64_t v = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (v >= m * vec) return;
  const int64_t t = v / vec, col = (v - t * vec) * 8;
  const int left = static_cast<int>(rows - col < 8 ? rows - col : 8);
  const bool whole = left == 8 && (rows & 7) == 0;
  float z[8];
  lin::load_bias(z, ep, col, left);
  float bias[8];
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    bias[c] = z[c];
    z[c] = 0.0f;
  }
  const float* p = part + t * rows + col;
  for (int s = 0; s < splits; ++s, p += m * rows) {
    if (whole) {
      const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
      z[0] += a.x; z[1] += a.y; z[2] += a.z; z[3] += a.w;
      z[4] += b.x; z[5] += b.y; z[6] += b.z; z[7] += b.w;
    } else {
#pragma unroll
      for (int c = 0; c < 8; ++c)
        if (c < left) z[c] += p[c];
    }
  }
#pragma unroll
  for (int c = 0; c < 8; ++c) z[c] += bias[c];
  lin::finish8(ep, y, t * rows + col, z, left, whole);
}

template <int MI>
void launch(const MidArgs& a, const MidPlan& p, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>((a.rows + kCols - 1) / kCols), static_cast<unsigned>(p.tiles), static_cast<unsigned>(p.splits)), block(kThreads);
  if (a.sc.absmax) hipLaunchKernelGGL((k_linear_mid<MI, false, false>), grid, block, 0, s, a);
  else if (a.sc.f8) hipLaunchKernelGGL((k_linear_mid<MI, true, true>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((k_linear_mid<MI, true, false>), grid, block, 0, s, a);
}

}  // namespace

// Tiles of up to 96 rows; splits so that about a workgroup per compute unit (of a
// full chip) has work, but each wave at least two groups of steps.
MidPlan mid_plan(int64_t m, int64_t rows, int64_t cols) {
  MidPlan p{};
  p.tiles = static_cast<int>((m + 95) / 96);
  const int64_t bands = (m + 31) / 32;
  p.mi = static_cast<int>((bands + p.tiles - 1) / p.tiles);
  p.tiles = static_cast<int>((bands + p.mi - 1) / p.mi);
  const int64_t groups = (rows + kCols - 1) / kCols * p.tiles, nk = cols / kBK;
  int64_t splits = groups >= 256 ? 1 : 256 / groups;
  const int64_t most = nk / (kWaves * 2 * kGroup);
  splits = splits < most ? splits : most;
  p.splits = static_cast<int>(splits < 1 ? 1 : splits < 16 ? splits : 16);
  int64_t per = (nk + p.splits * kWaves - 1) / (p.splits * kWaves);
  p.per = static_cast<int>((per + 2 * kGroup - 1) / (2 * kGroup) * (2 * kGroup));
  p.splits = static_cast<int>((nk + static_cast<int64_t>(p.per) * kWaves - 1) / (static_cast<int64_t>(p.per) * kWaves));
  return p;
}

hipError_t launch_linear_mid(const MidPlan& p, const uint8_t* packed, int64_t rows, int64_t cols, Scales sc, const uint16_t* x16,
                             const int32_t* xe, const int32_t* we, int64_t m, uint16_t* y, const Epilogue& ep, const uint16_t* u,
                             const uint16_t* lora_b, int r, float* part, hipStream_t s) {
  MidArgs a{};
  a.packed = packed; a.rows = rows; a.cols = cols; a.sc = sc; a.x = x16; a.xe = xe; a.we = we; a.m = m; a.y = y; a.ep = ep;
  a.u = u; a.lb = lora_b; a.r = r; a.r_pad = (r + 15) / 16 * 16; a.kl = static_cast<int>(gemm_lora_cols(r));
  a.splits = p.splits; a.per = p.per; a.part = part;
  a.cb = codebook(sc.fp4);
  if (p.mi == 1) launch<1>(a, p, s);
  else if (p.mi == 2) launch<2>(a, p, s);
  else launch<3>(a, p, s);
  if (p.splits > 1) {
    const int64_t v = m * ((rows + 7) / 8);
    hipLaunchKernelGGL(k_linear_join, dim3(static_cast<unsigned>((v + 255) / 256)), dim3(256), 0, s, part, p.splits, m, rows, y, ep);
  }
  return hipGetLastError();
}

}  // namespace nf4i
