// The input gradient grouped by expert for few tiles:
//
//   dx[p] = dy[p] . deq(W_e)     for offsets[e] <= p < offsets[e + 1]
//
// The reduction runs over the weight's rows, along which the codes are not
// contiguous.  Here no tile is turned in LDS: a lane loads 4 bytes (8 columns)
// of 8 consecutive weight rows and so holds, for each of its 8 columns, the 8
// values that v_mfma_f32_16x16x32_bf16 wants in one lane.  Product j of a step
// (32 weight rows x 128 columns of a wave) takes column j of every lane, i.e.
// columns 8 ln + j (ln = lane % 16); lane group g = lane / 16 brings weight
// rows 8 g .. 8 g + 7.  Of two rows' bytes, two bit-field inserts make bytes
// whose halves are one column's codes in both rows; such a byte indexes a table
// of float32 level pairs in LDS, each level is multiplied by its row's block
// scale and the pair rounded once to bfloat16 (a scale per row of the reduction
// cannot wait for the sums).
//
// Bound: reading the codes, so waves work on their own (no barrier in the loop)
// with the next steps' loads on their way; a workgroup's 8 waves are 1 or 2
// column chunks x 8 or 4 slices of the reduction, whose partial tiles are added
// in slice order at the end.  16 rows over 8 experts of 14336x4096: 84 us (47 us
// at the rate of a large copy); 256 rows, evenly spread: 108 us.  A lane's 4-byte
// loads cost 723 load instructions a wave where the forward product has 260.  In
// tall tiles the loads of dy, 16 lines each, add up to as much as the products.
#include "expert_tiles.h"
#include "skinny_tile.h"

namespace nf4i {
namespace {

using sk::floatx4;
using sk::u32x4;

// Waves of a workgroup, one workgroup per compute unit: tiles of 128 rows take
// all the registers of a SIMD for one wave.
template <int kRt>
constexpr int dx_waves() { return kRt == 8 ? 4 : 8; }
constexpr int kChunkCols = 128;        // columns of a wave
constexpr int kStepRows = 32;
constexpr int kCopies = 32;            // of the pair table: 64 KB, lane l reads copy l % 32

struct SkinnyDxArgs {
  const uint8_t* packed;
  int64_t rows, cols;  // of one expert
  Scales sc;
  ExpertRows er;
  const uint16_t* dy;  // [m][rows]
  uint16_t* dx;        // [m][cols]
  Codebook cb;
  int chunks;          // column chunks of a workgroup: 1 or 2; its waves are chunks x slices of the reduction
};

// One step's loads: 8 weight rows x 8 columns, and the scale of weight row
// lane % 32 in block lane / 32 of the chunk.
template <bool kDQ>
struct DxStep {
  uint32_t w[8];
  int8_t q;
  float s;
};
// Its kRt x 8 values of dy.
template <int kRt>
struct DxRows {
  u32x4 v[kRt];
};

// kRt: tiles of 16 rows of dy.
template <int kRt, bool kDQ, bool kF8>
__global__ __launch_bounds__(64 * dx_waves<kRt>(), dx_waves<kRt>() / 4) void k_expert_skinny_dx(SkinnyDxArgs a) {
  constexpr int kDxWaves = dx_waves<kRt>(), kDxThreads = 64 * kDxWaves;
  constexpr int kTm = 16 * kRt;
  __shared__ __align__(16) float2 tab[256 * kCopies];
  __shared__ __align__(16) float scl_all[kDxWaves][64];
  __shared__ __align__(16) floatx4 part[kDxWaves][8 * 64];
  __shared__ float rtab[kF8 ? 256 : 1];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int ln = lane & 15, g = lane >> 4;
  const int chunks = a.chunks, slices = kDxWaves / chunks;
  const int chunk = wave & (chunks - 1), slice = wave / chunks;
  const int64_t unit_cols = chunks * kChunkCols;
  float* scl = scl_all[wave];
  const char* tabc = reinterpret_cast<const char*>(tab);
  const uint32_t slot = static_cast<uint32_t>(lane & (kCopies - 1)) << 3;

  const ExpertScan scan = scan_experts(a.er, kTm, lane);
  const int64_t per_tile = (a.cols + unit_cols - 1) / unit_cols;
  const int64_t units = per_tile * scan.tiles;
  if (static_cast<int64_t>(blockIdx.x) >= units) return;
  {
    // entry e is levels e / 16 and e % 16: the threads write those of one first level in kPass passes
    constexpr int kPass = 16 * kCopies / kDxThreads;
    float second[kPass];
#pragma unroll
    for (int q = 0; q < kPass; ++q) second[q] = a.cb.level[(q * kDxThreads + threadIdx.x) / kCopies];
#pragma unroll
    for (int p = 0; p < 16 * kPass; ++p) tab[p * kDxThreads + threadIdx.x] = make_float2(a.cb.level[p / kPass], second[p % kPass]);
  }
  if constexpr (kF8)
    for (int i = threadIdx.x; i < 256; i += kDxThreads) rtab[i] = kE4m3Ratio.v[i];
  const float mean = kDQ ? *a.sc.mean : 0.0f;
  sk::lds_barrier();

  const uint32_t row_bytes = static_cast<uint32_t>(a.cols / 2), nblk = static_cast<uint32_t>(a.cols / 64);
  const int64_t steps_all = (a.rows + kStepRows - 1) / kStepRows;
  const int64_t per_slice = (steps_all + slices - 1) / slices;
  const int64_t n_lo = slice * per_slice * kStepRows;
  const int64_t n_hi = n_lo + per_slice * kStepRows < a.rows ? n_lo + per_slice * kStepRows : a.rows;
  const int nsteps = n_lo < n_hi ? static_cast<int>((n_hi - n_lo + kStepRows - 1) / kStepRows) : 0;

  const int nrows = n_lo < n_hi ? static_cast<int>(n_hi - n_lo) : 0;
  const int chunk0 = chunk * kChunkCols;

  // A unit: one tile's rows, unit_cols columns.
  int64_t row0, col0, w0;  // its first row of dx, first column, the wave's first weight row
  int cnt;                 // its rows
  uint32_t cl, cb, dyo[kRt];
  auto take_unit = [&](int64_t u) {
    const int64_t id = xcd_run(u, units);
    const ExpertTile tile = find_expert_tile(a.er, scan, kTm, id / per_tile, lane);
    row0 = tile.row0;
    col0 = id % per_tile * unit_cols;
    w0 = tile.e * a.rows + n_lo;
    cnt = static_cast<int>(tile.hi - tile.row0 < kTm ? tile.hi - tile.row0 : kTm);
    // columns past the end read the last ones and are not stored
    const int64_t c0 = col0 + chunk0;
    cl = static_cast<uint32_t>(c0 + 8 * ln < a.cols ? c0 + 8 * ln : a.cols - 8);
    cb = static_cast<uint32_t>(c0 / 64) + (lane >> 5) < nblk ? static_cast<uint32_t>(c0 / 64) + (lane >> 5) : nblk - 1;
#pragma unroll
    for (int r = 0; r < kRt; ++r)  // rows past the tile's repeat its last: not stored
      dyo[r] = static_cast<uint32_t>(16 * r + ln < cnt ? 16 * r + ln : cnt - 1) * static_cast<uint32_t>(a.rows);
  };

  constexpr int kDepth = kRt == 4 ? 2 : 4;    // steps of codes on their way
  constexpr int kDyDepth = kRt == 2 ? 4 : kRt == 4 ? 1 : 2;  // and of dy, which the caches hold
  DxStep<kDQ> set[kDepth];
  DxRows<kRt> dys[kDyDepth];
  auto load_dy = [&](DxRows<kRt>& st, int step) {
    const int n = (step < nsteps ? step : nsteps - 1) * kStepRows;
    const int left = nrows - n, k = 8 * g < left ? 8 * g : left - 8;
    const uint16_t* dy0 = a.dy + (row0 * a.rows + n_lo + n);
#pragma unroll
    for (int r = 0; r < kRt; ++r) st.v[r] = *reinterpret_cast<const u32x4*>(dy0 + (dyo[r] + k));
  };
  auto load_step = [&](DxStep<kDQ>& st, int step) {
    // steps past the slice's last repeat it (no branch around a load).  The
    // expert's rows are a multiple of 8: a lane group's 8 exist or none does, and
    // then it reads the last 8, which meet zeros of dy.
    const int n = (step < nsteps ? step : nsteps - 1) * kStepRows;
    const int left = nrows - n, k = 8 * g < left ? 8 * g : left - 8;
    const uint8_t* p = a.packed + (w0 + n) * row_bytes;
    const uint32_t wo = static_cast<uint32_t>(k) * row_bytes + (cl >> 1);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      st.w[i] = *reinterpret_cast<const uint32_t*>(p + static_cast<int64_t>(i) * row_bytes + wo);
    const int64_t b0 = (w0 + n) * nblk;
    const uint32_t bo = static_cast<uint32_t>((lane & 31) < left ? (lane & 31) : left - 1) * nblk + cb;
    if constexpr (kDQ) {
      st.q = (a.sc.q + b0)[bo];
      st.s = a.sc.absmax2[(static_cast<uint32_t>(b0) + bo) >> 8];  // fewer than 2^31 blocks
    } else {
      st.s = (a.sc.absmax + b0)[bo];
    }
  };
  auto start_unit = [&](int64_t u) {
    take_unit(u);
    if (nsteps > 0) {
#pragma unroll
      for (int i = 0; i < kDepth; ++i) {
        if (i < kDyDepth) load_dy(dys[i], i);
        load_step(set[i], i);
      }
    }
  };

  start_unit(blockIdx.x);
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    floatx4 acc[kRt][8];
#pragma unroll
    for (int r = 0; r < kRt; ++r)
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[r][j] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};

    auto multiply = [&](DxStep<kDQ>& st, DxRows<kRt>& dy, int step) {
      // codes of rows 2 t, 2 t + 1 as bytes: even columns, odd columns
      uint32_t ev[4], od[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        ev[t] = (st.w[2 * t] & 0xF0F0F0F0u) | ((st.w[2 * t + 1] >> 4) & 0x0F0F0F0Fu);
        od[t] = ((st.w[2 * t] << 4) & 0xF0F0F0F0u) | (st.w[2 * t + 1] & 0x0F0F0F0Fu);
      }
      const bool in = step * kStepRows + 8 * g < nrows;
      u32x4 af[kRt];
#pragma unroll
      for (int r = 0; r < kRt; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c) af[r][c] = in ? dy.v[r][c] : 0u;
      float s;
      if constexpr (kDQ) s = (kF8 ? rtab[st.q & 0xFF] : div127(st.q)) * st.s + mean;  // a_hat, three roundings
      else s = st.s;
      scl[lane] = s;
      load_dy(dy, step + kDyDepth);
      load_step(st, step + kDepth);
      sk::wave_lds_order();
      // the scales of rows 8 g .. in the lane's block
      const floatx4 s0 = *reinterpret_cast<const floatx4*>(scl + (ln >> 3) * 32 + 8 * g);
      const floatx4 s1 = *reinterpret_cast<const floatx4*>(scl + (ln >> 3) * 32 + 8 * g + 4);
      float2 lk[2][4];
      auto look_up = [&](int j) {
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const uint32_t at = __builtin_amdgcn_perm((j & 1) ? od[t] : ev[t], slot, 0x0C0C0000u | ((4u + (j >> 1)) << 8));
          lk[j & 1][t] = *reinterpret_cast<const float2*>(tabc + at);
        }
      };
      look_up(0);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (j < 7) look_up(j + 1);
        __builtin_amdgcn_sched_barrier(0);
        u32x4 b;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const float f0 = t < 2 ? s0[2 * t] : s1[2 * t - 4], f1 = t < 2 ? s0[2 * t + 1] : s1[2 * t - 3];
          typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
          const bf16x2 v = {static_cast<__bf16>(lk[j & 1][t].x * f0), static_cast<__bf16>(lk[j & 1][t].y * f1)};  // to nearest even
          b[t] = __builtin_bit_cast(uint32_t, v);
        }
#pragma unroll
        for (int r = 0; r < kRt; ++r) acc[r][j] = sk::mfma<false>(af[r], b, acc[r][j]);
      }
      sk::wave_lds_order();
    };

    for (int step = 0; step < nsteps; step += kDepth) {
#pragma unroll
      for (int i = 0; i < kDepth; ++i)
        if (step + i < nsteps) multiply(set[i], dys[i % kDyDepth], step + i);
    }
    // The next unit's first loads, then this one's slices added up, 16 rows at a
    // time: lane (ln, g) holds rows 4 g .. + 3 of columns 8 ln + j.
    const int64_t out_row = row0, out_col = col0;
    const int out_cnt = cnt;
    if (u + gridDim.x < units) start_unit(u + gridDim.x);
#pragma unroll
    for (int r = 0; r < kRt; ++r) {
#pragma unroll
      for (int j = 0; j < 8; ++j) part[wave][j * 64 + lane] = acc[r][j];
      sk::lds_barrier();
      for (int t = opaque(threadIdx.x); t < chunks * 256; t += kDxThreads) {
        const int ch = t >> 8, l = t & 63, i = (t >> 6) & 3;
        const int row = 16 * r + 4 * (l >> 4) + i;
        const int64_t col = out_col + ch * kChunkCols + 8 * (l & 15);
        if (row < out_cnt && col < a.cols) {
          float v[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            v[j] = part[ch][j * 64 + l][i];
#pragma unroll
            for (int k = 1; k < kDxWaves / 2; ++k) v[j] += part[k * chunks + ch][j * 64 + l][i];
          }
          if (chunks == 1) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
              for (int k = kDxWaves / 2; k < kDxWaves; ++k) v[j] += part[k][j * 64 + l][i];
          }
          *reinterpret_cast<u32x4*>(a.dx + (out_row + row) * a.cols + col) =
              u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
        }
      }
      sk::lds_barrier();
    }
  }
}

template <int kRt>
void launch(SkinnyDxArgs a, hipStream_t s) {
  const int64_t tiles = (a.er.m + 16 * kRt - 1) / (16 * kRt) + (a.er.m < a.er.experts ? a.er.m : a.er.experts);  // at most
  a.chunks = tiles * ((a.cols + 255) / 256) >= 2 * device_cus() ? 2 : 1;
  const int64_t most = tiles * ((a.cols + a.chunks * kChunkCols - 1) / (a.chunks * kChunkCols));
  const dim3 gd(static_cast<unsigned>(most < device_cus() ? most : device_cus())), bd(64 * dx_waves<kRt>());
  if (a.sc.absmax) hipLaunchKernelGGL((k_expert_skinny_dx<kRt, false, false>), gd, bd, 0, s, a);
  else if (a.sc.f8) hipLaunchKernelGGL((k_expert_skinny_dx<kRt, true, true>), gd, bd, 0, s, a);
  else hipLaunchKernelGGL((k_expert_skinny_dx<kRt, true, false>), gd, bd, 0, s, a);
}

}  // namespace

hipError_t launch_expert_skinny_dx(const uint8_t* packed, int64_t rows, int64_t cols, Scales sc, const ExpertRows& er,
                                   const uint16_t* dy, uint16_t* dx, hipStream_t s) {
  SkinnyDxArgs a{};
  a.packed = packed; a.rows = rows; a.cols = cols; a.sc = sc; a.er = er; a.dy = dy; a.dx = dx;
  a.cb = codebook(sc.fp4);
  // Taller tiles expand the weights for more rows, but an expert's last tile is
  // emptier and a step takes longer.  Measured in us, rows evenly spread, stacks
  // changing from call to call: tiles of 32, 64 and 128 rows.
  //   8 experts of 14336x4096, mean   2:   89   97  148
  //                                  32:  105  109  141
  //   4 of 2048x8192,          mean   4:   22   22   29
  //                                  32:   27   26   30
  //   2 of 14336x4096,         mean  64:   88  118  137
  //                                 256:  155  112  162
  //   2 of 4096x2048,          mean 450:   50   37   51
  //   1 of 14336x8192,         mean 280:  226  193  142
  //   1 of 16384x4096,         mean 600:  237  201  164
  // While one round of the compute units takes all tiles, lower ones are as fast
  // or faster; where they need another round, taller ones are.  The mean is a
  // rough sign of that: it errs where few experts have their rows in one round
  // (2 of 14336x4096 at 256: 128-row tiles, 162 us).
  const int64_t mean = er.m / er.experts;
  if (mean < 16) launch<2>(a, s);
  else if (mean < 96) launch<4>(a, s);
  else launch<8>(a, s);
  return hipGetLastError();
}

}  // namespace nf4i
