// The input gradient grouped by expert for few rows per expert:
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
// with the next two steps' loads on their way; a workgroup's 8 waves are 2
// column chunks x 4 slices of the reduction, whose partial tiles are added in
// slice order at the end.
#include "expert_tiles.h"
#include "skinny_tile.h"

namespace nf4i {
namespace {

using sk::floatx4;
using sk::u32x4;

constexpr int kDxThreads = 512;
constexpr int kSlices = 4;             // of the reduction
constexpr int kChunks = 2;             // of columns
constexpr int kChunkCols = 128;        // columns of a wave
constexpr int kUnitCols = kChunks * kChunkCols;
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
};

// One step's loads: 8 weight rows x 8 columns, kRt x 8 values of dy, and the
// scale of weight row lane % 32 in block lane / 32 of the chunk.
template <int kRt, bool kDQ>
struct DxStep {
  uint32_t w[8];
  u32x4 dy[kRt];
  int8_t q;
  float s;
};

// kRt: tiles of 16 rows of dy.
template <int kRt, bool kDQ, bool kF8>
__global__ __launch_bounds__(kDxThreads, 2) void k_expert_skinny_dx(SkinnyDxArgs a) {
  constexpr int kTm = 16 * kRt;
  __shared__ __align__(16) float2 tab[256 * kCopies];
  __shared__ __align__(16) float scl_all[8][64];
  __shared__ __align__(16) floatx4 part[8][8 * 64];
  __shared__ float rtab[kF8 ? 256 : 1];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int ln = lane & 15, g = lane >> 4;
  const int chunk = wave & (kChunks - 1), slice = wave / kChunks;
  float* scl = scl_all[wave];
  const char* tabc = reinterpret_cast<const char*>(tab);
  const uint32_t slot = static_cast<uint32_t>(lane & (kCopies - 1)) << 3;

  const ExpertScan scan = scan_experts(a.er, kTm, lane);
  const int64_t per_tile = (a.cols + kUnitCols - 1) / kUnitCols;
  const int64_t units = per_tile * scan.tiles;
  if (static_cast<int64_t>(blockIdx.x) >= units) return;
  {
    // entry e is levels e / 16 and e % 16: a pass of the threads writes the 16 of one first level
    static_assert(kDxThreads == 16 * kCopies, "a pass is 16 entries");
    const float second = a.cb.level[threadIdx.x / kCopies];
#pragma unroll
    for (int p = 0; p < 16; ++p) tab[p * kDxThreads + threadIdx.x] = make_float2(a.cb.level[p], second);
  }
  if constexpr (kF8)
    for (int i = threadIdx.x; i < 256; i += kDxThreads) rtab[i] = kE4m3Ratio.v[i];
  const float mean = kDQ ? *a.sc.mean : 0.0f;
  sk::lds_barrier();

  const uint32_t row_bytes = static_cast<uint32_t>(a.cols / 2), nblk = static_cast<uint32_t>(a.cols / 64);
  const int64_t steps_all = (a.rows + kStepRows - 1) / kStepRows;
  const int64_t per_slice = (steps_all + kSlices - 1) / kSlices;
  const int64_t n_lo = slice * per_slice * kStepRows;
  const int64_t n_hi = n_lo + per_slice * kStepRows < a.rows ? n_lo + per_slice * kStepRows : a.rows;
  const int nsteps = n_lo < n_hi ? static_cast<int>((n_hi - n_lo + kStepRows - 1) / kStepRows) : 0;

  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int64_t id = xcd_run(u, units);
    const ExpertTile tile = find_expert_tile(a.er, scan, kTm, static_cast<int>(id / per_tile), lane);
    const int64_t c0 = id % per_tile * kUnitCols + chunk * kChunkCols;  // the wave's first column
    const int cnt = static_cast<int>(tile.hi - tile.row0 < kTm ? tile.hi - tile.row0 : kTm);
    // columns past the end read the last ones and are not stored
    const uint32_t cl = static_cast<uint32_t>(c0 + 8 * ln < a.cols ? c0 + 8 * ln : a.cols - 8);
    const uint32_t cb = static_cast<uint32_t>(c0 / 64) + (lane >> 5) < nblk ? static_cast<uint32_t>(c0 / 64) + (lane >> 5) : nblk - 1;
    const int64_t w0 = tile.e * a.rows + n_lo;  // the wave's first weight row
    const uint16_t* dy0 = a.dy + tile.row0 * a.rows + n_lo;
    uint32_t dyo[kRt];
#pragma unroll
    for (int r = 0; r < kRt; ++r)  // rows past the tile's repeat its last: not stored
      dyo[r] = static_cast<uint32_t>(16 * r + ln < cnt ? 16 * r + ln : cnt - 1) * static_cast<uint32_t>(a.rows);
    const int nrows = static_cast<int>(n_hi - n_lo);

    DxStep<kRt, kDQ> set[2];
    auto load_step = [&](DxStep<kRt, kDQ>& st, int step) {
      // steps past the slice's last repeat it (no branch around a load).  The
      // expert's rows are a multiple of 8: a lane group's 8 exist or none does, and
      // then it reads the last 8, which meet zeros of dy.
      const int n = (step < nsteps ? step : nsteps - 1) * kStepRows;
      const int left = nrows - n, k = 8 * g < left ? 8 * g : left - 8;
      const uint8_t* p = a.packed + (w0 + n) * row_bytes;
      const uint32_t wo = static_cast<uint32_t>(k) * row_bytes + (cl >> 1);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        st.w[i] = __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(p + static_cast<int64_t>(i) * row_bytes + wo));
#pragma unroll
      for (int r = 0; r < kRt; ++r) st.dy[r] = *reinterpret_cast<const u32x4*>(dy0 + n + (dyo[r] + k));
      const int64_t b0 = (w0 + n) * nblk;
      const uint32_t bo = static_cast<uint32_t>((lane & 31) < left ? (lane & 31) : left - 1) * nblk + cb;
      if constexpr (kDQ) {
        st.q = (a.sc.q + b0)[bo];
        st.s = a.sc.absmax2[(static_cast<uint32_t>(b0) + bo) >> 8];  // fewer than 2^31 blocks
      } else {
        st.s = (a.sc.absmax + b0)[bo];
      }
    };

    floatx4 acc[kRt][8];
#pragma unroll
    for (int r = 0; r < kRt; ++r)
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[r][j] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};

    auto multiply = [&](DxStep<kRt, kDQ>& st, int step, int ahead) {
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
        for (int c = 0; c < 4; ++c) af[r][c] = in ? st.dy[r][c] : 0u;
      float s;
      if constexpr (kDQ) s = (kF8 ? rtab[st.q & 0xFF] : div127(st.q)) * st.s + mean;  // a_hat, three roundings
      else s = st.s;
      scl[lane] = s;
      load_step(st, ahead);
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

    if (nsteps > 0) {
      load_step(set[0], 0);
      load_step(set[1], 1);
      for (int step = 0; step < nsteps; step += 2) {
        multiply(set[0], step, step + 2);
        if (step + 1 < nsteps) multiply(set[1], step + 1, step + 3);
      }
    }
    // The slices' partial tiles, 16 rows at a time: lane (ln, g) holds rows 4 g .. + 3
    // of columns 8 ln + j.
#pragma unroll
    for (int r = 0; r < kRt; ++r) {
#pragma unroll
      for (int j = 0; j < 8; ++j) part[wave][j * 64 + lane] = acc[r][j];
      sk::lds_barrier();
      for (int t = opaque(threadIdx.x); t < kChunks * 256; t += kDxThreads) {
        const int ch = t >> 8, l = t & 63, i = (t >> 6) & 3;
        const int row = 16 * r + 4 * (l >> 4) + i;
        const int64_t col = id % per_tile * kUnitCols + ch * kChunkCols + 8 * (l & 15);
        if (row < cnt && col < a.cols) {
          uint32_t o[4];
          float v[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            v[j] = 0.0f;
#pragma unroll
            for (int k = 0; k < kSlices; ++k) v[j] += part[k * kChunks + ch][j * 64 + l][i];
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) o[j] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
          *reinterpret_cast<u32x4*>(a.dx + (tile.row0 + row) * a.cols + col) = u32x4{o[0], o[1], o[2], o[3]};
        }
      }
      sk::lds_barrier();
    }
  }
}

template <int kRt>
void launch(const SkinnyDxArgs& a, hipStream_t s) {
  const int64_t tiles = (a.er.m + 16 * kRt - 1) / (16 * kRt) + (a.er.m < a.er.experts ? a.er.m : a.er.experts);
  const int64_t most = tiles * ((a.cols + kUnitCols - 1) / kUnitCols);
  const dim3 gd(static_cast<unsigned>(most < device_cus() ? most : device_cus())), bd(kDxThreads);
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
  const int64_t mean = er.m / er.experts;
  if (mean < 12) launch<1>(a, s);
  else if (mean < 28) launch<2>(a, s);
  else launch<4>(a, s);
  return hipGetLastError();
}

}  // namespace nf4i
