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
// A byte of codes indexes a table of level pairs in LDS, each level as two
// bfloat16 parts (hi = round(level), lo = round(level - hi): 16 significant
// bits), and both parts are multiplied: the matrix cores have time for twice
// the products.  The sums of a 64-block are scaled in float32.  So nothing but
// the levels' 2^-17 is rounded before y.
#include "expert_tiles.h"
#include "skinny_tile.h"

namespace nf4i {
namespace {

using sk::Codes;
using sk::floatx4;
using sk::kSeg;
using sk::kWaves;
using sk::u32x4;

constexpr int kNb = kSeg / 64;   // blocks of a weight row per step
constexpr int kPer = kNb / 4;    // of which a lane brings the scales
constexpr int kCopies = 32;      // of the level table: lane l reads copy l % 32

struct SkinnyArgs {
  const uint8_t* packed;
  int64_t rows, cols;  // of one expert
  Scales sc;
  ExpertRows er;
  ExpertX ex;
  uint16_t* y;         // [m][rows]
  Codebook cb;
  sk::Plan pl;
};

template <bool kDQ>
struct Step {
  Codes codes;
  int8_t q[kPer];     // second-level code and its group's scale, or the absmax
  float s[kPer];
};

// kG: groups of 16 weight rows a wave takes per batch, x being read once for
// all of them; kOnce: a wave's columns are one segment, whose x is read once
// per tile.
template <bool kDQ, bool kF8, int kG, bool kOnce>
__global__ __launch_bounds__(sk::kThreads, 2) void k_expert_skinny(SkinnyArgs a) {
  __shared__ __align__(16) uint2 tab[256 * kCopies];
  __shared__ __align__(16) char stage_all[kWaves][sk::kStageBytes];
  __shared__ __align__(16) float scl_all[kWaves][sk::kRows * kNb];
  __shared__ __align__(16) floatx4 part[kWaves * kG * 64];
  __shared__ float rtab[kF8 ? 256 : 1];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int ln = lane & 15, g = lane >> 4;
  const sk::Plan& pl = a.pl;

  // the workgroup's run of the groups of all tiles
  const int64_t ngr = (a.rows + 15) / 16;  // groups of a tile
  const int64_t all = ngr * expert_tiles(a.er, sk::kRows, lane);
  int64_t at = all * blockIdx.x / gridDim.x;
  const int64_t end = all * (blockIdx.x + 1) / gridDim.x;
  if (at >= end) return;

  for (int i = threadIdx.x; i < 256 * kCopies; i += sk::kThreads) {
    const int e = i / kCopies;
    const float l0 = a.cb.level[e >> 4], l1 = a.cb.level[e & 15];
    const uint32_t h0 = f32_to_bf16(l0), h1 = f32_to_bf16(l1);
    tab[i] = make_uint2(h0 | (h1 << 16), pack_bf16x2(l0 - bf16_to_f32(h0), l1 - bf16_to_f32(h1)));
  }
  if constexpr (kF8)
    for (int i = threadIdx.x; i < 256; i += sk::kThreads) rtab[i] = kE4m3Ratio.v[i];
  const float mean = kDQ ? *a.sc.mean : 0.0f;
  __syncthreads();

  const int kw = wave % pl.ks, rw = wave / pl.ks;  // the wave's share of the columns, of the groups
  const bool live = rw < pl.rs;
  char* stage = stage_all[wave];
  float* scl = scl_all[wave];
  const char* tabc = reinterpret_cast<const char*>(tab);
  const uint32_t slot = static_cast<uint32_t>(lane & (kCopies - 1)) << 3;
  const uint32_t row_bytes = static_cast<uint32_t>(a.cols / 2), nblk = static_cast<uint32_t>(a.cols / 64);
  const int64_t klo = kw * pl.per, khi = klo + pl.per < a.cols ? klo + pl.per : a.cols;
  const int kspan = static_cast<int>(khi - klo);
  const int nseg = (kspan + kSeg - 1) / kSeg;
  const int64_t group_bytes = int64_t{16} * row_bytes, group_blocks = int64_t{16} * nblk;
  const sk::CodeLane cl = sk::code_lane(row_bytes, lane);
  const uint32_t srow = static_cast<uint32_t>(ln) * nblk + g * kPer;

  // the part of the run that lies in one tile
  for (int64_t next; at < end; at = next) {
    const int64_t tid = at / ngr, j0 = at - tid * ngr;
    const ExpertTile tile = find_expert_tile(a.er, sk::kRows, static_cast<int>(tid), lane);
    next = at + (ngr - j0) < end ? at + (ngr - j0) : end;
    const int ng = static_cast<int>(next - at);
    const int cnt = static_cast<int>(tile.hi - tile.row0 < sk::kRows ? tile.hi - tile.row0 : sk::kRows);  // rows of x
    const int64_t rows_left = a.rows - j0 * 16;
    const int tail = static_cast<int>(rows_left - (ng - 1) * 16 < 16 ? rows_left - (ng - 1) * 16 : 16);
    const int64_t row0 = tile.e * a.rows + j0 * 16;
    const uint8_t* codes0 = a.packed + row0 * row_bytes + klo / 2;
    const int64_t block0 = row0 * nblk + klo / 64;
    // the lane's row of x; rows past the tile's repeat its last and are not stored
    const uint16_t* xr;
    {
      const int64_t p = tile.row0 + (ln < cnt ? ln : cnt - 1);
      int64_t r = p;
      if (a.ex.index) {
        r = a.ex.index[p] / a.ex.slots;
        r = r < 0 ? 0 : r < a.ex.rows ? r : a.ex.rows - 1;
      }
      xr = a.ex.x + r * a.cols + klo;
    }

    Step<kDQ> set[2];
    auto load_step = [&](Step<kDQ>& st, int group, int seg, bool wanted) {
      const int rows = group == ng - 1 ? tail : 16;
      const int left = kspan - seg * kSeg;
      sk::load_codes(st.codes, codes0 + (group * group_bytes + seg * (kSeg / 2)), cl, row_bytes, rows, left / 32, wanted, lane);
      const int64_t b0 = block0 + (group * group_blocks + seg * kNb);  // the step's first block
      const bool whole = rows == 16 && left >= kSeg;
      const int lq = (left < kSeg ? left : kSeg) / 64 - 1;
      const uint32_t trow = static_cast<uint32_t>(ln < rows ? ln : rows - 1) * nblk;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int q = g * kPer + j;
        const uint32_t o = (whole ? srow + j : trow + (q < lq ? q : lq)) & (wanted ? ~0u : 0u);
        if constexpr (kDQ) {
          st.q[j] = (a.sc.q + b0)[o];
          st.s[j] = a.sc.absmax2[(b0 + o) >> 8];
        } else {
          st.s[j] = (a.sc.absmax + b0)[o];
        }
      }
    };

    u32x4 xv[kNb][2];
    auto load_x = [&](int seg) {
#pragma unroll
      for (int b = 0; b < kNb; ++b)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int k = seg * kSeg + 64 * b + 16 * g + 8 * u;
          xv[b][u] = *reinterpret_cast<const u32x4*>(xr + (k < kspan ? k : kspan - 8));
        }
      if (seg * kSeg + kSeg > kspan) {
#pragma unroll
        for (int b = 0; b < kNb; ++b)
#pragma unroll
          for (int u = 0; u < 2; ++u)
            if (seg * kSeg + 64 * b >= kspan) xv[b][u] = u32x4{0u, 0u, 0u, 0u};
      }
    };

    // as in the int4 GEMV: position p of the walk is group p % kG of segment
    // p / kG of the batch, two steps on their way in two register sets
    const int batch = pl.rs * kG;
    auto load_at = [&](Step<kDQ>& st, int base, int seg, int gi) {
      if (seg >= nseg) {
        seg -= nseg;
        base += batch;
      }
      const int group = base + gi * pl.rs + rw;
      load_step(st, group < ng ? group : ng - 1, seg, group < ng);
    };
    if constexpr (kOnce) load_x(0);
    load_at(set[0], 0, 0, 0);
    load_at(set[1], 0, 0, 1);
    for (int base = 0; base < ng; base += batch) {
      floatx4 acc[kG];
#pragma unroll
      for (int i = 0; i < kG; ++i) acc[i] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
      for (int seg = 0; live && seg < nseg; ++seg) {
        if constexpr (!kOnce) load_x(seg);
#pragma unroll
        for (int gi = 0; gi < kG; ++gi) {
          Step<kDQ>& st = set[gi & 1];
          const bool here = base + gi * pl.rs + rw < ng;
          if (here) {
            sk::stage_codes(st.codes, stage, lane);
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
              float s;
              if constexpr (kDQ) s = (kF8 ? rtab[st.q[j] & 0xFF] : div127(st.q[j])) * st.s[j] + mean;  // a_hat, three roundings
              else s = st.s[j];
              scl[ln * kNb + g * kPer + j] = s;
            }
          }
          load_at(st, base, gi + 2 < kG ? seg : seg + 1, (gi + 2) % kG);
          if (!here) continue;
          sk::wave_lds_order();
          const floatx4 f0 = *reinterpret_cast<const floatx4*>(scl + ln * kNb), f1 = *reinterpret_cast<const floatx4*>(scl + ln * kNb + 4);
#pragma unroll
          for (int b = 0; b < kNb; ++b) {
            const uint2 w = *reinterpret_cast<const uint2*>(stage + sk::slot_of(ln, 2 * b + (g >> 1)) + 8 * (g & 1));
            u32x4 hi[2], lo[2];
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                const uint32_t addr = __builtin_amdgcn_perm(u ? w.y : w.x, slot, 0x0C0C0000u | ((4u + c) << 8));
                const uint2 t = *reinterpret_cast<const uint2*>(tabc + addr);
                hi[u][c] = t.x;
                lo[u][c] = t.y;
              }
            floatx4 d = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
            d = sk::mfma<false>(xv[b][0], lo[0], d);
            d = sk::mfma<false>(xv[b][1], lo[1], d);
            d = sk::mfma<false>(xv[b][0], hi[0], d);
            d = sk::mfma<false>(xv[b][1], hi[1], d);
            const float f = b < 4 ? f0[b & 3] : f1[b & 3];
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[gi][i] = fmaf(f, d[i], acc[gi][i]);
          }
          sk::wave_lds_order();
        }
      }
      // the waves' partial tiles, added in wave order
      if (live) {
#pragma unroll
        for (int gi = 0; gi < kG; ++gi) part[(wave * kG + gi) * 64 + lane] = acc[gi];
      }
      sk::lds_barrier();
      for (int t = threadIdx.x; t < batch * 64; t += sk::kThreads) {
        const int l = t & 63, gi = (t >> 6) % kG, r = (t >> 6) / kG;
        const int group = base + gi * pl.rs + r;
        if (group >= ng) continue;
        floatx4 v = part[(r * pl.ks * kG + gi) * 64 + l];
        for (int k = 1; k < pl.ks; ++k) v += part[((r * pl.ks + k) * kG + gi) * 64 + l];
        const int64_t row = (j0 + group) * 16 + (l & 15);
        if (row >= a.rows) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int xm = 4 * (l >> 4) + i;
          if (xm < cnt) a.y[(tile.row0 + xm) * a.rows + row] = static_cast<uint16_t>(f32_to_bf16(v[i]));
        }
      }
      sk::lds_barrier();
    }
  }
}

template <bool kDQ, bool kF8>
void launch(const SkinnyArgs& a, hipStream_t s) {
  const int64_t ngr = (a.rows + 15) / 16;
  const int64_t tiles = a.er.m < a.er.experts ? a.er.m : a.er.experts;  // about; the offsets are device data
  const int64_t want = (ngr * tiles + a.pl.rs - 1) / a.pl.rs;
  int64_t grid = want < device_cus() ? want : device_cus();
  while (ngr / grid >= (int64_t{1} << 26)) grid *= 2;
  const dim3 gd(static_cast<unsigned>(grid)), bd(sk::kThreads);
  if (a.pl.per <= kSeg) hipLaunchKernelGGL((k_expert_skinny<kDQ, kF8, 4, true>), gd, bd, 0, s, a);
  else hipLaunchKernelGGL((k_expert_skinny<kDQ, kF8, 4, false>), gd, bd, 0, s, a);
}

}  // namespace

hipError_t launch_expert_skinny(const uint8_t* packed, int64_t rows, int64_t cols, Scales sc, const ExpertRows& er,
                                const ExpertX& ex, uint16_t* y, hipStream_t s) {
  SkinnyArgs a{};
  a.packed = packed; a.rows = rows; a.cols = cols; a.sc = sc; a.er = er; a.ex = ex; a.y = y;
  a.cb = codebook(sc.fp4);
  a.pl = sk::make_plan(cols);
  if (sc.absmax) launch<false, false>(a, s);
  else if (sc.f8) launch<true, true>(a, s);
  else launch<true, false>(a, s);
  return hipGetLastError();
}

}  // namespace nf4i
