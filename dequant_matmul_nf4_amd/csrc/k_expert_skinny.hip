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
// A byte of codes indexes a table of level pairs in LDS, rounded to float16 (11
// significant bits: off by less than 2^-11 of a level), and the sums of a
// 64-block are scaled in float32, so no scaled weight is rounded to 16 bits.
// x becomes float16 exactly: a wave scales its columns of a row by the power
// of two that brings their largest value to [2^14, 2^15) and scales the sums
// back (values 2^-29 of the largest and below lose bits; a block scale of 2^104
// could overflow the sum of a segment, 8 blocks of 64 products below 2^15).  Two
// bfloat16 parts per level instead were exact to 2^-17 but moved two registers per
// lookup to line up the operands: 66 against 57 us (16 rows over 8 experts of
// 14336x4096).
//
// That product takes 49 us now where 7 of the 8 experts have rows (4.4 TB/s; the
// codes and scales of 7 take 42 us at the rate of a large copy), 56 us where all
// have (47 us).  One row alone takes 15 us (6 us), where launch, offsets, index and
// x follow each other.  Measured without gain: 16 waves with steps of 256 columns,
// three or four steps on their way, codes kept in the caches, groups taken in
// rotated order.  Rows of more than 4096 columns re-read x for every batch of groups
// (8 experts of 4096x14336, 16 rows: 72 us).
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
constexpr int kCopies = 64;      // of the level table (64 KB): each lane has its own, no two meet in a bank

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

__device__ __forceinline__ uint32_t half_pair(float a, float b) {
  typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, half2_t{static_cast<_Float16>(a), static_cast<_Float16>(b)});
}

// The level pairs of a lane's 8 code bytes: one permute puts a byte above the
// lane's copy (an entry is 256 bytes), one LDS read brings the pair.
__device__ __forceinline__ void look_up(u32x4 (&t)[2], const uint2& w, const char* tab, uint32_t slot) {
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const uint32_t at = __builtin_amdgcn_perm(c < 4 ? w.x : w.y, slot, 0x0C0C0000u | ((4u + (c & 3)) << 8));
    t[c >> 2][c & 3] = *reinterpret_cast<const uint32_t*>(tab + at);
  }
}

// kG: groups of 16 weight rows a wave takes per batch, x being read once for
// all of them; kOnce: a wave's columns are one segment, whose x is read once
// per tile.
template <bool kDQ, bool kF8, int kG, bool kOnce>
__global__ __launch_bounds__(sk::kThreads, 2) void k_expert_skinny(SkinnyArgs a) {
  __shared__ __align__(16) uint32_t tab[256 * kCopies];
  __shared__ __align__(16) char stage_all[kWaves][sk::kStageBytes];
  __shared__ __align__(16) float scl_all[kWaves][sk::kRows * kNb];
  __shared__ __align__(16) floatx4 part[kWaves * kG * 64];
  __shared__ float rtab[kF8 ? 256 : 1];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int ln = lane & 15, g = lane >> 4;
  const sk::Plan& pl = a.pl;

  // the workgroup's run of the groups of all tiles
  const ExpertScan scan = scan_experts(a.er, sk::kRows, lane);
  const int64_t ngr = (a.rows + 15) / 16;  // groups of a tile
  const int64_t all = ngr * scan.tiles;
  int64_t at = all * blockIdx.x / gridDim.x;
  const int64_t end = all * (blockIdx.x + 1) / gridDim.x;
  if (at >= end) return;

  // Entry e of the table is levels e / 16 and e % 16: two passes of the threads
  // write the 16 entries of one first level.
  static_assert(sk::kThreads == 8 * kCopies, "a pass is 8 entries");
  {
    const float second[2] = {a.cb.level[threadIdx.x / kCopies], a.cb.level[8 + threadIdx.x / kCopies]};
#pragma unroll
    for (int p = 0; p < 32; ++p) tab[p * sk::kThreads + threadIdx.x] = half_pair(a.cb.level[p >> 1], second[p & 1]);
  }
  if constexpr (kF8)
    for (int i = threadIdx.x; i < 256; i += sk::kThreads) rtab[i] = kE4m3Ratio.v[i];
  const float mean = kDQ ? *a.sc.mean : 0.0f;
  sk::lds_barrier();

  const int kw = wave % pl.ks, rw = wave / pl.ks;  // the wave's share of the columns, of the groups
  const bool live = rw < pl.rs;
  char* stage = stage_all[wave];
  float* scl = scl_all[wave];
  const char* tabc = reinterpret_cast<const char*>(tab);
  const uint32_t slot = static_cast<uint32_t>(lane & (kCopies - 1)) << 2;
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
    const ExpertTile tile = find_expert_tile(a.er, scan, sk::kRows, tid, lane);
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
    floatx4 back;  // the powers of two that scale the sums of x rows 4 g .. back
    auto load_x = [&](int seg) {
      uint32_t top = 0;  // of the row's magnitudes in the segment, as bfloat16 bits
      const int left = kspan - seg * kSeg;
      if (left >= kSeg) {
        const uint16_t* p = xr + (seg * kSeg + 16 * g);
#pragma unroll
        for (int b = 0; b < kNb; ++b)
#pragma unroll
          for (int u = 0; u < 2; ++u) xv[b][u] = *reinterpret_cast<const u32x4*>(p + 64 * b + 8 * u);
      } else {
        const uint16_t* p = xr + seg * kSeg;
        const int g16 = 16 * static_cast<int>(opaque(g));
#pragma unroll
        for (int b = 0; b < kNb; ++b)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int k = 64 * b + g16 + 8 * u;
            xv[b][u] = *reinterpret_cast<const u32x4*>(p + (k < left ? k : left - 8));
          }
      }
#pragma unroll
      for (int b = 0; b < kNb; ++b)
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint32_t v = xv[b][u][c], lo = (v << 16) & 0x7FFF0000u, hi = v & 0x7FFF0000u;
            const uint32_t m = lo > hi ? lo : hi;
            top = m > top ? m : top;
          }
#pragma unroll
      for (int off = 16; off < 64; off <<= 1) {
        const uint32_t o = __shfl_xor(top, off, 64);
        top = o > top ? o : top;
      }
      // 2^e <= top < 2^(e + 1): the row times 2^(14 - e), its sums times 2^(e - 14).  The exponent
      // is kept in -112 .. 127, where both factors are normal numbers
      const int e = static_cast<int>(top >> 23) - 127 < -112 ? -112 : static_cast<int>(top >> 23) - 127;
      const float up = __uint_as_float(static_cast<uint32_t>(14 - e + 127) << 23);
#pragma unroll
      for (int b = 0; b < kNb; ++b) {
        const float f = seg * kSeg + 64 * b < kspan ? up : 0.0f;  // zeros past the columns' end
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int c = 0; c < 4; ++c)
            xv[b][u][c] = half_pair(bf16_to_f32(xv[b][u][c] & 0xFFFFu) * f, __uint_as_float(xv[b][u][c] & 0xFFFF0000u) * f);
      }
      const float down = __uint_as_float(static_cast<uint32_t>(e - 14 + 127) << 23);
#pragma unroll
      for (int i = 0; i < 4; ++i) back[i] = __shfl(down, 4 * g + i, 64);  // lane 4 g + i holds row 4 g + i
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
          // the codes of block b + 2 and the lookups of block b + 1 on their
          // way while block b is multiplied
          floatx4 sum = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
          uint2 w[3];
          auto read_codes = [&](int b) {
            w[b % 3] = *reinterpret_cast<const uint2*>(stage + sk::slot_of(ln, 2 * b + (g >> 1)) + 8 * (g & 1));
          };
          read_codes(0);
          read_codes(1);
          const floatx4 f0 = *reinterpret_cast<const floatx4*>(scl + ln * kNb), f1 = *reinterpret_cast<const floatx4*>(scl + ln * kNb + 4);
          u32x4 lk[2][2];
          look_up(lk[0], w[0], tabc, slot);
#pragma unroll
          for (int b = 0; b < kNb; ++b) {
            if (b + 2 < kNb) read_codes(b + 2);
            if (b + 1 < kNb) look_up(lk[(b + 1) & 1], w[(b + 1) % 3], tabc, slot);
            __builtin_amdgcn_sched_barrier(0);
            floatx4 d = sk::mfma<true>(xv[b][0], lk[b & 1][0], floatx4{0.0f, 0.0f, 0.0f, 0.0f});
            d = sk::mfma<true>(xv[b][1], lk[b & 1][1], d);
            const float f = b < 4 ? f0[b & 3] : f1[b & 3];
#pragma unroll
            for (int i = 0; i < 4; ++i) sum[i] = fmaf(f, d[i], sum[i]);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[gi][i] = fmaf(back[i], sum[i], acc[gi][i]);
          sk::wave_lds_order();
        }
      }
      // the waves' partial tiles, added in wave order
      if (live) {
#pragma unroll
        for (int gi = 0; gi < kG; ++gi) part[(wave * kG + gi) * 64 + lane] = acc[gi];
      }
      sk::lds_barrier();
      for (int t = opaque(threadIdx.x); t < batch * 64; t += sk::kThreads) {
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
