// y = x . W^T for 1 <= m <= 16 rows of x and uniform 4-bit weights with a
// scale s (and zero point z) per group of 32, 64 or 128 columns of a row:
//
//   y[i][r] = sum over groups G of s[r][G] (sum_{c in G} q[r][c] x[i][c] - z[r][G] sum_{c in G} x[i][c])
//
// A code q is put into the four leading fraction bits of a 16-bit 1.0: the
// operand is 1 + q / 16, exact in bfloat16 and in float16, two codes per
// and-or.  With d the products' sum in float32 and X the sum of x over the
// group (one product of x with ones per step, kept while x is),
//   sum (q - z) x = 16 (d - (1 + z / 16) X),
// so a group costs two fused multiply-adds per output and nothing is rounded
// below float32.  The 16 goes to the finished sums: 16 s would overflow for the
// largest float32 scales.  (An offset of 1 on q / 16 in [0, 1) costs the sum about two
// bits; 128 + q, whose offset needs no shift, would cost five.)
//
// Bound: reading the codes; skinny_tile.h has the walk.  With weights that change
// from call to call 28672x8192 takes 29 us at m = 1 with groups of 128 (4.2 TB/s),
// 39 us at m = 16 with groups of 64 and zero points (3.3 TB/s; 25 us at the rate of
// a large copy; the VALU is busy 39% of the time, a step of 4 KiB takes 359 of its
// instructions); groups of 32 53 us: each scale costs 8 multiply-adds of a lane.
// 4096x4096 takes 7 us: launch, x, one step and the join follow each other.
#include "expert_int4.h"
#include "skinny_tile.h"

namespace nf4i {
namespace {

using sk::Codes;
using sk::floatx4;
using sk::kSeg;
using sk::kWaves;
using sk::u32x4;

struct Int4Args {
  const uint8_t* packed;
  int64_t rows, cols;
  const void* scales;
  int scale_type;         // 0 float32, 1 bfloat16, 2 float16
  const uint8_t* zeros;   // or null: 8 everywhere
  const uint16_t* x;
  int m;
  void* y;
  int y_type;             // as scale_type
  sk::Plan pl;
};

// Eight codes of a word (element 2 j in the high half of byte j) as four
// operand words holding elements (1, 5), (0, 4), (3, 7), (2, 6).
template <bool kF16>
__device__ __forceinline__ u32x4 expand(uint32_t c) {
  if constexpr (kF16) {
    constexpr uint32_t mask = 0x03C003C0u, one = 0x3C003C00u;
    return u32x4{((c << 6) & mask) | one, ((c << 2) & mask) | one, ((c >> 2) & mask) | one, ((c >> 6) & mask) | one};
  } else {
    constexpr uint32_t mask = 0x00780078u, one = 0x3F803F80u;
    return u32x4{((c << 3) & mask) | one, ((c >> 1) & mask) | one, ((c >> 5) & mask) | one, ((c >> 9) & mask) | one};
  }
}

// x in the same order.
__device__ __forceinline__ u32x4 pair_order(const u32x4& v) {
  return u32x4{__builtin_amdgcn_perm(v[2], v[0], 0x07060302u), __builtin_amdgcn_perm(v[2], v[0], 0x05040100u),
               __builtin_amdgcn_perm(v[3], v[1], 0x07060302u), __builtin_amdgcn_perm(v[3], v[1], 0x05040100u)};
}

// The value of a scale as it is stored (converted where it is used, so that
// its load stays in flight).
template <bool kWide>
__device__ __forceinline__ float scale_value(uint32_t b, int type) {
  if constexpr (kWide) return __uint_as_float(b);
  const float f16 = static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(b))), bf16 = bf16_to_f32(b);
  return type == 1 ? bf16 : f16;
}

__device__ __forceinline__ void store_y(void* y, int type, int64_t i, float v) {
  if (type == 0) static_cast<float*>(y)[i] = v;
  else if (type == 1) static_cast<uint16_t*>(y)[i] = static_cast<uint16_t>(f32_to_bf16(v));
  else static_cast<_Float16*>(y)[i] = static_cast<_Float16>(v);
}

// What one step brings: codes, and the scales and zero points that the lane
// converts (row ln, scale groups g kPer .. of the step) in their stored types: a
// value widened where it is loaded is waited for there.
template <bool kWide>
struct ScaleBits { typedef uint16_t type; };
template <>
struct ScaleBits<true> { typedef uint32_t type; };

template <int kPer, bool kWide>
struct Step {
  Codes codes;
  typename ScaleBits<kWide>::type s[kPer];
  uint8_t z[kPer];
};

// kGrp: columns per scale; kWide: float32 scales; kG: groups of 16 rows a wave
// takes per batch, x being read once for all of them; kOnce: a wave's columns
// are one segment, whose x is read once for all batches.  In batches of two the
// next segment's x is on its way while this one is multiplied, where the
// registers allow it.
template <bool kF16, int kGrp, bool kWide, int kG, bool kOnce>
__global__ __launch_bounds__(sk::kThreads, 2) void k_int4_gemv(Int4Args a) {
  constexpr int kPw = kGrp / 32;        // code words a lane takes per scale group
  constexpr int kNs = kSeg / kGrp;      // scale groups per step
  constexpr int kPer = kNs / 4;
  constexpr bool kAhead = !kOnce && kG == 2 && kGrp >= 64;
  __shared__ __align__(16) char stage_all[kWaves][sk::kStageBytes];
  __shared__ __align__(16) float2 scl_all[kWaves][sk::kRows * kNs];
  __shared__ __align__(16) floatx4 xsum_all[kWaves][kNs * 4];
  __shared__ __align__(16) floatx4 part[kWaves * kG * 64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int ln = lane & 15, g = lane >> 4;
  const sk::Plan& pl = a.pl;
  const int kw = wave % pl.ks, rw = wave / pl.ks;  // the wave's share of the columns, of the groups
  const bool live = rw < pl.rs;
  char* stage = stage_all[wave];
  float2* scl = scl_all[wave];
  floatx4* xsum = xsum_all[wave];
  const uint32_t row_bytes = static_cast<uint32_t>(a.cols / 2);
  const uint32_t ngrp = static_cast<uint32_t>(a.cols / kGrp);

  // the workgroup's groups, counted from its first; rows are left from there
  const int64_t ngroups = (a.rows + 15) / 16;
  const int64_t gb = ngroups * blockIdx.x / gridDim.x;
  const int ng = static_cast<int>(ngroups * (blockIdx.x + 1) / gridDim.x - gb);
  const int64_t klo = kw * pl.per, khi = klo + pl.per < a.cols ? klo + pl.per : a.cols;
  const int kspan = static_cast<int>(khi - klo);
  const int nseg = (kspan + kSeg - 1) / kSeg;
  const int64_t rows_left = a.rows - gb * 16;
  const int tail = static_cast<int>(rows_left - (ng - 1) * 16 < 16 ? rows_left - (ng - 1) * 16 : 16);  // rows of the last group
  const uint8_t* codes0 = a.packed + gb * 16 * row_bytes + klo / 2;
  const int64_t scale0 = gb * 16 * ngrp + klo / kGrp;
  const int64_t group_bytes = int64_t{16} * row_bytes, group_scales = int64_t{16} * ngrp;
  const sk::CodeLane cl = sk::code_lane(row_bytes, lane);
  const uint32_t srow = static_cast<uint32_t>(ln) * ngrp + g * kPer;

  Step<kPer, kWide> set[2];
  auto load_step = [&](Step<kPer, kWide>& st, int group, int seg, bool wanted) {
    const int rows = group == ng - 1 ? tail : 16;
    const int left = kspan - seg * kSeg;
    sk::load_codes(st.codes, codes0 + (group * group_bytes + seg * (kSeg / 2)), cl, row_bytes, rows, left / 32, wanted, lane);
    const int64_t at = scale0 + (group * group_scales + seg * kNs);  // the step's first scale
    const bool whole = rows == 16 && left >= kSeg;
    const int lq = (left < kSeg ? left : kSeg) / kGrp - 1;
    const uint32_t trow = static_cast<uint32_t>(ln < rows ? ln : rows - 1) * ngrp;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int q = g * kPer + j;
      const uint32_t o = (whole ? srow + j : trow + (q < lq ? q : lq)) & (wanted ? ~0u : 0u);
      if constexpr (kWide) st.s[j] = (static_cast<const uint32_t*>(a.scales) + at)[o];
      else st.s[j] = (static_cast<const uint16_t*>(a.scales) + at)[o];
      st.z[j] = (a.zeros ? a.zeros + at : a.packed)[o & (a.zeros ? ~0u : 0u)];
    }
  };

  // x of a segment: as it is read, and as the operand with the groups' sums
  u32x4 xn[kNs][kPw], xv[kNs][kPw];
  auto load_x = [&](int seg) {
    // rows past m repeat row m - 1: they reach only rows of the result that are not stored
    const uint16_t* xr = a.x + (static_cast<int64_t>(ln < a.m ? ln : a.m - 1) * a.cols + klo);
    const int left = kspan - seg * kSeg;
    if (left >= kSeg) {
      const uint16_t* p = xr + (seg * kSeg + 8 * kPw * g);
#pragma unroll
      for (int s = 0; s < kNs; ++s)
#pragma unroll
        for (int u = 0; u < kPw; ++u) xn[s][u] = *reinterpret_cast<const u32x4*>(p + s * kGrp + 8 * u);
    } else {
      const uint16_t* p = xr + seg * kSeg;
      const int gk = 8 * kPw * static_cast<int>(opaque(g));
#pragma unroll
      for (int s = 0; s < kNs; ++s)
#pragma unroll
        for (int u = 0; u < kPw; ++u) {
          const int k = s * kGrp + gk + 8 * u;
          xn[s][u] = *reinterpret_cast<const u32x4*>(p + (k < left ? k : left - 8));
        }
    }
  };
  auto take_x = [&](int seg) {
    const u32x4 ones = kF16 ? u32x4{0x3C003C00u, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u}
                            : u32x4{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
#pragma unroll
    for (int s = 0; s < kNs; ++s) {
      floatx4 sum = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int u = 0; u < kPw; ++u) {
        const bool in = seg * kSeg + s * kGrp < kspan;
        const u32x4 v = pair_order(xn[s][u]);
        xv[s][u] = u32x4{in ? v[0] : 0u, in ? v[1] : 0u, in ? v[2] : 0u, in ? v[3] : 0u};
        sum = sk::mfma<kF16>(xv[s][u], ones, sum);
      }
      xsum[s * 4 + g] = sum;  // the same in the 16 lanes of g
    }
  };

  // Position p of a wave's walk is group p % kG of segment p / kG of the batch.
  // Two steps are on their way at any time, in the two register sets by the
  // parity of p; a position past the workgroup's groups is not multiplied.
  const int batch = pl.rs * kG;
  auto load_at = [&](Step<kPer, kWide>& st, int base, int seg, int gi) {
    if (seg >= nseg) {
      seg -= nseg;
      base += batch;
    }
    const int group = base + gi * pl.rs + rw;
    load_step(st, group < ng ? group : ng - 1, seg, group < ng);
  };
  if constexpr (kOnce || kAhead) load_x(0);
  load_at(set[0], 0, 0, 0);
  load_at(set[1], 0, 0, 1);
  if constexpr (kOnce) take_x(0);
  for (int base = 0; base < ng; base += batch) {
    floatx4 acc[kG];
#pragma unroll
    for (int i = 0; i < kG; ++i) acc[i] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int seg = 0; live && seg < nseg; ++seg) {
      if constexpr (!kOnce) {
        if constexpr (!kAhead) load_x(seg);
        take_x(seg);
        if constexpr (kAhead) load_x(seg + 1 < nseg ? seg + 1 : 0);
      }
#pragma unroll
      for (int gi = 0; gi < kG; ++gi) {
        Step<kPer, kWide>& st = set[gi & 1];
        const bool here = base + gi * pl.rs + rw < ng;
        if (here) {
          // this step's codes and scales into LDS
          sk::stage_codes(st.codes, stage, lane);
#pragma unroll
          for (int j = 0; j < kPer; ++j)
            scl[ln * kNs + g * kPer + j] =
                make_float2(scale_value<kWide>(st.s[j], a.scale_type), a.zeros ? -1.0f - static_cast<float>(st.z[j]) * 0.0625f : -1.5f);
        }
        load_at(st, base, gi + 2 < kG ? seg : seg + 1, (gi + 2) % kG);
        if (!here) continue;
        sk::wave_lds_order();
#pragma unroll
        for (int s = 0; s < kNs; ++s) {
          uint32_t w[kPw];
          if constexpr (kPw == 1) {
            w[0] = *reinterpret_cast<const uint32_t*>(stage + sk::slot_of(ln, s) + 4 * g);
          } else if constexpr (kPw == 2) {
            const uint2 v = *reinterpret_cast<const uint2*>(stage + sk::slot_of(ln, 2 * s + (g >> 1)) + 8 * (g & 1));
            w[0] = v.x;
            w[1] = v.y;
          } else {
            const u32x4 v = *reinterpret_cast<const u32x4*>(stage + sk::slot_of(ln, 4 * s + g));
#pragma unroll
            for (int u = 0; u < 4; ++u) w[u] = v[u];
          }
          const float2 f = scl[ln * kNs + s];
          const floatx4 xs = xsum[s * 4 + g];
          floatx4 d = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int u = 0; u < kPw; ++u) d = sk::mfma<kF16>(xv[s][u], expand<kF16>(w[u]), d);
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[gi][i] = fmaf(f.x, fmaf(f.y, xs[i], d[i]), acc[gi][i]);
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
    for (int t = opaque(threadIdx.x); t < batch * 64; t += sk::kThreads) {
      const int l = t & 63, gi = (t >> 6) % kG, r = (t >> 6) / kG;
      const int group = base + gi * pl.rs + r;
      if (group >= ng) continue;
      floatx4 v = part[(r * pl.ks * kG + gi) * 64 + l];
      for (int k = 1; k < pl.ks; ++k) v += part[((r * pl.ks + k) * kG + gi) * 64 + l];
      const int64_t row = (gb + group) * 16 + (l & 15);
      if (row >= a.rows) continue;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int xm = 4 * (l >> 4) + i;
        if (xm < a.m) store_y(a.y, a.y_type, xm * a.rows + row, 16.0f * v[i]);
      }
    }
    sk::lds_barrier();
  }
}

template <bool kF16, int kGrp, bool kWide>
void launch(const Int4Args& a, dim3 gd, hipStream_t s) {
  // A wave's columns in one segment: x is read once and the batch only decides
  // how often partial tiles are added up.  Otherwise x is read once a batch:
  // about as many groups as a wave has, 2 or 8 (groups of 64 at m = 16, 2, 4 and
  // 8 a batch: 28672x8192, 7 groups a wave, 63, 46 and 38 us; 16384x8192, 4
  // groups, 36, 26 and 29 us; 8192x28672, 2 groups, 56, 62 and 69 us).
  const int64_t groups = (a.rows + 15) / 16, each = groups / (static_cast<int64_t>(gd.x) * a.pl.rs);
  const dim3 bd(sk::kThreads);
  if (a.pl.per <= kSeg) hipLaunchKernelGGL((k_int4_gemv<kF16, kGrp, kWide, 4, true>), gd, bd, 0, s, a);
  else if (each >= 3) hipLaunchKernelGGL((k_int4_gemv<kF16, kGrp, kWide, 8, false>), gd, bd, 0, s, a);
  else hipLaunchKernelGGL((k_int4_gemv<kF16, kGrp, kWide, 2, false>), gd, bd, 0, s, a);
}

template <bool kF16>
void launch(const Int4Args& a, int group, dim3 gd, hipStream_t s) {
  const bool wide = a.scale_type == 0;
  if (group == 32) wide ? launch<kF16, 32, true>(a, gd, s) : launch<kF16, 32, false>(a, gd, s);
  else if (group == 64) wide ? launch<kF16, 64, true>(a, gd, s) : launch<kF16, 64, false>(a, gd, s);
  else wide ? launch<kF16, 128, true>(a, gd, s) : launch<kF16, 128, false>(a, gd, s);
}

}  // namespace

hipError_t launch_int4_gemv(const Int4Weight& w, const uint16_t* x, int x_f16, int64_t m, void* y, int y_type,
                            hipStream_t s) {
  Int4Args a{};
  a.packed = w.packed; a.rows = w.rows; a.cols = w.cols; a.scales = w.scales; a.scale_type = w.scale_type;
  a.zeros = w.zeros; a.x = x; a.m = static_cast<int>(m); a.y = y; a.y_type = y_type;
  a.pl = sk::make_plan(w.cols);
  // one workgroup per compute unit, fewer where there are not `rs` groups for
  // each; more where a workgroup's groups would not be counted in 31 bits
  const int64_t groups = (w.rows + 15) / 16, want = (groups + a.pl.rs - 1) / a.pl.rs;
  int64_t grid = want < device_cus() ? want : device_cus();
  while (groups / grid >= (int64_t{1} << 26)) grid *= 2;
  const dim3 gd(static_cast<unsigned>(grid));
  if (x_f16) launch<true>(a, w.group, gd, s);
  else launch<false>(a, w.group, gd, s);
  return hipGetLastError();
}

}  // namespace nf4i
