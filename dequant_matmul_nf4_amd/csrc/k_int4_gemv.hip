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
// below float32.  (An offset of 1 on q / 16 in [0, 1) costs the sum about two
// bits; the usual 128 + q would cost five.)
//
// Bound: reading the codes.  See skinny_tile.h for the walk and skinny
// products' staging.
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

// A scale as it is stored (converted where it is used, so that the load stays in flight).
__device__ __forceinline__ uint32_t scale_bits(const void* p, int type, int64_t i) {
  return type == 0 ? static_cast<const uint32_t*>(p)[i] : static_cast<const uint16_t*>(p)[i];
}
__device__ __forceinline__ float scale_value(uint32_t b, int type) {
  const float f16 = static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(b)));
  return type == 0 ? __uint_as_float(b) : type == 1 ? bf16_to_f32(b) : f16;
}

__device__ __forceinline__ void store_y(void* y, int type, int64_t i, float v) {
  if (type == 0) static_cast<float*>(y)[i] = v;
  else if (type == 1) static_cast<uint16_t*>(y)[i] = static_cast<uint16_t>(f32_to_bf16(v));
  else static_cast<_Float16*>(y)[i] = static_cast<_Float16>(v);
}

constexpr int kG = 4;  // groups of 16 rows a wave takes per batch: x is read once for all of them

// kGrp: columns per scale.
template <bool kF16, int kGrp>
__global__ __launch_bounds__(sk::kThreads) void k_int4_gemv(Int4Args a) {
  constexpr int kPw = kGrp / 32;        // code words a lane takes per scale group
  constexpr int kNs = kSeg / kGrp;      // scale groups per step
  __shared__ __align__(16) char stage_all[kWaves][sk::kStageBytes];
  __shared__ __align__(16) float2 scl_all[kWaves][sk::kRows * kNs];
  __shared__ __align__(16) floatx4 part[kWaves * kG * 64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int ln = lane & 15, g = lane >> 4;
  const sk::Plan& pl = a.pl;
  const int kw = wave % pl.ks, rw = wave / pl.ks;  // the wave's share of the columns, of the groups
  const bool live = rw < pl.rs;
  char* stage = stage_all[wave];
  float2* scl = scl_all[wave];
  const int64_t row_bytes = a.cols / 2, ngrp = a.cols / kGrp;

  const int64_t ngroups = (a.rows + 15) / 16;
  const int64_t gb = ngroups * blockIdx.x / gridDim.x, ge = ngroups * (blockIdx.x + 1) / gridDim.x;
  const int64_t klo = kw * pl.per, khi = klo + pl.per < a.cols ? klo + pl.per : a.cols;
  const int nseg = static_cast<int>((khi - klo + kSeg - 1) / kSeg);

  Codes codes;
  uint32_t sc[kNs >= 4 ? kNs / 4 : 1], zp[kNs >= 4 ? kNs / 4 : 1];
  // The loads of one step; lane (ln, g) takes the scales of row ln, groups g, g + 4, ...
  auto load_step = [&](int64_t group, int seg) {
    const int64_t k0 = klo + static_cast<int64_t>(seg) * kSeg;
    codes = sk::load_codes(a.packed, row_bytes, group * 16, a.rows, k0, khi, lane);
    const int64_t row = group * 16 + ln < a.rows ? group * 16 + ln : a.rows - 1;
    const int64_t last = (khi - k0) / kGrp - 1;
#pragma unroll
    for (int j = 0; j < (kNs >= 4 ? kNs / 4 : 1); ++j) {
      int64_t q = kNs >= 4 ? g + 4 * j : (g % kNs);
      q = q < last ? q : last;
      const int64_t at = row * ngrp + k0 / kGrp + q;
      sc[j] = scale_bits(a.scales, a.scale_type, at);
      zp[j] = a.zeros ? a.zeros[at] : 8u;
    }
  };

  u32x4 xv[kNs][kPw];
  floatx4 xsum[kNs];
  auto load_x = [&](int seg) {
    const int64_t k0 = klo + static_cast<int64_t>(seg) * kSeg;
    // rows past m repeat row m - 1: they reach only rows of the result that are not stored
    const uint16_t* xr = a.x + static_cast<int64_t>(ln < a.m ? ln : a.m - 1) * a.cols;
    const u32x4 ones = kF16 ? u32x4{0x3C003C00u, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u}
                            : u32x4{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
#pragma unroll
    for (int s = 0; s < kNs; ++s)
#pragma unroll
      for (int u = 0; u < kPw; ++u) {
        const int64_t k = k0 + s * kGrp + 8 * kPw * g + 8 * u;
        xv[s][u] = *reinterpret_cast<const u32x4*>(xr + (k < khi ? k : khi - 8));
      }
#pragma unroll
    for (int s = 0; s < kNs; ++s) {
      xsum[s] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int u = 0; u < kPw; ++u) {
        const bool in = k0 + s * kGrp < khi;
        const u32x4 v = pair_order(xv[s][u]);
        xv[s][u] = u32x4{in ? v[0] : 0u, in ? v[1] : 0u, in ? v[2] : 0u, in ? v[3] : 0u};
        xsum[s] = sk::mfma<kF16>(xv[s][u], ones, xsum[s]);
      }
    }
  };

  int have = -1;  // the segment whose x is held
  if (live && gb + rw < ge) load_step(gb + rw, 0);
  for (int64_t base = gb; base < ge; base += static_cast<int64_t>(pl.rs) * kG) {
    floatx4 acc[kG];
#pragma unroll
    for (int i = 0; i < kG; ++i) acc[i] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int seg = 0; live && seg < nseg; ++seg) {
      if (seg != have) {
        load_x(seg);
        have = seg;
      }
#pragma unroll
      for (int gi = 0; gi < kG; ++gi) {
        const int64_t group = base + static_cast<int64_t>(gi) * pl.rs + rw;
        if (group >= ge) continue;
        // this step's codes and scales into LDS, then the next step's loads
        sk::stage_codes(codes, stage, lane);
#pragma unroll
        for (int j = 0; j < (kNs >= 4 ? kNs / 4 : 1); ++j) {
          const int q = kNs >= 4 ? g + 4 * j : (g % kNs);
          scl[ln * kNs + q] = make_float2(16.0f * scale_value(sc[j], a.scale_type), -1.0f - static_cast<float>(zp[j]) * 0.0625f);
        }
        {
          int64_t ng = group + pl.rs;
          int ns = seg;
          if (gi + 1 == kG || ng >= ge) {  // the batch's next segment, or the next batch
            ng = base + rw;
            if (++ns == nseg) {
              ns = 0;
              ng += static_cast<int64_t>(pl.rs) * kG;
            }
          }
          if (ng < ge) load_step(ng, ns);
        }
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
          floatx4 d = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int u = 0; u < kPw; ++u) d = sk::mfma<kF16>(xv[s][u], expand<kF16>(w[u]), d);
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[gi][i] = fmaf(f.x, fmaf(f.y, xsum[s][i], d[i]), acc[gi][i]);
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
    for (int t = threadIdx.x; t < pl.rs * kG * 64; t += sk::kThreads) {
      const int l = t & 63, gi = (t >> 6) % kG, r = (t >> 6) / kG;
      const int64_t group = base + static_cast<int64_t>(gi) * pl.rs + r;
      if (group >= ge) continue;
      floatx4 v = part[(r * pl.ks * kG + gi) * 64 + l];
      for (int k = 1; k < pl.ks; ++k) v += part[((r * pl.ks + k) * kG + gi) * 64 + l];
      const int64_t row = group * 16 + (l & 15);
      if (row >= a.rows) continue;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int xm = 4 * (l >> 4) + i;
        if (xm < a.m) store_y(a.y, a.y_type, xm * a.rows + row, v[i]);
      }
    }
    sk::lds_barrier();
  }
}

}  // namespace

hipError_t launch_int4_gemv(const Int4Weight& w, const uint16_t* x, int x_f16, int64_t m, void* y, int y_type,
                            hipStream_t s) {
  Int4Args a{};
  a.packed = w.packed; a.rows = w.rows; a.cols = w.cols; a.scales = w.scales; a.scale_type = w.scale_type;
  a.zeros = w.zeros; a.x = x; a.m = static_cast<int>(m); a.y = y; a.y_type = y_type;
  const int64_t groups = (w.rows + 15) / 16;
  // one workgroup per compute unit, fewer where there are not `rs` groups for each
  sk::Plan pl = sk::make_plan(w.cols, 0);
  const int64_t want = (groups + pl.rs - 1) / pl.rs;
  pl.grid = static_cast<int>(want < device_cus() ? want : device_cus());
  a.pl = pl;
  const dim3 gd(static_cast<unsigned>(pl.grid)), bd(sk::kThreads);
#define NF4_INT4(F16) \
  do { \
    if (w.group == 32) hipLaunchKernelGGL((k_int4_gemv<F16, 32>), gd, bd, 0, s, a); \
    else if (w.group == 64) hipLaunchKernelGGL((k_int4_gemv<F16, 64>), gd, bd, 0, s, a); \
    else hipLaunchKernelGGL((k_int4_gemv<F16, 128>), gd, bd, 0, s, a); \
  } while (0)
  if (x_f16) NF4_INT4(true);
  else NF4_INT4(false);
#undef NF4_INT4
  return hipGetLastError();
}

}  // namespace nf4i
