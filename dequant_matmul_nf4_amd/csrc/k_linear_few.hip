// A layer's product with its epilogue for a decode batch, and for more rows where
// there is little work: tiles of 16 rows of x and 16 of the weight.
//
// A product of v_mfma_f32_16x16x32 spans half a block of each of its 16 weight
// rows: the weight enters as its levels in float16 (rounded by 2^-11 at most), the two
// products of a block run into an accumulator of their own, and the block's scale is
// applied to that in float32, so no scaled weight is rounded.  x enters exactly but
// for values 2^-29 of the largest of its row's 256 columns: scaled by a power of two of
// those columns, taken back on their sums.
//
// Few rows are bound by reading the codes, small weights by latency, so a
// workgroup of 16 waves (one per compute unit, 4 waves to a SIMD) covers up to 4096
// columns at once: a wave takes 256 of them, holds x's share in registers and walks
// over groups of 16 weight rows in steps of 2 KiB of codes, two steps on their way.
// Every load's lanes lie side by side in memory, and codes, x and scales are
// turned into operand order in the wave's own LDS: with a row to each lane the address
// unit took 64 clocks a load, and 4096x4096 with 16 rows 23 us instead of 10.  Longer
// rows have a wave take several segments, x of the next asked for before the
// codes after it, because loads return in order.  The waves' partial tiles meet in
// LDS and are added in wave order; then every output value has a thread of its own
// for the epilogue (four to a thread spilled the walk's registers).
//
// Measured (int8 scales, time in a graph over changing weights): 16 rows of 512x512
// 4.9 us, of 4096x4096 9.8, of 14336x4096 16.7, of 4096x14336 22, of 28672x8192 42 to 44
// (2.8 TB/s: issue bounds it, 191 vector and 49 LDS instructions a step in all, x's
// conversion among them, which a wave of two segments makes for each of its two batches
// of groups, four times in 14 steps; codes that stay in cache take 29); 8 waves of 512
// columns 11.4, 12.1, 15.4, 31 and 51, 8 waves of 256 with x a segment ahead and four
// steps on their way 43.9 for the last.
#include "linear_epilogue.h"
#include "linear_f16.h"
#include "skinny_tile.h"

namespace nf4i {
namespace {

using sk::floatx4;
using sk::u32x4;

constexpr int kWaves = 16;
constexpr int kThreads = 64 * kWaves;
constexpr int kRows = 16;    // of the weight and of x per product
constexpr int kNb = 4;       // blocks of a weight row per step
constexpr int kCopies = 64;  // of the level table (64 KB): each lane has its own, no two meet in a bank

struct FewArgs {
  const uint8_t* packed;
  int64_t rows;
  Scales sc;
  Codebook cb;
  const uint16_t* x;   // [m][cols]
  int64_t m;
  int nblk;            // blocks of a weight row
  int ks, rs, segs;    // waves that share a group's columns, groups at a time (a power of two), steps of a wave
  int64_t each, more;  // groups of a workgroup; the first `more` workgroups take one more
  lin::FewOut out;
};

// LDS of a wave: x, then each step's codes in operand order; the scales of a step.
constexpr int kStage = 4096;
constexpr int kLoads = 2;  // 16-byte loads of a lane per step

template <bool kDQ>
struct Step {
  u32x4 c[kLoads];  // rows 8 i + lane / 8
  int8_t q;         // of row lane / 4, block lane % 4: second-level code and its group's scale, or the absmax
  float s;
};

// Codes of 16 rows x 256 columns: row r holds 16-byte piece p at slot p ^ (r % 8) of its 128 bytes.
__device__ __forceinline__ int code_row(int i, int lane) { return 8 * i + (lane >> 3); }
__device__ __forceinline__ int code_piece(int i, int lane) { return (lane & 7) ^ (code_row(i, lane) & 7); }
__device__ __forceinline__ uint32_t code_slot(int row, int piece) {
  return static_cast<uint32_t>(row * 128 + ((piece ^ (row & 7)) << 4));
}

__device__ __forceinline__ uint32_t half_pair(float a, float b) {
  typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, half2_t{static_cast<_Float16>(a), static_cast<_Float16>(b)});
}
// Two bf16 values times a power of two (one instruction each).
__device__ __forceinline__ uint32_t scaled_pair(uint32_t v, float f) {
  return half_pair(__builtin_fmaf(bf16_to_f32(v & 0xFFFFu), f, 0.0f), __builtin_fmaf(__uint_as_float(v & 0xFFFF0000u), f, 0.0f));
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

// The table comes first: at address 0 the permute makes a lookup's whole address.
template <bool kF8>
struct __attribute__((aligned(16))) FewLds {
  uint32_t tab[256 * kCopies];
  char stage[kWaves][kStage];
  float scales[kWaves][kRows * kNb];
  float rtab[kF8 ? 256 : 1];
};

// kG: groups of 16 weight rows a wave takes per batch, x being read once for all of them.
template <bool kDQ, bool kF8, int kG>
__global__ __launch_bounds__(kThreads, 4) void k_linear_few(FewArgs a) {
  __shared__ FewLds<kF8> shared;
  auto& tab = shared.tab;
  auto& lds = shared.stage;
  auto& rtab = shared.rtab;
  static_assert(kG * 1024 <= kStage, "a wave's partial tiles take its codes' place");
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int ln = lane & 15, g = lane >> 4;
  const uint32_t level = half_pair(a.cb.level[ln], 0.0f);
  const float mean = kDQ ? *a.sc.mean : 0.0f;
  const int64_t w = blockIdx.x;
  const int ng = static_cast<int>(a.each + (w < a.more ? 1 : 0));  // groups w, w + gridDim.x, ..
  const int64_t row0 = static_cast<int64_t>(blockIdx.y) * kRows;   // of x
  const int cnt = static_cast<int>(a.m - row0 < kRows ? a.m - row0 : kRows);
  int rw = 0;  // the wave's share of the groups, of the columns
#pragma unroll
  for (int i = 1; i < kWaves; ++i) rw += wave >= i * a.ks ? 1 : 0;
  const int kw = wave - rw * a.ks;
  const int batch = a.rs * kG;
  const bool live = rw < a.rs && rw < ng;
  const uint32_t nblk = static_cast<uint32_t>(a.nblk), row_bytes = nblk * 32;
  const int first = kw * a.segs * kNb;  // the wave's first block
  const int span = a.nblk - first < a.segs * kNb ? a.nblk - first : a.segs * kNb;  // its blocks
  const int nseg = (span + kNb - 1) / kNb;
  const char* tabc = reinterpret_cast<const char*>(tab);
  char* stage = lds[wave];
  float* scl = shared.scales[wave];
  const uint32_t slot = static_cast<uint32_t>(lane) << 2;
  // every load's lanes lie side by side in a few lines (one whose every lane is in another line
  // takes the address unit a clock for each)
  const int sn = lane >> 2, sj = lane & 3;
  uint32_t coff[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) coff[i] = code_row(i, lane) * row_bytes + 16 * code_piece(i, lane);
  const uint32_t soff = sn * nblk + sj;
  const char* const x0 = reinterpret_cast<const char*>(a.x + (row0 * a.nblk + first) * 64);

  auto load_step = [&](Step<kDQ>& st, int k, int seg) {
    const bool wanted = k < ng;
    const int64_t group = w + static_cast<int64_t>(wanted ? k : 0) * gridDim.x;
    const int64_t left = a.rows - group * kRows;
    const int nb = span - seg * kNb;
    const int64_t b0 = group * kRows * a.nblk + first + seg * kNb;
    uint32_t off[kLoads], so = soff;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) off[i] = coff[i];
    if (left < kRows || nb < kNb) {  // what lies past the last repeats it
      const int l2 = opaque(lane), rows = left < kRows ? static_cast<int>(left) : kRows, blocks = nb < kNb ? nb : kNb;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int row = code_row(i, l2), piece = code_piece(i, l2);
        off[i] = (row < rows ? row : rows - 1) * row_bytes + 16 * (piece < 2 * blocks ? piece : 2 * blocks - 1);
      }
      const int row = l2 >> 2, j = l2 & 3;
      so = (row < rows ? row : rows - 1) * nblk + (j < blocks ? j : blocks - 1);
    }
    const uint32_t keep = wanted ? ~0u : 0u;  // no branch around a load; one that is not wanted reads one place
    const uint8_t* codes = a.packed + b0 * 32;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) st.c[i] = *reinterpret_cast<const u32x4*>(codes + (off[i] & keep));
    so &= keep;
    if constexpr (kDQ) {
      st.q = (a.sc.q + b0)[so];
      st.s = a.sc.absmax2[(b0 + so) >> 8];
    } else {
      st.s = (a.sc.absmax + b0)[so];
    }
  };

  u32x4 xv[kNb][2];
  floatx4 back;  // the powers of two that scale the sums of x rows 4 g .. back
  auto fetch_x = [&](int seg) {
    // 256 bytes of 4 rows per load; load i of a half takes row 4 i + g, the piece that belongs in
    // slot ln of it.  Rows past the tile's repeat its last and are not stored.  The offsets are made
    // here: kept, they take registers that the steps want
    const int l2 = opaque(lane), last = 8 * (span - seg * kNb) - 1;
    const char* p = x0 + seg * (kNb * 128);
    uint32_t off[4], at[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = sk::code_row(i, l2);
      off[i] = static_cast<uint32_t>(row < cnt ? row : cnt - 1) * (nblk * 128);
      at[i] = sk::code_piece(i, l2);
    }
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int piece = 16 * c + static_cast<int>(at[i]);
        xv[2 * c + (i >> 1)][i & 1] = *reinterpret_cast<const u32x4*>(p + (off[i] + 16 * (piece < last ? piece : last)));
      }
  };
  auto convert_x = [&](int seg) {
    // turned in the wave's LDS: lane (row ln, g) takes columns 16 g .. + 15 of each block
#pragma unroll
    for (int c = 0; c < 2; ++c) {
#pragma unroll
      for (int i = 0; i < 4; ++i) *reinterpret_cast<u32x4*>(stage + i * 1024 + lane * 16) = xv[2 * c + (i >> 1)][i & 1];
      sk::wave_lds_order();
#pragma unroll
      for (int i = 0; i < 4; ++i)
        xv[2 * c + (i >> 1)][i & 1] = *reinterpret_cast<const u32x4*>(stage + sk::slot_of(ln, 8 * (i >> 1) + 2 * g + (i & 1)));
      sk::wave_lds_order();
    }
    // the largest of the row's magnitudes in the segment, as bfloat16 bits
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    const int nb = span - seg * kNb;
    u16x2 top2 = {0, 0};
#pragma unroll
    for (int b = 0; b < kNb; ++b)
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int c = 0; c < 4; ++c) top2 = __builtin_elementwise_max(top2, __builtin_bit_cast(u16x2, xv[b][u][c] & 0x7FFF7FFFu));
    uint32_t top = static_cast<uint32_t>(top2.x > top2.y ? top2.x : top2.y) << 16;
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
    for (int b = 0; b < kNb; ++b)
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int c = 0; c < 4; ++c) xv[b][u][c] = scaled_pair(xv[b][u][c], up);
    if (nb < kNb) {  // zeros past the columns' end, whose loads repeat the last (times zero an infinity would be NaN)
#pragma unroll
      for (int b = 1; b < kNb; ++b)
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int c = 0; c < 4; ++c) xv[b][u][c] = b < nb ? xv[b][u][c] : 0u;
    }
    const float down = __uint_as_float(static_cast<uint32_t>(e - 14 + 127) << 23);
#pragma unroll
    for (int i = 0; i < 4; ++i) back[i] = __shfl(down, 4 * g + i, 64);  // lane 4 g + i holds row 4 g + i
  };

  // two steps on their way in two register sets: step p of a batch is group p % kG of segment p / kG
  Step<kDQ> set[2];
  auto load_at = [&](Step<kDQ>& st, int base, int seg, int gi) {
    if (seg >= nseg) {
      seg -= nseg;
      base += batch;
    }
    load_step(st, base + gi * a.rs + rw, seg < nseg ? seg : 0);
  };
  auto multiply = [&](floatx4& acc) {
    sk::wave_lds_order();
    const floatx4 f = *reinterpret_cast<const floatx4*>(scl + ln * kNb);
    floatx4 sum = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
    uint2 cw[kNb];
#pragma unroll
    for (int b = 0; b < kNb; ++b) cw[b] = *reinterpret_cast<const uint2*>(stage + code_slot(ln, 2 * b + (g >> 1)) + 8 * (g & 1));
    u32x4 lk[2][2];
    look_up(lk[0], cw[0], tabc, slot);
#pragma unroll
    for (int b = 0; b < kNb; ++b) {
      // the lookups of block b + 1 on their way while block b is multiplied
      if (b + 1 < kNb) look_up(lk[(b + 1) & 1], cw[b + 1], tabc, slot);
      __builtin_amdgcn_sched_barrier(0);
      floatx4 d = sk::mfma<true>(xv[b][0], lk[b & 1][0], floatx4{0.0f, 0.0f, 0.0f, 0.0f});
      d = sk::mfma<true>(xv[b][1], lk[b & 1][1], d);
#pragma unroll
      for (int i = 0; i < 4; ++i) sum[i] = fmaf(f[b], d[i], sum[i]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = fmaf(back[i], sum[i], acc[i]);
    sk::wave_lds_order();
  };
  auto stepped = [&](Step<kDQ>& st, floatx4& acc, int base, int seg, int gi) {
    const bool here = base + gi * a.rs + rw < ng;
    if (here) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) *reinterpret_cast<u32x4*>(stage + i * 1024 + lane * 16) = st.c[i];
      if constexpr (kDQ) scl[lane] = (kF8 ? rtab[st.q & 0xFF] : div127(st.q)) * st.s + mean;  // a_hat, three roundings
      else scl[lane] = st.s;
    }
    // the next segment's x goes out ahead of the codes after it: loads return in order
    const bool turn = gi == kG - 1 && nseg > 1;
    if (!turn) load_at(st, base, seg + (gi + 2) / kG, (gi + 2) % kG);
    if (here) multiply(acc);
    if (turn) {
      fetch_x(seg + 1 < nseg ? seg + 1 : 0);
      load_at(st, base, seg + (gi + 2) / kG, (gi + 2) % kG);
    }
  };
  if (live) {
    fetch_x(0);
    load_at(set[0], 0, 0, 0);
    load_at(set[1], 0, 1 / kG, 1 % kG);
  }
  {
    // Entry e of the table is levels e / 16 and e % 16; 16 lanes write an entry's copies, so
    // a pass of the threads writes 64 entries, a lane those of one second level.
    const uint32_t second = static_cast<uint32_t>(__shfl(static_cast<int>(level), (4 * wave + g) & 15, 64)) << 16;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const uint32_t e = static_cast<uint32_t>(__builtin_amdgcn_readlane(level, 4 * p + (wave >> 2))) | second;
      *reinterpret_cast<u32x4*>(tab + p * 4 * kThreads + 4 * threadIdx.x) = u32x4{e, e, e, e};
    }
    if constexpr (kF8)
      if (threadIdx.x < 256) rtab[threadIdx.x] = kE4m3Ratio.v[threadIdx.x];
    sk::lds_barrier();
  }
  for (int base = 0; base < ng; base += batch) {
    if (live) {
      floatx4 acc[kG];
#pragma unroll
      for (int i = 0; i < kG; ++i) acc[i] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
      auto segment = [&](int seg, int odd) {
        if (nseg > 1 || base == 0) convert_x(seg);
#pragma unroll
        for (int gi = 0; gi < kG; ++gi) stepped(set[(odd * kG + gi) & 1], acc[gi], base, seg, gi);
      };
      for (int seg = 0; seg < nseg; ++seg) {
        segment(seg, 0);
        if constexpr (kG % 2 != 0) {
          if (++seg < nseg) segment(seg, 1);
        }
      }
      sk::wave_lds_order();
#pragma unroll
      for (int gi = 0; gi < kG; ++gi) *reinterpret_cast<floatx4*>(stage + (gi * 64 + lane) * 16) = acc[gi];
    }
    sk::lds_barrier();
    // the waves' partial tiles, added in wave order
    const int here = ng - base < batch ? ng - base : batch;
    const int rs_log = __builtin_ctz(a.rs);
    for (int t = opaque(threadIdx.x); t < here * 256; t += kThreads) {
      const int l = t & 63, i = (t >> 6) & 3, k = t >> 8, gi = k >> rs_log, r = k & (a.rs - 1);
      const char* from = lds[r * a.ks] + (gi * 64 + l) * 16 + 4 * i;
      float z[1] = {*reinterpret_cast<const float*>(from)};
      for (int q = 1; q < a.ks; ++q) z[0] += *reinterpret_cast<const float*>(from + q * kStage);
      const int64_t row = (w + static_cast<int64_t>(base + k) * gridDim.x) * kRows + (l & 15);
      const int xm = 4 * (l >> 4) + i;
      if (row < a.rows && xm < cnt) a.out.store(row0 + xm, 1, row, z);
    }
    if constexpr (kG == 1) break;  // one batch
    sk::lds_barrier();
  }
}

template <bool kDQ, bool kF8>
void launch(const FewArgs& a, dim3 grid, hipStream_t s) {
  // A workgroup's groups in one go of one a wave, of two, or batches of four: what is held for more
  // groups costs registers and loads that find nothing (4096x4096 with 16 rows 10.1 us by the first,
  // 15 by the last; with 32 rows 11.4 by the second, 12.4 by the last).
  const int64_t groups = a.each + (a.more > 0 ? 1 : 0);
  if (groups <= a.rs) hipLaunchKernelGGL((k_linear_few<kDQ, kF8, 1>), grid, dim3(kThreads), 0, s, a);
  else if (groups <= 2 * a.rs) hipLaunchKernelGGL((k_linear_few<kDQ, kF8, 2>), grid, dim3(kThreads), 0, s, a);
  else hipLaunchKernelGGL((k_linear_few<kDQ, kF8, 4>), grid, dim3(kThreads), 0, s, a);
}

}  // namespace

hipError_t launch_linear_few(const uint8_t* packed, int64_t rows, int64_t cols, Scales sc, const uint16_t* x, int64_t m,
                             uint16_t* y, const Epilogue& ep, const uint16_t* u, const uint16_t* lora_b, int r, hipStream_t s) {
  FewArgs a{};
  a.packed = packed; a.rows = rows; a.sc = sc; a.cb = codebook(sc.fp4); a.x = x; a.m = m;
  a.nblk = static_cast<int>(cols / 64);
  const int segs = (a.nblk + kNb - 1) / kNb;
  a.segs = (segs + kWaves - 1) / kWaves;
  a.ks = (segs + a.segs - 1) / a.segs;
  for (a.rs = 1; 2 * a.rs * a.ks <= kWaves; a.rs *= 2) {}
  const int64_t ngr = (rows + kRows - 1) / kRows, tiles = (m + kRows - 1) / kRows, room = device_cus() / tiles;
  int64_t wpt = ngr < room ? ngr : room > 0 ? room : 1;
  while (ngr / wpt >= (int64_t{1} << 24)) wpt *= 2;
  a.each = ngr / wpt;
  a.more = ngr % wpt;
  a.out = lin::few_out(rows, y, ep, u, lora_b, r);
  const dim3 grid(static_cast<unsigned>(wpt), static_cast<unsigned>(tiles));
  if (sc.absmax) launch<false, false>(a, grid, s);
  else if (sc.f8) launch<true, true>(a, grid, s);
  else launch<true, false>(a, grid, s);
  return hipGetLastError();
}

}  // namespace nf4i
