// The streaming matrix-core product of a few rows of x (at most 16) with
// 4-bit weights, shared by the int4 GEMV (k_int4_gemv.hip) and the expert
// product of few rows (k_expert_skinny.hip).
//
// What bounds it is reading the codes, so everything serves keeping reads in
// flight: a workgroup of 16 waves (the most its registers allow) cuts the
// columns over its waves, and a wave walks "steps" of 16 weight rows x 256
// columns (2 KiB of codes), the codes of the next step on their way while it
// multiplies this one.
//
// A wave loads a step as 16 pieces of 128 contiguous bytes (a whole line per
// weight row) and turns it in 2 KiB of LDS of its own into the operand's
// order: the weights are the B operand of v_mfma_f32_16x16x32, so lane
// (row ln = lane % 16, g = lane / 16) needs 8 values of its row per product.
// One product spans 32 columns, and the products that share one scale run
// into an accumulator of their own, to which the scale is then applied in
// float32: the operands are codes or levels alone, and no scaled weight is
// rounded.  LDS row r holds 16-byte piece p at slot p ^ ((r / 2) % 8), which
// spreads the reads of 16 rows over the banks.
//
// The waves of one group of 16 rows leave their partial tiles in LDS; they are
// added in wave order, so results do not depend on timing.
#pragma once

#include "nf4_device.h"

namespace nf4i {
namespace sk {

typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 halfx8 __attribute__((ext_vector_type(8)));

constexpr int kWaves = 16;
constexpr int kThreads = 64 * kWaves;
constexpr int kSeg = 256;              // columns of a step
constexpr int kRows = 16;              // weight rows of a step, and the most rows of x
constexpr int kStageBytes = kRows * kSeg / 2;

// x, weights: 8 values of one type each
template <bool kF16>
__device__ __forceinline__ floatx4 mfma(const u32x4& x, const u32x4& w, const floatx4& c) {
  if constexpr (kF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(halfx8, x), __builtin_bit_cast(halfx8, w), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x), __builtin_bit_cast(bf16x8, w), c, 0, 0, 0);
}

// A workgroup barrier for LDS data only: global loads stay in flight across it.
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// Orders this wave's LDS stores before the LDS reads of its other lanes (the
// LDS serves a wave's accesses in order; this stops the compiler alone).
__device__ __forceinline__ void wave_lds_order() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

__device__ __forceinline__ uint32_t slot_of(int row, int piece) {
  return static_cast<uint32_t>(row * (kSeg / 2) + ((piece ^ ((row >> 1) & 7)) << 4));
}

// The codes a lane moves per step: rows lane / 8 and 8 + lane / 8 of the
// group, the 16-byte piece that belongs in slot lane % 8 of each.
struct Codes {
  u32x4 c[2];
};

// One step's loads: weight rows row0 .. row0 + 15 (clamped to the last row),
// columns k0 .. k0 + 255 (pieces clamped to the last one before kend; the x
// operand is zero there).  The codes are read once: non-temporal.
__device__ __forceinline__ Codes load_codes(const uint8_t* packed, int64_t row_bytes, int64_t row0, int64_t rows,
                                            int64_t k0, int64_t kend, int lane) {
  Codes r;
  const int64_t last = (kend - k0) / 32 - 1;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int tr = 8 * i + (lane >> 3);
    const int64_t row = row0 + tr < rows ? row0 + tr : rows - 1;
    int64_t piece = (lane & 7) ^ ((tr >> 1) & 7);
    piece = piece < last ? piece : last;
    r.c[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(packed + row * row_bytes + k0 / 2 + piece * 16));
  }
  return r;
}

__device__ __forceinline__ void stage_codes(const Codes& r, char* stage, int lane) {
#pragma unroll
  for (int i = 0; i < 2; ++i) *reinterpret_cast<u32x4*>(stage + i * 1024 + lane * 16) = r.c[i];
}

// How a launch cuts its work: `ks` waves share a group's columns, the others
// take other groups (`rs` groups at a time).
struct Plan {
  int ks, rs;
  int64_t per;     // columns of a wave (a multiple of kSeg, except where the row ends)
  int grid;
};

// At least one step per wave; ks * rs <= 16.
inline Plan make_plan(int64_t cols, int grid) {
  Plan p{};
  const int64_t nseg = (cols + kSeg - 1) / kSeg;
  p.ks = static_cast<int>(nseg < kWaves ? nseg : kWaves);
  const int64_t unit = nseg >= kWaves ? 128 : kSeg;  // wide rows are cut evenly, at multiples of 128 columns
  const int64_t units = (cols + unit - 1) / unit;
  p.per = (units + p.ks - 1) / p.ks * unit;
  p.ks = static_cast<int>((cols + p.per - 1) / p.per);
  p.rs = kWaves / p.ks;
  p.grid = grid;
  return p;
}

}  // namespace sk
}  // namespace nf4i
