// The streaming matrix-core product of a few rows of x (at most 16) with
// 4-bit weights, shared by the int4 GEMV (k_int4_gemv.hip) and the expert
// product of few rows (k_expert_skinny.hip).
//
// What bounds it is reading the codes, so everything serves keeping reads in
// flight: a workgroup of 8 waves (one per compute unit, as its registers
// allow) cuts the columns over its waves, and a wave walks "steps" of 16
// weight rows x 512 columns (4 KiB of codes), the codes of the next two steps
// on their way while it multiplies this one.
//
// A wave loads a step as 256 contiguous bytes of each weight row (two whole
// lines) and turns it in 4 KiB of LDS of its own into the operand's
// order: the weights are the B operand of v_mfma_f32_16x16x32, so lane
// (row ln = lane % 16, g = lane / 16) needs 8 values of its row per product.
// One product spans 32 columns, and the products that share one scale run
// into an accumulator of their own, to which the scale is then applied in
// float32: the operands are codes or levels alone, and no scaled weight is
// rounded.  LDS row r holds 16-byte piece p at slot p ^ r, which spreads the
// reads of 16 rows over the banks.
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

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;
constexpr int kSeg = 512;              // columns of a step
constexpr int kRows = 16;              // weight rows of a step, and the most rows of x
constexpr int kStageBytes = kRows * kSeg / 2;
constexpr int kLoads = kStageBytes / 1024;  // 16-byte loads of a lane per step

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
  return static_cast<uint32_t>(row * (kSeg / 2) + ((piece ^ row) << 4));
}

// The codes a lane moves per step: load i takes row 4 i + lane / 16 of the
// group, the 16-byte piece that belongs in slot lane % 16 of it.
struct Codes {
  u32x4 c[kLoads];
};

__device__ __forceinline__ int code_row(int i, int lane) { return 4 * i + (lane >> 4); }
__device__ __forceinline__ int code_piece(int i, int lane) { return (lane & 15) ^ code_row(i, lane); }

// The offset of load i from the step's first byte (rows of row_bytes < 2^27
// bytes).  `rows` and `pieces` are left from there, at least one of each: what
// lies past the last repeats it (such products meet zeros or are not stored).
__device__ __forceinline__ uint32_t code_offset(int i, uint32_t row_bytes, int rows, int pieces, int lane) {
  const int tr = code_row(i, lane), tp = code_piece(i, lane);
  const uint32_t row = tr < rows ? tr : rows - 1, piece = tp < pieces ? tp : pieces - 1;
  return row * row_bytes + (piece << 4);
}

// The offsets of whole steps, kept.
struct CodeLane {
  uint32_t off[kLoads];
};

__device__ __forceinline__ CodeLane code_lane(uint32_t row_bytes, int lane) {
  CodeLane r;
#pragma unroll
  for (int i = 0; i < kLoads; ++i) r.off[i] = code_offset(i, row_bytes, kRows, kSeg / 32, lane);
  return r;
}

// One step's loads.  They are issued whatever the step (no branch around a
// load): only then does the compiler know how many loads are younger than the
// ones it waits for, and waits for no more.  One that is not wanted reads 16
// bytes.  The codes are read once: non-temporal.
__device__ __forceinline__ void load_codes(Codes& r, const uint8_t* step, const CodeLane& l, uint32_t row_bytes,
                                           int rows, int pieces, bool wanted, int lane) {
  const bool whole = rows >= kRows && pieces >= kSeg / 32;
  uint32_t off[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) off[i] = l.off[i];
  if (!whole) {
    const int l2 = opaque(lane);  // rare: nothing of this is worth keeping in registers
#pragma unroll
    for (int i = 0; i < kLoads; ++i) off[i] = code_offset(i, row_bytes, rows, pieces, l2);
  }
  const uint32_t keep = wanted ? ~0u : 0u;
#pragma unroll
  for (int i = 0; i < kLoads; ++i)
    r.c[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(step + (off[i] & keep)));
}

__device__ __forceinline__ void stage_codes(const Codes& r, char* stage, int lane) {
#pragma unroll
  for (int i = 0; i < kLoads; ++i) *reinterpret_cast<u32x4*>(stage + i * 1024 + lane * 16) = r.c[i];
}

// How a launch cuts its work: `ks` waves share a group's columns, the others
// take other groups (`rs` groups at a time).
struct Plan {
  int ks, rs;
  int64_t per;     // columns of a wave (where the row ends: fewer)
};

// At least one step per wave; ks * rs <= kWaves.
inline Plan make_plan(int64_t cols) {
  Plan p{};
  const int64_t nseg = (cols + kSeg - 1) / kSeg;
  p.ks = static_cast<int>(nseg < kWaves ? nseg : kWaves);
  const int64_t unit = nseg >= kWaves ? 128 : kSeg;  // wide rows are cut evenly, at multiples of 128 columns
  const int64_t units = (cols + unit - 1) / unit;
  p.per = (units + p.ks - 1) / p.ks * unit;
  p.ks = static_cast<int>((cols + p.per - 1) / p.per);
  p.rs = kWaves / p.ks;
  return p;
}

}  // namespace sk
}  // namespace nf4i
