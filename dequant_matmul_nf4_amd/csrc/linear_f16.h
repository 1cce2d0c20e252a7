// The float16 operands of the linear kernels: weights as level times scale, the
// power of two of a weight row, the table of level pairs, and the kernel that
// brings x to float16 (k_linear_prep.hip).
#pragma once

#include "layer_ops.h"
#include "nf4_device.h"

namespace nf4i {
namespace f16 {

typedef _Float16 half2 __attribute__((ext_vector_type(2)));
typedef _Float16 halfx8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// Scaled values lie below 2^(kTop + 1): room for the largest of a row in float16.
constexpr int kTop = 14;
// 256 level pairs (element 2j = high nibble in the low half), one copy per lane:
// entry e of lane l at byte 256 e + 4 l, so no two lanes meet in a bank and, with the
// table at LDS address 0, one permute is a lookup's address.
constexpr int kCopies = 64;
constexpr int kTabWords = 256 * kCopies;

__device__ __forceinline__ void wave_lds_order() {
  // a wave's LDS accesses are served in order; this keeps the compiler to it
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// A workgroup barrier for LDS data only: global loads stay in flight across it.
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// 2^e for -126 <= e <= 127.
__device__ __forceinline__ float power(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// The exponent e such that v 2^-e lies in [2^kTop, 2^(kTop + 1)), at least `low`
// (smaller v lie lower): what keeps 2^-e a normal number, but for the weight's rows
// beside adapters, which are brought to the same power and need room beside rows of
// zeros.
constexpr int kLow = -112, kLowAdapted = -60;
__device__ __forceinline__ int exponent_of(float v, int low) {
  const int e = static_cast<int>((__float_as_uint(v) >> 23) & 0xFF) - 127 - kTop;
  return e < low ? low : e;
}

__device__ __forceinline__ half2 twice(float s) {
  const _Float16 h = static_cast<_Float16>(s);
  return half2{h, h};
}

template <int kThreads>
__device__ __forceinline__ void fill_table(uint32_t* tab, const Codebook& cb) {
  // a pass of the threads writes kThreads / kCopies entries
  constexpr int kPer = kThreads / kCopies;
  static_assert(kPer <= 16 && 16 % kPer == 0, "whole passes per first level");
  const int e0 = threadIdx.x / kCopies;
  float second[16 / kPer];
#pragma unroll
  for (int i = 0; i < 16 / kPer; ++i) second[i] = cb.level[i * kPer + e0];
#pragma unroll
  for (int p = 0; p < 256 / kPer; ++p) {
    const half2 h = {static_cast<_Float16>(cb.level[p * kPer / 16]), static_cast<_Float16>(second[p % (16 / kPer)])};
    tab[p * kThreads + threadIdx.x] = __builtin_bit_cast(uint32_t, h);
  }
}

// The level pair of byte b of a word of codes: a permute puts it above the lane's slot.
__device__ __forceinline__ uint32_t table_slot(int lane) { return static_cast<uint32_t>(lane) << 2; }
__device__ __forceinline__ uint32_t look_up(uint32_t word, int b, const char* tab, uint32_t slot) {
  return *reinterpret_cast<const uint32_t*>(tab + __builtin_amdgcn_perm(word, slot, 0x0C0C0000u | ((4u + b) << 8)));
}

// A level pair times the block's scale.
__device__ __forceinline__ uint32_t times(uint32_t pair, half2 s) {
  return __builtin_bit_cast(uint32_t, __builtin_bit_cast(half2, pair) * s);
}

// Four level pairs times the block's scale: an operand of eight weights.
__device__ __forceinline__ halfx8 expand(const uint32_t (&l)[4], half2 s) {
  u32x4 v;
#pragma unroll
  for (int b = 0; b < 4; ++b) v[b] = times(l[b], s);
  return __builtin_bit_cast(halfx8, v);
}

}  // namespace f16

// The adapters' columns of x: u[t] = (hi | lo | 0), kl values, with hi + lo = s x[t] . A^T in two
// bf16 parts of r_pad values each (zeros past r); A [r][cols].
struct AdapterU {
  const uint16_t* a;
  int r, r_pad, kl;
  float s;
  uint16_t* u;
};
hipError_t launch_adapter_u(const uint16_t* x, int64_t m, int64_t cols, const AdapterU& ad, hipStream_t s);

// x16 = x[t] 2^-xe[t] in float16 for the m rows of x [m][cols] (cols % 64 == 0), in
// blocks: the 16 bytes of row t, columns 64 k + 32 h + 8 s .. + 7 (h < 2, s < 4) are
// number ((t / 32 cols / 64 + k) 4 + s) 64 + 32 h + t % 32 of x16, which holds m
// rounded up to 32 rows (what lies past row m is not written).  we: the exponents of
// the weight's rows.
// ad: what the adapters' thin product needs, also left by this call where r > 0.
constexpr int64_t x16_rows(int64_t m) { return (m + 31) / 32 * 32; }
hipError_t launch_linear_prep(const uint16_t* x, int64_t m, int64_t cols, uint16_t* x16, int32_t* xe, const Scales& sc,
                              int64_t rows, int32_t* we, const AdapterU& ad, hipStream_t s);

// The linear product of one or two rows of x (k_gemv.hip) and of a decode batch
// (k_linear_few.hip): x as it is, no exponents.
bool linear_row_fits(int64_t m, int64_t rows, int64_t cols);
hipError_t launch_linear_row(const uint8_t* packed, int64_t rows, int64_t cols, Scales sc, const uint16_t* x, int64_t m,
                             uint16_t* y, const Epilogue& ep, const uint16_t* u, const uint16_t* lora_b, int r, hipStream_t s);
hipError_t launch_linear_few(const uint8_t* packed, int64_t rows, int64_t cols, Scales sc, const uint16_t* x, int64_t m,
                             uint16_t* y, const Epilogue& ep, const uint16_t* u, const uint16_t* lora_b, int r, hipStream_t s);

// The linear product for up to a few hundred rows (k_linear_mid.hip).
struct MidPlan {
  int mi, tiles;     // 32-row bands of a workgroup, workgroups along the rows of x
  int splits, per;   // of the reduction over workgroups, steps of a wave
};
MidPlan mid_plan(int64_t m, int64_t rows, int64_t cols);
hipError_t launch_linear_mid(const MidPlan& p, const uint8_t* packed, int64_t rows, int64_t cols, Scales sc, const uint16_t* x16,
                             const int32_t* xe, const int32_t* we, int64_t m, uint16_t* y, const Epilogue& ep, const uint16_t* u,
                             const uint16_t* lora_b, int r, float* part, hipStream_t s);

}  // namespace nf4i
