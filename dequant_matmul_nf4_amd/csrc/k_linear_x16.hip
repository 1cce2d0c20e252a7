// Rows of x from bf16 to float16 for the linear kernels: each row is scaled by
// the power of two that brings its largest magnitude to [2^14, 2^15), so bf16's 8
// significant bits stay whole but for values 2^-29 of that and below.  A wave
// takes a row; its bf16 values stay in registers between finding the largest and
// scaling where the row has at most 4096 columns, else they are read again from
// the caches.
#include "linear_f16.h"

namespace nf4i {
namespace {

constexpr int kThreads = 256;
constexpr int kKeep = 8;  // 16-byte pieces of a lane

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ uint32_t larger(uint32_t top, const u32x4& v) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const uint32_t lo = (v[c] << 16) & 0x7FFF0000u, hi = v[c] & 0x7FFF0000u;
    const uint32_t m = lo > hi ? lo : hi;
    top = m > top ? m : top;
  }
  return top;
}

__device__ __forceinline__ u32x4 scaled(const u32x4& v, float up) {
  u32x4 o;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const f16::half2 h = {static_cast<_Float16>(bf16_to_f32(v[c] & 0xFFFFu) * up),
                          static_cast<_Float16>(__uint_as_float(v[c] & 0xFFFF0000u) * up)};
    o[c] = __builtin_bit_cast(uint32_t, h);
  }
  return o;
}

template <bool kWhole>
__global__ __launch_bounds__(kThreads) void k_x16(const uint16_t* x, int64_t m, int64_t cols, uint16_t* x16, int32_t* xe) {
  const int lane = threadIdx.x & 63;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (kThreads / 64) + (threadIdx.x >> 6);
  if (t >= m) return;
  const u32x4* p = reinterpret_cast<const u32x4*>(x + t * cols);
  u32x4* q = reinterpret_cast<u32x4*>(x16 + t * cols);
  const int64_t n = cols / 8;
  u32x4 v[kKeep];
  uint32_t top = 0;
  if constexpr (kWhole) {
#pragma unroll
    for (int i = 0; i < kKeep; ++i) v[i] = i * 64 + lane < n ? p[i * 64 + lane] : u32x4{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < kKeep; ++i) top = larger(top, v[i]);
  } else {
#pragma unroll 8
    for (int64_t i = lane; i < n; i += 64) top = larger(top, p[i]);
  }
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const uint32_t o = __shfl_xor(top, off, 64);
    top = o > top ? o : top;
  }
  const int e = f16::exponent_of(__uint_as_float(top));
  const float up = f16::power(-e);
  if (lane == 0) xe[t] = e;
  if constexpr (kWhole) {
#pragma unroll
    for (int i = 0; i < kKeep; ++i)
      if (i * 64 + lane < n) q[i * 64 + lane] = scaled(v[i], up);
  } else {
#pragma unroll 4
    for (int64_t i = lane; i < n; i += 64) q[i] = scaled(p[i], up);
  }
}

}  // namespace

hipError_t launch_x16(const uint16_t* x, int64_t m, int64_t cols, uint16_t* x16, int32_t* xe, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>((m + kThreads / 64 - 1) / (kThreads / 64))), block(kThreads);
  if (cols <= 64 * 8 * kKeep) hipLaunchKernelGGL((k_x16<true>), grid, block, 0, s, x, m, cols, x16, xe);
  else hipLaunchKernelGGL((k_x16<false>), grid, block, 0, s, x, m, cols, x16, xe);
  return hipGetLastError();
}

}  // namespace nf4i
