// Rows of x from bf16 to float16 for the linear kernels: each row is scaled by
// the power of two that brings its largest magnitude to [2^14, 2^15), so bf16's 8
// significant bits stay whole but for values 2^-29 of that and below.
//
// The output lies in the order in which the matrix cores take it: blocks of 1 KB for
// 32 rows x 16 columns of a 64-column step, lane l's 16 bytes at 16 l (row l % 32,
// columns 32 (l / 32) + 8 s .. + 7 of the step for block s of 4), so that the linear
// kernels read and move whole lines.  A workgroup of 16 waves takes 8 rows, a wave
// instruction 8 rows x 64 columns (8 lines in, 8 lines out); the waves take the
// steps in turn, keep theirs in registers between finding the largest and scaling
// where the row has at most 8192 columns, and read them again where it has more.
#include "linear_f16.h"

namespace nf4i {
namespace {

constexpr int kWaves = 16, kThreads = 64 * kWaves;
constexpr int kRows = 8;
constexpr int kKeep = 8;  // steps of a wave kept in registers, at most

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

// N: steps of a wave, at most, kept; 0: read twice.
template <int N>
__global__ __launch_bounds__(kThreads) void k_x16(const uint16_t* x, int64_t m, int64_t cols, uint16_t* x16, int32_t* xe) {
  __shared__ uint32_t tops[kWaves][kRows];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 7, p = lane >> 3;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kRows + r, tc = t < m ? t : m - 1;
  const int64_t nk = cols / 64;
  const u32x4* in = reinterpret_cast<const u32x4*>(x + tc * cols) + p;  // piece p of a step: columns 8 p .. + 7
  u32x4* out = reinterpret_cast<u32x4*>(x16) + (t / 32 * nk * 4 + (p & 3)) * 64 + (p >> 2) * 32 + (t & 31);
  uint32_t top = 0;
  u32x4 v[N > 0 ? N : 1];
  if constexpr (N > 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int64_t k = wave + i * kWaves;
      v[i] = k < nk ? in[k * 8] : u32x4{0, 0, 0, 0};
    }
#pragma unroll
    for (int i = 0; i < N; ++i) top = larger(top, v[i]);
  } else {
#pragma unroll 8
    for (int64_t k = wave; k < nk; k += kWaves) top = larger(top, in[k * 8]);
  }
#pragma unroll
  for (int off = 8; off < 64; off <<= 1) {  // the row's 8 lanes
    const uint32_t o = __shfl_xor(top, off, 64);
    top = o > top ? o : top;
  }
  if (p == 0) tops[wave][r] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWaves; ++w) top = tops[w][r] > top ? tops[w][r] : top;
  const int e = f16::exponent_of(__uint_as_float(top));
  const float up = f16::power(-e);
  if (t >= m) return;
  if (threadIdx.x < kRows) xe[t] = e;
  if constexpr (N > 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int64_t k = wave + i * kWaves;
      if (k < nk) out[k * 256] = scaled(v[i], up);
    }
  } else {
#pragma unroll 4
    for (int64_t k = wave; k < nk; k += kWaves) out[k * 256] = scaled(in[k * 8], up);
  }
}

}  // namespace

hipError_t launch_x16(const uint16_t* x, int64_t m, int64_t cols, uint16_t* x16, int32_t* xe, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>((m + kRows - 1) / kRows)), block(kThreads);
  const int64_t per = (cols / 64 + kWaves - 1) / kWaves;
  if (per <= 4) hipLaunchKernelGGL((k_x16<4>), grid, block, 0, s, x, m, cols, x16, xe);
  else if (per <= kKeep) hipLaunchKernelGGL((k_x16<kKeep>), grid, block, 0, s, x, m, cols, x16, xe);
  else hipLaunchKernelGGL((k_x16<0>), grid, block, 0, s, x, m, cols, x16, xe);
  return hipGetLastError();
}

}  // namespace nf4i
