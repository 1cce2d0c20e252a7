// What the linear kernels' float16 operands need, in one launch before them.
//
// Rows of x from bf16 to float16: each row is scaled by the power of two that
// brings its largest magnitude to [2^14, 2^15), so bf16's 8 significant bits stay
// whole but for values 2^-29 of that and below.  The output lies in the order in
// which the matrix cores take it: blocks of 1 KB for 32 rows x 16 columns of a
// 64-column step, lane l's 16 bytes at 16 l (row l % 32, columns 32 (l / 32) + 8 s ..
// + 7 of the step for block s of 4), so that the linear kernels read and move whole
// lines.  Of few rows, one to a workgroup: latency counts.  Of many, a workgroup of 16
// waves takes 8, a wave instruction 8 rows x 64 columns (8 lines in, 8 lines out).
//
// The adapters' thin product, for the same rows: a workgroup takes a row of x and 16
// rows of A, whole lines of both, and its waves' sums meet in LDS.  4096x14336 with rank
// 16 pays 4 us for it with 96 rows and 8 with 16; on the matrix cores with a row to a
// lane, as the product of many rows forms it, 27.
//
// The weight rows' exponents: that of the largest block scale, or with double
// quantization of a bound on it, the largest of the row's group scales plus the
// mean; a row per wave.
#include "linear_f16.h"

namespace nf4i {
namespace {

constexpr int kWaves = 16, kThreads = 64 * kWaves;
constexpr int kRows = 8;
constexpr int kWeightRows = 64;   // of a workgroup
constexpr int64_t kFewRows = 512;  // of x: one to a workgroup

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

struct PrepArgs {
  const uint16_t* x;
  int64_t m, cols;
  uint16_t* x16;
  int32_t* xe;
  Scales sc;
  int64_t rows;      // of the weight
  int32_t* we;
  int64_t xgroups, wgroups;  // workgroups of x, behind them those of the weight, then the adapters'
  AdapterU ad;
};

__device__ __forceinline__ void weight_rows(const PrepArgs& a, int64_t group) {
  const int lane = threadIdx.x & 63;
  const int64_t nblk = a.cols / 64;
  const float mean = a.sc.absmax ? 0.0f : fabsf(*a.sc.mean);
#pragma unroll
  for (int i = 0; i < kWeightRows / kWaves; ++i) {
    const int64_t n = group * kWeightRows + i * kWaves + (threadIdx.x >> 6);
    if (n >= a.rows) return;
    float top = 0.0f;
    if (a.sc.absmax) {
      for (int64_t b = lane; b < nblk; b += 64) top = fmaxf(top, fabsf(a.sc.absmax[n * nblk + b]));
    } else {
      for (int64_t g = (n * nblk >> 8) + lane; g <= (n * nblk + nblk - 1) >> 8; g += 64) top = fmaxf(top, fabsf(a.sc.absmax2[g]));
    }
    top = group_max<64>(top) + mean;
    if (lane == 0) a.we[n] = f16::exponent_of(top, a.ad.r > 0 ? f16::kLowAdapted : f16::kLow);
  }
}

// Sums of 16 values over the 64 lanes: half of them given away at a time, so that lane l ends
// with the sum of value 8 l5 + 4 l4 + 2 l3 + l2 (the bits of l).
template <int off, int N>
__device__ __forceinline__ void halve(float (&v)[16], bool upper) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float give = upper ? v[i] : v[N + i];
    v[i] = (upper ? v[N + i] : v[i]) + __shfl_xor(give, off, 64);
  }
}

// A row of x times 16 rows of A: (s T hi | s T lo) of them.  Products of bf16 values are exact in
// float32, the sums are float32.  All of a workgroup's loads are whole lines; A comes from L2 for
// all rows of x but the first.
__device__ __forceinline__ void adapter_row(const PrepArgs& a, int64_t group, float (&red)[kWaves][16]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const AdapterU& d = a.ad;
  const int chunks = d.r_pad / 16;
  const int64_t t = group / chunks, n = a.cols / 8;
  const int j0 = static_cast<int>(group - t * chunks) * 16;
  const u32x4* in = reinterpret_cast<const u32x4*>(a.x + t * a.cols);
  const u32x4* la = reinterpret_cast<const u32x4*>(d.a);
  float v[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) v[j] = 0.0f;
  for (int64_t k = threadIdx.x; k < n; k += kThreads) {
    const u32x4 x = in[k];
    u32x4 w[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) w[j] = la[(j0 + j < d.r ? j0 + j : d.r - 1) * n + k];
#pragma unroll
    for (int j = 0; j < 16; ++j)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        v[j] = fmaf(bf16_to_f32(x[c] & 0xFFFFu), bf16_to_f32(w[j][c] & 0xFFFFu), v[j]);
        v[j] = fmaf(__uint_as_float(x[c] & 0xFFFF0000u), __uint_as_float(w[j][c] & 0xFFFF0000u), v[j]);
      }
  }
  halve<32, 8>(v, lane & 32);
  halve<16, 4>(v, lane & 16);
  halve<8, 2>(v, lane & 8);
  halve<4, 1>(v, lane & 4);
  v[0] += __shfl_xor(v[0], 2, 64);
  v[0] += __shfl_xor(v[0], 1, 64);
  if ((lane & 3) == 0) red[wave][(lane >> 5) * 8 + (lane >> 4 & 1) * 4 + (lane >> 3 & 1) * 2 + (lane >> 2 & 1)] = v[0];
  __syncthreads();
  uint16_t* u = d.u + t * d.kl;
  if (threadIdx.x < 16) {
    const int j = j0 + threadIdx.x;
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) sum += red[w][threadIdx.x];
    sum = j < d.r ? d.s * sum : 0.0f;
    const uint32_t hi = f32_to_bf16(sum);
    u[j] = static_cast<uint16_t>(hi);
    u[d.r_pad + j] = static_cast<uint16_t>(f32_to_bf16(rest_of(sum, bf16_to_f32(hi))));
  }
  if (j0 == 0)
    for (int c = 2 * d.r_pad + threadIdx.x; c < d.kl; c += kThreads) u[c] = 0;
}

// The adapters' columns of x alone, for the kernels that take x as it is.
__global__ __launch_bounds__(kThreads) void k_adapter_rows(PrepArgs a) {
  __shared__ float red[kWaves][16];
  adapter_row(a, blockIdx.x, red);
}

// One row of x: 16-byte pieces threadIdx, + 1024, ..: N of a thread, kept; 0: read twice.
template <int N>
__global__ __launch_bounds__(kThreads) void k_prep_row(PrepArgs a) {
  __shared__ uint32_t tops[kWaves];
  __shared__ float red[kWaves][16];
  if (static_cast<int64_t>(blockIdx.x) >= a.xgroups + a.wgroups) return adapter_row(a, blockIdx.x - a.xgroups - a.wgroups, red);
  if (static_cast<int64_t>(blockIdx.x) >= a.xgroups) return weight_rows(a, blockIdx.x - a.xgroups);
  const int64_t t = blockIdx.x, n = a.cols / 8, nk = a.cols / 64;
  const u32x4* in = reinterpret_cast<const u32x4*>(a.x + t * a.cols);
  char* out = reinterpret_cast<char*>(a.x16) + t / 32 * nk * 4096 + (t & 31) * 16;
  const auto store = [&](int64_t i, const u32x4& w) {  // piece p = i % 8 of step i / 8
    *reinterpret_cast<u32x4*>(out + (i >> 3) * 4096 + (i & 3) * 1024 + (i >> 2 & 1) * 512) = w;
  };
  uint32_t top = 0;
  u32x4 v[N > 0 ? N : 1];
  if constexpr (N > 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int64_t k = threadIdx.x + i * kThreads;
      v[i] = in[k < n ? k : n - 1];
    }
#pragma unroll
    for (int i = 0; i < N; ++i) top = larger(top, v[i]);
  } else {
#pragma unroll 4
    for (int64_t k = threadIdx.x; k < n; k += kThreads) top = larger(top, in[k]);
  }
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const uint32_t o = __shfl_xor(top, off, 64);
    top = o > top ? o : top;
  }
  if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWaves; ++w) top = tops[w] > top ? tops[w] : top;
  const int e = f16::exponent_of(__uint_as_float(top), f16::kLow);
  const float up = f16::power(-e);
  if (threadIdx.x == 0) a.xe[t] = e;
  if constexpr (N > 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int64_t k = threadIdx.x + i * kThreads;
      if (k < n) store(k, scaled(v[i], up));
    }
  } else {
#pragma unroll 2
    for (int64_t k = threadIdx.x; k < n; k += kThreads) store(k, scaled(in[k], up));
  }
}

// Eight rows of x.  N: steps of a wave, at most, kept; 0: read twice.
template <int N>
__global__ __launch_bounds__(kThreads) void k_prep_rows(PrepArgs a) {
  __shared__ uint32_t tops[kWaves][kRows];
  if (static_cast<int64_t>(blockIdx.x) >= a.xgroups) return weight_rows(a, blockIdx.x - a.xgroups);
  const int64_t m = a.m, cols = a.cols;
  const uint16_t* x = a.x;
  const int lane = threadIdx.x & 63, r = lane & 7, p = lane >> 3;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kRows, t = t0 + r;
  const int64_t nk = cols / 64;
  // offsets from the first of the 8 rows, which lie in one band of 32: piece p of a step is its columns 8 p .. + 7
  const char* in = reinterpret_cast<const char*>(x + t0 * cols);
  char* out = reinterpret_cast<char*>(a.x16) + t0 / 32 * nk * 4096;
  const uint32_t from = static_cast<uint32_t>((t < m ? r : m - 1 - t0) * cols) * 2 + 16 * p;
  const uint32_t to = (p & 3) * 1024 + (p >> 2) * 512 + static_cast<uint32_t>(t & 31) * 16;
  const auto load = [&](int64_t k) { return *reinterpret_cast<const u32x4*>(in + k * 128 + from); };
  const auto store = [&](int64_t k, const u32x4& w) { *reinterpret_cast<u32x4*>(out + k * 4096 + to) = w; };
  uint32_t top = 0;
  u32x4 v[N > 0 ? N : 1];
  if constexpr (N > 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int64_t k = wave + i * kWaves;
      v[i] = load(k < nk ? k : nk - 1);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) top = larger(top, v[i]);
  } else {
#pragma unroll 8
    for (int64_t k = wave; k < nk; k += kWaves) top = larger(top, load(k));
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
  const int e = f16::exponent_of(__uint_as_float(top), f16::kLow);
  const float up = f16::power(-e);
  if (t >= m) return;
  if (threadIdx.x < kRows) a.xe[t] = e;
  if constexpr (N > 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int64_t k = wave + i * kWaves;
      if (k < nk) store(k, scaled(v[i], up));
    }
  } else {
#pragma unroll 4
    for (int64_t k = wave; k < nk; k += kWaves) store(k, scaled(load(k), up));
  }
}

}  // namespace

hipError_t launch_adapter_u(const uint16_t* x, int64_t m, int64_t cols, const AdapterU& ad, hipStream_t s) {
  if (m > kFewRows) return launch_lora_u(x, ad.a, m, cols, ad.r, ad.s, ad.u, s);
  PrepArgs a{};
  a.x = x; a.m = m; a.cols = cols; a.ad = ad;
  hipLaunchKernelGGL(k_adapter_rows, dim3(static_cast<unsigned>(m * (ad.r_pad / 16))), dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_linear_prep(const uint16_t* x, int64_t m, int64_t cols, uint16_t* x16, int32_t* xe, const Scales& sc,
                              int64_t rows, int32_t* we, const AdapterU& ad, hipStream_t s) {
  const bool few = m <= kFewRows;
  if (!few && ad.r > 0)
    if (hipError_t e = launch_lora_u(x, ad.a, m, cols, ad.r, ad.s, ad.u, s)) return e;
  const int64_t ug = few && ad.r > 0 ? m * (ad.r_pad / 16) : 0;
  const int64_t xg = few ? m : (m + kRows - 1) / kRows, wg = (rows + kWeightRows - 1) / kWeightRows;
  if (xg + wg + ug > 0x7FFFFFFF) return hipErrorInvalidValue;
  const PrepArgs a{x, m, cols, x16, xe, sc, rows, we, xg, wg, ad};
  const dim3 grid(static_cast<unsigned>(xg + wg + ug)), block(kThreads);
  const int64_t per = few ? (cols / 8 + kThreads - 1) / kThreads : (cols / 64 + kWaves - 1) / kWaves;
  if (few && per <= 2) hipLaunchKernelGGL((k_prep_row<2>), grid, block, 0, s, a);
  else if (few) hipLaunchKernelGGL((k_prep_row<0>), grid, block, 0, s, a);
  else if (per <= 4) hipLaunchKernelGGL((k_prep_rows<4>), grid, block, 0, s, a);
  else if (per <= 8) hipLaunchKernelGGL((k_prep_rows<8>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((k_prep_rows<0>), grid, block, 0, s, a);
  return hipGetLastError();
}

}  // namespace nf4i
