// The epilogue of a product, shared by its kernels:
//   z = sum + bias;  pre = bf16(z);  y = bf16(act(z) + residual).
// z reaches the activation in float32; y and pre are rounded once each.
#pragma once

#include "epilogue.h"
#include "layer_ops.h"

namespace nf4i {
namespace lin {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  const bf16x2 p = {static_cast<__bf16>(lo), static_cast<__bf16>(hi)};
  return __builtin_bit_cast(uint32_t, p);
}

// N bias values of columns col .., `left` of which exist (zeros past them and without a bias).
template <int N>
__device__ __forceinline__ void load_bias(float (&b)[N], const Epilogue& ep, int64_t col, int left) {
#pragma unroll
  for (int c = 0; c < N; ++c) b[c] = 0.0f;
  if (!ep.bias) return;
  if (ep.bias_f32) {
#pragma unroll
    for (int c = 0; c < N; ++c)
      if (c < left) b[c] = static_cast<const float*>(ep.bias)[col + c];
  } else {
#pragma unroll
    for (int c = 0; c < N; ++c)
      if (c < left) b[c] = bf16_to_f32(static_cast<const uint16_t*>(ep.bias)[col + c]);
  }
}

// act(z) of N values: one branch around code made for each activation.
template <int N>
__device__ __forceinline__ void apply_act(int act, float (&z)[N]) {
  switch (act) {
    case kActNone: break;
    case kActRelu:
#pragma unroll
      for (int c = 0; c < N; ++c) z[c] = act_value<kActRelu>(z[c]);
      break;
    case kActSilu:
#pragma unroll
      for (int c = 0; c < N; ++c) z[c] = act_value<kActSilu>(z[c]);
      break;
    case kActGelu:
#pragma unroll
      for (int c = 0; c < N; ++c) z[c] = act_value<kActGelu>(z[c]);
      break;
    default:
#pragma unroll
      for (int c = 0; c < N; ++c) z[c] = act_value<kActGeluTanh>(z[c]);
  }
}

// N values of one column, `step` apart from `at` on, the first `n` of which exist.
template <int N>
__device__ __forceinline__ void finish_column(const Epilogue& ep, uint16_t* y, int64_t at, int64_t step, int n, float (&z)[N]) {
  float res[N];
  if (ep.residual) {
#pragma unroll
    for (int c = 0; c < N; ++c) res[c] = c < n ? bf16_to_f32(ep.residual[at + c * step]) : 0.0f;
  }
  const auto put = [&](uint16_t* to) {
#pragma unroll
    for (int c = 0; c < N; ++c)
      if (c < n) to[at + c * step] = static_cast<uint16_t>(bf16_pair(z[c], 0.0f));
  };
  if (ep.pre) put(ep.pre);
  apply_act(ep.act, z);
  if (ep.residual) {
#pragma unroll
    for (int c = 0; c < N; ++c) z[c] += res[c];
  }
  put(y);
}

// Eight consecutive values of a row, the first `left` of which exist; `whole`:
// all do, and 16-byte accesses are aligned.
__device__ __forceinline__ void finish8(const Epilogue& ep, uint16_t* y, int64_t at, float (&z)[8], int left, bool whole) {
  u32x4 res{};
  if (ep.residual) {
    if (whole) {
      res = *reinterpret_cast<const u32x4*>(ep.residual + at);
    } else {
#pragma unroll
      for (int c = 0; c < 8; ++c)
        if (c < left) res[c >> 1] |= static_cast<uint32_t>(ep.residual[at + c]) << (16 * (c & 1));
    }
  }
  const auto put = [&](uint16_t* to) {
    const u32x4 o = {bf16_pair(z[0], z[1]), bf16_pair(z[2], z[3]), bf16_pair(z[4], z[5]), bf16_pair(z[6], z[7])};
    if (whole) {
      *reinterpret_cast<u32x4*>(to + at) = o;
    } else {
#pragma unroll
      for (int c = 0; c < 8; ++c)
        if (c < left) to[at + c] = static_cast<uint16_t>(o[c >> 1] >> (16 * (c & 1)));
    }
  };
  if (ep.pre) put(ep.pre);
  apply_act(ep.act, z);
  if (ep.residual) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      z[2 * c] += bf16_to_f32(res[c] & 0xFFFFu);
      z[2 * c + 1] += __uint_as_float(res[c] & 0xFFFF0000u);
    }
  }
  put(y);
}

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// Eight bf16 values times a power of two.
__device__ __forceinline__ bf16x8 times(const u32x4& v, float by) {
  u32x4 o;
#pragma unroll
  for (int k = 0; k < 4; ++k) o[k] = bf16_pair(bf16_to_f32(v[k] & 0xFFFFu) * by, __uint_as_float(v[k] & 0xFFFF0000u) * by);
  return __builtin_bit_cast(bf16x8, o);
}

// Operands of the adapters' product, times a power of two: columns c .. c + 7 of
// (B | B | 0) of weight row n (B [rows][r], halves of r_pad columns) ...
__device__ __forceinline__ bf16x8 adapter_w(const uint16_t* lb, int r, int r_pad, int64_t n, int c, float by) {
  typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
  const int j0 = c < r_pad ? c : c - r_pad;
  const uint16_t* b = lb + n * r + j0;
  u32x4 v = {0, 0, 0, 0};
  if (j0 + 8 <= r) {
    v = *reinterpret_cast<const u32x4_any*>(b);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (j0 + i < r) v[i >> 1] |= static_cast<uint32_t>(b[i]) << (16 * (i & 1));
  }
  return times(v, by);
}
// ... and eight columns of a row of (s T hi | s T lo).
__device__ __forceinline__ bf16x8 adapter_x(const uint16_t* u, float by) { return times(*reinterpret_cast<const u32x4*>(u), by); }

// What takes the sums of a few rows of x: N rows from t on, n of which exist, and
// weight row `row`.
struct FewOut {
  static constexpr bool kZeroTail = true;
  int64_t rows;
  uint16_t* y;
  Epilogue ep;
  const uint16_t* u;   // adapter columns of x: [m][kl] (s T hi | s T lo | 0)
  const uint16_t* lb;  // B [rows][r]
  int r, r_pad, kl;    // 0 without adapters

  template <int N>
  __device__ __forceinline__ void store(int64_t t, int n, int64_t row, float (&z)[N]) const {
    if (r > 0) adapters(t, n, row, z);
    float bias[1];
    load_bias(bias, ep, row, 1);
#pragma unroll
    for (int c = 0; c < N; ++c) z[c] += bias[0];
    finish_column(ep, y, t * rows + row, rows, n, z);
  }
  // z[c] += sum_j (hi + lo)[t + c][j] B[row][j]
  template <int N>
  __device__ __forceinline__ void adapters(int64_t t, int n, int64_t row, float (&z)[N]) const {
    typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
    const uint16_t* h = u + t * kl;
    const uint16_t* b = lb + row * r;
    for (int j = 0; j < r; j += 8) {
      u32x4 w = {0, 0, 0, 0}, hi[N], lo[N];
#pragma unroll
      for (int c = 0; c < N; ++c) {
        const uint16_t* hc = h + (c < n ? c : n - 1) * kl + j;
        hi[c] = *reinterpret_cast<const u32x4*>(hc);
        lo[c] = *reinterpret_cast<const u32x4*>(hc + r_pad);
      }
      if (j + 8 <= r) {
        w = *reinterpret_cast<const u32x4_any*>(b + j);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (j + i < r) w[i >> 1] |= static_cast<uint32_t>(b[j + i]) << (16 * (i & 1));
      }
#pragma unroll
      for (int c = 0; c < N; ++c)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          z[c] = fmaf(bf16_to_f32(hi[c][k] & 0xFFFFu) + bf16_to_f32(lo[c][k] & 0xFFFFu), bf16_to_f32(w[k] & 0xFFFFu), z[c]);
          z[c] = fmaf(__uint_as_float(hi[c][k] & 0xFFFF0000u) + __uint_as_float(lo[c][k] & 0xFFFF0000u), __uint_as_float(w[k] & 0xFFFF0000u), z[c]);
        }
    }
  }
};
inline FewOut few_out(int64_t rows, uint16_t* y, const Epilogue& ep, const uint16_t* u, const uint16_t* lora_b, int r) {
  return FewOut{rows, y, ep, u, lora_b, r, (r + 15) / 16 * 16, static_cast<int>(gemm_lora_cols(r))};
}

}  // namespace lin
}  // namespace nf4i
