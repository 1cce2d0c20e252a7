// The epilogue of a product, shared by its kernels:
//   z = sum + bias;  pre = bf16(z);  y = bf16(act(z) + residual).
// z reaches the activation in float32; y and pre are rounded once each.
#pragma once

#include <type_traits>

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

__device__ __forceinline__ float bias_at(const Epilogue& ep, int64_t col) {
  if (!ep.bias) return 0.0f;
  return ep.bias_f32 ? static_cast<const float*>(ep.bias)[col] : bf16_to_f32(static_cast<const uint16_t*>(ep.bias)[col]);
}

// f(integral constant of the activation): one branch around code made for each.
template <class F>
__device__ __forceinline__ void with_act(int act, const F& f) {
  switch (act) {
    case kActNone: f(std::integral_constant<int, kActNone>{}); break;
    case kActRelu: f(std::integral_constant<int, kActRelu>{}); break;
    case kActSilu: f(std::integral_constant<int, kActSilu>{}); break;
    case kActGelu: f(std::integral_constant<int, kActGelu>{}); break;
    default: f(std::integral_constant<int, kActGeluTanh>{});
  }
}

// One value at `at` of the outputs.
template <int A>
__device__ __forceinline__ void finish1(const Epilogue& ep, uint16_t* y, int64_t at, float z) {
  if (ep.pre) ep.pre[at] = static_cast<uint16_t>(bf16_pair(z, 0.0f));
  float v = act_value<A>(z);
  if (ep.residual) v += bf16_to_f32(ep.residual[at]);
  y[at] = static_cast<uint16_t>(bf16_pair(v, 0.0f));
}

// Eight consecutive values of a row, `at` a multiple of 8 and the buffers 16-byte aligned.
template <int A>
__device__ __forceinline__ void finish8(const Epilogue& ep, uint16_t* y, int64_t at, const float (&z)[8]) {
  u32x4 res{};
  if (ep.residual) res = *reinterpret_cast<const u32x4*>(ep.residual + at);
  if (ep.pre) {
    const u32x4 p = {bf16_pair(z[0], z[1]), bf16_pair(z[2], z[3]), bf16_pair(z[4], z[5]), bf16_pair(z[6], z[7])};
    *reinterpret_cast<u32x4*>(ep.pre + at) = p;
  }
  u32x4 o;
#pragma unroll
  for (int c = 0; c < 4; ++c)
    o[c] = bf16_pair(act_value<A>(z[2 * c]) + bf16_to_f32(res[c] & 0xFFFFu),
                     act_value<A>(z[2 * c + 1]) + __uint_as_float(res[c] & 0xFFFF0000u));
  *reinterpret_cast<u32x4*>(y + at) = o;
}

}  // namespace lin
}  // namespace nf4i
