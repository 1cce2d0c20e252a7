// Quantization to uniform 4-bit codes with a scale (and zero point) per group
// of 32, 64 or 128 consecutive values of a row, and the way back.
//
//   symmetric   s = round(max |x| / 7)                       q = clamp(rint(x / s) + 8, 0, 15)
//   asymmetric  lo = min(0, min x), hi = max(0, max x)
//               s = round((hi - lo) / 15), z = clamp(rint(-lo / s), 0, 15)
//                                                            q = clamp(rint(x / s) + z, 0, 15)
//   back        w = (q - z) s                                (z = 8 where symmetric)
//
// round() is to the scales' type; quotients are IEEE float32 divisions and
// rint() is to even.  A group whose s is 0 gets q = z (asymmetric: 0).
//
// Both are bound by HBM: a value is touched once (28672x8192 bf16: quantizer
// 117 us, 5.1 TB/s; expanded to float32 143 us, written non-temporally at 6.6
// TB/s, 274 us with plain stores).  The groups tile the
// flattened weight (cols is a multiple of the group), so a lane takes 16
// consecutive values, a group is 2, 4 or 8 lanes, and its extremes are found
// with that many lanes' permutes.
#include "expert_int4.h"
#include "nf4_device.h"

namespace nf4i {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float floatx4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float half_bits_to_f32(uint32_t b) {
  return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(b)));
}

// 16 consecutive values in float32.  The 16-bit types are read non-temporally:
// the codes just written then stay in the last-level cache for whoever reads
// them next (28672x8192 bf16 quantized and expanded: 113 + 143 us, 103 + 219 us
// without).  float32 is not, as a lane's four loads share a line that would be
// fetched again (4096x4096: 14 against 22 us).
template <int kType>
__device__ __forceinline__ void load16(const void* x, int64_t i, float (&v)[16]) {
  if constexpr (kType == 0) {
    const floatx4* p = reinterpret_cast<const floatx4*>(static_cast<const float*>(x) + i);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const floatx4 t = p[k];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[4 * k + e] = t[e];
    }
  } else {
    const u32x4* p = reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(x) + i);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const u32x4 t = __builtin_nontemporal_load(p + k);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[8 * k + 2 * e] = kType == 1 ? bf16_to_f32(t[e] & 0xFFFFu) : half_bits_to_f32(t[e]);
        v[8 * k + 2 * e + 1] = kType == 1 ? __uint_as_float(t[e] & 0xFFFF0000u) : half_bits_to_f32(t[e] >> 16);
      }
    }
  }
}

// The scale in its type, stored by one lane, and its value.
__device__ __forceinline__ float round_scale(float s, int type) {
  if (type == 0) return s;
  if (type == 1) return bf16_to_f32(f32_to_bf16(s));
  return fminf(static_cast<float>(static_cast<_Float16>(s)), 65504.0f);
}
__device__ __forceinline__ void store_scale(void* scales, int type, int64_t i, float s) {
  if (type == 0) static_cast<float*>(scales)[i] = s;
  else if (type == 1) static_cast<uint16_t*>(scales)[i] = static_cast<uint16_t>(f32_to_bf16(s));
  else static_cast<_Float16*>(scales)[i] = static_cast<_Float16>(s);
}

template <int kType>
__global__ __launch_bounds__(256) void k_int4_quantize(const void* __restrict__ x, int64_t n, int shift,
                                                       uint8_t* __restrict__ packed, void* __restrict__ scales,
                                                       int scale_type, uint8_t* __restrict__ zeros) {
  const int64_t i = (block_number() * 256 + threadIdx.x) * 16;
  // groups are whole: the lanes of one are all here or all past the end
  if (i >= n) return;
  float v[16];
  load16<kType>(x, i, v);
  float lo = v[0], hi = v[0];
#pragma unroll
  for (int k = 1; k < 16; ++k) {
    lo = fminf(lo, v[k]);
    hi = fmaxf(hi, v[k]);
  }
  for (int off = 1; off < 1 << (shift - 4); off <<= 1) {
    lo = fminf(lo, __shfl_xor(lo, off, kWave));
    hi = fmaxf(hi, __shfl_xor(hi, off, kWave));
  }
  float s, z;
  if (zeros) {
    lo = fminf(lo, 0.0f);
    hi = fmaxf(hi, 0.0f);
    s = round_scale((hi - lo) / 15.0f, scale_type);
    z = s > 0.0f ? fminf(fmaxf(rintf(-lo / s), 0.0f), 15.0f) : 0.0f;
  } else {
    s = round_scale(fmaxf(fabsf(lo), fabsf(hi)) / 7.0f, scale_type);
    z = 8.0f;
  }
  uint32_t w[2] = {0u, 0u};
  // rint(x / s): with r = fl32(1 / s), q0 = fl32(x r) and the exact remainder
  // x - q0 s, fl32(q0 + (x - q0 s) r) is the IEEE quotient (Markstein) while
  // nothing under- or overflows on the way; smaller quotients round to 0 both ways.
  // (Under a float16 scale, which saturates, a value can be infinite and s not:
  // its remainder would be a NaN, where the quotient is infinite.)
  const bool fast = s >= 0x1p-80f && s <= 0x1p100f && fmaxf(fabsf(lo), fabsf(hi)) <= 0x1.fffffep127f;
  const float r = 1.0f / s;
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    float t;
    if (fast) {
      const float q0 = v[k] * r;
      t = rintf(fmaf(fmaf(-q0, s, v[k]), r, q0));
    } else {
      t = s > 0.0f ? rintf(v[k] / s) : 0.0f;
    }
    const uint32_t q = static_cast<uint32_t>(fminf(fmaxf(t + z, 0.0f), 15.0f));
    w[k >> 3] |= q << (8 * ((k & 7) >> 1) + ((k & 1) ? 0 : 4));
  }
  *reinterpret_cast<u32x2*>(packed + i / 2) = u32x2{w[0], w[1]};
  if ((i & ((1 << shift) - 1)) == 0) {
    store_scale(scales, scale_type, i >> shift, s);
    if (zeros) zeros[i >> shift] = static_cast<uint8_t>(z);
  }
}

__device__ __forceinline__ float scale_at(const void* p, int type, int64_t i) {
  if (type == 0) return static_cast<const float*>(p)[i];
  const uint32_t h = static_cast<const uint16_t*>(p)[i];
  return type == 1 ? bf16_to_f32(h) : half_bits_to_f32(h);
}

// A vector: eight values for the 16-bit types, four for float32, one 16-byte
// store either way.  A thread takes kUnroll vectors, their loads issued first.
constexpr int kUnroll = 4;

template <int kType>
__global__ __launch_bounds__(256) void k_int4_dequantize(Int4Weight w, int shift, int64_t n, void* __restrict__ out) {
  constexpr int kPer = kType == 0 ? 4 : 8;
  const int64_t i0 = (block_number() * (256 * kUnroll) + threadIdx.x) * kPer;
  uint32_t c[kUnroll];
  float s[kUnroll];
  int z[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int64_t at = i0 + u * 256 * kPer, i = at < n ? at : n - kPer;
    c[u] = kType == 0 ? *reinterpret_cast<const uint16_t*>(w.packed + i / 2) : *reinterpret_cast<const uint32_t*>(w.packed + i / 2);
    s[u] = scale_at(w.scales, w.scale_type, i >> shift);
    z[u] = w.zeros ? w.zeros[i >> shift] : 8;
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int64_t i = i0 + u * 256 * kPer;
    if (i >= n) continue;
    float v[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int q = static_cast<int>((c[u] >> (8 * (k >> 1) + ((k & 1) ? 0 : 4))) & 15u);
      // (opaque: a product fused with its conversion to float16 would be rounded once, not twice)
      v[k] = __uint_as_float(opaque(__float_as_uint(static_cast<float>(q - z[u]) * s[u])));
    }
    if constexpr (kType == 0) {
      __builtin_nontemporal_store(floatx4{v[0], v[1], v[2], v[3]}, reinterpret_cast<floatx4*>(static_cast<float*>(out) + i));
    } else {
      u32x4 o;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if constexpr (kType == 1) {
          o[k] = pack_bf16x2(v[2 * k], v[2 * k + 1]);
        } else {
          const uint16_t a = __builtin_bit_cast(uint16_t, static_cast<_Float16>(v[2 * k]));
          const uint16_t b = __builtin_bit_cast(uint16_t, static_cast<_Float16>(v[2 * k + 1]));
          o[k] = a | (static_cast<uint32_t>(b) << 16);
        }
      }
      __builtin_nontemporal_store(o, reinterpret_cast<u32x4*>(static_cast<uint16_t*>(out) + i));
    }
  }
}

}  // namespace

static int shift_of(int group) { return group == 32 ? 5 : group == 64 ? 6 : 7; }

hipError_t launch_int4_quantize(const void* x, int x_type, int64_t n, int group, uint8_t* packed, void* scales,
                                int scale_type, uint8_t* zeros, hipStream_t s) {
  const int64_t blocks = (n + 4095) / 4096;
  const int shift = shift_of(group);
  const dim3 gd = block_grid(blocks), bd(256);
  if (x_type == 0) hipLaunchKernelGGL((k_int4_quantize<0>), gd, bd, 0, s, x, n, shift, packed, scales, scale_type, zeros);
  else if (x_type == 1) hipLaunchKernelGGL((k_int4_quantize<1>), gd, bd, 0, s, x, n, shift, packed, scales, scale_type, zeros);
  else hipLaunchKernelGGL((k_int4_quantize<2>), gd, bd, 0, s, x, n, shift, packed, scales, scale_type, zeros);
  return hipGetLastError();
}

hipError_t launch_int4_dequantize(const Int4Weight& w, void* out, int out_type, hipStream_t s) {
  const int64_t n = w.rows * w.cols;
  const int per = (out_type == 0 ? 1024 : 2048) * kUnroll;
  const int64_t blocks = (n + per - 1) / per;
  const dim3 gd = block_grid(blocks), bd(256);
  if (out_type == 0) hipLaunchKernelGGL((k_int4_dequantize<0>), gd, bd, 0, s, w, shift_of(w.group), n, out);
  else if (out_type == 1) hipLaunchKernelGGL((k_int4_dequantize<1>), gd, bd, 0, s, w, shift_of(w.group), n, out);
  else hipLaunchKernelGGL((k_int4_dequantize<2>), gd, bd, 0, s, w, shift_of(w.group), n, out);
  return hipGetLastError();
}

}  // namespace nf4i
