// The norm over many gradients and their scaling to a largest norm:
//
//   norm = sqrt(sum over all tensors of g^2),   scale = min(1, max_norm / (norm + 1e-6))
//   out = rnd(g scale)                 (in float32, rounded once to out's type)
//
// Reading the gradients bounds it: once for the norm, once more to scale them.
// Squares are added in float64, which is as fast as float32 here, so that no
// finite gradient overflows or vanishes in its square.
//
// The tensors are cut into chunks of kChunk values, numbered over all tensors;
// a workgroup takes one contiguous run of them, finds its first tensor by
// bisection and walks on from there.  It leaves one sum in the workspace; the
// scaling kernel's workgroups each add all those sums in one order, so every one
// of them has the same norm, whatever the timing.  The scaling kernel walks its
// runs backwards: what the norm read last is still in the last-level cache.
// Up to kInline tensors travel in the kernels' arguments; more are first
// written into a table in the workspace by small launches that carry them in
// theirs, so that a call copies nothing from host memory and can be captured.
//
// Measured: 1120 float32 gradients of 828 MB, clipped into a flat tensor: norm 184 us
// (4.5 TB/s), scaling 337 (4.9 TB/s), the table's ten launches 17 and their gaps.
#include "layer_ops.h"
#include "nf4.h"
#include "nf4_device.h"

namespace nf4i {
namespace {

constexpr int kThreads = 256;
constexpr int kVec = 8;                            // values of a thread per step
constexpr int kStep = kThreads * kVec;
constexpr int kChunk = 8 * kStep;                  // 16384 values
constexpr int kMaxGroups = 2048;
constexpr int kInline = 112;

enum { kF32 = 0, kBf16 = 1, kF16 = 2 };

struct Entry {
  const void* grad;
  void* out;
  int64_t n;
  int64_t first;  // number of its first chunk, its types in the upper 8 bits
};
constexpr int kTypeShift = 56;

struct Inline {
  Entry e[kInline];
};

struct Table {
  int count;
  int64_t chunks;
};

typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4_any4 __attribute__((ext_vector_type(4), aligned(4)));

__device__ __forceinline__ int64_t first_of(const Entry& e) { return e.first & ((int64_t{1} << kTypeShift) - 1); }
__device__ __forceinline__ int type_of(const Entry& e) { return static_cast<int>(e.first >> kTypeShift) & 3; }
__device__ __forceinline__ int out_type_of(const Entry& e) { return static_cast<int>(e.first >> (kTypeShift + 2)) & 3; }

__device__ __forceinline__ float half_to_f32(uint32_t b) {
  return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(b)));
}

template <int T>
__device__ __forceinline__ void load8(float (&v)[kVec], const void* p, int64_t i) {
  if constexpr (T == kF32) {
    const u32x4_any4* q = reinterpret_cast<const u32x4_any4*>(static_cast<const float*>(p) + i);
    const u32x4_any4 a = q[0], b = q[1];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[k] = __uint_as_float(a[k]);
      v[4 + k] = __uint_as_float(b[k]);
    }
  } else {
    const u32x4_any a = *reinterpret_cast<const u32x4_any*>(static_cast<const uint16_t*>(p) + i);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (T == kBf16) {
        v[2 * k] = __uint_as_float(a[k] << 16);
        v[2 * k + 1] = __uint_as_float(a[k] & 0xFFFF0000u);
      } else {
        v[2 * k] = half_to_f32(a[k] & 0xFFFFu);
        v[2 * k + 1] = half_to_f32(a[k] >> 16);
      }
    }
  }
}

template <int T>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
  if constexpr (T == kF32) return static_cast<const float*>(p)[i];
  else if constexpr (T == kBf16) return bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
  else return half_to_f32(static_cast<const uint16_t*>(p)[i]);
}

template <int T>
__device__ __forceinline__ uint32_t to16(float v) {
  if constexpr (T == kBf16) return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
  else return __builtin_bit_cast(uint16_t, static_cast<_Float16>(v));
}

template <int T>
__device__ __forceinline__ void store8(const float (&v)[kVec], void* p, int64_t i) {
  if constexpr (T == kF32) {
    u32x4_any4* q = reinterpret_cast<u32x4_any4*>(static_cast<float*>(p) + i);
    u32x4_any4 a, b;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      a[k] = __float_as_uint(v[k]);
      b[k] = __float_as_uint(v[4 + k]);
    }
    q[0] = a;
    q[1] = b;
  } else {
    u32x4_any a;
#pragma unroll
    for (int k = 0; k < 4; ++k) a[k] = to16<T>(v[2 * k]) | (to16<T>(v[2 * k + 1]) << 16);
    *reinterpret_cast<u32x4_any*>(static_cast<uint16_t*>(p) + i) = a;
  }
}

template <int T>
__device__ __forceinline__ void store1(float v, void* p, int64_t i) {
  if constexpr (T == kF32) static_cast<float*>(p)[i] = v;
  else static_cast<uint16_t*>(p)[i] = static_cast<uint16_t>(to16<T>(v));
}

// The last tensor whose first chunk is at or before chunk c (tensors without
// values have none: their first chunk is the next one's).
__device__ __forceinline__ int find_tensor(const Entry* e, int count, int64_t c) {
  int lo = 0, hi = count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (first_of(e[mid]) <= c) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Four sums of a thread: consecutive values do not wait for each other.
struct Sums {
  double s[4];
};

template <int T>
__device__ __forceinline__ void add_squares(Sums& s, const void* p, int64_t i0, int64_t i1) {
  const int64_t whole = i0 + (i1 - i0) / kStep * kStep;
  if (i1 - i0 == kChunk) {
    // the whole chunk's loads in two halves, so that many are on their way
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float v[4][kVec];
#pragma unroll
      for (int u = 0; u < 4; ++u) load8<T>(v[u], p, i0 + (4 * h + u) * kStep + threadIdx.x * kVec);
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int k = 0; k < kVec; ++k) s.s[k & 3] = fma(static_cast<double>(v[u][k]), static_cast<double>(v[u][k]), s.s[k & 3]);
    }
    return;
  }
  for (int64_t i = i0 + threadIdx.x * kVec; i < whole; i += kStep) {
    float v[kVec];
    load8<T>(v, p, i);
#pragma unroll
    for (int k = 0; k < kVec; ++k) s.s[k & 3] = fma(static_cast<double>(v[k]), static_cast<double>(v[k]), s.s[k & 3]);
  }
  for (int64_t i = whole + threadIdx.x; i < i1; i += kThreads) {
    const double v = load1<T>(p, i);
    s.s[0] = fma(v, v, s.s[0]);
  }
}

// Sum over the workgroup, the same in every thread.
__device__ __forceinline__ double group_sum(double v, double* red) {
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) v += __shfl_xor(v, off, 64);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  return (red[0] + red[1]) + (red[2] + red[3]);
}

__device__ void norm_part(const Entry* e, const Table& t, double* part, double* red) {
  const int64_t c0 = t.chunks * blockIdx.x / gridDim.x, c1 = t.chunks * (blockIdx.x + 1) / gridDim.x;
  Sums s{};
  int j = c0 < c1 ? find_tensor(e, t.count, c0) : 0;
  for (int64_t c = c0; c < c1; ++c) {
    while (j + 1 < t.count && first_of(e[j + 1]) <= c) ++j;
    const Entry& q = e[j];
    const int64_t i0 = (c - first_of(q)) * kChunk, i1 = q.n - i0 < kChunk ? q.n : i0 + kChunk;
    const int ty = type_of(q);
    if (ty == kF32) add_squares<kF32>(s, q.grad, i0, i1);
    else if (ty == kBf16) add_squares<kBf16>(s, q.grad, i0, i1);
    else add_squares<kF16>(s, q.grad, i0, i1);
  }
  const double v = group_sum((s.s[0] + s.s[1]) + (s.s[2] + s.s[3]), red);
  if (threadIdx.x == 0) part[blockIdx.x] = v;
}

__global__ __launch_bounds__(kThreads) void k_norm_inline(Inline in, Table t, double* part) {
  __shared__ double red[4];
  norm_part(in.e, t, part, red);
}
__global__ __launch_bounds__(kThreads) void k_norm_table(const Entry* e, Table t, double* part) {
  __shared__ double red[4];
  norm_part(e, t, part, red);
}

// sqrt of the parts' sum, in every thread.
__device__ __forceinline__ double norm_of(const double* part, int parts, double* red) {
  double s = 0.0;
  for (int i = threadIdx.x; i < parts; i += kThreads) s += part[i];
  return sqrt(group_sum(s, red));
}

__global__ __launch_bounds__(kThreads) void k_norm_join(const double* part, int parts, float* norm) {
  __shared__ double red[4];
  const double n = norm_of(part, parts, red);
  if (threadIdx.x == 0) *norm = static_cast<float>(n);
}

// B: float, or double where the scale is below float32's normal numbers.
template <class B>
__device__ __forceinline__ float scaled(float v, B by) { return static_cast<float>(static_cast<B>(v) * by); }

template <int T, int O, class B>
__device__ __forceinline__ void scale_chunk(const void* p, void* out, int64_t i0, int64_t i1, B by) {
  const int64_t whole = i0 + (i1 - i0) / kStep * kStep;
  if (i1 - i0 == kChunk) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float v[4][kVec];
#pragma unroll
      for (int u = 0; u < 4; ++u) load8<T>(v[u], p, i0 + (4 * h + u) * kStep + threadIdx.x * kVec);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
#pragma unroll
        for (int k = 0; k < kVec; ++k) v[u][k] = scaled(v[u][k], by);
        store8<O>(v[u], out, i0 + (4 * h + u) * kStep + threadIdx.x * kVec);
      }
    }
    return;
  }
  for (int64_t i = i0 + threadIdx.x * kVec; i < whole; i += kStep) {
    float v[kVec];
    load8<T>(v, p, i);
#pragma unroll
    for (int k = 0; k < kVec; ++k) v[k] = scaled(v[k], by);
    store8<O>(v, out, i);
  }
  for (int64_t i = whole + threadIdx.x; i < i1; i += kThreads) store1<O>(scaled(load1<T>(p, i), by), out, i);
}

template <int T, class B>
__device__ __forceinline__ void scale_to(const Entry& q, int64_t i0, int64_t i1, B by) {
  const int o = out_type_of(q);
  if (o == kF32) scale_chunk<T, kF32>(q.grad, q.out, i0, i1, by);
  else if (o == kBf16) scale_chunk<T, kBf16>(q.grad, q.out, i0, i1, by);
  else scale_chunk<T, kF16>(q.grad, q.out, i0, i1, by);
}

struct ScaleArgs {
  const double* part;  // parts sums of squares, or null: the norm is *total
  int parts;
  const float* total;
  float max_norm;
  float* norm;         // out, or null
};

__device__ void scale_part(const Entry* e, const Table& t, const ScaleArgs& a, double* red) {
  const double n = a.part ? norm_of(a.part, a.parts, red) : static_cast<double>(*a.total);
  if (a.norm && blockIdx.x == 0 && threadIdx.x == 0) *a.norm = static_cast<float>(n);
  const double ratio = static_cast<double>(a.max_norm) / (n + 1e-6);
  const float by = ratio > 1.0 ? 1.0f : static_cast<float>(ratio);  // NaN stays NaN
  const int64_t c0 = t.chunks * blockIdx.x / gridDim.x, c1 = t.chunks * (blockIdx.x + 1) / gridDim.x;
  if (c0 >= c1) return;
  int j = find_tensor(e, t.count, c1 - 1);
  for (int64_t c = c1 - 1; c >= c0; --c) {
    while (first_of(e[j]) > c || e[j].n == 0) --j;
    const Entry& q = e[j];
    const int ty = type_of(q);
    if (by == 1.0f && q.out == q.grad && ty == out_type_of(q)) continue;  // g * 1 is there already
    const int64_t i0 = (c - first_of(q)) * kChunk, i1 = q.n - i0 < kChunk ? q.n : i0 + kChunk;
    if (ratio < 0x1p-126) {
      if (ty == kF32) scale_to<kF32>(q, i0, i1, ratio);
      else if (ty == kBf16) scale_to<kBf16>(q, i0, i1, ratio);
      else scale_to<kF16>(q, i0, i1, ratio);
    } else if (ty == kF32) {
      scale_to<kF32>(q, i0, i1, by);
    } else if (ty == kBf16) {
      scale_to<kBf16>(q, i0, i1, by);
    } else {
      scale_to<kF16>(q, i0, i1, by);
    }
  }
}

__global__ __launch_bounds__(kThreads) void k_scale_inline(Inline in, Table t, ScaleArgs a) {
  __shared__ double red[4];
  scale_part(in.e, t, a, red);
}
__global__ __launch_bounds__(kThreads) void k_scale_table(const Entry* e, Table t, ScaleArgs a) {
  __shared__ double red[4];
  scale_part(e, t, a, red);
}

__global__ __launch_bounds__(128) void k_write_table(Inline in, int n, Entry* to) {
  if (static_cast<int>(threadIdx.x) < n) to[threadIdx.x] = in.e[threadIdx.x];
}

}  // namespace

size_t grad_workspace(int count) {
  return kMaxGroups * sizeof(double) + (count > kInline ? static_cast<size_t>(count) * sizeof(Entry) : 0);
}

hipError_t launch_grads(const nf4_grad* grads, int count, bool clip, float max_norm, const float* total_norm, float* norm,
                        void* ws, hipStream_t s) {
  double* part = static_cast<double*>(ws);
  Entry* table = reinterpret_cast<Entry*>(part + kMaxGroups);
  Inline in{};
  Table t{count, 0};
  const bool far = count > kInline;
  for (int i = 0; i < count; ++i) {
    const nf4_grad& g = grads[i];
    Entry& e = in.e[i % kInline];
    e = Entry{g.grad, g.out, g.n, t.chunks | (static_cast<int64_t>(g.dtype | (clip ? g.out_dtype << 2 : 0)) << kTypeShift)};
    t.chunks += (g.n + kChunk - 1) / kChunk;
    if (far && (i % kInline == kInline - 1 || i == count - 1))
      hipLaunchKernelGGL(k_write_table, dim3(1), dim3(128), 0, s, in, i % kInline + 1, table + i / kInline * kInline);
  }
  const int64_t most = 8 * static_cast<int64_t>(device_cus()) < kMaxGroups ? 8 * static_cast<int64_t>(device_cus()) : kMaxGroups;
  const int64_t want = t.chunks < most ? t.chunks : most;
  const dim3 grid(static_cast<unsigned>(want > 0 ? want : 1)), block(kThreads);
  if (!clip || !total_norm) {
    if (far) hipLaunchKernelGGL(k_norm_table, grid, block, 0, s, table, t, part);
    else hipLaunchKernelGGL(k_norm_inline, grid, block, 0, s, in, t, part);
  }
  if (!clip) {
    hipLaunchKernelGGL(k_norm_join, dim3(1), block, 0, s, part, static_cast<int>(grid.x), norm);
  } else {
    const ScaleArgs a{total_norm ? nullptr : part, static_cast<int>(grid.x), total_norm, max_norm, norm};
    if (far) hipLaunchKernelGGL(k_scale_table, grid, block, 0, s, table, t, a);
    else hipLaunchKernelGGL(k_scale_inline, grid, block, 0, s, in, t, a);
  }
  return hipGetLastError();
}

}  // namespace nf4i
