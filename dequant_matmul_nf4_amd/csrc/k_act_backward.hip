// The backward pass of the product's epilogue, y = act(z) + residual:
//
//   dz[t][n] = dy[t][n] act'(z[t][n])   (rounded once to bf16)
//   dbias[n] = sum_t dy[t][n] act'(z[t][n])   (float32, before that rounding)
//
// Reading dy and z and writing dz bounds it (6 bytes an element).  A thread
// takes 8 consecutive columns (16 bytes) and walks down a chunk of rows, so the
// bias's sums stay in its registers; the threads of a workgroup that share
// columns add theirs in LDS, each chunk leaves one row of sums in the workspace
// and a second kernel adds the chunks in order (results do not depend on timing).
// Rows of any length: loads and stores of 16 bytes need no alignment but the
// element's, and the columns past the last whole 8 are taken one by one.
//
// Measured: 4096 x 14336 with gelu_tanh 70 us and 4.8 for the chunks' sums (352 MB, 5.0
// TB/s); 333 x 11007 with gelu 13.4 and 3.9 (22 MB in one round of loads: latency).
// 64 threads across, not 256: a fourth of the chunks, and so of their sums.
#include "epilogue.h"
#include "layer_ops.h"

namespace nf4i {
namespace {

constexpr int kThreads = 256;
constexpr int kCols = 8;        // columns of a thread
constexpr int kUnroll = 4;      // rows on their way at a time
constexpr int kTail = 2;        // of them where the columns are taken one by one
constexpr int kMaxTx = 64;      // threads across the columns
constexpr int kMaxChunks = 256;

typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

struct Plan {
  int tx;            // threads across the columns (a power of two up to kMaxTx)
  int ctiles;        // workgroups across the columns
  int chunks;        // workgroups along the rows
  int64_t per;       // rows of a chunk
};

Plan make_plan(int64_t m, int64_t rows) {
  Plan p{};
  const int64_t vec = (rows + kCols - 1) / kCols;
  p.tx = 1;
  while (p.tx < kMaxTx && p.tx < vec) p.tx *= 2;
  const int64_t ctiles = (vec + p.tx - 1) / p.tx;
  const int ty = kThreads / p.tx;
  // about 8 workgroups per compute unit of a full chip, each with at least kUnroll rows per thread
  const int64_t want = ctiles > 2048 ? 1 : 2048 / ctiles, most = (m + ty * kUnroll - 1) / (ty * kUnroll);
  int64_t chunks = want < most ? want : most;
  chunks = chunks < kMaxChunks ? chunks : kMaxChunks;
  chunks = chunks > 1 ? chunks : 1;
  p.per = (m + chunks - 1) / chunks;
  p.per = (p.per + ty - 1) / ty * ty;
  p.chunks = static_cast<int>((m + p.per - 1) / p.per);
  p.ctiles = static_cast<int>(ctiles);
  return p;
}

__device__ __forceinline__ uint32_t pair(float lo, float hi) {
  const bf16x2 p = {static_cast<__bf16>(lo), static_cast<__bf16>(hi)};
  return __builtin_bit_cast(uint32_t, p);
}

template <int A, bool kDz, bool kBias>
__global__ __launch_bounds__(kThreads) void k_act_backward(const uint16_t* dy, const uint16_t* pre, int64_t m, int64_t rows,
                                                           uint16_t* dz, float* part, Plan pl) {
  __shared__ float red[kBias ? kThreads * kCols : 1];
  const int x = threadIdx.x & (pl.tx - 1), yy = threadIdx.x / pl.tx, ty = kThreads / pl.tx;
  const int64_t col = (static_cast<int64_t>(blockIdx.x) * pl.tx + x) * kCols;
  const int left = static_cast<int>(rows - col < kCols ? rows - col : kCols);  // columns of this thread
  const int64_t t0 = static_cast<int64_t>(blockIdx.y) * pl.per;
  const int64_t t1 = t0 + pl.per < m ? t0 + pl.per : m;
  float sum[kCols];
#pragma unroll
  for (int c = 0; c < kCols; ++c) sum[c] = 0.0f;

  if (left == kCols) {
    auto one = [&](const u32x4& d, const u32x4& z, int64_t at) {
      u32x4 o;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        float lo = bf16_to_f32(d[c] & 0xFFFFu), hi = __uint_as_float(d[c] & 0xFFFF0000u);
        if constexpr (A != kActNone) {
          lo *= act_slope<A>(bf16_to_f32(z[c] & 0xFFFFu));
          hi *= act_slope<A>(__uint_as_float(z[c] & 0xFFFF0000u));
        }
        if constexpr (kBias) {
          sum[2 * c] += lo;
          sum[2 * c + 1] += hi;
        }
        o[c] = pair(lo, hi);
      }
      if constexpr (kDz) *reinterpret_cast<u32x4_any*>(dz + at) = o;
    };
    int64_t t = t0 + yy;
    for (; t + (kUnroll - 1) * ty < t1; t += kUnroll * ty) {
      u32x4 d[kUnroll], z[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int64_t at = (t + u * ty) * rows + col;
        d[u] = *reinterpret_cast<const u32x4_any*>(dy + at);
        if constexpr (A != kActNone) z[u] = *reinterpret_cast<const u32x4_any*>(pre + at);
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) one(d[u], z[u], (t + u * ty) * rows + col);
    }
    for (; t < t1; t += ty) {
      const int64_t at = t * rows + col;
      u32x4 z{};
      if constexpr (A != kActNone) z = *reinterpret_cast<const u32x4_any*>(pre + at);
      const u32x4 d = *reinterpret_cast<const u32x4_any*>(dy + at);
      one(d, z, at);
    }
  } else {
    // the columns past the last whole 8: all that a few rows need is asked for before the first is stored
    // (dz may be dy, so the compiler would not; one at a time these threads took longer than all others)
    for (int64_t t = t0 + yy; t < t1; t += kTail * ty) {
      uint16_t d[kTail][kCols] = {}, z[kTail][kCols] = {};
#pragma unroll
      for (int u = 0; u < kTail; ++u)
#pragma unroll
        for (int c = 0; c < kCols; ++c)
          if (c < left && t + u * ty < t1) {
            const int64_t at = (t + u * ty) * rows + col + c;
            d[u][c] = dy[at];
            if constexpr (A != kActNone) z[u][c] = pre[at];
          }
#pragma unroll
      for (int u = 0; u < kTail; ++u)
#pragma unroll
        for (int c = 0; c < kCols; ++c)
          if (c < left && t + u * ty < t1) {
            float v = bf16_to_f32(d[u][c]);
            if constexpr (A != kActNone) v *= act_slope<A>(bf16_to_f32(z[u][c]));
            if constexpr (kBias) sum[c] += v;
            if constexpr (kDz) dz[(t + u * ty) * rows + col + c] = static_cast<uint16_t>(pair(v, 0.0f));
          }
    }
  }

  if constexpr (kBias) {
    for (int h = ty / 2; h >= 1; h /= 2) {  // the threads of one column pairwise
      if (yy >= h && yy < 2 * h)
#pragma unroll
        for (int c = 0; c < kCols; ++c) red[c * kThreads + threadIdx.x] = sum[c];
      __syncthreads();
      if (yy < h)
#pragma unroll
        for (int c = 0; c < kCols; ++c) sum[c] += red[c * kThreads + threadIdx.x + h * pl.tx];
      __syncthreads();
    }
    if (yy == 0)
#pragma unroll
      for (int c = 0; c < kCols; ++c)
        if (c < left) part[blockIdx.y * rows + col + c] = sum[c];
  }
}

// dbias[n] = the chunks' sums in order: four threads a column, each a quarter of the chunks.
__global__ __launch_bounds__(kThreads) void k_bias_join(const float* part, int64_t rows, int chunks, float* dbias) {
  __shared__ float red[kThreads];
  const int c = threadIdx.x & 63, q = threadIdx.x >> 6;
  const int64_t n = static_cast<int64_t>(blockIdx.x) * 64 + c;
  const int k0 = chunks * q / 4, k1 = chunks * (q + 1) / 4;
  float s = 0.0f;
  if (n < rows)
#pragma unroll 8
    for (int k = k0; k < k1; ++k) s += part[k * rows + n];
  red[threadIdx.x] = s;
  __syncthreads();
  if (q == 0 && n < rows) dbias[n] = ((s + red[64 + c]) + red[128 + c]) + red[192 + c];
}

template <int A>
void launch(const uint16_t* dy, const uint16_t* pre, int64_t m, int64_t rows, uint16_t* dz, float* part, const Plan& pl,
            hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(pl.ctiles), static_cast<unsigned>(pl.chunks)), block(kThreads);
  if (dz && part) hipLaunchKernelGGL((k_act_backward<A, true, true>), grid, block, 0, s, dy, pre, m, rows, dz, part, pl);
  else if (dz) hipLaunchKernelGGL((k_act_backward<A, true, false>), grid, block, 0, s, dy, pre, m, rows, dz, part, pl);
  else hipLaunchKernelGGL((k_act_backward<A, false, true>), grid, block, 0, s, dy, pre, m, rows, dz, part, pl);
}

}  // namespace

size_t act_backward_workspace(int64_t m, int64_t rows) {
  const Plan pl = make_plan(m, rows);
  return pl.chunks > 1 ? static_cast<size_t>(pl.chunks) * static_cast<size_t>(rows) * sizeof(float) : 0;
}

hipError_t launch_act_backward(const uint16_t* dy, const uint16_t* pre, int64_t m, int64_t rows, int act, uint16_t* dz,
                               float* dbias, float* ws, hipStream_t s) {
  const Plan pl = make_plan(m, rows);
  float* part = dbias && pl.chunks > 1 ? ws : dbias;
  switch (act) {
    case kActNone: launch<kActNone>(dy, pre, m, rows, dz, part, pl, s); break;
    case kActRelu: launch<kActRelu>(dy, pre, m, rows, dz, part, pl, s); break;
    case kActSilu: launch<kActSilu>(dy, pre, m, rows, dz, part, pl, s); break;
    case kActGelu: launch<kActGelu>(dy, pre, m, rows, dz, part, pl, s); break;
    default: launch<kActGeluTanh>(dy, pre, m, rows, dz, part, pl, s);
  }
  if (dbias && pl.chunks > 1)
    hipLaunchKernelGGL(k_bias_join, dim3(static_cast<unsigned>((rows + 63) / 64)), dim3(kThreads), 0, s, part, rows,
                       pl.chunks, dbias);
  return hipGetLastError();
}

}  // namespace nf4i
