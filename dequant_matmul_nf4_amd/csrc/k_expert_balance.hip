// The routers' balance loss of a mixture-of-experts layer and its gradient.
//
//   p[t] = softmax(logits[t])            (zeros where every logit is -inf)
//   counts[e] = slots of the kept tokens that chose expert e;  T = kept tokens
//   P[e] = sum over the kept t of p[t][e] / T
//   loss = coef E sum_e counts[e] / (T slots) P[e]
//   dlogits[t][e] = dloss coef E / (T^2 slots) p[t][e] (counts[e] - sum_j counts[j] p[t][j])
//
// Reading the logits bounds both (writing the gradient too).  A row belongs to
// a group of L lanes (a power of two), each lane holding kV consecutive
// experts (16 bytes) per step of L kV experts, so a wave works on 64 / L rows
// at a time and the row's maximum and sums are exchanged inside the group.  In
// the forward pass a lane's experts stay the same from row to row: the sums of
// probabilities stay in its registers, are added over the workgroup's waves in
// LDS and leave one row per workgroup in the workspace, as do the counts
// (integers, counted in LDS).  A second kernel adds the workgroups' rows, 64
// experts to a workgroup, and the last of its workgroups to arrive adds their
// shares of the loss in order; results do not depend on timing.  Few logits
// take one launch of one workgroup.  Measured: 131072 tokens of 128 experts in bf16
// with 8 slots 15.5 us and 5.2 for the joining (37.7 MB: 7.4 us at a copy's rate;
// exponentials and sums take 5 of the time, the launch and the sums over the workgroup most of the
// rest); the gradient of 16384 of 256 in float32 9.9 us (33.5 MB, 6.5).
//
// All counts have much in common, which cancels in the gradient as p sums to 1:
// their mean, an integer, is taken off first, so that what is left of the
// difference keeps float32's precision.
#include <type_traits>

#include "epilogue.h"
#include "layer_ops.h"

namespace nf4i {
namespace {

constexpr int kWaves = 16;
constexpr int kThreads = 64 * kWaves;
constexpr int kMaxE = 1024;
constexpr int kMaxGroups = 256;       // workgroups of the forward pass
constexpr int kJoinCols = 64;         // experts of a joining workgroup

typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4_any4 __attribute__((ext_vector_type(4), aligned(4)));

enum { kF32 = 0, kBf16 = 1, kF16 = 2 };

__device__ __forceinline__ float from16(uint32_t bits, int type) {
  if (type == kBf16) return bf16_to_f32(bits);
  return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(bits)));
}

// kV logits of a row from column c on; columns past the row's end are -inf.  kWhole: rows of
// a multiple of kV, so that no lane's columns are cut and no branch stands around a load (with
// one, every load is waited for before the next is asked for).
template <int T>
struct Row {
  static constexpr int kV = T == kF32 ? 4 : 8;
  template <bool kWhole>
  static __device__ __forceinline__ void load(float (&v)[kV], const void* base, int64_t row, int experts, int c) {
    if constexpr (kWhole) {
      const int64_t at = row * experts + (c < experts ? c : 0);
      if constexpr (T == kF32) {
        const u32x4_any4 w = *reinterpret_cast<const u32x4_any4*>(static_cast<const float*>(base) + at);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(w[i]);
      } else {
        const u32x4_any w = *reinterpret_cast<const u32x4_any*>(static_cast<const uint16_t*>(base) + at);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[2 * i] = from16(w[i] & 0xFFFFu, T);
          v[2 * i + 1] = from16(w[i] >> 16, T);
        }
      }
#pragma unroll
      for (int i = 0; i < kV; ++i) v[i] = c < experts ? v[i] : -INFINITY;
    } else if constexpr (T == kF32) {
      const float* p = static_cast<const float*>(base) + row * experts + c;
      if (c + kV <= experts) {
        const u32x4_any4 w = *reinterpret_cast<const u32x4_any4*>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(w[i]);
      } else {
#pragma unroll
        for (int i = 0; i < kV; ++i) v[i] = c + i < experts ? p[i] : -INFINITY;
      }
    } else {
      const uint16_t* p = static_cast<const uint16_t*>(base) + row * experts + c;
      if (c + kV <= experts) {
        const u32x4_any w = *reinterpret_cast<const u32x4_any*>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[2 * i] = from16(w[i] & 0xFFFFu, T);
          v[2 * i + 1] = from16(w[i] >> 16, T);
        }
      } else {
#pragma unroll
        for (int i = 0; i < kV; ++i) v[i] = c + i < experts ? from16(p[i], T) : -INFINITY;
      }
    }
  }
  static __device__ __forceinline__ void store(const float (&v)[kV], void* base, int64_t row, int experts, int c) {
    if constexpr (T == kF32) {
      float* p = static_cast<float*>(base) + row * experts + c;
      if (c + kV <= experts) {
        u32x4_any4 w;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(v[i]);
        *reinterpret_cast<u32x4_any4*>(p) = w;
      } else {
#pragma unroll
        for (int i = 0; i < kV; ++i)
          if (c + i < experts) p[i] = v[i];
      }
    } else {
      uint16_t b[kV];
#pragma unroll
      for (int i = 0; i < kV; ++i) {
        if constexpr (T == kBf16) b[i] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(v[i]));
        else b[i] = __builtin_bit_cast(uint16_t, static_cast<_Float16>(v[i]));
      }
      uint16_t* p = static_cast<uint16_t*>(base) + row * experts + c;
      if (c + kV <= experts) {
        u32x4_any w;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = b[2 * i] | (static_cast<uint32_t>(b[2 * i + 1]) << 16);
        *reinterpret_cast<u32x4_any*>(p) = w;
      } else {
#pragma unroll
        for (int i = 0; i < kV; ++i)
          if (c + i < experts) p[i] = b[i];
      }
    }
  }
};

// The value of another lane: within 16 lanes by the operand's own lane patterns (pairs and
// fours exchanged; halves of 8 and rows of 16 mirrored, which is as good once all lanes of a
// half agree), beyond through LDS.  With every step through LDS its latency was most of a row's time.
template <int off>
__device__ __forceinline__ float across(float v) {
  constexpr int kPattern = off == 1 ? 0xB1 : off == 2 ? 0x4E : off == 4 ? 0x141 : 0x140;
  if constexpr (off < 16)
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), kPattern, 0xF, 0xF, true));
  else
    return __shfl_xor(v, off, 64);
}
template <int L, int off = 1>
__device__ __forceinline__ float lanes_sum(float v) {
  if constexpr (off < L) return lanes_sum<L, 2 * off>(v + across<off>(v));
  else return v;
}
template <int L, int off = 1>
__device__ __forceinline__ float lanes_max(float v) {
  if constexpr (off < L) return lanes_max<L, 2 * off>(fmaxf(v, across<off>(v)));
  else return v;
}

// The softmax of a group's row in place; rows without any probability become zeros.
template <int kV, int IT, int L>
__device__ __forceinline__ void softmax(float (&v)[IT][kV]) {
  float top = -INFINITY;
#pragma unroll
  for (int it = 0; it < IT; ++it)
#pragma unroll
    for (int i = 0; i < kV; ++i) top = fmaxf(top, v[it][i]);
  top = lanes_max<L>(top);
  const float base = top == -INFINITY ? 0.0f : top;
  float sum = 0.0f;
#pragma unroll
  for (int it = 0; it < IT; ++it)
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      v[it][i] = exp_fast(v[it][i] - base);
      sum += v[it][i];
    }
  sum = lanes_sum<L>(sum);
  const float by = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
  for (int it = 0; it < IT; ++it)
#pragma unroll
    for (int i = 0; i < kV; ++i) v[it][i] *= by;
}

// Shares of the workspace: sums of probabilities and counts by workgroup, the
// joining workgroups' shares of the loss, their ticket.
struct Ws {
  float* probs;      // [groups][E]
  int32_t* counts;   // [groups][E + 1]
  double* share;     // [joining workgroups]
  uint32_t* ticket;
};

// Column E of the counts holds the kept tokens.
struct Args {
  const void* logits;
  const int32_t* ids;
  const uint8_t* mask;
  int64_t tokens;
  int experts, slots;
  float coef;
  float* loss;
  int32_t* counts;
  float* mean_probs;
  Ws ws;
};

__device__ __forceinline__ double loss_of(const Args& a, double sum, double kept) {
  return kept > 0 ? static_cast<double>(a.coef) * a.experts * sum / (kept * a.slots) : 0.0;
}

template <int T, int IT, int L>
__global__ __launch_bounds__(kThreads) void k_balance(Args a) {
  constexpr int kV = Row<T>::kV, kStep = L * kV;
  constexpr int kRows = 64 / L;      // rows of a wave at a time
  constexpr int kUnroll = IT > 1 ? 1 : kV > 4 ? 8 : 4;
  __shared__ float probs[kWaves][IT * kStep];
  __shared__ int32_t hist[4][kMaxE + 1];
  __shared__ double red[kWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane / L, l = lane & (L - 1);
  const int E = a.experts;
  for (int i = threadIdx.x; i < 4 * (kMaxE + 1); i += kThreads) hist[i / (kMaxE + 1)][i % (kMaxE + 1)] = 0;
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.ws.ticket = 0;
  __syncthreads();

  const int64_t t0 = a.tokens * blockIdx.x / gridDim.x, t1 = a.tokens * (blockIdx.x + 1) / gridDim.x;
  // a thread's first slots and whether their tokens are kept, asked for before the logits
  constexpr int kIds = 4;
  const int64_t slots0 = t0 * a.slots, slots1 = t1 * a.slots;
  const int turn = kThreads / a.slots, rest = kThreads - turn * a.slots;  // a thread's next slot is of the token `turn` on, or the next
  int64_t slot = slots0 + threadIdx.x, token = t0 + threadIdx.x / a.slots;
  int place = threadIdx.x % a.slots;
  auto next_ids = [&](int (&id)[kIds]) {
#pragma unroll
    for (int i = 0; i < kIds; ++i) {
      const bool have = slot < slots1;
      const int got = a.ids[have ? slot : 0];
      const bool keep = have && (!a.mask || a.mask[token < t1 ? token : 0]);
      id[i] = keep && got >= 0 && got < E ? got : -1;
      slot += kThreads;
      token += turn;
      place += rest;
      if (place >= a.slots) {
        place -= a.slots;
        ++token;
      }
    }
  };
  int id[kIds];
  next_ids(id);
  float sum[IT][kV];
#pragma unroll
  for (int it = 0; it < IT; ++it)
#pragma unroll
    for (int i = 0; i < kV; ++i) sum[it][i] = 0.0f;
  const uint8_t* const mask = a.mask ? a.mask : reinterpret_cast<const uint8_t*>(a.ids);  // read either way
  auto rows = [&](auto whole) {
    for (int64_t t = t0 + (wave * kUnroll) * kRows; t < t1; t += kWaves * kUnroll * kRows) {
      float v[kUnroll][IT][kV];
      bool live[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int64_t r = t + u * kRows + g;
        const uint8_t keep = mask[!a.mask ? 0 : r < t1 ? r : t1 - 1];
        live[u] = r < t1 && (!a.mask || keep);
#pragma unroll
        for (int it = 0; it < IT; ++it) Row<T>::template load<decltype(whole)::value>(v[u][it], a.logits, r < t1 ? r : t1 - 1, E, it * kStep + l * kV);
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        softmax<kV, IT, L>(v[u]);
#pragma unroll
        for (int it = 0; it < IT; ++it)
#pragma unroll
          for (int i = 0; i < kV; ++i) sum[it][i] += live[u] ? v[u][it][i] : 0.0f;
      }
    }
  };
  if (E % kV == 0) rows(std::true_type{});
  else rows(std::false_type{});
  // the counts: four tables, so that fewer of a wave's lanes meet in one place
  int kept = 0;
  for (int64_t t = t0 + threadIdx.x; t < t1; t += kThreads) kept += !a.mask || a.mask[t];
  for (;;) {
#pragma unroll
    for (int i = 0; i < kIds; ++i)
      if (id[i] >= 0) atomicAdd(&hist[threadIdx.x & 3][id[i]], 1);
    if (slot >= slots1) break;
    next_ids(id);
  }
  if (kept) atomicAdd(&hist[threadIdx.x & 3][E], kept);
  // a lane's columns over the wave's rows, then over the waves
#pragma unroll
  for (int it = 0; it < IT; ++it)
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      float s = sum[it][i];
#pragma unroll
      for (int off = L; off < 64; off <<= 1) s += __shfl_xor(s, off, 64);
      if (g == 0) probs[wave][it * kStep + l * kV + i] = s;
    }
  __syncthreads();
  const bool alone = gridDim.x == 1;
  const int total = hist[0][E] + hist[1][E] + hist[2][E] + hist[3][E];
  double share = 0.0;
  for (int e = threadIdx.x; e <= E; e += kThreads) {
    const int c = hist[0][e] + hist[1][e] + hist[2][e] + hist[3][e];
    float s = 0.0f;
    if (e < E)
#pragma unroll
      for (int w = 0; w < kWaves; ++w) s += probs[w][e];
    if (alone) {
      a.counts[e] = c;
      if (e < E) {
        const float mean = total > 0 ? s / static_cast<float>(total) : 0.0f;
        a.mean_probs[e] = mean;
        share += static_cast<double>(c) * static_cast<double>(mean);
      }
    } else {
      a.ws.counts[static_cast<int64_t>(blockIdx.x) * (E + 1) + e] = c;
      if (e < E) a.ws.probs[static_cast<int64_t>(blockIdx.x) * E + e] = s;
    }
  }
  if (!alone) return;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) share += __shfl_xor(share, off, 64);
  if (lane == 0) red[wave] = share;
  __syncthreads();
  if (threadIdx.x == 0) {
    double s = 0.0;
    for (int w = 0; w < kWaves; ++w) s += red[w];
    *a.loss = static_cast<float>(loss_of(a, s, total));
  }
}

// Adds the workgroups' rows: kJoinCols experts to a workgroup, its waves each a
// part of the rows.
__global__ __launch_bounds__(kThreads) void k_balance_join(Args a, int groups) {
  __shared__ double probs[kWaves][kJoinCols];
  __shared__ int32_t counts[kWaves][kJoinCols];
  __shared__ int32_t kept[kWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int E = a.experts, e = blockIdx.x * kJoinCols + lane;
  const int g0 = groups * wave / kWaves, g1 = groups * (wave + 1) / kWaves;
  double p = 0.0;
  int c = 0, k = 0;
  const int at = e < E ? e : E - 1;
#pragma unroll 4
  for (int g = g0; g < g1; ++g) {
    p += static_cast<double>(a.ws.probs[static_cast<int64_t>(g) * E + at]);
    c += a.ws.counts[static_cast<int64_t>(g) * (E + 1) + at];
  }
  for (int g = g0 + lane; g < g1; g += 64) k += a.ws.counts[static_cast<int64_t>(g) * (E + 1) + E];
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) k += __shfl_xor(k, off, 64);
  probs[wave][lane] = p;
  counts[wave][lane] = c;
  if (lane == 0) kept[wave] = k;
  __syncthreads();
  if (wave == 0) {
    int total = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) total += kept[w];
    p = 0.0;
    c = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      p += probs[w][lane];
      c += counts[w][lane];
    }
    const float mean = total > 0 ? static_cast<float>(p / total) : 0.0f;
    double share = 0.0;
    if (e < E) {
      a.counts[e] = c;
      a.mean_probs[e] = mean;
      share = total > 0 ? static_cast<double>(c) * (p / total) : 0.0;
    }
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) share += __shfl_xor(share, off, 64);
    if (lane == 0) {
      if (blockIdx.x == 0) a.counts[E] = total;
      if (gridDim.x == 1) {
        *a.loss = static_cast<float>(loss_of(a, share, total));
      } else {
        // the share is visible before the ticket says so; the last to arrive sees all of them
        __hip_atomic_store(&a.ws.share[blockIdx.x], share, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        const uint32_t last = __hip_atomic_fetch_add(a.ws.ticket, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
        if (last == gridDim.x - 1) {
          double s = 0.0;
          for (unsigned b = 0; b < gridDim.x; ++b)
            s += __hip_atomic_load(&a.ws.share[b], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
          *a.loss = static_cast<float>(loss_of(a, s, total));
        }
      }
    }
  }
}

struct BackArgs {
  const void* logits;
  const int32_t* counts;
  const uint8_t* mask;
  int64_t tokens;
  int experts, slots;
  float coef;
  const float* dloss;
  void* dlogits;
};

template <int T, int IT, int L>
__global__ __launch_bounds__(256) void k_balance_backward(BackArgs a) {
  constexpr int kV = Row<T>::kV, kStep = L * kV;
  constexpr int kRows = 64 / L;
  constexpr int kUnroll = IT > 1 ? 1 : 2;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane / L, l = lane & (L - 1);
  const int E = a.experts;
  const int64_t waves = static_cast<int64_t>(gridDim.x) * 4, at = static_cast<int64_t>(blockIdx.x) * 4 + wave;
  // the lane's counts without their mean, the factor of every gradient
  int32_t c[IT][kV];
  int64_t all = 0;
#pragma unroll
  for (int it = 0; it < IT; ++it)
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      const int e = it * kStep + l * kV + i;
      c[it][i] = e < E ? a.counts[e] : 0;
      all += c[it][i];
    }
#pragma unroll
  for (int off = 1; off < L; off <<= 1) all += __shfl_xor(all, off, 64);
  const int32_t mean = static_cast<int32_t>(all / E);
  float w[IT][kV];
#pragma unroll
  for (int it = 0; it < IT; ++it)
#pragma unroll
    for (int i = 0; i < kV; ++i) w[it][i] = it * kStep + l * kV + i < E ? static_cast<float>(c[it][i] - mean) : 0.0f;
  const double kept = a.counts[E];
  const double dl = a.dloss ? static_cast<double>(*a.dloss) : 1.0;
  const float by = kept > 0 ? static_cast<float>(dl * a.coef * E / (kept * kept * a.slots)) : 0.0f;

  const uint8_t* const mask = a.mask ? a.mask : reinterpret_cast<const uint8_t*>(a.counts);  // read either way
  auto rows = [&](auto whole) {
    for (int64_t t = at * kUnroll * kRows; t < a.tokens; t += waves * kUnroll * kRows) {
      float v[kUnroll][IT][kV];
      bool live[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int64_t r = t + u * kRows + g, rc = r < a.tokens ? r : a.tokens - 1;
        const uint8_t keep = mask[a.mask ? rc : 0];
        live[u] = !a.mask || keep;
#pragma unroll
        for (int it = 0; it < IT; ++it) Row<T>::template load<decltype(whole)::value>(v[u][it], a.logits, rc, E, it * kStep + l * kV);
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int64_t r = t + u * kRows + g;
        softmax<kV, IT, L>(v[u]);
        float dot = 0.0f;
#pragma unroll
        for (int it = 0; it < IT; ++it)
#pragma unroll
          for (int i = 0; i < kV; ++i) dot = fmaf(v[u][it][i], w[it][i], dot);
        dot = lanes_sum<L>(dot);
#pragma unroll
        for (int it = 0; it < IT; ++it) {
#pragma unroll
          for (int i = 0; i < kV; ++i) v[u][it][i] = live[u] ? by * v[u][it][i] * (w[it][i] - dot) : 0.0f;
          const int col = it * kStep + l * kV;
          if (r < a.tokens && col < E) Row<T>::store(v[u][it], a.dlogits, r, E, col);
        }
      }
    }
  };
  if (E % kV == 0) rows(std::true_type{});
  else rows(std::false_type{});
}

// Calls f<T, IT, L>() for a row of `experts` logits of `type`.
template <int T, class F>
void by_width(int experts, const F& f) {
  constexpr int kV = Row<T>::kV;
  const int vec = (experts + kV - 1) / kV;
  if (vec <= 1) f(std::integral_constant<int, 1>{}, std::integral_constant<int, 1>{});
  else if (vec <= 2) f(std::integral_constant<int, 1>{}, std::integral_constant<int, 2>{});
  else if (vec <= 4) f(std::integral_constant<int, 1>{}, std::integral_constant<int, 4>{});
  else if (vec <= 8) f(std::integral_constant<int, 1>{}, std::integral_constant<int, 8>{});
  else if (vec <= 16) f(std::integral_constant<int, 1>{}, std::integral_constant<int, 16>{});
  else if (vec <= 32) f(std::integral_constant<int, 1>{}, std::integral_constant<int, 32>{});
  else if (vec <= 64) f(std::integral_constant<int, 1>{}, std::integral_constant<int, 64>{});
  else if (vec <= 128) f(std::integral_constant<int, 2>{}, std::integral_constant<int, 64>{});
  else if constexpr (T == kF32) f(std::integral_constant<int, 4>{}, std::integral_constant<int, 64>{});
}

template <class F>
void by_type(int type, int experts, const F& f) {
  if (type == kF32) by_width<kF32>(experts, [&](auto it, auto l) { f(std::integral_constant<int, kF32>{}, it, l); });
  else if (type == kBf16) by_width<kBf16>(experts, [&](auto it, auto l) { f(std::integral_constant<int, kBf16>{}, it, l); });
  else by_width<kF16>(experts, [&](auto it, auto l) { f(std::integral_constant<int, kF16>{}, it, l); });
}

constexpr int64_t kAlone = 1 << 15;  // logits that one workgroup takes

int balance_groups(int64_t tokens, int experts) {
  if (tokens * experts <= kAlone) return 1;
  const int64_t want = (tokens * experts + kAlone / 4 - 1) / (kAlone / 4);
  return static_cast<int>(want < kMaxGroups ? want : kMaxGroups);
}

}  // namespace

size_t expert_balance_workspace(int64_t tokens, int experts) {
  const int g = balance_groups(tokens, experts);
  const size_t rows = g > 1 ? (static_cast<size_t>(g) * (2 * experts + 1) * 4 + 7) / 8 * 8 : 0;
  return rows + kMaxE / kJoinCols * sizeof(double) + 8;
}

hipError_t launch_expert_balance(const void* logits, int type, const int32_t* ids, const uint8_t* mask, int64_t tokens,
                                 int experts, int slots, float coef, float* loss, int32_t* counts, float* mean_probs,
                                 void* ws, hipStream_t s) {
  const int groups = balance_groups(tokens, experts);
  Args a{logits, ids, mask, tokens, experts, slots, coef, loss, counts, mean_probs, {}};
  a.ws.share = static_cast<double*>(ws);
  a.ws.ticket = reinterpret_cast<uint32_t*>(a.ws.share + kMaxE / kJoinCols);
  a.ws.probs = reinterpret_cast<float*>(a.ws.ticket + 2);
  a.ws.counts = reinterpret_cast<int32_t*>(a.ws.probs + static_cast<int64_t>(groups) * experts);
  by_type(type, experts, [&](auto t, auto it, auto l) {
    hipLaunchKernelGGL((k_balance<decltype(t)::value, decltype(it)::value, decltype(l)::value>), dim3(groups), dim3(kThreads), 0, s, a);
  });
  if (groups > 1)
    hipLaunchKernelGGL(k_balance_join, dim3((experts + kJoinCols - 1) / kJoinCols), dim3(kThreads), 0, s, a, groups);
  return hipGetLastError();
}

hipError_t launch_expert_balance_backward(const void* logits, int type, const int32_t* counts, const uint8_t* mask,
                                          int64_t tokens, int experts, int slots, float coef, const float* dloss,
                                          void* dlogits, hipStream_t s) {
  const BackArgs a{logits, counts, mask, tokens, experts, slots, coef, dloss, dlogits};
  by_type(type, experts, [&](auto t, auto it, auto l) {
    constexpr int kRows = (decltype(it)::value > 1 ? 1 : 2) * (64 / decltype(l)::value);
    const int64_t want = (tokens + 4 * kRows - 1) / (4 * kRows), most = 16 * device_cus();
    const unsigned grid = static_cast<unsigned>(want < most ? want : most);
    hipLaunchKernelGGL((k_balance_backward<decltype(t)::value, decltype(it)::value, decltype(l)::value>), dim3(grid), dim3(256), 0, s, a);
  });
  return hipGetLastError();
}

}  // namespace nf4i
