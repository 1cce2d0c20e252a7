// The routing around a mixture-of-experts product: which rows go to which
// expert (expert_plan), and the weighted sum of the experts' rows back into
// the tokens with its gradients (expert_combine).
//
// A "slot" is one of a token's choices of an expert: slot t * k + j is the
// j-th choice of token t.  The plan is a stable counting sort of the slots by
// expert: offsets[e] .. offsets[e + 1] are the sorted rows of expert e,
// order[p] the slot at row p and position[s] the row of slot s (-1: the id is
// outside 0 .. experts - 1, the slot is dropped).  Ranks come from ballots
// and prefix sums, never from the order in which atomics arrive.  The plan is
// launches and latency (64 slots: one launch, 3.1 us; 131072 slots over 128 experts:
// two, 2.5 + 7.0 us).  The sums are bound by HBM: 32768 rows of 4096 columns into
// 16384 tokens 78 us (5.2 TB/s), backward 134 us (4.8 TB/s).
#include "expert_int4.h"
#include "nf4_device.h"

namespace nf4i {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kPlanThreads = 1024;
constexpr int kPlanWaves = kPlanThreads / 64;
constexpr int kPlanMaxBlocks = 256;

// Lanes of the wave with this lane's key, over the `bits` that the experts
// use: one ballot per bit.
__device__ __forceinline__ uint64_t same_key(int key, int bits) {
  uint64_t m = ~uint64_t(0);
  for (int b = 0; b < bits; ++b) {
    const bool one = (key >> b) & 1;
    const uint64_t v = __ballot(one);
    m &= one ? v : ~v;
  }
  return m;
}

// Exclusive prefix sum over the 1024 threads of a workgroup; *total gets the sum.
__device__ __forceinline__ int block_prefix(int v, int* wsum, int* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int s = v;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int t = __shfl_up(s, off, 64);
    if (lane >= off) s += t;
  }
  if (lane == 63) wsum[wave] = s;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kPlanWaves; ++w) {
    before += w < wave ? wsum[w] : 0;
    all += wsum[w];
  }
  __syncthreads();
  *total = all;
  return before + s - v;
}

// counts[block][e]: the block's slots per expert.
__global__ __launch_bounds__(kPlanThreads) void k_plan_count(const int32_t* __restrict__ ids, int64_t n, int experts,
                                                             int64_t chunk, int32_t* __restrict__ counts) {
  __shared__ int hist[kMaxExperts];
  hist[threadIdx.x] = 0;
  __syncthreads();
  const int64_t lo = blockIdx.x * chunk, hi = lo + chunk < n ? lo + chunk : n;
  for (int64_t i = lo + threadIdx.x; i < hi; i += kPlanThreads) {
    const int id = ids[i];
    if (id >= 0 && id < experts) atomicAdd(&hist[id], 1);
  }
  __syncthreads();
  if (threadIdx.x < experts) counts[static_cast<int64_t>(blockIdx.x) * experts + threadIdx.x] = hist[threadIdx.x];
}

// kOne: the one block of a small plan counts for itself.
template <bool kOne>
__global__ __launch_bounds__(kPlanThreads) void k_plan_place(const int32_t* __restrict__ ids, int64_t n, int experts,
                                                             int bits, int64_t chunk, const int32_t* __restrict__ counts,
                                                             int32_t* __restrict__ order, int32_t* __restrict__ position,
                                                             int32_t* __restrict__ offsets) {
  __shared__ int base[kMaxExperts];                  // the next row of each expert
  __shared__ uint16_t wcnt[kPlanWaves][kMaxExperts + 1];
  __shared__ int wsum[kPlanWaves];
  __shared__ int sums[2][kOne ? 1 : kPlanThreads];
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int64_t lo = blockIdx.x * chunk, hi = lo + chunk < n ? lo + chunk : n;
  int next = lo + t < hi ? ids[lo + t] : -1;  // this thread's id of the next round
  int mine = 0, before = 0;                   // expert t: all slots, those of earlier blocks
  for (int w = 0; t < experts && w < kPlanWaves; ++w) wcnt[w][t] = 0;
  if constexpr (kOne) {
    base[t] = 0;
    __syncthreads();
    for (int64_t i = t; i < n; i += kPlanThreads) {
      const int id = ids[i];
      if (id >= 0 && id < experts) atomicAdd(&base[id], 1);
    }
    __syncthreads();
    mine = base[t];
    __syncthreads();
  } else {
    // the threads read the blocks' counts, 2^bits of them one block at a time
    const int e = t & ((1 << bits) - 1), lanes = kPlanThreads >> bits;
    int all = 0, early = 0;
    if (e < experts) {
#pragma unroll 4
      for (int b = t >> bits; b < static_cast<int>(gridDim.x); b += lanes) {
        const int c = counts[static_cast<int64_t>(b) * experts + e];
        all += c;
        early += b < static_cast<int>(blockIdx.x) ? c : 0;
      }
    }
    sums[0][t] = all;
    sums[1][t] = early;
    __syncthreads();
    for (int k = t; t < experts && k < kPlanThreads; k += 1 << bits) {
      mine += sums[0][k];
      before += sums[1][k];
    }
  }
  int total;
  const int first = block_prefix(mine, wsum, &total);
  base[t] = first + before;
  if (blockIdx.x == 0) {
    if (t < experts) offsets[t] = first;
    if (t == 0) offsets[experts] = total;
  }
  // rows past the last kept slot
  for (int64_t i = lo + t; i < hi; i += kPlanThreads)
    if (i >= total) order[i] = -1;
  for (int64_t i0 = lo; i0 < hi; i0 += kPlanThreads) {
    const int64_t i = i0 + t;
    const int key = next >= 0 && next < experts ? next : kMaxExperts;
    next = i + kPlanThreads < hi ? ids[i + kPlanThreads] : -1;
    const uint64_t kept = __ballot(key < kMaxExperts);
    const uint64_t mask = same_key(key, bits) & kept;
    const int rank = __popcll(mask & ((uint64_t(1) << lane) - 1));
    if (key < kMaxExperts && rank == 0) wcnt[wave][key] = static_cast<uint16_t>(__popcll(mask));
    __syncthreads();
    // per expert: the waves' counts into their prefix, and the tile's sum onto base
    int sum = 0;
    if (t < experts) {
#pragma unroll
      for (int w = 0; w < kPlanWaves; ++w) {
        const int c = wcnt[w][t];
        wcnt[w][t] = static_cast<uint16_t>(sum);
        sum += c;
      }
    }
    __syncthreads();
    if (i < hi) {
      int p = -1;
      if (key < kMaxExperts) {
        p = base[key] + wcnt[wave][key] + rank;
        order[p] = static_cast<int32_t>(i);
      }
      position[i] = p;
    }
    __syncthreads();
    if (t < experts) {
      base[t] += sum;
      for (int w = 0; w < kPlanWaves; ++w) wcnt[w][t] = 0;
    }
    __syncthreads();
  }
}

// ----------------------------------------------------------------- combine

__device__ __forceinline__ void unpack8(const u32x4& v, float (&f)[8]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    f[2 * k] = bf16_to_f32(v[k] & 0xFFFFu);
    f[2 * k + 1] = __uint_as_float(v[k] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ u32x4 pack8(const float (&f)[8]) {
  return u32x4{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7])};
}

// out[t] = sum_j weights[t][j] y[position[t][j]], summed in float32 in the
// order of j and rounded once.  `lanes` threads per token, 8 columns each.
__global__ __launch_bounds__(256) void k_combine(const uint16_t* __restrict__ y, int64_t m,
                                                 const int32_t* __restrict__ position, int64_t tokens, int slots,
                                                 int64_t cols, const float* __restrict__ weights,
                                                 uint16_t* __restrict__ out, int lanes) {
  const int64_t token = block_number() * (256 / lanes) + threadIdx.x / lanes;
  if (token >= tokens) return;
  const int32_t* pos = position + token * slots;
  const float* wt = weights ? weights + token * slots : nullptr;
  for (int64_t c = (threadIdx.x & (lanes - 1)) * 8; c < cols; c += lanes * 8) {
    float acc[8] = {};
    for (int j = 0; j < slots; ++j) {
      const int64_t p = pos[j];
      if (p < 0 || p >= m) continue;
      const float w = wt ? wt[j] : 1.0f;
      float f[8];
      unpack8(*reinterpret_cast<const u32x4*>(y + p * cols + c), f);
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[k] = fmaf(w, f[k], acc[k]);
    }
    __builtin_nontemporal_store(pack8(acc), reinterpret_cast<u32x4*>(out + token * cols + c));
  }
}

// A wave per slot s of token t at row p: dy[p] = weights[s] dout[t] and
// dweights[s] = <dout[t], y[p]>.
__global__ __launch_bounds__(256) void k_combine_backward(const uint16_t* __restrict__ dout,
                                                          const uint16_t* __restrict__ y, int64_t m,
                                                          const int32_t* __restrict__ position, int64_t n, int slots,
                                                          int64_t cols, const float* __restrict__ weights,
                                                          uint16_t* __restrict__ dy, float* __restrict__ dweights) {
  const int lane = threadIdx.x & 63;
  const int64_t s = block_number() * 4 + (threadIdx.x >> 6);
  if (s >= n) return;
  const int64_t p = position[s], token = s / slots;
  const bool live = p >= 0 && p < m;
  float dot = 0.0f;
  if (live) {
    const float w = weights ? weights[s] : 1.0f;
    for (int64_t c = lane * 8; c < cols; c += 512) {
      float g[8], f[8], d[8];
      unpack8(*reinterpret_cast<const u32x4*>(dout + token * cols + c), g);
      if (dweights) {
        unpack8(*reinterpret_cast<const u32x4*>(y + p * cols + c), f);
#pragma unroll
        for (int k = 0; k < 8; ++k) dot = fmaf(g[k], f[k], dot);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) d[k] = w * g[k];
      if (dy) __builtin_nontemporal_store(pack8(d), reinterpret_cast<u32x4*>(dy + p * cols + c));
    }
  }
  if (dweights) {
    dot = wave_sum(dot);
    if (lane == 0) dweights[s] = dot;
  }
}

}  // namespace

// Blocks of a plan, at most kPlanMaxBlocks (their counts are the workspace),
// each of whole rounds of kPlanThreads slots.
static int64_t plan_chunk(int64_t n) {
  const int64_t rounds = (n + kPlanThreads - 1) / kPlanThreads;
  return (rounds + kPlanMaxBlocks - 1) / kPlanMaxBlocks * kPlanThreads;
}
constexpr int64_t kPlanOne = 4096;  // at most this many slots: one block, one launch

size_t expert_plan_workspace(int64_t n, int experts) {
  if (n <= kPlanOne) return 0;
  const int64_t chunk = plan_chunk(n);
  return static_cast<size_t>((n + chunk - 1) / chunk) * experts * sizeof(int32_t);
}

hipError_t launch_expert_plan(const int32_t* ids, int64_t n, int experts, int32_t* order, int32_t* position,
                              int32_t* offsets, void* ws, hipStream_t s) {
  int bits = 0;
  while ((1 << bits) < experts) ++bits;
  if (n <= kPlanOne) {
    hipLaunchKernelGGL((k_plan_place<true>), dim3(1), dim3(kPlanThreads), 0, s, ids, n, experts, bits, n, nullptr, order,
                       position, offsets);
    return hipGetLastError();
  }
  const int64_t chunk = plan_chunk(n);
  const unsigned blocks = static_cast<unsigned>((n + chunk - 1) / chunk);
  int32_t* counts = static_cast<int32_t*>(ws);
  hipLaunchKernelGGL(k_plan_count, dim3(blocks), dim3(kPlanThreads), 0, s, ids, n, experts, chunk, counts);
  hipLaunchKernelGGL((k_plan_place<false>), dim3(blocks), dim3(kPlanThreads), 0, s, ids, n, experts, bits, chunk, counts,
                     order, position, offsets);
  return hipGetLastError();
}

hipError_t launch_expert_combine(const uint16_t* y, int64_t m, const int32_t* position, int64_t tokens, int slots,
                                 int64_t cols, const float* weights, uint16_t* out, hipStream_t s) {
  int lanes = 8;
  while (lanes < 256 && lanes * 8 < cols) lanes <<= 1;
  const int64_t blocks = (tokens + 256 / lanes - 1) / (256 / lanes);
  hipLaunchKernelGGL(k_combine, block_grid(blocks), dim3(256), 0, s, y, m, position, tokens, slots, cols,
                     weights, out, lanes);
  return hipGetLastError();
}

hipError_t launch_expert_combine_backward(const uint16_t* dout, const uint16_t* y, int64_t m, const int32_t* position,
                                          int64_t tokens, int slots, int64_t cols, const float* weights, uint16_t* dy,
                                          float* dweights, hipStream_t s) {
  const int64_t n = tokens * slots;
  const int64_t blocks = (n + 3) / 4;
  hipLaunchKernelGGL(k_combine_backward, block_grid(blocks), dim3(256), 0, s, dout, y, m, position, n,
                     slots, cols, weights, dy, dweights);
  return hipGetLastError();
}

}  // namespace nf4i
