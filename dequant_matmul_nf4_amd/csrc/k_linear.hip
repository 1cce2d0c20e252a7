// A layer's product with its epilogue for many rows of x (prompts, training):
//
//   z = x . deq(W)^T + s (x . A^T) . B^T + bias;   y = act(z) + residual
//
// The K loop is the forward GEMM's (gemm_fwd.h; its schedule, operands and work
// units are described in k_gemm.hip), the weight rounded once to bf16 after
// scaling.  The adapters are extra K columns, as there; B is read from its own
// rows, which only this kernel's last step or two need.
//
// The epilogue: the matrix cores leave a lane with 4 consecutive columns of 32
// rows, 8 bytes of bf16 each, which as they are would touch a line of memory per
// row with every store.  A wave turns its 64 columns in LDS instead, 64 rows at a
// time in a quarter of the stages that is its own (free after the last step), and
// takes them back as 8 columns of 8 rows, so that residual, pre and y move in
// whole lines and the lane's bias stays in registers.  16-byte piece p of row r
// sits at slot p ^ (r % 16): no two rows of a store meet in a bank.
#include "gemm_fwd.h"
#include "linear_epilogue.h"

namespace nf4i {
namespace {

using gt::bf16x8;
using gt::floatx16;
using gt::kCopies;
using gt::kThreads;

constexpr int kBN = gt::kTileN, kBK = gt::kStep;
constexpr int kMI = 8;
constexpr int kBM = 32 * kMI;
constexpr int kStageBytes = gt::act_stage_bytes<kBM>();
constexpr int kTurnRows = 64;
static_assert(kTurnRows * 64 * 4 * 4 == 2 * kStageBytes, "four waves' quarters fill both stages");

struct LinearArgs {
  const uint8_t* packed;
  int64_t rows, cols;
  Scales sc;
  const uint16_t* x;
  int64_t m;
  uint16_t* y;
  Epilogue ep;
  const uint16_t* u;   // adapter columns of x: [m][kl] (s T hi | s T lo | 0), or null
  const uint16_t* lb;  // B [rows][r]
  int r, r_pad, kl;
  int64_t whole, units;  // as in the forward GEMM
  Codebook cb;
};

// Eight adapter columns c .. c + 7 of weight row n: (B | B | 0).
__device__ __forceinline__ bf16x8 adapter_frag(const LinearArgs& a, int64_t n, int c) {
  const int j0 = c < a.r_pad ? c : c - a.r_pad;
  const uint16_t* b = a.lb + n * a.r;
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint32_t h[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int j = j0 + 2 * k + i;
      h[i] = j < a.r ? b[j] : 0u;  // c past 2 r_pad: j >= r there too
    }
    w[k] = h[0] | (h[1] << 16);
  }
  const gt::u32x4 v = {w[0], w[1], w[2], w[3]};
  return __builtin_bit_cast(bf16x8, v);
}

template <int MI>
__device__ __forceinline__ void epilogue(const floatx16 (&acc)[MI][2], const LinearArgs& a, int64_t m0, int64_t n0, char* turn,
                                         int wave, int lane) {
  const int64_t col = n0 + wave * 64 + 8 * (lane & 7);
  const bool vec = (a.rows & 7) == 0;  // every row of the outputs 16-byte aligned
  const int left = static_cast<int>(a.rows - col < 8 ? a.rows - col : 8);
  float bias[8];
#pragma unroll
  for (int c = 0; c < 8; ++c) bias[c] = c < left ? lin::bias_at(a.ep, col + c) : 0.0f;
#pragma unroll
  for (int rd = 0; rd < MI / 2; ++rd) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int row = 32 * i + (lane & 31), p = 8 * j + 2 * g + (lane >> 5);
          const floatx16& t = acc[2 * rd + i][j];
          *reinterpret_cast<float4*>(turn + row * 256 + ((p ^ (row & 15)) << 4)) =
              make_float4(t[4 * g], t[4 * g + 1], t[4 * g + 2], t[4 * g + 3]);
        }
    // the wave's own LDS accesses are served in order; this keeps the compiler to it
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    lin::with_act(a.ep.act, [&](auto act) {
#pragma unroll 2
      for (int it = 0; it < 8; ++it) {
        const int row = 8 * it + (lane >> 3), p = 2 * (lane & 7);
        const int64_t t = m0 + 64 * rd + row;
        const float4 lo = *reinterpret_cast<const float4*>(turn + row * 256 + ((p ^ (row & 15)) << 4));
        const float4 hi = *reinterpret_cast<const float4*>(turn + row * 256 + (((p + 1) ^ (row & 15)) << 4));
        if (t >= a.m || left <= 0) continue;
        const float z[8] = {lo.x + bias[0], lo.y + bias[1], lo.z + bias[2], lo.w + bias[3],
                            hi.x + bias[4], hi.y + bias[5], hi.z + bias[6], hi.w + bias[7]};
        const int64_t at = t * a.rows + col;
        if (vec) {
          lin::finish8<decltype(act)::value>(a.ep, a.y, at, z);
        } else {
#pragma unroll
          for (int c = 0; c < 8; ++c)
            if (c < left) lin::finish1<decltype(act)::value>(a.ep, a.y, at + c, z[c]);
        }
      }
    });
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  }
}

// One work unit: the (32 MI) x 256 tile of y at rows m0.., columns n0..
template <int MI, bool kDQ, bool kF8>
__device__ __forceinline__ void linear_unit(const LinearArgs& a, int64_t m0, int64_t n0, char* xs, const char* tabc,
                                            uint32_t slot, float mean, int wave, int lane) {
  char *xs0 = xs, *xs1 = xs + kStageBytes;
  const gt::ActPtrs<MI> xp = gt::make_act_ptrs<MI, 32 * MI>(a.x, a.cols, a.m, m0, wave, lane);
  gt::WPtrs wp;
  int64_t nrow[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int64_t n = n0 + wave * 64 + j * 32 + (lane & 31);
    nrow[j] = n < a.rows ? n : a.rows - 1;  // rows past the end: never stored
    wp.c[j] = a.packed + nrow[j] * (a.cols / 2) + (lane >> 5) * 16;
    wp.blk[j] = nrow[j] * (a.cols / 64);
  }
  floatx16 acc[MI][2];
  gt::zero_acc(acc);
  gt::fwd_steps<MI, kDQ, kF8>(
      a.sc, a.cols / kBK, [&](int64_t ks, char* stage) { gt::dma_act(xp, ks, stage, wave); }, wp, xs0, xs1, tabc, slot, mean,
      lane, acc);
  if (a.kl > 0) {
    const gt::ActPtrs<MI> up = gt::make_act_ptrs<MI, 32 * MI>(a.u, a.kl, a.m, m0, wave, lane);
    const uint32_t sw = ((lane & 31) >> 1) & 7, h4 = (lane >> 5) * 4;
    for (int k0 = 0; k0 < a.kl; k0 += kBK) {
      gt::dma_act(up, k0 / kBK, xs0, wave);  // xs0 was last read before the previous barrier
      bf16x8 bl[4][2];
#pragma unroll
      for (int s4 = 0; s4 < 4; ++s4)
#pragma unroll
        for (int j = 0; j < 2; ++j) bl[s4][j] = adapter_frag(a, nrow[j], k0 + 8 * static_cast<int>(h4) + 8 * s4);
      gt::wait_vmem();
      __syncthreads();
      const char* xa = xs0 + (lane & 31) * gt::kActRowBytes;
#pragma unroll
      for (int s4 = 0; s4 < 4; ++s4) {
        bf16x8 af[MI];
        gt::read_act(xa, s4, sw, h4, af);
        gt::mfma16(af, bl[s4], acc);
      }
      __syncthreads();
    }
  }
  epilogue<MI>(acc, a, m0, n0, xs + wave * (2 * kStageBytes / 4), wave, lane);
  __syncthreads();  // the next unit's first stage may lie in another wave's quarter
}

template <bool kDQ, bool kF8>
__global__ __launch_bounds__(kThreads, 1) void k_linear(LinearArgs a) {
  __shared__ __align__(16) char xs[2 * kStageBytes];
  __shared__ __align__(16) float2 tab[256 * kCopies];
  const char* tabc = reinterpret_cast<const char*>(tab);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  static_assert(kCopies == 32, "a copy's slot");
  const uint32_t slot = static_cast<uint32_t>(lane & (kCopies - 1)) << 3;
  gt::fill_level_pairs<kCopies>(tab, a.cb);  // ends with a barrier
  const float mean = kDQ ? *a.sc.mean : 0.0f;
  const int64_t tiles_n = (a.rows + kBN - 1) / kBN;
  const int64_t tiles = tiles_n * ((a.m + kBM - 1) / kBM);
  for (int64_t u = blockIdx.x; u < a.units; u += gridDim.x) {
    const bool half = u >= a.whole;
    const int64_t tile = half ? a.whole + (u - a.whole) / 2 : u;
    int64_t tid = tile;
    if (tiles % 8 == 0) tid = (tile % 8) * (tiles / 8) + tile / 8;
    const int64_t m0 = (tid / tiles_n) * kBM;
    const int64_t n0 = (tid % tiles_n) * kBN;
    if (!half) {
      linear_unit<kMI, kDQ, kF8>(a, m0, n0, xs, tabc, slot, mean, wave, lane);
    } else {
      const int64_t mh = m0 + ((u - a.whole) & 1) * (kBM / 2);
      if (mh < a.m) linear_unit<kMI / 2, kDQ, kF8>(a, mh, n0, xs, tabc, slot, mean, wave, lane);
    }
  }
}

}  // namespace

size_t linear_workspace(int64_t m, int64_t rows, int64_t cols, int r) {
  (void)rows;
  (void)cols;
  return r > 0 ? static_cast<size_t>(m) * gemm_lora_cols(r) * sizeof(uint16_t) : 0;
}

hipError_t launch_linear(const uint8_t* packed, int64_t rows, int64_t cols, Scales sc, const uint16_t* x, int64_t m,
                         uint16_t* y, const Epilogue& ep, const uint16_t* lora_a, const uint16_t* lora_b, int r,
                         float lora_scale, void* ws, hipStream_t s) {
  LinearArgs a{};
  a.packed = packed; a.rows = rows; a.cols = cols; a.sc = sc; a.x = x; a.m = m; a.y = y; a.ep = ep;
  a.cb = codebook(sc.fp4);
  if (r > 0) {
    a.u = static_cast<const uint16_t*>(ws);
    a.lb = lora_b;
    a.r = r;
    a.r_pad = (r + 15) / 16 * 16;
    a.kl = static_cast<int>(gemm_lora_cols(r));
    if (hipError_t e = launch_lora_u(x, lora_a, m, cols, r, lora_scale, static_cast<uint16_t*>(ws), s)) return e;
  }
  const int64_t tiles = ((rows + kBN - 1) / kBN) * ((m + kBM - 1) / kBM);
  const int64_t slots = device_cus();
  const int64_t last = tiles - tiles / slots * slots;
  const bool halve = last > 0 && 2 * last <= slots && m > kBM / 2;
  a.whole = halve ? tiles - last : tiles;
  a.units = halve ? tiles + last : tiles;
  const unsigned grid = static_cast<unsigned>(a.units < slots ? a.units : slots);
  if (sc.absmax) hipLaunchKernelGGL((k_linear<false, false>), dim3(grid), dim3(kThreads), 0, s, a);
  else if (sc.f8) hipLaunchKernelGGL((k_linear<true, true>), dim3(grid), dim3(kThreads), 0, s, a);
  else hipLaunchKernelGGL((k_linear<true, false>), dim3(grid), dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace nf4i
