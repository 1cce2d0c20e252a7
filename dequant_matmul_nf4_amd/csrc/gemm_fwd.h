// The K loop of the forward products y = x . deq(W)^T on the matrix cores,
// shared by the GEMM (k_gemm.hip, where its schedule and operands are
// described) and the 64-row tiles of the product grouped by expert
// (k_expert_gemm.hip): a workgroup
// of 4 waves accumulates a (32 MI) x 256 tile, x through two LDS stages that
// the caller's `dma` fills, the weights' codes straight into operands.
#pragma once

#include "gemm_tiles.h"

namespace nf4i {
namespace gt {

constexpr int kCopies = 32;  // of the level-pair table: 64 KB

// The 256 level pairs (element 2j = high nibble first), C interleaved copies:
// entry e of copy c at byte e * 8 C + c * 8.  Ends with a barrier.
template <int C>
__device__ __forceinline__ void fill_level_pairs(float2* tab, const Codebook& cb) {
  if (threadIdx.x < 256) {
    const int e = threadIdx.x;
    const float2 v = make_float2(cb.level[e >> 4], cb.level[e & 15]);
#pragma unroll
    for (int c = 0; c < C; ++c) tab[e * C + c] = v;
  }
  __syncthreads();
}

// The codes a lane expands in one K step: for its two W rows (j = 0, 1) the
// 16 bytes of columns 32 h .. 32 h + 31, and the rows' block scale inputs.
struct WRegs {
  u32x4 w[2];
  float am[2];   // absmax (plain scales)
  int q[2];      // int8 scale code (double quant)
  float s2[2];
};

struct WPtrs {
  const uint8_t* c[2];    // codes of row j at step 0, lane half's 16 bytes
  int64_t blk[2];         // block index of row j at step 0
};

template <bool kDQ>
__device__ __forceinline__ void load_w(WRegs& r, const WPtrs& p, const Scales& sc, int64_t ks) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    r.w[j] = *reinterpret_cast<const u32x4*>(p.c[j] + ks * (kStep / 2));
    const int64_t blk = p.blk[j] + ks;
    if constexpr (kDQ) {
      r.q[j] = sc.q[blk];
      r.s2[j] = sc.absmax2[blk >> 8];
    } else {
      r.am[j] = sc.absmax[blk];
    }
  }
}

// Level pairs of code bytes 4 s .. 4 s + 3 of a lane's 16 bytes (one k step
// of one W row): four LDS reads.  The byte permute puts the code byte at
// bits 8..15 next to the lane's slot; a shift scales it to the entry size
// 8 C (slot = (lane % C) << (8 - log2 C)).
struct Lookups {
  float2 l[2][4];
};

template <int C>
__device__ __forceinline__ void lookup_step(Lookups& lk, const u32x4 (&w)[2], int s, const char* tab,
                                            uint32_t slot) {
  constexpr int kShift = C == 32 ? 0 : C == 16 ? 1 : 2;
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const uint32_t addr = __builtin_amdgcn_perm(w[j][s], slot, 0x0C0C0000u | ((4u + b) << 8)) >> kShift;
      lk.l[j][b] = *reinterpret_cast<const float2*>(tab + addr);
    }
}

// Each level times the block scale, each pair rounded once to bf16.
__device__ __forceinline__ bf16x8 expand_frag(const float2 (&l)[4], float sa) {
  const u32x4 v = {bf16_pair(l[0].x * sa, l[0].y * sa), bf16_pair(l[1].x * sa, l[1].y * sa),
                   bf16_pair(l[2].x * sa, l[2].y * sa), bf16_pair(l[3].x * sa, l[3].y * sa)};
  return __builtin_bit_cast(bf16x8, v);
}

// Spreads the work issued next to the MFMAs of one 16-wide k step between
// them: per MFMA V VALU operations and L LDS accesses.
template <int N, int V, int L>
__device__ __forceinline__ void mfma_interleave() {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // MFMA
    __builtin_amdgcn_sched_group_barrier(0x002, V, 0);  // VALU
    __builtin_amdgcn_sched_group_barrier(0x080, L, 0);  // LDS read or write
  }
}

// The scale form is a template parameter (plain, int8, float8): a runtime
// choice would put a global-memory table load behind a branch, and the wait
// the compiler places after it would also wait for the next step's loads.
template <bool kDQ, bool kF8>
__device__ __forceinline__ void block_scales(const WRegs& wr, float mean, float (&sa)[2]) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    if constexpr (kDQ) sa[j] = (code_ratio(wr.q[j], kF8 ? 1 : 0) * wr.s2[j]) + mean;  // a_hat, three roundings
    else sa[j] = wr.am[j];
  }
}

// acc += x . deq(W)^T over nk steps.  dma(ks, stage) requests the x tile of
// step ks into a stage (direct global-to-LDS loads, 1 KB per wave instruction).
// Every LDS stage is read before a barrier that all waves pass before this returns.
template <int MI, bool kDQ, bool kF8, class Dma>
__device__ __forceinline__ void fwd_steps(const Scales& sc, int64_t nk, const Dma& dma, const WPtrs& wp, char* xs0,
                                          char* xs1, const char* tabc, uint32_t slot, float mean, int lane,
                                          floatx16 (&acc)[MI][2]) {
  // Per MFMA: the expansion and lookups of the next 16-wide k step are the
  // same for all tile heights, spread over 2 MI MFMAs.
  constexpr int kV = 24 / MI, kL = 8 / MI;
  // K step k: MFMAs from x stage k % 2 and the codes of step k (wc), in
  // four 16-wide k steps s.  Software pipeline: while the MFMAs of s run,
  // the wave expands the B fragments of s + 1 (looked up one k step
  // earlier) and issues the LDS reads of s + 2; during s = 3 it expands
  // the next step's s = 0, so that after the barrier the MFMAs can start at
  // once.  The global loads of step k + 1 (clamped on the last step: x to
  // the other stage, codes to registers) go out at the top of step k.
  WRegs wc, wnx;
  dma(0, xs0);
  load_w<kDQ>(wc, wp, sc, 0);
  float sa[2];
  bf16x8 bf[2][2];
  Lookups lk[3];
  bf16x8 af[3][MI];
  const uint32_t sw = ((lane & 31) >> 1) & 7, h4 = (lane >> 5) * 4;
  block_scales<kDQ, kF8>(wc, mean, sa);
  lookup_step<kCopies>(lk[0], wc.w, 0, tabc, slot);
  bf[0][0] = expand_frag(lk[0].l[0], sa[0]);
  bf[0][1] = expand_frag(lk[0].l[1], sa[1]);
  wait_vmem();
  __syncthreads();
  for (int64_t ks = 0; ks < nk; ++ks) {
    const int64_t kn = ks + 1 < nk ? ks + 1 : ks;
    dma(kn, (ks & 1) ? xs0 : xs1);  // the other stage was last read before the previous barrier
    load_w<kDQ>(wnx, wp, sc, kn);
    __builtin_amdgcn_sched_barrier(0);
    const char* xa = ((ks & 1) ? xs1 : xs0) + (lane & 31) * kActRowBytes;
    read_act(xa, 0, sw, h4, af[0]);
    read_act(xa, 1, sw, h4, af[1]);
    lookup_step<kCopies>(lk[1], wc.w, 1, tabc, slot);
    __builtin_amdgcn_sched_barrier(0);
    // s = 0
    mfma16(af[0], bf[0], acc);
    bf[1][0] = expand_frag(lk[1].l[0], sa[0]);
    bf[1][1] = expand_frag(lk[1].l[1], sa[1]);
    read_act(xa, 2, sw, h4, af[2]);
    lookup_step<kCopies>(lk[2], wc.w, 2, tabc, slot);
    mfma_interleave<2 * MI, kV, kL>();
    __builtin_amdgcn_sched_barrier(0);
    // s = 1
    mfma16(af[1], bf[1], acc);
    bf[0][0] = expand_frag(lk[2].l[0], sa[0]);
    bf[0][1] = expand_frag(lk[2].l[1], sa[1]);
    read_act(xa, 3, sw, h4, af[0]);
    lookup_step<kCopies>(lk[0], wc.w, 3, tabc, slot);
    mfma_interleave<2 * MI, kV, kL>();
    __builtin_amdgcn_sched_barrier(0);
    // s = 2
    mfma16(af[2], bf[0], acc);
    bf[1][0] = expand_frag(lk[0].l[0], sa[0]);
    bf[1][1] = expand_frag(lk[0].l[1], sa[1]);
    mfma_interleave<2 * MI, kV, kL>();
    __builtin_amdgcn_sched_barrier(0);
    // s = 3, with the next step's s = 0 expansion
    mfma16(af[0], bf[1], acc);
    block_scales<kDQ, kF8>(wnx, mean, sa);
    lookup_step<kCopies>(lk[1], wnx.w, 0, tabc, slot);
    bf[0][0] = expand_frag(lk[1].l[0], sa[0]);
    bf[0][1] = expand_frag(lk[1].l[1], sa[1]);
    mfma_interleave<2 * MI, kV, kL>();
    __builtin_amdgcn_sched_barrier(0);
    wait_vmem();
    __syncthreads();
    wc = wnx;
  }
}

}  // namespace gt
}  // namespace nf4i
