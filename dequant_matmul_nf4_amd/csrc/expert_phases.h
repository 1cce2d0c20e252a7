// The matrix-core loop of the products grouped by expert (k_expert_gemm.hip and its
// input gradient, k_expert_gemm_dx.hip): four phases of 16 reduction indices per
// step, and direct global-to-LDS loads whose waits are counted by hand.
#pragma once

#include "gemm_fwd.h"
#include "skinny_tile.h"

namespace nf4i {
namespace gt {

// Direct global-to-LDS loads of a wave: lane l's 16 (4, 1) bytes at base + off
// to lds + 16 l (4 l, 4 l).  Inline assembly, since the compiler lets reads of LDS
// wait for all loads to LDS that it knows of.
__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const char*)(const char*)p));
}
__device__ __forceinline__ void request16(const void* base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base), "s"(lds) : "memory", "m0");
}
__device__ __forceinline__ void request16(const void* p, uint32_t lds) {  // an address per lane
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(p), "s"(lds) : "memory", "m0");
}
__device__ __forceinline__ void request4(const void* base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dword %0, %1" ::"v"(off), "s"(base), "s"(lds) : "memory", "m0");
}
__device__ __forceinline__ void request1(const void* base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_ubyte %0, %1" ::"v"(off), "s"(base), "s"(lds) : "memory", "m0");
}
// Until at most N of the wave's loads are on their way.
template <int N>
__device__ __forceinline__ void wait_requests() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// The operands of the products in flight: bf[s % 2], af[s % 2] are those of the
// 16 reduction indices s, lk[s % 2] the levels that bf[s % 2] is expanded from.
template <int MI>
struct Operands {
  bf16x8 bf[2][2], af[2][MI];
  Lookups lk[2];
};

// The products of s, and spelled out between them what the wave does meanwhile:
// expands the weights of s + 1 (looked up one s earlier; expand(j, t, levels)
// makes pair t of fragment j), reads activations of s + 1 (piece `at` of xa's rows)
// and looks up s + 2 (word `word` of the codes w).  more(q): what else goes
// behind product q.  Left to the compiler all of this collects behind the
// products, and a wave that is alone on its SIMD leaves the matrix core idle.
template <int MI, int C, class Expand, class More>
__device__ __forceinline__ void mfma_phase(int s, Operands<MI>& o, floatx16 (&acc)[MI][2], const u32x4 (&w)[2], int word,
                                           const char* xa, int at, uint32_t sw, uint32_t h4, const char* tab,
                                           uint32_t slot, const Expand& expand, const More& more) {
  constexpr int kShift = C == 32 ? 0 : C == 16 ? 1 : 2;
  const int cur = s & 1, nxt = cur ^ 1;
  const char* p = xa + (((h4 + at) ^ sw) << 4);
  u32x4 v[2];
#pragma unroll
  for (int q = 0; q < 2 * MI; ++q) {
    // a transposed output tile, as in mfma16
    acc[q >> 1][q & 1] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(o.bf[cur][q & 1], o.af[cur][q >> 1], acc[q >> 1][q & 1], 0, 0, 0);
    __builtin_amdgcn_sched_barrier(0);
    more(q);
#pragma unroll
    for (int e = 8 * q / (2 * MI); e < 8 * (q + 1) / (2 * MI); ++e) {
      v[e >> 2][e & 3] = opaque(expand(e >> 2, e & 3, o.lk[nxt].l[e >> 2][e & 3]));  // here, not where it is used
    }
#pragma unroll
    for (int e = (8 * q + 2 * MI - 1) / (2 * MI); e < (8 * (q + 1) + 2 * MI - 1) / (2 * MI); ++e) {
      const uint32_t addr = __builtin_amdgcn_perm(w[e >> 2][word], slot, 0x0C0C0000u | ((4u + (e & 3)) << 8)) >> kShift;
      o.lk[cur].l[e >> 2][e & 3] = *reinterpret_cast<const float2*>(tab + addr);
    }
#pragma unroll
    for (int i = (q + 1) / 2; i < (q + 2) / 2; ++i) o.af[nxt][i] = lds_frag(p + i * 32 * kActRowBytes);
    __builtin_amdgcn_sched_barrier(0);
  }
  o.bf[nxt][0] = __builtin_bit_cast(bf16x8, v[0]);
  o.bf[nxt][1] = __builtin_bit_cast(bf16x8, v[1]);
}

// What the first phase finds: the operands of s = 0, the lookups of s = 1.
template <int MI, int C, class Expand>
__device__ __forceinline__ void first_operands(Operands<MI>& o, const u32x4 (&w)[2], const char* xa, uint32_t sw,
                                               uint32_t h4, const char* tab, uint32_t slot, const Expand& expand) {
  read_act(xa, 0, sw, h4, o.af[0]);
  lookup_step<C>(o.lk[0], w, 0, tab, slot);
  lookup_step<C>(o.lk[1], w, 1, tab, slot);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    u32x4 v;
#pragma unroll
    for (int t = 0; t < 4; ++t) v[t] = expand(j, t, o.lk[0].l[j][t]);
    o.bf[0][j] = __builtin_bit_cast(bf16x8, v);
  }
}

}  // namespace gt
}  // namespace nf4i
