// A layer's product with its epilogue for a decode batch (up to 32 rows of x): the
// streaming walk over the codes that the product grouped by expert takes for few
// rows (skinny_walk.h, skinny_tile.h), one weight, with the epilogue where the
// waves' sums have met.  Levels enter in float16, x exactly (scaled by a power of two
// per row and up to 512 columns), scales in float32 on the blocks' sums.
#include "linear_epilogue.h"
#include "linear_f16.h"
#include "skinny_walk.h"

namespace nf4i {
namespace {

struct FewArgs {
  sk::WalkArgs walk;
  const uint16_t* x;   // [m][cols]
  int64_t m;
  lin::FewOut out;
};

struct FewJob {
  const FewArgs& a;
  struct Tile {
    int64_t e, row0;
    int cnt;
  };
  __device__ __forceinline__ int64_t tiles() const { return (a.m + sk::kRows - 1) / sk::kRows; }
  __device__ __forceinline__ Tile tile(int64_t tid) const {
    const int64_t row0 = tid * sk::kRows;
    return Tile{0, row0, static_cast<int>(a.m - row0 < sk::kRows ? a.m - row0 : sk::kRows)};
  }
  __device__ __forceinline__ const uint16_t* x_row(int64_t p) const { return a.x + p * a.walk.cols; }
  __device__ __forceinline__ void store(int64_t p, int64_t row, float v) const { a.out.store(p, row, v); }
};

template <bool kDQ, bool kF8, bool kOnce>
__global__ __launch_bounds__(sk::kThreads, 2) void k_linear_few(FewArgs a) {
  __shared__ sk::WalkLds<4, kF8> lds;
  sk::walk<kDQ, kF8, 4, kOnce>(a.walk, lds, FewJob{a});
}

template <bool kDQ, bool kF8>
void launch(const FewArgs& a, hipStream_t s) {
  const int64_t ngr = (a.walk.rows + 15) / 16, tiles = (a.m + sk::kRows - 1) / sk::kRows;
  const int64_t want = (ngr * tiles + a.walk.pl.rs - 1) / a.walk.pl.rs;
  int64_t grid = want < device_cus() ? want : device_cus();
  while (ngr / grid >= (int64_t{1} << 26)) grid *= 2;
  const dim3 gd(static_cast<unsigned>(grid)), bd(sk::kThreads);
  if (a.walk.pl.per <= sk::kSeg) hipLaunchKernelGGL((k_linear_few<kDQ, kF8, true>), gd, bd, 0, s, a);
  else hipLaunchKernelGGL((k_linear_few<kDQ, kF8, false>), gd, bd, 0, s, a);
}

}  // namespace

hipError_t launch_linear_few(const uint8_t* packed, int64_t rows, int64_t cols, Scales sc, const uint16_t* x, int64_t m,
                             uint16_t* y, const Epilogue& ep, const uint16_t* u, const uint16_t* lora_b, int r, hipStream_t s) {
  const FewArgs a{sk::WalkArgs{packed, rows, cols, sc, codebook(sc.fp4), sk::make_plan(cols)}, x, m,
                  lin::few_out(rows, y, ep, u, lora_b, r)};
  if (sc.absmax) launch<false, false>(a, s);
  else if (sc.f8) launch<true, true>(a, s);
  else launch<true, false>(a, s);
  return hipGetLastError();
}

}  // namespace nf4i
