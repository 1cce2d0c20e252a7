// How the decode walk over weight rows (k_gemv.hip) is spread over the chip, and
// what it has room for: host code alone, so that it can be checked without a GPU.
#pragma once

#include <cstdint>

namespace nf4i {

constexpr int kRowsMaxWg = 512;   // rows per workgroup for one row of x (LDS for the partial sums)
constexpr int kSegMax = 16;       // column segments per workgroup (cols <= 65536)

// Weight rows of a workgroup that a walk with mc rows of x has room for: its kernel
// holds rows_room(mc) * kSegMax * mc partial sums.
constexpr int rows_room(int mc) { return kRowsMaxWg / mc; }

struct RowsPlan {
  int grid;          // number of workgroups
  int nseg;          // column segments
  int seg_blocks;    // blocks per segment (<= 64)
  int wpr;           // waves per segment (row parts)
};

// Rows split evenly over at least one workgroup per CU (at most rows_room(mc)
// rows each), columns into the fewest segments of at most 64 blocks, balanced,
// and the waves spread over the segments.
inline RowsPlan rows_plan(int64_t rows, int64_t cols, int waves, int mc, int64_t cus) {
  const int64_t nblk = cols / 64;
  RowsPlan pl{};
  pl.nseg = static_cast<int>((nblk + 63) / 64);
  pl.seg_blocks = static_cast<int>((nblk + pl.nseg - 1) / pl.nseg);
  pl.wpr = waves / pl.nseg;
  // grid: one workgroup per CU, more if a workgroup would own more rows than it has
  // room for (wpr parts of ceil(rows / (grid * wpr)) rows each)
  int64_t g = cus;
  while (pl.wpr > 0 && pl.wpr * ((rows + g * pl.wpr - 1) / (g * pl.wpr)) > rows_room(mc)) ++g;
  pl.grid = static_cast<int>(g);
  return pl;
}

// Whether the kernel for mc rows of x can take the plan: its segments, every
// workgroup's rows, and the 32-bit offsets within a row.
inline bool rows_plan_fits(const RowsPlan& pl, int64_t rows, int64_t cols, int mc) {
  if (pl.nseg > kSegMax || pl.wpr < 1 || pl.grid < 1 || (cols / 64) * 32 >= (int64_t{1} << 32)) return false;
  const int64_t parts = static_cast<int64_t>(pl.grid) * pl.wpr;
  return pl.wpr * ((rows + parts - 1) / parts) <= rows_room(mc);
}

}  // namespace nf4i
