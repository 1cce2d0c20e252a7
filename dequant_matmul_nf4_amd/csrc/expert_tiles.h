// Which expert a tile of the grouped products belongs to.  The rows of expert
// e are offsets[e] .. offsets[e + 1] - 1 (device data), cut into tiles of TM
// rows; tiles are numbered expert by expert.  Offsets are clamped to 0 .. m
// and to ascend, so that no offset makes a kernel leave its buffers.
#pragma once

#include "expert_int4.h"
#include "nf4_device.h"

namespace nf4i {

struct ExpertTile {
  int e;            // expert, -1: no such tile
  int64_t lo, hi;   // its rows
  int64_t row0;     // the tile's first row
};

__device__ __forceinline__ int wave_prefix(int v, int lane) {
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int t = __shfl_up(v, off, 64);
    if (lane >= off) v += t;
  }
  return v;
}

// Rows of expert 64 c + lane (none past the last expert).
__device__ __forceinline__ void expert_range(const ExpertRows& er, int c, int lane, int64_t& lo, int64_t& hi) {
  const int e = 64 * c + lane;
  const int64_t a = er.offsets[e < er.experts ? e : er.experts];
  const int64_t b = er.offsets[e < er.experts ? e + 1 : er.experts];
  lo = a < 0 ? 0 : a < er.m ? a : er.m;
  hi = b < lo ? lo : b < er.m ? b : er.m;
}

// Tiles of kCoverRows rows, the last one more than half full.
__device__ __forceinline__ int cover_tiles(int64_t rows) { return static_cast<int>((rows + kCoverRows / 2 - 1) / kCoverRows); }

// How many of these the first of two kernels takes: full rounds of its
// workgroups, and a last round that fills most of them.
__device__ __forceinline__ int64_t covered_tiles(const ExpertRows& er, int lane) {
  int64_t all = 0;
  for (int c = 0; 64 * c < er.experts; ++c) {
    int64_t lo, hi;
    expert_range(er, c, lane, lo, hi);
    all += __builtin_amdgcn_readlane(wave_prefix(cover_tiles(hi - lo), lane), 63);
  }
  const int64_t units = all * er.cover_units, full = units / er.cover_slots * er.cover_slots;
  return 3 * (units - full) > 2 * er.cover_slots ? all : full / er.cover_units;
}

// Tiles of the experts 64 c .. 64 c + 63, one expert per lane.
struct ExpertLane {
  int64_t lo, hi;
  int tiles;        // this lane's expert
  int upto;         // of lanes 0 .. this
};

// covered: of the cover_tiles, counted expert by expert, the first ones that
// another kernel takes; the expert's rows begin behind them.
__device__ __forceinline__ ExpertLane expert_lane(const ExpertRows& er, int c, int tm, int lane, int64_t covered = 0) {
  ExpertLane r;
  if (covered > 0) {
    int64_t before = 0;
    for (int b = 0; b <= c; ++b) {
      expert_range(er, b, lane, r.lo, r.hi);
      const int own = cover_tiles(r.hi - r.lo), upto = wave_prefix(own, lane);
      if (b == c) {
        const int64_t mine = covered - before - (upto - own);
        r.lo += (mine < 0 ? 0 : mine < own ? mine : own) * kCoverRows;
        r.lo = r.lo < r.hi ? r.lo : r.hi;
      }
      before += __builtin_amdgcn_readlane(upto, 63);
    }
  } else {
    expert_range(er, c, lane, r.lo, r.hi);
  }
  r.tiles = static_cast<int>((r.hi - r.lo + tm - 1) / tm);
  r.upto = wave_prefix(r.tiles, lane);
  return r;
}

// The offsets of the first 64 experts stay in the lanes' registers, so that few
// experts are read once.  Every lane of a wave calls these.  Offsets
// that go up and down can give all rows to every other expert: the tiles of 64
// experts still fit 31 bits (tiles of fewer than 64 rows are for few rows), those
// of all take 64.
struct ExpertScan {
  ExpertLane first;
  int64_t tiles;    // all tiles
  int64_t covered;  // tiles that another kernel takes
};

__device__ __forceinline__ ExpertScan scan_experts(const ExpertRows& er, int tm, int lane, int64_t covered = 0) {
  ExpertScan s;
  s.covered = covered;
  s.first = expert_lane(er, 0, tm, lane, covered);
  s.tiles = __builtin_amdgcn_readlane(s.first.upto, 63);
  for (int c = 1; 64 * c < er.experts; ++c) s.tiles += __builtin_amdgcn_readlane(expert_lane(er, c, tm, lane, covered).upto, 63);
  return s;
}

__device__ __forceinline__ ExpertTile find_expert_tile(const ExpertRows& er, const ExpertScan& s, int tm, int64_t tile, int lane) {
  ExpertTile t{-1, 0, 0, 0};
  ExpertLane r = s.first;
  for (int c = 0;; r = expert_lane(er, c, tm, lane, s.covered)) {
    const int here = __builtin_amdgcn_readlane(r.upto, 63);
    if (tile < here) {
      const int l = __builtin_ctzll(__ballot(r.upto > static_cast<int>(tile)));
      t.e = 64 * c + l;
      t.lo = __builtin_amdgcn_readlane(static_cast<int>(r.lo), l);
      t.hi = __builtin_amdgcn_readlane(static_cast<int>(r.hi), l);
      t.row0 = t.lo + (tile - (__builtin_amdgcn_readlane(r.upto, l) - __builtin_amdgcn_readlane(r.tiles, l))) * tm;
      return t;
    }
    tile -= here;
    if (64 * ++c >= er.experts) return t;
  }
}

// Number `tile` of the cover_tiles (there are more than that).
__device__ __forceinline__ ExpertTile find_cover_tile(const ExpertRows& er, int64_t tile, int lane) {
  ExpertTile t{0, 0, 0, 0};
  for (int c = 0; 64 * c < er.experts; ++c) {
    int64_t lo, hi;
    expert_range(er, c, lane, lo, hi);
    const int own = cover_tiles(hi - lo), upto = wave_prefix(own, lane), here = __builtin_amdgcn_readlane(upto, 63);
    if (tile < here) {
      const int l = __builtin_ctzll(__ballot(upto > static_cast<int>(tile)));
      t.e = 64 * c + l;
      t.lo = __builtin_amdgcn_readlane(static_cast<int>(lo), l);
      t.hi = __builtin_amdgcn_readlane(static_cast<int>(hi), l);
      tile -= __builtin_amdgcn_readlane(upto, l) - __builtin_amdgcn_readlane(own, l);
      t.row0 = t.lo + tile * kCoverRows;
      return t;
    }
    tile -= here;
  }
  return t;
}

// Unit u of n dealt round-robin over the 8 XCDs (as workgroups are): each XCD
// gets one contiguous run of the units, so that the units it works on at one
// time are neighbours.
__device__ __forceinline__ int64_t xcd_run(int64_t u, int64_t n) {
  const int64_t x = u & 7, q = n >> 3, r = n & 7;
  return x * q + (x < r ? x : r) + (u >> 3);
}

}  // namespace nf4i
