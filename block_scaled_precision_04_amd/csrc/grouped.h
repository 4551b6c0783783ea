// Parts that the W4A4 and the W8A8 GEMMs share: the row tiles of a grouped
// problem, and the places of 64-byte activation rows in LDS.
#pragma once
#include <algorithm>
#include <type_traits>

#include "common.h"

namespace {

// Inclusive sum over the wave's lanes: within rows of 16 by row shifts, then row
// totals broadcast to the rows after (DPP moves, no LDS round trips).
BS_INLINE int wave_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, true);   // row_shr:1
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, true);   // row_shr:2
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, true);   // row_shr:4
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, true);   // row_shr:8
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);  // row 0 -> 1, 2 -> 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);  // rows 0-1 -> 2-3
  return v;
}

// The `tile`-th row tile of the grouped problem: the slots of expert e are cut
// into runs of up to BM.  Lane l looks at experts 4l .. 4l+3 of each 256; a
// wave-wide scan of their tile counts finds the tile.  Offsets are clamped to
// [0, S], so whatever they hold no slot outside the buffers is named.
// Returns false past the last tile.
template <int BM>
BS_INLINE bool find_tile(const int* __restrict__ offsets, int E, int S, int tile, int& expert, int& r0, int& r1) {
  const int l = threadIdx.x & 63;
  int run = 0;
  for (int b = 0; b < E; b += 256) {
    int o[5], cnt[4], mine = 0;
#pragma unroll
    for (int i = 0; i < 5; ++i) o[i] = min(max(offsets[min(b + 4 * l + i, E)], 0), S);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      cnt[i] = o[i + 1] > o[i] ? (o[i + 1] - o[i] + BM - 1) / BM : 0;
      mine += cnt[i];
    }
    const int incl = wave_scan(mine);
    const int total = __builtin_amdgcn_readlane(incl, 63);
    if (tile < run + total) {
      int before = run + incl - mine;
      int fe = -1, f0 = 0, f1 = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (tile >= before && tile < before + cnt[i]) {
          fe = b + 4 * l + i;
          f0 = o[i] + (tile - before) * BM;
          f1 = min(f0 + BM, o[i + 1]);
        }
        before += cnt[i];
      }
      const int src = __builtin_ctzll(__ballot(fe >= 0));
      expert = __builtin_amdgcn_readlane(fe, src);
      r0 = __builtin_amdgcn_readlane(f0, src);
      r1 = __builtin_amdgcn_readlane(f1, src);
      return true;
    }
    run += total;
  }
  return false;
}

// ceil(count / BM) summed over experts is largest when as many experts as
// possible hold one row: with A = min(S, E) of them, A + (S - A) / BM.
inline int tile_bound(int S, int E, int BM) {
  const int A = std::min(S, E);
  return A + (S - A) / BM;
}

// 16-byte chunk swizzle of a 64-byte activation row in LDS: the 16 rows of a
// fragment read take one chunk each, four rows per 256-byte line.
BS_INLINE int swz4(int row, int chunk) { return chunk ^ ((row >> 2) & 3); }

// Workgroup -> grouped tile (row tile id / n_tiles, columns id % n_tiles).
// Workgroups go round the XCDs one by one, so with n_tiles a multiple of 8 the
// row tiles of an expert already meet on one XCD for each tile of columns and
// share its weight in that L2; else runs of four row tiles with all their
// columns stay together (64 experts K = 2048: N = 1280 49 us instead of 61, N =
// 2304 76 instead of 96).  Where every column falls on two XCDs and a run's
// weight is more than an L2 holds, it stays as it is (N = 7168 98 us, runs 105).
BS_INLINE uint32_t xcd_runs(uint32_t id, uint32_t grid, uint32_t n_tiles) {
  const uint32_t run = 4 * n_tiles;
  if (n_tiles % (n_tiles > 16 ? 4 : 8) == 0 || id >= grid / (8 * run) * (8 * run)) return id;
  const uint32_t xcd = id & 7, i = id >> 3;
  return (i / run * 8 + xcd) * run + i % run;
}

template <int V>
using Int = std::integral_constant<int, V>;

}  // namespace
