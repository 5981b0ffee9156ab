// The work of kv_attend_prompt: which row and which of its query tiles a block
// has. Plain C++ too, so that its arithmetic can be checked on the host.
#pragma once
#ifdef __CUDACC__
#define PROMPT_TILES __device__ __forceinline__
#else
#include <algorithm>
#define PROMPT_TILES inline
#endif

namespace mtp {

#ifndef __CUDACC__
using std::max;
using std::min;
#endif

// A row of the packed positions: where it begins, and how many it has.
PROMPT_TILES void prompt_row(const int* start, int tokens, int r, int& a0, int& n) {
  a0 = min(max(start[r], 0), tokens);
  n = min(max(start[r + 1], a0), tokens) - a0;
}

// Query tiles of n query rows, `tile` each.
PROMPT_TILES int prompt_tiles(int n, int tile) { return (n + tile - 1) / tile; }

// The row and the query tile of tile number `left` of the rows from r on; false behind the last row. (64 bits: rows
// whose starts go up and down hold the same positions many times.)
PROMPT_TILES bool prompt_tile_from(const int* start, int tokens, int rows, int tile, int r, long long left, int& a0, int& n, int& j) {
  for (; r < rows; ++r) {
    prompt_row(start, tokens, r, a0, n);
    const int t = prompt_tiles(n, tile);
    if (left < t) {
      j = (int)left;
      return true;
    }
    left -= t;
  }
  return false;
}

// Blocks that hold all rows' query tiles of `tile` query rows, G a position,
// whatever the rows' lengths are: a row's last tile may be short, so rows add one
// each at the most.
inline long long prompt_most_tiles(int tokens, int rows, int G, int tile) {
  return (long long)tokens * G / tile + (tokens < rows ? tokens : rows);
}

// Two warps (one of each group, `slot` 0 and 1) meet twice at the end of a unit: each arrives on a barrier of its own
// (which counts to one) and waits for the other's. A warp goes on as soon as the other has arrived, which may not have
// looked yet: were both times on one barrier, its second arrival could end the phase that the other still waits to see
// ended, and each would wait for the other. With a barrier for each time, a warp is back at the first only behind the
// second, where the other arrives after it has seen the first.
constexpr int kMeets = 16;  // 2 times, 2 groups, 4 warps of a group
PROMPT_TILES int meet_barrier(int time, int slot, int quarter) { return (time * 2 + slot) * 4 + quarter; }
// The parity of the phase that the block's unit number `unit` ends there.
PROMPT_TILES unsigned meet_parity(int /*time*/, int unit) { return unit & 1; }

}  // namespace mtp
