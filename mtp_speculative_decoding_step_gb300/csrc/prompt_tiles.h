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

// Blocks that hold all rows' query tiles of `tile` query rows, G a position,
// whatever the rows' lengths are: a row's last tile may be short, so rows add one
// each at the most.
inline long long prompt_most_tiles(int tokens, int rows, int G, int tile) {
  return (long long)tokens * G / tile + (tokens < rows ? tokens : rows);
}

}  // namespace mtp
