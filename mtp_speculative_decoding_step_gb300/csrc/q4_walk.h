// The work of kv_q4_attend as a row of tasks, (row, KV head, query tile,
// 128-position tile) each, of which every block owns an equal stretch. Plain
// C++ too, so that its arithmetic can be checked at lengths that no run reaches.
#pragma once
#ifdef __CUDACC__
#define Q4_WALK __device__
#else
#include <algorithm>
#define Q4_WALK
#endif

namespace mtp {

#ifndef __CUDACC__
using std::max;
using std::min;
#endif

constexpr int kT = 128;  // positions per tile

// A block's share of one (row, KV head, query tile). Query row f of the row's
// position-major order is (position f / G, head f % G of the KV head's G); tile
// j holds f in [j RT, (j + 1) RT).
struct Run {
  int r, g, j;         // row, KV head, query tile
  int a0, n, pos;      // first packed position, positions, the first one's place in the cache
  int lo, end;         // cached positions that some query row sees: [lo, end)
  int first, tile, nt; // the query tile's first 128-position tile; this share's tiles
  int p0, p1;          // places of the first and the last query row
  int flags;           // 1: begins here, 2: ends here, 4: the block's last share
  int last;            // the block that ends it

  // whether some (row, position) pair of a tile may be out of sight
  Q4_WALK bool edge(int t, int window) const {
    return t * kT + kT - 1 > p0 || (window > 0 && t * kT <= max(p1, -1) - window);
  }
  // its number among the edge tiles: p0 and p1 lie less than kT apart, so two
  // tiles at most hold a causal border, and two a window's
  Q4_WALK int edge_index(int t) const {
    return t * kT + kT - 1 > p0 ? min(max(t - p0 / kT, 0), 1) : 2 + min(t - first, 1);
  }
};

// Args: start, len, tokens, max_pages, page, window of the call.
template <class Args>
struct Walk {
  const Args* a;
  int G, RT;       // query heads per KV head, query rows per tile

  Q4_WALK void row(int r, int& a0, int& n, int& L) const {
    a0 = min(max(a->start[r], 0), a->tokens);
    n = min(max(a->start[r + 1], a0), a->tokens) - a0;
    L = min(max(a->len[r], 0), a->max_pages * a->page);
  }
  Q4_WALK int tiles(int n) const { return (n * G + RT - 1) / RT; }
  Q4_WALK void span(int n, int L, int j, int& lo, int& end, int& t0, int& cnt) const {
    const int i0 = j * RT / G, i1 = (min(n * G, (j + 1) * RT) - 1) / G;
    end = max(L - n + i1 + 1, 0);
    // (from 0 at the least before the window goes off: a first place below 0 less a window near 2^31 would wrap)
    lo = a->window > 0 ? max(0, max(0, L - n + i0 + 1) - a->window) : 0;
    t0 = 0;
    cnt = 1;  // one tile at least: rows that see nothing are written too
    if (lo < end) {
      t0 = lo / kT;
      cnt = (end - 1) / kT - t0 + 1;
    } else {
      end = lo;
    }
  }
  Q4_WALK long long per_head(int n, int L) const {
    long long sum = 0;  // (past 2^31 for prompts of millions of positions)
#pragma unroll 1
    for (int j = 0; j < tiles(n); ++j) {
      int lo, end, t0, cnt;
      span(n, L, j, lo, end, t0, cnt);
      sum += cnt;
    }
    return sum;
  }
  // Task x of a row whose KV heads have ph tasks each: its head, and its number there.
  Q4_WALK void find(long long x, long long ph, int& g, long long& o) const {
    if ((x | ph) >> 32 == 0) {
      g = (int)((unsigned)x / (unsigned)ph);
      o = (unsigned)x % (unsigned)ph;
    } else {  // (at most n_kv steps; a 64-bit division costs more code than the few such rows are worth)
      for (g = 0; x >= ph; x -= ph) ++g;
      o = x;
    }
  }
};

}  // namespace mtp
