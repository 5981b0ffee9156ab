// Arguments of kv_attend_prompt's kernels, and which row and query tile a block has.
#pragma once
#include "common.cuh"
#include "prompt_tiles.h"

namespace mtp {

struct PromptArgs {
  const void *q, *k, *v;
  long long ts[3], hs[3];  // strides of Q, K, V in elements
  const int32_t* start;
  void* out;
  float* lse;
  int32_t* status;
  int rows, n_q, n_kv, tokens, window;
  float scale;
  int group;  // bf16: heads to a query tile
  int out_whole;  // bf16: every 32 bytes of an output row are one sector
};

// The row and the query tile (of `tile` positions) of tile number x, counted from the last row's last tile (a row's
// later tiles are its longest); false past the first. By a whole warp, rows in consecutive groups per lane.
__device__ __forceinline__ bool find_tile(const PromptArgs& a, int tile, int x, int& a0, int& n, int& j) {
  const int lane = threadIdx.x & 31, per = (a.rows + 31) / 32, r0 = min(lane * per, a.rows), r1 = min(r0 + per, a.rows);
  long long sum = 0;
  int b0, m;
#pragma unroll 4
  for (int r = r0; r < r1; ++r) {
    prompt_row(a.start, a.tokens, r, b0, m);
    sum += prompt_tiles(m, tile);
  }
  long long inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xFFFFFFFFu, inc, o);
    if (lane >= o) inc += u;
  }
  const long long all = __shfl_sync(0xFFFFFFFFu, inc, 31), y = all - 1 - x;
  if (y < 0) return false;
  const int owner = __ffs(__ballot_sync(0xFFFFFFFFu, inc - sum <= y && y < inc)) - 1;
  const long long at = __shfl_sync(0xFFFFFFFFu, inc - sum, owner);
  return prompt_tile_from(a.start, a.tokens, a.rows, tile, __shfl_sync(0xFFFFFFFFu, r0, owner), y - at, a0, n, j);
}

cudaError_t launch_prompt_tc(PromptArgs a, int head_dim, cudaStream_t s);

}  // namespace mtp
