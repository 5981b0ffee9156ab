// Where kv_attend_prompt's warps meet and which tile a block has, for the tests, as host code.
#include "../mtp_speculative_decoding_step_gb300/csrc/prompt_tiles.h"

extern "C" {

int meets(void) { return mtp::kMeets; }
int meet_barrier(int time, int slot, int quarter) { return mtp::meet_barrier(time, slot, quarter); }
int meet_parity(int time, int unit) { return (int)mtp::meet_parity(time, unit); }

int tile_from(const int* start, int tokens, int rows, int tile, int r, long long left, int* out) {
  return mtp::prompt_tile_from(start, tokens, rows, tile, r, left, out[0], out[1], out[2]);
}

}  // extern "C"
