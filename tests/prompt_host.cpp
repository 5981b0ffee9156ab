// Where kv_attend_prompt's warps meet, for the tests, as host code.
#include "../mtp_speculative_decoding_step_gb300/csrc/prompt_tiles.h"

extern "C" {

int meets(void) { return mtp::kMeets; }
int meet_barrier(int time, int slot, int quarter) { return mtp::meet_barrier(time, slot, quarter); }
int meet_parity(int time, int unit) { return (int)mtp::meet_parity(time, unit); }

}  // extern "C"
