// The task walk of kv_q4_attend_tree and the bound on kv_attend_prompt's blocks for the tests, as host code.
#include "../mtp_speculative_decoding_step_gb300/csrc/prompt_tiles.h"
#include "../mtp_speculative_decoding_step_gb300/csrc/q4_walk.h"

namespace {
struct Args {
  const int *start, *len;
  int tokens, max_pages, page, window;
};
}  // namespace

extern "C" {

void tree_row(const int* start, const int* len, int tokens, int max_pages, int page, int r, int* out) {
  const Args a{start, len, tokens, max_pages, page, 0};
  mtp::Walk<Args, true>{&a, 1, 16}.row(r, out[0], out[1], out[2]);
}

void tree_span(int n, int L, int G, int RT, int window, int j, int* out) {
  const Args a{nullptr, nullptr, n, 1, 1, window};
  mtp::Walk<Args, true>{&a, G, RT}.span(n, L, j, out[0], out[1], out[2], out[3]);
}

int tree_edge(int n, int L, int first, int t, int window, int* index) {
  mtp::Run s{};
  s.p0 = L - n - 1;
  s.p1 = L - 1;
  s.first = first;
  *index = s.edge_index(t);
  return s.edge(t, window);
}

long long most_tiles(int tokens, int rows, int G, int tile) { return mtp::prompt_most_tiles(tokens, rows, G, tile); }

void prompt_row(const int* start, int tokens, int r, int* out) { mtp::prompt_row(start, tokens, r, out[0], out[1]); }

}  // extern "C"
