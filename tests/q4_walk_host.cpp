// The task walk of kv_q4_attend for the tests, as host code.
#include "../mtp_speculative_decoding_step_gb300/csrc/q4_walk.h"

namespace {
struct Args {
  const int *start, *len;
  int tokens, max_pages, page, window;
};
}  // namespace

extern "C" {

long long walk_per_head(int n, int L, int G, int RT, int window) {
  const Args a{nullptr, nullptr, n, 1, 1, window};
  return mtp::Walk<Args>{&a, G, RT}.per_head(n, L);
}

void walk_find(long long x, long long ph, int* g, long long* o) {
  const Args a{};
  decltype(mtp::Walk<Args>{}.per_head(0, 0)) in{};
  mtp::Walk<Args>{&a, 1, 16}.find(x, ph, *g, in);
  *o = in;
}

}  // extern "C"

extern "C" {

void walk_span(int n, int L, int G, int RT, int window, int j, int* out) {
  const Args a{nullptr, nullptr, n, 1, 1, window};
  mtp::Walk<Args>{&a, G, RT}.span(n, L, j, out[0], out[1], out[2], out[3]);
}

int walk_edge(int p0, int p1, int t, int window) {
  mtp::Run s{};
  s.p0 = p0;
  s.p1 = p1;
  return s.edge(t, window);
}

}  // extern "C"
