// Log probabilities of given tokens, ranks, entropy and alternatives
// (spec_logprobs).
//
// One block per row: the maximum, then the sums
//   S = sum e^(x-m),  T = sum (x-m) e^(x-m),  rank = #{j before t},
// then the alternatives one by one.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace mtp {

namespace {

constexpr int kLpThreads = 512;
constexpr int kLpMaxTop = 64;

struct LpArgs {
  const void* x;
  long long stride;
  const int32_t* tok;
  float *lp, *ent, *top_lp;
  int32_t *rank, *top_id, *status;
  int n, V, top;
};

template <int DT>
__global__ void __launch_bounds__(kLpThreads) k_logprobs(const __grid_constant__ LpArgs a) {
  __shared__ float s_v[32];
  __shared__ int s_i[32];
  __shared__ float red[32];
  pdl_wait();
  pdl_trigger();
  const int r = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long base = r * a.stride;
  // argmax of the elements after (v, id) in the order
  auto next = [&](float lv, int li, float& bv, int& bi) {
    bv = -INFINITY;
    bi = -1;
    for (int j = threadIdx.x; j < a.V; j += kLpThreads) {
      const float x = load_elem(a.x, DT, base + j);
      if (li >= 0 && !better(lv, li, x, j)) continue;
      if (bi < 0 ? x > -INFINITY : better(x, j, bv, bi)) { bv = x; bi = j; }
    }
    if (bi < 0) bi = 0x7FFFFFFF;
    warp_argmax(bv, bi);
    __syncthreads();
    if (lane == 0) { s_v[warp] = bv; s_i[warp] = bi; }
    __syncthreads();
    bv = lane < kLpThreads / 32 ? s_v[lane] : -INFINITY;
    bi = lane < kLpThreads / 32 ? s_i[lane] : 0x7FFFFFFF;
    warp_argmax(bv, bi);
    if (bi == 0x7FFFFFFF) bi = -1;
  };
  float m;
  int mi;
  next(0.f, -1, m, mi);
  const int t = a.tok[r];
  const bool given = t >= 0 && t < a.V;
  if (!given && t != -1 && threadIdx.x == 0) flag_status(a.status, MTP_ERR_BAD_ARG);
  const float xt = given ? load_elem(a.x, DT, base + t) : 0.f;
  float S = 0.f, T = 0.f, cnt = 0.f;
  bool bad = false;
  for (int j = threadIdx.x; j < a.V; j += kLpThreads) {
    const float x = load_elem(a.x, DT, base + j);
    bad |= !(x < INFINITY);
    const float e = mi < 0 ? 0.f : expf(x - m);
    S += e;
    if (e > 0.f) T += (x - m) * e;
    cnt += better(x, j, xt, t) ? 1.f : 0.f;
  }
  S = block_sum(S, red);
  T = block_sum(T, red);
  cnt = block_sum(cnt, red);
  if (bad) flag_status(a.status, MTP_ERR_NONFINITE);
  const float ls = logf(S);
  if (threadIdx.x == 0) {
    a.lp[r] = given ? (mi < 0 ? -INFINITY : xt - m - ls) : 0.f;
    if (a.rank) a.rank[r] = given ? (int)cnt : -1;
    if (a.ent) a.ent[r] = mi < 0 ? 0.f : ls - T / S;
  }
  float v = m;
  int id = mi;
  for (int k = 0; k < a.top; ++k) {
    if (threadIdx.x == 0) {
      a.top_id[(long long)r * a.top + k] = id;
      a.top_lp[(long long)r * a.top + k] = id < 0 ? -INFINITY : v - m - ls;
    }
    if (id >= 0 && k + 1 < a.top) {
      float nv;
      int ni;
      next(v, id, nv, ni);
      v = nv;
      id = ni;
    }
  }
}

}  // namespace
}  // namespace mtp

using namespace mtp;

extern "C" {

size_t spec_logprobs_workspace_bytes(int32_t n, int32_t vocab, int32_t top) {
  if (n < 1 || vocab < 1 || top < 0 || top > kLpMaxTop) return 0;
  return 256;
}

mtp_status spec_logprobs(mtp_stream stream, int32_t n, int32_t vocab, const void* d_logits, int64_t row_stride,
                         int32_t dtype, const int32_t* d_tok, int32_t top, float* d_logprob, int32_t* d_rank,
                         float* d_entropy, int32_t* d_top_id, float* d_top_lp, int32_t* d_status, void* d_workspace) {
  if (n < 0 || vocab < 1 || vocab > (1 << 20) || top < 0 || top > kLpMaxTop ||
      (dtype != MTP_DTYPE_BF16 && dtype != MTP_DTYPE_F32))
    return MTP_ERR_BAD_ARG;
  if (n == 0) return MTP_OK;
  const int es = dtype == MTP_DTYPE_BF16 ? 2 : 4;
  if (!d_logits || !d_tok || !d_logprob || !d_workspace || (top > 0 && (!d_top_id || !d_top_lp)) ||
      (n > 1 && row_stride < vocab) || (reinterpret_cast<uintptr_t>(d_logits) & (es - 1)) != 0 ||
      (reinterpret_cast<uintptr_t>(d_workspace) & 15) != 0)
    return MTP_ERR_BAD_ARG;
  LpArgs a{d_logits, row_stride, d_tok, d_logprob, d_entropy, d_top_lp, d_rank, d_top_id, d_status, n, vocab, top};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = launch_pdl(dtype == MTP_DTYPE_BF16 ? k_logprobs<MTP_DTYPE_BF16> : k_logprobs<MTP_DTYPE_F32>,
                                   dim3(n), dim3(kLpThreads), 0, s, a);
  count_launch();
  return e == cudaSuccess ? MTP_OK : MTP_ERR_CUDA;
}

}  // extern "C"
