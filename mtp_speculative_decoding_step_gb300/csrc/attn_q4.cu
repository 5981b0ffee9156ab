// Attention over the paged 4-bit cache (kv_q4_attend).
//
// One warp per (query position, query head): the lanes share the head
// dimension, keys go by one at a time with a running maximum and sum in fp32.
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "kernels.h"
#include "q4.cuh"

namespace mtp {

namespace {

struct Q4AttnArgs {
  const uint8_t *kc, *vc;
  const int32_t *k_exp, *v_exp, *table, *start, *len;
  const void* q;
  long long ts, hs;
  void* out;
  float* lse;
  int32_t* status;
  int rows, n_q, n_kv, page, n_pages, max_pages, tokens, window;
  float scale;
};

template <int DH, int DT>
__global__ void __launch_bounds__(128) k_q4_attn(const __grid_constant__ Q4AttnArgs a) {
  constexpr int E = DH / 32, kRow = q4_row_bytes(DH);
  const int lane = threadIdx.x & 31;
  pdl_wait();
  pdl_trigger();
  const long long w = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int h = (int)(w % a.n_q), t = (int)(w / a.n_q);
  if (t >= a.tokens) return;
  int lo = 0, hi = a.rows;  // last row whose start is <= t
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.start[mid] <= t) lo = mid;
    else hi = mid;
  }
  const int r = lo;
  const int n = min(a.start[r + 1], a.tokens) - a.start[r], i = t - a.start[r];
  if (i < 0 || i >= n) return;
  const int L = (int)min((long long)max(a.len[r], 0), (long long)a.max_pages * a.page);
  if (L != a.len[r]) flag_status(a.status, MTP_ERR_BAD_ARG);
  const int pos = L - n + i;
  const int first = a.window > 0 ? max(0, pos - a.window + 1) : 0;
  const int g = h / (a.n_q / a.n_kv);
  float q[E], o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = load_elem(a.q, DT, t * a.ts + h * a.hs + lane * E + e) * a.scale * pow2i(head_exp(a.k_exp, g));
    o[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int j = first; j <= pos; ++j) {
    const int id = a.table[(long long)r * a.max_pages + j / a.page];
    if (id < 0 || id >= a.n_pages) {
      flag_status(a.status, MTP_ERR_BAD_ARG);
      continue;
    }
    const long long at = (((long long)id * a.n_kv + g) * a.page + j % a.page) * kRow;
    auto elem = [&](const uint8_t* c, float (&v)[E]) {
      const float s = f16x2_to_f(e4m3x2_to_f16x2(c[at + DH / 2 + lane * E / 16])).x;
#pragma unroll
      for (int e = 0; e < E / 2; ++e) {
        uint32_t x[4];
        e2m1x8_to_f16(c[at + lane * E / 2 + e], x);
        const float2 f = f16x2_to_f(x[0]);
        v[2 * e] = f.x * s;
        v[2 * e + 1] = f.y * s;
      }
    };
    float k[E], v[E], s = 0.f;
    elem(a.kc, k);
#pragma unroll
    for (int e = 0; e < E; ++e) s = fmaf(q[e], k[e], s);
    s = warp_sum(s);
    elem(a.vc, v);
    const float mn = s > m ? s : m;
    const float f = m == -INFINITY ? 0.f : expf(m - mn), p = expf(s - mn);
    l = l * f + p;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = fmaf(p, v[e], o[e] * f);
    m = mn;
  }
  const float up = pow2i(head_exp(a.v_exp, g));
#pragma unroll
  for (int e = 0; e < E; ++e)
    store_elem(a.out, DT, ((long long)t * a.n_q + h) * DH + lane * E + e, l != 0.f ? o[e] / l * up : 0.f);
  if (lane == 0 && a.lse) a.lse[(long long)t * a.n_q + h] = l != 0.f ? m + logf(l) : -INFINITY;
}

}  // namespace
}  // namespace mtp

using namespace mtp;

extern "C" {

size_t kv_q4_attend_workspace_bytes(const kv_q4_cache* c, int32_t n_q, int32_t max_q, int32_t dtype) {
  if (!c || kv_q4_row_bytes(c->head_dim) == 0 || c->n_kv < 1 || n_q < c->n_kv || max_q < 1 ||
      (dtype != MTP_DTYPE_BF16 && dtype != MTP_DTYPE_F32))
    return 0;
  return 256;
}

mtp_status kv_q4_attend(mtp_stream stream, const kv_q4_cache* c, int32_t rows, int32_t n_q, int32_t tokens,
                        const void* d_q, int64_t tok_stride, int64_t head_stride, int32_t dtype,
                        const int32_t* d_table, int32_t max_pages, const int32_t* d_start, const int32_t* d_len,
                        int32_t max_q, float scale, int32_t window, void* d_out, float* d_lse, int32_t* d_status,
                        void* d_workspace) {
  if (!q4_cache_ok(c) || rows < 1 || rows > 4096 || n_q < 1 || n_q > 1024 || n_q % c->n_kv != 0 || tokens < 0 ||
      max_pages < 1 || (long long)max_pages * c->page >= (1LL << 31) || max_q < 1 || window < 0 ||
      !std::isfinite(scale) || (dtype != MTP_DTYPE_BF16 && dtype != MTP_DTYPE_F32))
    return MTP_ERR_BAD_ARG;
  if (tokens == 0) return MTP_OK;
  const int es = dtype == MTP_DTYPE_BF16 ? 2 : 4;
  if (!d_q || !d_table || !d_start || !d_len || !d_out || !d_workspace ||
      (reinterpret_cast<uintptr_t>(d_q) & (es - 1)) != 0 || (reinterpret_cast<uintptr_t>(d_out) & 15) != 0 ||
      (reinterpret_cast<uintptr_t>(d_workspace) & 15) != 0)
    return MTP_ERR_BAD_ARG;
  Q4AttnArgs a{static_cast<const uint8_t*>(c->k), static_cast<const uint8_t*>(c->v), c->k_exp, c->v_exp, d_table,
               d_start, d_len, d_q, tok_stride, head_stride, d_out, d_lse, d_status, rows, n_q, c->n_kv, c->page,
               c->n_pages, max_pages, tokens, window, scale};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  void (*k)(Q4AttnArgs) = nullptr;
  const bool b = dtype == MTP_DTYPE_BF16;
  if (c->head_dim == 64) k = b ? k_q4_attn<64, MTP_DTYPE_BF16> : k_q4_attn<64, MTP_DTYPE_F32>;
  if (c->head_dim == 128) k = b ? k_q4_attn<128, MTP_DTYPE_BF16> : k_q4_attn<128, MTP_DTYPE_F32>;
  if (c->head_dim == 256) k = b ? k_q4_attn<256, MTP_DTYPE_BF16> : k_q4_attn<256, MTP_DTYPE_F32>;
  const long long warps = (long long)tokens * n_q;
  const cudaError_t e = launch_pdl(k, dim3((unsigned)((warps + 3) / 4)), dim3(128), 0, s, a);
  count_launch();
  return e == cudaSuccess ? MTP_OK : MTP_ERR_CUDA;
}

}  // extern "C"
