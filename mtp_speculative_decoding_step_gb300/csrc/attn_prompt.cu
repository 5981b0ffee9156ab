// Causal attention of whole packed prompts over unrounded keys and values
// (kv_attend_prompt): checks, and the fp32 kernel. (bf16: attn_prompt_tc.cu.)
//
//   s_ij = scale q_i . k_j,  out_i = sum_j softmax(s_i)_j v_j,  j <= i (and > i - window)
//
// in one pass over the keys with the running maximum and sum of each query.
#include <algorithm>
#include <cmath>
#include <mutex>

#include "attn_prompt.h"
#include "common.cuh"
#include "kernels.h"
#include "prompt_tiles.h"
#include "ranges.h"

namespace mtp {

namespace {

// ------------------------------------------------------------ CUDA cores

constexpr int kSimtThreads = 256;

// R: queries of a thread.
template <int DH, int R>
struct Simt {
  static constexpr int kRows = 16 * R;  // queries of a block
  static constexpr int kKeys = DH == 256 ? 32 : 64;  // of a tile; two tiles of K and V fit
  static constexpr int kS = DH + 4, kPS = kKeys + 4;  // strides of rows, of P's
  static constexpr int kTile = kKeys * kS;
  static constexpr int kSmem = (kRows * kS + 4 * kTile + kRows * kPS) * 4;
  static_assert(kSmem <= 227 * 1024, "shared memory");
};

// 16 bytes to shared memory asynchronously; zeros where there is nothing to copy.
__device__ __forceinline__ void copy16(float* dst, const float* src, bool some) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(some ? 16 : 0) : "memory");
}

// 16 R queries of a head against 32 or 64 keys at a time, all in fp32; the next tile of K and V is copied meanwhile. Thread
// (ty, tx) of 16 x 16 has the scores of R queries with kKeys / 16 keys, then R queries' outputs in DH / 16 dimensions: 8
// loads of 16 bytes from shared memory per 64 products with 4 queries, which bound it. 1024 positions of 24 heads of 256: 440
// us, 29 TFLOP/s.
template <int DH, int R>
__global__ void __launch_bounds__(kSimtThreads) k_prompt_simt(const __grid_constant__ PromptArgs a) {
  using S = Simt<DH, R>;
  constexpr int kD = DH / 64, kB = S::kKeys / 16;
  extern __shared__ __align__(16) float smem[];
  float *sq = smem, *skv = sq + S::kRows * S::kS, *sp = skv + 4 * S::kTile;
  __shared__ int s_at[4];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4, h = blockIdx.x % a.n_q, g = h / (a.n_q / a.n_kv);
  if (tid < 32) {
    int a0 = 0, n = 0, j = 0;
    const bool some = find_tile(a, S::kRows, blockIdx.x / a.n_q, a0, n, j);
    if (tid == 0) {
      s_at[0] = a0;
      s_at[1] = some ? n : 0;
      s_at[2] = j;
    }
  }
  __syncthreads();
  const int a0 = s_at[0], n = s_at[1], i0 = s_at[2] * S::kRows;
  if (n == 0) return;
  const int rows = min(n - i0, S::kRows);
  auto stage = [&](float* dst, int side, const void* src, int head, int first, int count, int most) {
    for (int e = tid; e < most * (DH / 4); e += kSimtThreads) {
      const int r = e / (DH / 4), d = e % (DH / 4) * 4;
      const long long at = (long long)(a0 + first + min(r, max(count, 1) - 1)) * a.ts[side] + (long long)head * a.hs[side] + d;
      copy16(dst + r * S::kS + d, static_cast<const float*>(src) + at, r < count);
    }
  };
  const int first = a.window > 0 ? max(0, i0 - (a.window - 1)) / S::kKeys * S::kKeys : 0, last = i0 + rows;
  auto keys = [&](int t0, int buf) {
    stage(skv + 2 * buf * S::kTile, 1, a.k, g, t0, min(n - t0, S::kKeys), S::kKeys);
    stage(skv + (2 * buf + 1) * S::kTile, 2, a.v, g, t0, min(n - t0, S::kKeys), S::kKeys);
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  stage(sq, 0, a.q, h, i0, rows, S::kRows);
  keys(first, 0);
  const float c = a.scale * 1.44269504f;
  float m[R], l[R], o[R][kD][4];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    m[r] = -INFINITY;
    l[r] = 0.f;
#pragma unroll
    for (int d = 0; d < kD; ++d)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[r][d][e] = 0.f;
  }
  int buf = 0;
  for (int t0 = first; t0 < last; t0 += S::kKeys, buf ^= 1) {
    if (t0 + S::kKeys < last) {
      keys(t0 + S::kKeys, buf ^ 1);
      asm volatile("cp.async.wait_group 1;" ::: "memory");
    } else {
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
    __syncthreads();
    const float *sk = skv + 2 * buf * S::kTile, *sv = sk + S::kTile;
    float s[R][kB];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int b = 0; b < kB; ++b) s[r][b] = 0.f;
#pragma unroll 4
    for (int d = 0; d < DH; d += 4) {
      float4 qv[R], kv[kB];
#pragma unroll
      for (int r = 0; r < R; ++r) qv[r] = *reinterpret_cast<const float4*>(sq + (R * ty + r) * S::kS + d);
#pragma unroll
      for (int b = 0; b < kB; ++b) kv[b] = *reinterpret_cast<const float4*>(sk + (tx + 16 * b) * S::kS + d);
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int b = 0; b < kB; ++b)
          s[r][b] = fmaf(qv[r].x, kv[b].x, fmaf(qv[r].y, kv[b].y, fmaf(qv[r].z, kv[b].z, fmaf(qv[r].w, kv[b].w, s[r][b]))));
    }
    const bool edge = t0 + S::kKeys > i0 + 1 || (a.window > 0 && t0 <= i0 + S::kRows - 1 - a.window);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int i = i0 + R * ty + r;
      bool gone[kB];
      float mx = -INFINITY;
#pragma unroll
      for (int b = 0; b < kB; ++b) {
        const int t = t0 + tx + 16 * b;
        gone[b] = t > i || (a.window > 0 && t <= i - a.window);
        s[r][b] = gone[b] ? -INFINITY : s[r][b] * c;
        mx = fmaxf(mx, s[r][b]);
      }
#pragma unroll
      for (int w = 1; w < 16; w <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, w));
      const float nm = fmaxf(m[r], mx), from = nm == -INFINITY ? 0.f : nm;
      const float f = m[r] == nm ? 1.f : exp2f(m[r] - from);
      float sum = 0.f;
#pragma unroll
      for (int b = 0; b < kB; ++b) {
        const float p = exp2f(s[r][b] - from);
        if (!gone[b]) sum += p;
        sp[(R * ty + r) * S::kPS + tx + 16 * b] = gone[b] ? -1.f : p;  // (-1: out of sight, whatever V holds there)
      }
#pragma unroll
      for (int w = 1; w < 16; w <<= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, w);
      l[r] = fmaf(l[r], f, sum);
      m[r] = nm;
#pragma unroll
      for (int d = 0; d < kD; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[r][d][e] *= f;
    }
    __syncwarp();  // (a query's 16 threads are one warp's)
    auto add = [&](auto edges) {
#pragma unroll 2
      for (int t = 0; t < S::kKeys; t += 4) {
        float4 p[R];
#pragma unroll
        for (int r = 0; r < R; ++r) p[r] = *reinterpret_cast<const float4*>(sp + (R * ty + r) * S::kPS + t);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          float pu[R];
#pragma unroll
          for (int r = 0; r < R; ++r) pu[r] = u == 0 ? p[r].x : (u == 1 ? p[r].y : (u == 2 ? p[r].z : p[r].w));
#pragma unroll
          for (int d = 0; d < kD; ++d) {
            const float4 v = *reinterpret_cast<const float4*>(sv + (t + u) * S::kS + 64 * d + 4 * tx);
#pragma unroll
            for (int r = 0; r < R; ++r) {
              if (decltype(edges)::value && pu[r] < 0.f) continue;
              o[r][d][0] = fmaf(pu[r], v.x, o[r][d][0]);
              o[r][d][1] = fmaf(pu[r], v.y, o[r][d][1]);
              o[r][d][2] = fmaf(pu[r], v.z, o[r][d][2]);
              o[r][d][3] = fmaf(pu[r], v.w, o[r][d][3]);
            }
          }
        }
      }
    };
    if (edge) add(std::true_type{});
    else add(std::false_type{});
    __syncthreads();  // (before the copies of the tile after the next)
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int i = i0 + R * ty + r;
    if (i >= n) continue;
    const long long at = (long long)(a0 + i) * a.n_q + h;
    const float f = l[r] != 0.f ? 1.f / l[r] : 0.f;
    if (tx == 0 && a.lse) a.lse[at] = l[r] != 0.f ? (m[r] + log2f(l[r])) * 0.693147181f : -INFINITY;
#pragma unroll
    for (int d = 0; d < kD; ++d)
      *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at * DH + 64 * d + 4 * tx) =
          make_float4(o[r][d][0] * f, o[r][d][1] * f, o[r][d][2] * f, o[r][d][3] * f);
  }
}

// A kernel's dynamic shared memory limit, raised once per device.
template <typename K>
cudaError_t raise_smem(K k, int bytes, bool (&set)[kMaxDevices], std::mutex& mu) {
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= kMaxDevices) dev = 0;
  std::lock_guard<std::mutex> lock(mu);
  if (set[dev]) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) cudaGetLastError();
  else set[dev] = true;
  return e;
}

template <int DH, int R>
cudaError_t launch_simt(const PromptArgs& a, cudaStream_t s) {
  using S = Simt<DH, R>;
  static std::mutex mu;
  static bool set[kMaxDevices] = {};
  const cudaError_t e = raise_smem(k_prompt_simt<DH, R>, S::kSmem, set, mu);
  if (e != cudaSuccess) return e;
  count_launch();
  return launch_pdl(k_prompt_simt<DH, R>, dim3((unsigned)(prompt_most_tiles(a.tokens, a.rows, 1, S::kRows) * a.n_q)),
                    dim3(kSimtThreads), S::kSmem, s, a);
}

// Small query tiles where there are few: the block with a row's last queries has all of its keys, one tile after another, and a
// tile of keys takes it a third of the time with 16 queries that it takes with 64. With 64, 32 and 16 queries, in us: 3 rows of
// 131 of 4 heads of 64 (108 blocks of 16) 17.9, 13.5, 11.3; 300 positions of 8 heads of 128 (152) 45.0, 35.9, 29.4; 64 of 24
// heads of 256 (120) 22.0, 16.2, 14.1; 256 of those (408; 216 of 32) 76, 56, 74; 4 rows of 200 of 8 of 128 (432; 232) 36.9,
// 37.9, 40.7; 8 rows of 256 of 4 of 64 (544; 288) 23.4, 26.7, 34.3. The outputs are the same bits.
template <int DH>
cudaError_t launch_simt(const PromptArgs& a, cudaStream_t s) {
  auto blocks = [&](int tile) { return prompt_most_tiles(a.tokens, a.rows, 1, tile) * a.n_q; };
  if (blocks(16) <= device_sm_count()) return launch_simt<DH, 1>(a, s);
  if (2 * blocks(32) <= 3 * device_sm_count()) return launch_simt<DH, 2>(a, s);
  return launch_simt<DH, 4>(a, s);
}

}  // namespace
}  // namespace mtp

using namespace mtp;

extern "C" {

size_t kv_attend_prompt_workspace_bytes(int32_t tokens, int32_t rows) {
  if (tokens < 0 || rows < 1 || rows > 4096) return 0;
  return 16;
}

mtp_status kv_attend_prompt(mtp_stream stream, int32_t rows, int32_t n_q, int32_t n_kv, int32_t head_dim,
                            int32_t tokens, const void* d_q, int64_t q_tok_stride, int64_t q_head_stride,
                            const void* d_k, int64_t k_tok_stride, int64_t k_head_stride, const void* d_v,
                            int64_t v_tok_stride, int64_t v_head_stride, int32_t dtype, const int32_t* d_start,
                            int32_t max_len, float scale, int32_t window, void* d_out, float* d_lse,
                            int32_t* d_status, void* d_workspace) {
  if (rows < 1 || rows > 4096 || n_kv < 1 || n_q < 1 || n_q > 1024 || n_q % n_kv != 0 ||
      (head_dim != 64 && head_dim != 128 && head_dim != 256) || tokens < 0 || (long long)tokens * n_q >= (1LL << 31) ||
      max_len < 1 || window < 0 || !std::isfinite(scale) || (dtype != MTP_DTYPE_BF16 && dtype != MTP_DTYPE_F32))
    return MTP_ERR_BAD_ARG;
  if (tokens == 0) return MTP_OK;
  if (!d_q || !d_k || !d_v || !d_start || !d_out || !d_workspace) return MTP_ERR_BAD_ARG;
  const int es = dtype == MTP_DTYPE_BF16 ? 2 : 4;
  PromptArgs a{d_q, d_k, d_v, {q_tok_stride, k_tok_stride, v_tok_stride}, {q_head_stride, k_head_stride, v_head_stride},
               d_start, d_out, d_lse, d_status, rows, n_q, n_kv, tokens, window, scale};
  uintptr_t bits = reinterpret_cast<uintptr_t>(d_q) | reinterpret_cast<uintptr_t>(d_k) | reinterpret_cast<uintptr_t>(d_v) |
                   reinterpret_cast<uintptr_t>(d_out) | reinterpret_cast<uintptr_t>(d_workspace);
  for (int i = 0; i < 3; ++i) {
    const long long heads = i == 0 ? n_q : n_kv;
    // (the bf16 kernel's copies want strides above 0 and below 2^40 bytes; the same for both types)
    if (tokens > 1 && (a.ts[i] <= 0 || a.ts[i] >= (1LL << 40) / es)) return MTP_ERR_BAD_ARG;
    if (heads > 1 && (a.hs[i] <= 0 || a.hs[i] >= (1LL << 40) / es)) return MTP_ERR_BAD_ARG;
    bits |= (uintptr_t)a.ts[i] * es | (uintptr_t)a.hs[i] * es;
  }
  if ((bits & 15) != 0 || ((reinterpret_cast<uintptr_t>(d_lse) | reinterpret_cast<uintptr_t>(d_start)) & 3) != 0) return MTP_ERR_BAD_ARG;
  // an output over an input would be read after it is written
  const size_t n_out = (size_t)tokens * n_q * head_dim * es, n_lse = (size_t)tokens * n_q * 4, n_start = (size_t)(rows + 1) * 4;
  const void* in[3] = {d_q, d_k, d_v};
  for (int i = 0; i < 3; ++i) {
    Bytes x;
    if (!rows_range(in[i], tokens, a.ts[i], i == 0 ? n_q : n_kv, a.hs[i], head_dim, es, x) || cross(d_out, n_out, x.at, x.size) ||
        cross(d_lse, n_lse, x.at, x.size))
      return MTP_ERR_BAD_ARG;
  }
  if (cross(d_out, n_out, d_start, n_start) || cross(d_lse, n_lse, d_start, n_start) || cross(d_out, n_out, d_lse, n_lse))
    return MTP_ERR_BAD_ARG;
  a.out_whole = (reinterpret_cast<uintptr_t>(d_out) & 31) == 0;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (dtype == MTP_DTYPE_BF16) e = launch_prompt_tc(a, head_dim, s);
  else e = head_dim == 64 ? launch_simt<64>(a, s) : (head_dim == 128 ? launch_simt<128>(a, s) : launch_simt<256>(a, s));
  return e == cudaSuccess ? MTP_OK : MTP_ERR_CUDA;
}

}  // extern "C"
