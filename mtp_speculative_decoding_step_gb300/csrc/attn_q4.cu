// kv_q4_attend and kv_q4_attend_tree: checks, the choice of the kernel's shape, and the join of the
// partial results of query tiles that more than one block worked on.
#include <algorithm>
#include <cmath>

#include "attn_q4.cuh"

namespace mtp {

namespace {

constexpr int kJoinThreads = 128;  // small blocks: most find nothing to do
constexpr int kJoinFew = 4;        // parts that one warp joins by itself
constexpr int kJoinSome = 16;      // parts whose every load a block has in flight at once

// Block (b, y): the query tile that block b of the attention began and did not
// end; blocks b + 1 to `last` hold the rest of it. Row by row (y, y + gridDim.y,
// ...): the parts' weights, one thread per part, then their sum, a group of
// DH / 4 threads per part; up to 16 parts (one row of 16 nodes over 4096 positions: 13) with
// all loads at once, 25.4 us where three trips one after another took 27.5. A few parts (prompts: two) are a warp's work, four
// rows at a time without barriers: prompts' 40 MB of parts take 13 us, and took
// 37 by whole blocks.
template <int DH, int DT>
__global__ void __launch_bounds__(kJoinThreads) k_q4_join(const __grid_constant__ Q4AttnArgs a, int RT) {
  constexpr int kG = kJoinThreads / (DH / 4);
  __shared__ float s_w[kJoinThreads], s_red[2][kJoinThreads / 32];
  __shared__ float4 s_o[kG][DH / 4];
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int4 me = a.part_meta[2 * b + 1];
  if (me.w <= b) return;  // it began nothing that others went on with
  const int parts = me.w - b + 1, G = a.n_q / a.n_kv;
  const int a0 = min(max(a.start[me.x], 0), a.tokens);
  const int n = min(max(a.start[me.x + 1], a0), a.tokens) - a0;
  const float up = pow2i(head_exp(a.v_exp, me.y));
  // a part that saw nothing has m = -inf, the sum 0 and O = 0; one whose scores
  // were all NaN has m = -inf and the sum NaN. Parts whose weight is 0 are added
  // too: 0 x NaN is NaN, as where one block sums all of the row.
  auto at = [&](int p, int j) { return (long long)(2 * (b + p) + (p == 0)) * RT + j; };
  auto weight = [](float2 ml, float m) { return ml.x == -INFINITY ? (ml.y == 0.f ? 0.f : 1.f) : exp2f(ml.x - m); };
  auto place = [&](int f) { return (long long)(a0 + f / G) * a.n_q + me.y * G + f % G; };
  if (parts <= kJoinFew) {
    for (int j = blockIdx.y + gridDim.y * warp; j < RT; j += gridDim.y * (kJoinThreads / 32)) {
      const int f = me.z * RT + j;
      if (f >= n * G) return;
      float2 ml[kJoinFew];
      float4 v[kJoinFew][(DH + 127) / 128];
#pragma unroll
      for (int p = 0; p < kJoinFew; ++p) {
        ml[p] = p < parts ? a.part_ml[at(p, j)] : make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int i = 0; i < (DH + 127) / 128; ++i)
          if (p < parts && lane < DH / 4) v[p][i] = reinterpret_cast<const float4*>(a.part_o + at(p, j) * DH)[32 * i + lane];
      }
      float m = ml[0].x, l = 0.f, w[kJoinFew];
#pragma unroll
      for (int p = 1; p < kJoinFew; ++p) m = fmaxf(m, ml[p].x);
#pragma unroll
      for (int p = 0; p < kJoinFew; ++p) {
        w[p] = weight(ml[p], m);
        l = fmaf(w[p], ml[p].y, l);
      }
      const float scale = l != 0.f ? up / l : 0.f;
      const long long dst = place(f);
#pragma unroll
      for (int i = 0; i < (DH + 127) / 128; ++i) {
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int p = 0; p < kJoinFew; ++p)
          if (p < parts) {
            o.x = fmaf(w[p], v[p][i].x, o.x);
            o.y = fmaf(w[p], v[p][i].y, o.y);
            o.z = fmaf(w[p], v[p][i].z, o.z);
            o.w = fmaf(w[p], v[p][i].w, o.w);
          }
        if (l == 0.f) o = make_float4(0.f, 0.f, 0.f, 0.f);
        if (lane >= DH / 4) continue;
        if (DT == MTP_DTYPE_F32) {
          reinterpret_cast<float4*>(static_cast<float*>(a.out) + dst * DH)[32 * i + lane] =
              make_float4(o.x * scale, o.y * scale, o.z * scale, o.w * scale);
        } else {
          uint2 u;
          asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u.x) : "f"(o.y * scale), "f"(o.x * scale));
          asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u.y) : "f"(o.w * scale), "f"(o.z * scale));
          reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + dst * DH)[32 * i + lane] = u;
        }
      }
      if (lane == 0 && a.lse) a.lse[dst] = l != 0.f ? (m + log2f(l)) * 0.693147181f : -INFINITY;
    }
    return;
  }
  const int grp = tid / (DH / 4), d4 = tid % (DH / 4);
  if (parts <= kJoinSome) {
    for (int j = blockIdx.y; j < RT; j += gridDim.y) {
      // everything that a row needs in one trip to memory; each warp makes the weights for itself, a lane per part
      const float2 ml = lane < parts ? a.part_ml[at(lane, j)] : make_float2(-INFINITY, 0.f);
      float4 v[kJoinSome / kG];
#pragma unroll
      for (int q = 0; q < kJoinSome / kG; ++q)
        if (grp + kG * q < parts) v[q] = reinterpret_cast<const float4*>(a.part_o + at(grp + kG * q, j) * DH)[d4];
      const int f = me.z * RT + j;
      if (f >= n * G) return;
      const float m = warp_max(ml.x), w = lane < parts ? weight(ml, m) : 0.f, l = warp_sum(w * ml.y);
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int q = 0; q < kJoinSome / kG; ++q) {
        const float wq = __shfl_sync(0xFFFFFFFFu, w, (grp + kG * q) & 31);
        if (grp + kG * q >= parts) continue;
        o.x = fmaf(wq, v[q].x, o.x);
        o.y = fmaf(wq, v[q].y, o.y);
        o.z = fmaf(wq, v[q].z, o.z);
        o.w = fmaf(wq, v[q].w, o.w);
      }
      s_o[grp][d4] = o;
      __syncthreads();
      const long long dst = place(f);
      const float scale = up / l;
      for (int d = tid; d < DH; d += kJoinThreads) {
        float y = 0.f;
#pragma unroll
        for (int g = 0; g < kG; ++g) y += reinterpret_cast<const float*>(s_o[g])[d];
        store_elem(a.out, DT, dst * DH + d, l != 0.f ? y * scale : 0.f);
      }
      if (tid == 0 && a.lse) a.lse[dst] = l != 0.f ? (m + log2f(l)) * 0.693147181f : -INFINITY;
      __syncthreads();
    }
    return;
  }
  for (int j = blockIdx.y; j < RT; j += gridDim.y) {
    const int f = me.z * RT + j;
    if (f >= n * G) return;
    float m = -INFINITY;
    for (int p = tid; p < parts; p += kJoinThreads) m = fmaxf(m, a.part_ml[at(p, j)].x);
    m = warp_max(m);
    __syncthreads();
    if (lane == 0) s_red[0][warp] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kJoinThreads / 32; ++w) m = fmaxf(m, s_red[0][w]);
    float l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int p0 = 0; p0 < parts; p0 += kJoinThreads) {
      if (p0 + tid < parts) {
        const float2 ml = a.part_ml[at(p0 + tid, j)];
        const float w = weight(ml, m);
        s_w[tid] = w;
        l = fmaf(w, ml.y, l);
      }
      __syncthreads();
#pragma unroll 8
      for (int p = grp; p < min(parts - p0, kJoinThreads); p += kG) {
        const float w = s_w[p];
        const float4 v = reinterpret_cast<const float4*>(a.part_o + at(p0 + p, j) * DH)[d4];
        o.x = fmaf(w, v.x, o.x);
        o.y = fmaf(w, v.y, o.y);
        o.z = fmaf(w, v.z, o.z);
        o.w = fmaf(w, v.w, o.w);
      }
      __syncthreads();
    }
    l = warp_sum(l);
    if (lane == 0) s_red[1][warp] = l;
    s_o[grp][d4] = o;
    __syncthreads();
    l = 0.f;
#pragma unroll
    for (int w = 0; w < kJoinThreads / 32; ++w) l += s_red[1][w];
    const long long dst = place(f);
    for (int d = tid; d < DH; d += kJoinThreads) {
      float y = 0.f;
#pragma unroll
      for (int g = 0; g < kG; ++g) y += reinterpret_cast<const float*>(s_o[g])[d];
      store_elem(a.out, DT, dst * DH + d, l != 0.f ? y * (up / l) : 0.f);
    }
    if (tid == 0 && a.lse) a.lse[dst] = l != 0.f ? (m + log2f(l)) * 0.693147181f : -INFINITY;
  }
}

// Columns of the products: the query rows of a position block on one KV head,
// twice for fp32 queries, rounded up to 16, 32, 64 or 128 (fp32: 64). A wider
// tile than its rows fill costs MMA and softmax time, a narrower one reads and
// dequantises the cache again for every further tile. Times in us with 16, 32,
// 64 and 128 columns: 18 rows of one sequence 17.0, 15.0, 17.4, 19.5; 24 of
// eight 55.7, 38.2, 46.6, 58.7; 4 of 64 63.8, 71.3, 92.8, 114.5; 9000 and 12288
// (prompts) 2784, 1529, 982, 711.
int columns(int n_q, int n_kv, int max_q, bool wide) {
  const long long rows = (long long)max_q * (n_q / n_kv) * (wide ? 2 : 1);
  return rows <= 16 ? 16 : (rows <= 32 ? 32 : (rows <= 64 || wide ? 64 : 128));
}

// Trees: the query rows of one KV head are many (16 nodes of 6 heads fill 96 columns) and the rows of a call few, so
// that wide tiles leave blocks without work, or with one tile and all of its start, drain and join. Estimated from what
// was measured with 24 heads on 4 of 256, in us: a block's tiles at 1.3, 1.66 or 2.27 with 32, 64 or 128 columns, and 20,
// 28 or 32 for the rest. Times with these: one row of 16 nodes at 4096 positions 25.0, 28.6, 33.0; of 33 nodes 27.4,
// 37.0, 39.8; of 64 at 16,384 72.5, 67.4, 58.7; eight rows of 16 at 8192 70.9, 73.4, 64.0, of 33 147, 117, 92. (Eight rows
// of 33 of 8 heads on 2 of 128 are taken for equal: 56, 60, 62.) The lengths are taken to be what the block table holds
// (with room for 37,376 positions or more one row of 16 nodes takes 128 columns, however short it is);
// no more columns than the workspace has room for.
int tree_columns(int widest, long long query_rows, long long heads, long long tiles, int blocks) {
  constexpr float kTile[3] = {1.3f, 1.66f, 2.27f}, kRest[3] = {20.f, 28.f, 32.f};
  int best = widest;
  float least = INFINITY;
  for (int i = 0, n = 32; n <= widest; ++i, n *= 2) {
    const long long tasks = heads * tiles * ((query_rows + n - 1) / n);
    const float t = (float)((tasks + blocks - 1) / blocks) * kTile[i] + kRest[i];
    if (t < least) {
      least = t;
      best = n;
    }
  }
  return best;
}

}  // namespace
}  // namespace mtp

using namespace mtp;

extern "C" {

size_t kv_q4_attend_workspace_bytes(const kv_q4_cache* c, int32_t n_q, int32_t max_q, int32_t dtype) {
  if (!c || kv_q4_row_bytes(c->head_dim) == 0 || c->n_kv < 1 || n_q < c->n_kv || max_q < 1 ||
      (dtype != MTP_DTYPE_BF16 && dtype != MTP_DTYPE_F32))
    return 0;
  const bool wide = dtype == MTP_DTYPE_F32;
  const size_t rt = (size_t)columns(n_q, c->n_kv, max_q, wide) / (wide ? 2 : 1), slots = 2 * (size_t)device_sm_count();
  // (the parts' O and, for long shares, one more per block)
  return slots * (sizeof(int4) + rt * sizeof(float2)) + slots / 2 * 3 * rt * sizeof(float) * c->head_dim;
}

// Both entry points; d_mask makes the queries a tree's nodes.
static mtp_status attend(mtp_stream stream, const kv_q4_cache* c, int32_t rows, int32_t n_q, int32_t tokens,
                         const void* d_q, int64_t tok_stride, int64_t head_stride, int32_t dtype,
                         const int32_t* d_table, int32_t max_pages, const int32_t* d_start, const int32_t* d_len,
                         const int32_t* d_mask, const int32_t* d_place, int32_t max_q, float scale, int32_t window,
                         void* d_out, float* d_lse, int32_t* d_status, void* d_workspace) {
  if (!q4_cache_ok(c) || rows < 1 || rows > 4096 || n_q < 1 || n_q > 1024 || n_q % c->n_kv != 0 || tokens < 0 ||
      (long long)tokens * n_q >= (1LL << 31) || max_pages < 1 || (long long)max_pages * c->page >= (1LL << 31) ||
      max_q < 1 || window < 0 || !std::isfinite(scale) || (dtype != MTP_DTYPE_BF16 && dtype != MTP_DTYPE_F32))
    return MTP_ERR_BAD_ARG;
  if (tokens == 0) return MTP_OK;
  const bool wide = dtype == MTP_DTYPE_F32;
  const int es = wide ? 4 : 2;
  if (!d_q || !d_table || !d_start || !d_len || !d_out || !d_workspace ||
      (reinterpret_cast<uintptr_t>(d_q) & (es - 1)) != 0 || (reinterpret_cast<uintptr_t>(d_out) & 15) != 0 ||
      (reinterpret_cast<uintptr_t>(d_workspace) & 15) != 0)
    return MTP_ERR_BAD_ARG;
  const int blocks = device_sm_count();
  int n = columns(n_q, c->n_kv, max_q, wide);
  if (d_mask)
    n = tree_columns(n, (long long)max_q * (n_q / c->n_kv) * (wide ? 2 : 1), (long long)rows * c->n_kv,
                     ((long long)max_pages * c->page + kT - 1) / kT, blocks);
  const int rt = n / (wide ? 2 : 1);
  uint8_t* w = static_cast<uint8_t*>(d_workspace);
  int4* meta = reinterpret_cast<int4*>(w);
  w += sizeof(int4) * 2 * blocks;
  float2* ml = reinterpret_cast<float2*>(w);
  w += sizeof(float2) * 2 * blocks * rt;
  float* part_o = reinterpret_cast<float*>(w);
  Q4AttnArgs a{static_cast<const uint8_t*>(c->k), static_cast<const uint8_t*>(c->v), c->k_exp, c->v_exp, d_table,
               d_start, d_len, d_q, tok_stride, head_stride, d_out, d_lse, d_status, meta, ml,
               part_o, part_o + (size_t)2 * blocks * rt * c->head_dim, rows, n_q, c->n_kv, c->page, c->n_pages, max_pages, tokens, window, 0,
               scale, d_mask, d_place};
  const uintptr_t bits = reinterpret_cast<uintptr_t>(d_q) | (uintptr_t)(tok_stride * es) | (uintptr_t)(head_stride * es);
  a.q_vec = (bits & 15) == 0;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  auto launch = c->head_dim == 64    ? (d_mask ? launch_q4_tree_64 : launch_q4_attn_64)
                : c->head_dim == 128 ? (d_mask ? launch_q4_tree_128 : launch_q4_attn_128)
                                     : (d_mask ? launch_q4_tree_256 : launch_q4_attn_256);
  cudaError_t e = launch(a, n, wide, blocks, s);
  if (e != cudaSuccess) return MTP_ERR_CUDA;
  void (*join)(Q4AttnArgs, int) =
      c->head_dim == 64    ? (wide ? k_q4_join<64, MTP_DTYPE_F32> : k_q4_join<64, MTP_DTYPE_BF16>)
      : c->head_dim == 128 ? (wide ? k_q4_join<128, MTP_DTYPE_F32> : k_q4_join<128, MTP_DTYPE_BF16>)
                           : (wide ? k_q4_join<256, MTP_DTYPE_F32> : k_q4_join<256, MTP_DTYPE_BF16>);
  // (rows of a query tile that are used, as far as the caller knows)
  const int used = (int)std::min<long long>(std::min(rt, 32), (long long)max_q * (n_q / c->n_kv));
  e = launch_pdl(join, dim3(blocks, used), dim3(kJoinThreads), 0, s, a, rt);
  count_launch();
  return e == cudaSuccess ? MTP_OK : MTP_ERR_CUDA;
}

mtp_status kv_q4_attend(mtp_stream stream, const kv_q4_cache* c, int32_t rows, int32_t n_q, int32_t tokens,
                        const void* d_q, int64_t tok_stride, int64_t head_stride, int32_t dtype,
                        const int32_t* d_table, int32_t max_pages, const int32_t* d_start, const int32_t* d_len,
                        int32_t max_q, float scale, int32_t window, void* d_out, float* d_lse, int32_t* d_status,
                        void* d_workspace) {
  return attend(stream, c, rows, n_q, tokens, d_q, tok_stride, head_stride, dtype, d_table, max_pages, d_start, d_len,
                nullptr, nullptr, max_q, scale, window, d_out, d_lse, d_status, d_workspace);
}

mtp_status kv_q4_attend_tree(mtp_stream stream, const kv_q4_cache* c, int32_t rows, int32_t n_q, int32_t tokens,
                             const void* d_q, int64_t tok_stride, int64_t head_stride, int32_t dtype,
                             const int32_t* d_table, int32_t max_pages, const int32_t* d_start, const int32_t* d_len,
                             const int32_t* d_mask, const int32_t* d_pos, int32_t max_q, float scale, int32_t window,
                             void* d_out, float* d_lse, int32_t* d_status, void* d_workspace) {
  if (max_q > kTreeMost) return MTP_ERR_BAD_ARG;
  if (tokens > 0 && (!d_mask || (reinterpret_cast<uintptr_t>(d_mask) & 15) != 0 || (window > 0 && !d_pos))) return MTP_ERR_BAD_ARG;
  return attend(stream, c, rows, n_q, tokens, d_q, tok_stride, head_stride, dtype, d_table, max_pages, d_start, d_len,
                d_mask, window > 0 ? d_pos : nullptr, max_q, scale, window, d_out, d_lse, d_status, d_workspace);
}

}  // extern "C"
