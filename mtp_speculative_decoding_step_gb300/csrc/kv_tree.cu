// Trees of drafted tokens over the paged cache: positions and ancestor masks
// from the parents (kv_tree_plan), and the path that the target confirms, with
// its rows moved together in every layer's cache (kv_q4_tree_commit).
//
// Plan. A node's path to the root is doubled in length log2(depth) times: with
// m_i the nodes at distances [0, 2^k) above i and j_i the one at 2^k,
//   m_i |= m_{j_i},  j_i = j_{j_i}
// so a chain of 128 takes seven steps where walking it takes 127 dependent
// loads. A block per row, a thread per node; bound by latency: 8 trees of 16 nodes
// 1.8 us, 512 trees of up to 128 2.8 us, in a graph of such calls.
//
// Commit. next_i = the lowest child of i whose token is choice_i, found for all
// nodes at once; the path is then one dependent load per node. The row of the
// path's k-th node moves to place k. Parents come before their children, so
// k <= path[k] and path[] rises: a place that is written (k) is a source of
// later nodes only if path[m] = k for some m > k, which path[m] > path[k] >= k
// excludes; it may be one of an earlier node, so a thread takes its bytes of
// all of the path's rows in order, reading ahead of its writes. Every block of
// a row walks the path again (it is L2-resident and a few hundred cycles) and
// takes a part of the layers, sides and heads: one launch for all layers. 8 rows
// and one layer 3.3 us, 64 rows and 16 layers 4.6 us (4.8 MB).
#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "q4.cuh"

namespace mtp {

namespace {

constexpr int kMost = MTP_TREE_MAX;  // nodes of a row
constexpr int kWords = kMost / 32;

struct TreePlanArgs {
  const int32_t *parent, *start, *len;
  int32_t *pos, *mask, *status;
  int tokens, window;
};

__global__ void __launch_bounds__(kMost) k_tree_plan(const __grid_constant__ TreePlanArgs a) {
  __shared__ uint4 s_mask[2][kMost];
  __shared__ int s_jump[2][kMost];
  pdl_wait();
  pdl_trigger();
  const int r = blockIdx.x, i = threadIdx.x;
  const int a0 = min(max(a.start[r], 0), a.tokens), n = min(max(a.start[r + 1], a0), a.tokens) - a0;
  const int len = a.len[r];
  if (n == 0) return;
  if (n > kMost || len < n) {
    if (i == 0) flag_status(a.status, MTP_ERR_BAD_ARG);
    for (int t = i; t < n; t += kMost) {
      a.pos[a0 + t] = -1;
      reinterpret_cast<int4*>(a.mask)[a0 + t] = make_int4(0, 0, 0, 0);
    }
    return;
  }
  // -1: no parent, kMost: not a tree (its descendants come to it)
  uint32_t m[kWords] = {0, 0, 0, 0};
  int jump = -1;
  if (i < n) {
    jump = a.parent[a0 + i];
    m[i >> 5] = 1u << (i & 31);
    if (jump < -1 || jump >= i) jump = kMost;
  }
  s_mask[0][i] = make_uint4(m[0], m[1], m[2], m[3]);
  s_jump[0][i] = jump;
  int b = 0;
  while (__syncthreads_or(jump >= 0 && jump < kMost)) {
    if (jump >= 0 && jump < kMost) {
      const uint4 o = s_mask[b][jump];
      m[0] |= o.x;
      m[1] |= o.y;
      m[2] |= o.z;
      m[3] |= o.w;
      jump = s_jump[b][jump];
    }
    b ^= 1;
    s_mask[b][i] = make_uint4(m[0], m[1], m[2], m[3]);
    s_jump[b][i] = jump;
  }
  if (i >= n) return;
  if (jump == kMost) {
    flag_status(a.status, MTP_ERR_BAD_ARG);
    a.pos[a0 + i] = -1;
    reinterpret_cast<int4*>(a.mask)[a0 + i] = make_int4(0, 0, 0, 0);
    return;
  }
  const int depth = __popc(m[0]) + __popc(m[1]) + __popc(m[2]) + __popc(m[3]) - 1;
  if (a.window > 0 && depth >= a.window) {  // ancestors rise in depth with their number: drop the first depth + 1 - window
    int drop = depth + 1 - a.window;
#pragma unroll
    for (int w = 0; w < kWords; ++w)
      while (drop > 0 && m[w]) {
        m[w] &= m[w] - 1;
        --drop;
      }
  }
  a.pos[a0 + i] = len - n + depth;
  reinterpret_cast<int4*>(a.mask)[a0 + i] = make_int4(m[0], m[1], m[2], m[3]);
}

constexpr int kCommitThreads = 128;
constexpr int kCommitBatch = 8;  // rows of the path read before the first of them is written

struct CommitArgs {
  uint8_t* cache[MTP_MAX_CACHES][2];
  const int32_t *table, *start, *len, *parent, *tok, *choice;
  int32_t *n_acc, *out_tok, *keep, *path, *status;
  int n_caches, n_kv, page, n_pages, max_pages, tokens, max_path;
};

// U: a ninth of a cache row (dh / 2 codes and dh / 16 scales are 9 dh / 16 bytes).
template <typename U>
__global__ void __launch_bounds__(kCommitThreads) k_tree_commit(const __grid_constant__ CommitArgs a) {
  __shared__ int s_next[kMost], s_path[kMost], s_src[kMost], s_dst[kMost], s_n;
  __shared__ int s_choice[kMost];
  pdl_wait();
  pdl_trigger();
  const int r = blockIdx.x, i = threadIdx.x;
  const int a0 = min(max(a.start[r], 0), a.tokens), n = min(max(a.start[r + 1], a0), a.tokens) - a0;
  const int cover = a.len[r], base = max(cover, n) - n;
  const bool bad = n > kMost || cover < n || (a.n_caches > 0 && cover > a.max_pages * a.page);
  int par = -1, tok = 0;
  if (!bad && i < n) {
    par = a.parent[a0 + i];
    tok = a.tok[a0 + i];
    s_choice[i] = a.choice[a0 + i];
  }
  s_next[i] = kMost;
  __syncthreads();
  if (!bad && i < n) {
    if (par < -1 || par >= i) flag_status(a.status, MTP_ERR_BAD_ARG);
    else if (par >= 0 && tok == s_choice[par]) atomicMin(&s_next[par], i);
  }
  __syncthreads();
  if (i == 0) {
    int k = 0;
    if (bad) flag_status(a.status, MTP_ERR_BAD_ARG);
    else if (n > 0)
      for (int at = 0; at < kMost && k < a.max_path; at = s_next[at]) s_path[k++] = at;
    s_n = k;
  }
  __syncthreads();
  const int len = s_n;
  if (blockIdx.y == 0) {
    for (int k = i; k < a.max_path; k += kCommitThreads) {
      a.out_tok[(long long)r * a.max_path + k] = k < len ? s_choice[s_path[k]] : -1;
      if (a.path) a.path[(long long)r * a.max_path + k] = k < len ? s_path[k] : -1;
    }
    if (i == 0) {
      a.n_acc[r] = max(len - 1, 0);
      a.keep[r] = bad ? cover : base + len;
    }
  }
  if (a.n_caches == 0) return;
  // the moves: path[k] -> k
  if (i < len) {
    int at[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int p = base + (e == 0 ? s_path[i] : i), pg = p / a.page, id = a.table[(long long)r * a.max_pages + pg];
      at[e] = id >= 0 && id < a.n_pages ? id * a.page + (p - pg * a.page) : -1;
    }
    const bool stay = s_path[i] == i, lost = at[0] < 0 || at[1] < 0;
    if (!stay && lost && blockIdx.y == 0) flag_status(a.status, MTP_ERR_BAD_ARG);
    s_src[i] = stay || lost ? -1 : at[0];
    s_dst[i] = at[1];
  }
  __syncthreads();
  const int unit = blockIdx.y * kCommitThreads + i, col = unit % 9, head = unit / 9 % a.n_kv, side = unit / (9 * a.n_kv);
  if (side >= 2 * a.n_caches) return;
  U* cache = reinterpret_cast<U*>(a.cache[side >> 1][side & 1]) + col;
  auto row = [&](int slot) {
    const int pg = slot / a.page;
    return (((long long)pg * a.n_kv + head) * a.page + (slot - pg * a.page)) * 9;
  };
  for (int k0 = 1; k0 < len; k0 += kCommitBatch) {  // (place 0 stays)
    U v[kCommitBatch];
#pragma unroll
    for (int k = 0; k < kCommitBatch; ++k)
      if (k0 + k < len && s_src[k0 + k] >= 0) v[k] = cache[row(s_src[k0 + k])];
#pragma unroll
    for (int k = 0; k < kCommitBatch; ++k)
      if (k0 + k < len && s_src[k0 + k] >= 0) cache[row(s_dst[k0 + k])] = v[k];
  }
}

// Whether [a, a + na) and [b, b + nb) share an element.
bool meet(const int32_t* a, long long na, const int32_t* b, long long nb) {
  return a && b && na > 0 && nb > 0 && a < b + nb && b < a + na;
}

}  // namespace
}  // namespace mtp

using namespace mtp;

extern "C" {

mtp_status kv_tree_plan(mtp_stream stream, int32_t rows, int32_t tokens, const int32_t* d_parent,
                        const int32_t* d_start, const int32_t* d_len, int32_t window, int32_t* d_pos, int32_t* d_mask,
                        int32_t* d_status) {
  if (rows < 1 || rows > 4096 || tokens < 0 || window < 0) return MTP_ERR_BAD_ARG;
  if (tokens == 0) return MTP_OK;
  if (!d_parent || !d_start || !d_len || !d_pos || !d_mask || (reinterpret_cast<uintptr_t>(d_mask) & 15) != 0)
    return MTP_ERR_BAD_ARG;
  const int32_t* in[3] = {d_parent, d_start, d_len};
  const long long size[3] = {tokens, (long long)rows + 1, rows};
  for (int i = 0; i < 3; ++i)
    if (meet(d_pos, tokens, in[i], size[i]) || meet(d_mask, (long long)kWords * tokens, in[i], size[i])) return MTP_ERR_BAD_ARG;
  if (meet(d_pos, tokens, d_mask, (long long)kWords * tokens)) return MTP_ERR_BAD_ARG;
  const TreePlanArgs a{d_parent, d_start, d_len, d_pos, d_mask, d_status, tokens, window};
  count_launch();
  const cudaError_t e = launch_pdl(k_tree_plan, dim3(rows), dim3(kMost), 0, reinterpret_cast<cudaStream_t>(stream), a);
  return e == cudaSuccess ? MTP_OK : MTP_ERR_CUDA;
}

mtp_status kv_q4_tree_commit(mtp_stream stream, const kv_q4_cache* caches, int32_t n_caches, int32_t rows,
                             int32_t tokens, const int32_t* d_table, int32_t max_pages, const int32_t* d_start,
                             const int32_t* d_len, const int32_t* d_parent, const int32_t* d_tok,
                             const int32_t* d_choice, int32_t max_path, int32_t* d_n_acc, int32_t* d_out_tok,
                             int32_t* d_keep, int32_t* d_path, int32_t* d_status) {
  if (n_caches < 0 || n_caches > MTP_MAX_CACHES || (n_caches > 0 && !caches) || rows < 1 || rows > 4096 || tokens < 0 ||
      max_pages < 1 || max_path < 1 || max_path > kMost)
    return MTP_ERR_BAD_ARG;
  CommitArgs a = {};
  for (int i = 0; i < n_caches; ++i) {
    const kv_q4_cache& c = caches[i];
    if (!q4_cache_ok(&c) || c.n_kv != caches[0].n_kv || c.head_dim != caches[0].head_dim || c.page != caches[0].page ||
        c.n_pages != caches[0].n_pages)
      return MTP_ERR_BAD_ARG;
    a.cache[i][0] = static_cast<uint8_t*>(c.k);
    a.cache[i][1] = static_cast<uint8_t*>(c.v);
  }
  // one layer twice would be moved twice: rows that had moved would be taken for those that had not
  uint8_t* base[2 * MTP_MAX_CACHES];
  for (int i = 0; i < 2 * n_caches; ++i) base[i] = a.cache[i >> 1][i & 1];
  std::sort(base, base + 2 * n_caches);
  const int page = n_caches > 0 ? caches[0].page : 1;
  const size_t bytes = n_caches > 0 ? (size_t)caches[0].n_pages * caches[0].n_kv * page * q4_row_bytes(caches[0].head_dim) : 0;
  for (int i = 1; i < 2 * n_caches; ++i)
    if ((size_t)(base[i] - base[i - 1]) < bytes) return MTP_ERR_BAD_ARG;
  if (n_caches > 0 && (long long)max_pages * page >= (1LL << 31)) return MTP_ERR_BAD_ARG;
  if (!d_start || !d_len || !d_n_acc || !d_out_tok || !d_keep ||
      (tokens > 0 && (!d_parent || !d_tok || !d_choice)) || (n_caches > 0 && !d_table))
    return MTP_ERR_BAD_ARG;
  const int32_t *in[6] = {d_table, d_start, d_len, d_parent, d_tok, d_choice}, *out[4] = {d_n_acc, d_out_tok, d_keep, d_path};
  const long long n_in[6] = {(long long)rows * max_pages, (long long)rows + 1, rows, tokens, tokens, tokens};
  const long long n_out[4] = {rows, (long long)rows * max_path, rows, (long long)rows * max_path};
  for (int o = 0; o < 4; ++o) {
    for (int i = 0; i < 6; ++i)
      if (meet(out[o], n_out[o], in[i], n_in[i])) return MTP_ERR_BAD_ARG;
    for (int i = 0; i < o; ++i)
      if (meet(out[o], n_out[o], out[i], n_out[i])) return MTP_ERR_BAD_ARG;
  }
  a.table = d_table;
  a.start = d_start;
  a.len = d_len;
  a.parent = d_parent;
  a.tok = d_tok;
  a.choice = d_choice;
  a.n_acc = d_n_acc;
  a.out_tok = d_out_tok;
  a.keep = d_keep;
  a.path = d_path;
  a.status = d_status;
  a.n_caches = n_caches;
  a.n_kv = n_caches > 0 ? caches[0].n_kv : 1;
  a.page = page;
  a.n_pages = n_caches > 0 ? caches[0].n_pages : 0;
  a.max_pages = max_pages;
  a.tokens = tokens;
  a.max_path = max_path;
  const int units = 2 * n_caches * a.n_kv * 9;
  const dim3 grid(rows, std::max(1, (units + kCommitThreads - 1) / kCommitThreads));
  const int dh = n_caches > 0 ? caches[0].head_dim : 256;
  count_launch();
  const cudaError_t e = launch_pdl(dh == 256 ? k_tree_commit<uint4> : (dh == 128 ? k_tree_commit<uint2> : k_tree_commit<uint32_t>), grid,
                                   dim3(kCommitThreads), 0, reinterpret_cast<cudaStream_t>(stream), a);
  return e == cudaSuccess ? MTP_OK : MTP_ERR_CUDA;
}

}  // extern "C"
