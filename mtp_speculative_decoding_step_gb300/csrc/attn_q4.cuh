// Attention over the paged 4-bit cache (kv_q4_attend) on the 5th-generation
// tensor cores.
//
//   s_jt = c_j q_j . k_t,  out_j = sum_t softmax(s)_jt v_t
//
// for the query rows j of one KV head (positions x the query heads that share
// it), c_j = scale log2 e 2^(exponents). Both products are formed transposed,
// with 128 cached positions (or 128 head dimensions) as the MMA's M and the
// query rows as its N, so that a block of a few queries costs N = 16..64
// columns instead of a padded 128-row tile, and one kernel serves single
// tokens, verify blocks and prompts:
//
//   S^T[128 positions][N] = K[128][DH] . Q^T      A = K in tensor memory
//   O^T[DH][N]           += V^T[DH][128] . P^T    A = V in shared memory
//
// A block owns an equal run of (row, KV head, query tile, 128-position tile)
// tasks, whatever the rows' lengths are; a (row, head, query tile) that its run
// does not hold whole leaves a partial (O, running maximum, sum) that a second
// kernel joins. 16 warps:
//   warps 0, 3    copy the tile's 4-bit K and V rows (cp.async.bulk) into a ring each
//   warp 1        issues the MMAs; S runs one or two tiles ahead of P.V
//   warp 2        hands out the block's shares
//   dequantisers  thread = position: codes x scale as f16, exact (at most six
//                 significant bits). K goes to tensor memory (the thread's row
//                 is the operand's lane), V to 128B-swizzled shared memory
//                 (position-major, read by the MMA as an M-major operand)
//   softmax       reads S^T in the MMA fragment layout (a thread holds 8 rows x
//                 2 columns of a 16 x 8 patch), so column sums stay in registers
//                 and stmatrix.trans lays P^T out for the MMA
// The running maximum is lazy: weights are 2^(y - m) with m seven below a
// maximum seen, and m moves (O is rescaled in tensor memory) only when some y
// passes m + 15; until then a tile needs one vote and no reduction. f16 holds
// weights up to 2^15 and, 2^-14 being its smallest normal number, rounds all
// within 2^21 of the largest to 11 bits.
//
// What it measured (24 query heads on 4 KV heads of 256), and what is known of
// what bounds it:
//   prompts (two rows of 1500 and 2048 queries near 8192): 690 us, 950 TFLOP/s.
//     The tensor pipe is active 47 %, the issue slots 42 %: neither is full. With
//     128 columns tensor memory has room for one S and one K, so that expansion,
//     S, softmax and P.V of a block take turns
//   8 rows of 4 queries, 1k to 16k positions: 36 us, 2.4 TB/s. A block has 15.4
//     tiles of 2450 cycles, 20 us (1900 of the 2450 are shared-memory traffic: raw
//     rows in and out, V's f16 tile written by threads and read by the MMA, P);
//     the rest is a share's start, its drain of O and the join, not told apart
//   64 rows of one query, 2 KV heads of 128, pages of 16: 61 us, 2.4 TB/s. A
//     block has 54 tiles, 2200 cycles each with the starts and the join, where
//     shared memory accounts for 890 and the issue slots are 47 % busy: which wait
//     limits it is not known
//   1 row of 3 queries, 4096 positions (one tile a block): 14.4 us with the join,
//     one after another: shares 2700 cycles, page look-up and copy 2900, the two
//     products and the softmax between 3700, O 3300, together 6.5 us; a launch and
//     the join are some 4 more, and what is left of the 14.4 is not accounted for
//   fp32 queries, the same four: 1960, 46, 64 and 15 us
//   many short rows (8 query heads on 2 of 128): 512 of up to 1023 positions 62 us,
//     4096 of up to 127 282 us. Every block reads all rows' lengths, 32 at a time,
//     which at 4096 rows is 128 dependent steps; not measured by itself
//
// Trees (TREE, kv_q4_attend_tree): the queries are the nodes of a tree at a row's last positions. The tiles that hold them
// are edges, where a query's sight is a bit of its mask; everything before is the same. 8 rows of 20 to 33 nodes, 1k to 16k
// positions: 123 us, 405 TFLOP/s. A block has 30 tiles of 128 columns at some 5000 cycles, of which the softmax is busy 3400
// (S read, scaled and voted on 1840, weights 750, P^T stored 500), K and V are expanded in 3100 and the MMAs take 2050; a
// move of the maxima costs 9000 more, one to four a share; a share's start and first maxima are 15,000, the join 10 us.
// One row of 16 nodes at 4096 positions: 25 us, the join 6 of them.
//
// fp32 queries: q and the weights each enter as two f16 parts in separate
// columns (22 bits), N / 2 rows a tile.
//
// Every wait is bounded: on expiry the block raises the status word, waits for
// its copies, frees its tensor memory and returns.
#pragma once
#include <mutex>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"
#include "q4.cuh"
#include "q4_walk.h"
#include "tc_attn.cuh"

namespace mtp {

constexpr int kAttnThreads = 512;
constexpr float kUnset = -INFINITY;

struct Q4AttnArgs {
  const uint8_t *kc, *vc;
  const int32_t *k_exp, *v_exp, *table, *start, *len;
  const void* q;
  long long ts, hs;
  void* out;
  float* lse;
  int32_t* status;
  int4* part_meta;               // [2 * blocks] (row, head, query tile, block that ends it; -1 if it began elsewhere; 0 if none)
  float2* part_ml;               // [2 * blocks][rows of a tile] (m, sum)
  float* part_o;                 // [2 * blocks][rows of a tile][DH]
  float* far_o;                  // [blocks][rows of a tile][DH]: O of a long share's tiles before the last kFar
  int rows, n_q, n_kv, page, n_pages, max_pages, tokens, window;
  int q_vec;                     // 16-byte loads of q are aligned
  float scale;
  const int32_t *mask, *place;   // trees: bits of the nodes that a query sees; its position (NULL: no window)
};

// ------------------------------------------------------------ shape

constexpr int least(int a, int b) { return a < b ? a : b; }

template <int DH, int N, bool WIDE, bool TREE = false>
struct Shape {
  static constexpr int kRow = q4_row_bytes(DH);
  static constexpr int RT = WIDE ? N / 2 : N;            // query rows per tile
  static constexpr int SG = N == 128 ? 2 : 1;            // softmax warpgroups
  static constexpr int NW = N / SG;                      // columns per softmax warpgroup
  static constexpr int NC = WIDE ? NW / 2 : NW;          // query rows per softmax warpgroup
  // The tensor core's accumulation drops the bits past fp32's, 5e-7 of a sum per
  // tile: after kFar tiles O moves to memory, where it is added with rounding. (2e-6
  // of fp32 outputs are left then, 9e-5 of bf16's, whose own step is 40 times that;
  // a row of 131,072 positions summed by one block had lost 8e-4.)
  static constexpr int kFar = WIDE ? 8 : 128;
  static constexpr int MB = DH == 256 ? 2 : 1;           // M blocks of O^T (64 dims: duplicated rows)
  static constexpr int KC = DH / 2;                      // tensor-memory columns of a K operand
  static constexpr int SB = MB * N + 2 * N + 2 * KC <= 512 ? 2 : 1;  // S and K buffers
  static constexpr uint32_t cO = 0, cS = MB * N, cK = cS + SB * N, cEnd = cK + SB * KC;
  static constexpr uint32_t kCols = cEnd <= 128 ? 128 : (cEnd <= 256 ? 256 : 512);
  // shared memory
  static constexpr int kRaw = kT * kRow;                 // a tile's rows of K or V
  static constexpr int VB = DH == 256 ? 1 : 2;           // V tiles in shared memory
  static constexpr int kV = kT * DH * 2, kQ = N * DH * 2, kP = N * kT * 2;  // (SB buffers of P)
  static constexpr int kMetaBytes = 8704, kTreeBytes = TREE ? 128 * 16 : 0;  // (masks of a tile's query rows)
  static constexpr int kRoom = (227 * 1024 - kMetaBytes - kTreeBytes - VB * kV - kQ - SB * kP) / kRaw;
  // ring stages; even counts for two dequantising groups, so that each group
  // meets every phase of its stages' barriers
  static constexpr int kMost = 8;
  static constexpr int KS = least(kMost, SG == 2 ? (kRoom + 1) / 2 : (kRoom >= 8 ? kRoom / 4 * 2 : 2));
  static constexpr int VS = least(kMost, SG == 2 ? kRoom / 2 : (kRoom - KS) / 2 * 2);  // V waits longer than K
  static constexpr int oV = 0, oQ = VB * kV, oP = oQ + kQ, oRawK = oP + SB * kP, oRawV = oRawK + KS * kRaw;
  static constexpr int oMeta = (oRawV + VS * kRaw + 127) / 128 * 128;
  static constexpr int oTree = oMeta + kMetaBytes, kSmem = oTree + kTreeBytes;
  static_assert(VS >= 1 && KS <= kMost && VS <= kMost && KS + VS <= kRoom && cEnd <= 512 && (SG == 2 || (KS % 2 == 0 && VS % 2 == 0)), "shape");
};

constexpr int kRuns = 8;

// Small state of a block.
template <int DH>
struct Meta {
  uint64_t rawk_full[8], rawk_empty[8], rawv_full[8], rawv_empty[8];
  uint64_t k_full[2], k_empty[2], s_full[2], s_empty[2];
  // (a waiter has to meet every phase of its barrier, since a parity tells only
  // neighbouring ones apart: v_empty goes by the tile's parity, as the groups do)
  uint64_t v_full[4], v_empty[4], p_full[2], p_empty[2], q_full;
  uint32_t valid_k[8], valid_v[8];   // bit p: piece p of the stage was copied
  uint32_t tmem;
  int fail;
  uint64_t run_full[kRuns], run_empty[kRuns];
  Run run[kRuns];                    // the shares, written by one warp ahead of the other roles
  alignas(16) float cm[128][2];      // per query row: c, m
  float f[128];                      // per query row: factor of a moved m, then 1 / sum
  float far[128];                    // per query row: the m of what is in far_o
  alignas(16) int lim[128];          // per query row: its position
  int dst[128];                      // per query row: row of out and lse, or -1
  float red[4][128];                 // per warp of a softmax group and query row
  alignas(16) uint8_t zero[144];     // a row of zeros, read in the place of positions out of sight
  uint32_t copied[2];                // tiles of K and of V whose copies were issued
  uint64_t drain;                    // the MMAs of a run that gave up
  // Notes of NaN in V, in sets that the shares use in turn. V of a tile waits for
  // the products of the tile as many before it as there are V buffers; shares
  // have one tile at least, and those products wait for the softmax to have
  // begun on their share. So a share's notes are still being read while V of the
  // next one (one buffer) or of the next two is expanded, and no longer.
  static constexpr int kNotes = Shape<DH, 16, false>::VB + 1;
  uint32_t nan_run[kNotes];             // 1 + the last run that noted something in the set
  uint32_t nan_bits[kNotes][4][DH / 16][4];  // edge tile, 16 dimensions: positions whose V is NaN there
};
static_assert(sizeof(Meta<256>) <= 8704, "meta");

__device__ __forceinline__ __half2 as_half2(uint32_t u) { return *reinterpret_cast<const __half2*>(&u); }
__device__ __forceinline__ uint32_t as_bits(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }

// NW words of a cache row in shared memory, in the widest loads that rows of
// kRow bytes are aligned for.
template <int NW, int kRow>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[NW]) {
  if (kRow % 16 == 0 && NW % 4 == 0) {
#pragma unroll
    for (int i = 0; i < NW / 4; ++i) {
      const uint4 v = reinterpret_cast<const uint4*>(p)[i];
      w[4 * i] = v.x;
      w[4 * i + 1] = v.y;
      w[4 * i + 2] = v.z;
      w[4 * i + 3] = v.w;
    }
  } else if (kRow % 8 == 0 && NW % 2 == 0) {
#pragma unroll
    for (int i = 0; i < NW / 2; ++i) {
      const uint2 v = reinterpret_cast<const uint2*>(p)[i];
      w[2 * i] = v.x;
      w[2 * i + 1] = v.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < NW; ++i) w[i] = reinterpret_cast<const uint32_t*>(p)[i];
  }
}

// Whether a query at `pos` sees a position of an edge tile whose V is NaN in
// 16-dimension block b. (Trees: `mask` has the query's bits of the n positions from base on.)
template <int B, bool TREE>
__device__ __noinline__ bool sees_nan(int first, int t0, int cnt, int p0, int p1, const uint32_t (*bits)[B][4], int b, int pos,
                                      int window, const uint32_t* mask, int base, int n) {
  Run s;
  s.first = first;
  s.p0 = p0;
  s.p1 = p1;
  for (int tile = t0; tile < t0 + cnt; ++tile) {
    if (!s.edge(tile, window)) continue;
    for (int w = 0; w < 4; ++w) {
      uint32_t m = bits[s.edge_index(tile)][b][w];
      while (m) {
        const int t = tile * kT + 32 * w + __ffs(m) - 1;
        m &= m - 1;
        if (TREE && t >= base) {
          if (t - base < n && (mask[(t - base) >> 5] >> ((t - base) & 31) & 1)) return true;
        } else if (t <= pos && (window == 0 || pos - t < window)) {
          return true;
        }
      }
    }
  }
  return false;
}

// A softmax group's O of the tiles since the last call, added to what far_o has
// of those before (`first`: nothing), or back from there at the share's `end`.
// Out of line with all its addresses: few shares come here, and the loop over
// tiles needs the registers (with them inside, prompts took 760 us, not 713).
template <int DH, int N, bool WIDE, bool TREE>
__device__ __noinline__ void add_far(const Q4AttnArgs* a, Meta<DH>* M, int sg, bool first, bool end) {
  using S = Shape<DH, N, WIDE, TREE>;
  const int me = threadIdx.x & 127, quarter = me >> 5, c0 = sg * S::NC;
  if (me < S::NC) {
    const int col = c0 + me;
    const float was = M->far[col], m = M->cm[col][1];
    M->f[col] = first ? 0.f : (was == m ? 1.f : (was == kUnset ? 0.f : ex2(was - m)));
    M->far[col] = m;
  }
  group_sync(1 + sg);
  if (DH == 64 && quarter >= 2) return;  // (duplicated rows)
  const uint32_t t0 = M->tmem + S::cO + c0 + ((uint32_t)(32 * quarter) << 16);
  float* p0 = a->far_o + ((long long)blockIdx.x * S::RT + c0) * DH + me;
#pragma unroll 1
  for (int mb = 0; mb < S::MB; ++mb)
#pragma unroll 1
    for (int c = 0; c < S::NC; c += 8) {
      const uint32_t t = t0 + mb * N + c;
      float* p = p0 + c * DH + mb * 128;
      float o[8];
      tc::tmem_ld8(t, o);
      if (WIDE && !end) {
        float o2[8];
        tc::tmem_ld8(t + N / 2, o2);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] += o2[e];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (!first) o[e] = fmaf(p[e * DH], M->f[c0 + c + e], o[e]);
      if (end) {
        asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::"r"(__float_as_uint(o[0])),
                     "r"(__float_as_uint(o[1])), "r"(__float_as_uint(o[2])), "r"(__float_as_uint(o[3])),
                     "r"(__float_as_uint(o[4])), "r"(__float_as_uint(o[5])), "r"(__float_as_uint(o[6])),
                     "r"(__float_as_uint(o[7])), "r"(t));
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) p[e * DH] = o[e];
      }
    }
  if (end) tc_wait_st();
}

template <int DH, int N, bool WIDE, bool TREE>
__global__ void __launch_bounds__(kAttnThreads, 1) k_q4_attn(const __grid_constant__ Q4AttnArgs a) {
  using S = Shape<DH, N, WIDE, TREE>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];  // (swizzled operands go by address bits 7 to 9)
  uint8_t* const base = smem_raw;
  auto& M = *reinterpret_cast<Meta<DH>*>(base + S::oMeta);
  const int warp = __shfl_sync(0xFFFFFFFFu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  constexpr int kDq = S::SG == 2 ? 1 : 2;                // dequantising warpgroups
  constexpr int kSoftWarp = 4 + 4 * kDq;                 // first softmax warp
  constexpr int kSoftWarps = 4 * S::SG;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 8; ++i) {
      mbar_init(smem_u32(&M.rawk_full[i]), 1);
      mbar_init(smem_u32(&M.rawv_full[i]), 1);
      mbar_init(smem_u32(&M.rawk_empty[i]), 4);
      mbar_init(smem_u32(&M.rawv_empty[i]), 4);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(smem_u32(&M.v_full[i]), 4);
      mbar_init(smem_u32(&M.v_empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&M.k_full[i]), 4);
      mbar_init(smem_u32(&M.k_empty[i]), 1);
      mbar_init(smem_u32(&M.s_full[i]), 1);
      mbar_init(smem_u32(&M.s_empty[i]), kSoftWarps);
      mbar_init(smem_u32(&M.p_full[i]), kSoftWarps);
      mbar_init(smem_u32(&M.p_empty[i]), 1);
    }
    mbar_init(smem_u32(&M.q_full), kSoftWarps);
    M.fail = 0;
    M.copied[0] = M.copied[1] = 0;
    for (int i = 0; i < Meta<DH>::kNotes; ++i) M.nan_run[i] = 0;
    mbar_init(smem_u32(&M.drain), 1);
    for (int i = 0; i < kRuns; ++i) {
      mbar_init(smem_u32(&M.run_full[i]), 1);
      mbar_init(smem_u32(&M.run_empty[i]), 3 + 4 * kDq + kSoftWarps);  // copies (2), MMAs, the warps of the others
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (threadIdx.x >= 64 && threadIdx.x < 64 + S::kRow / 4) reinterpret_cast<uint32_t*>(M.zero)[threadIdx.x - 64] = 0u;
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&M.tmem)),
                 "r"(S::kCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = M.tmem;
  volatile int* fail = &M.fail;
  const int ps = a.page % kT == 0 ? kT : (a.page % 64 == 0 ? 64 : (a.page % 32 == 0 ? 32 : 16));  // slots per copy
  pdl_wait();
  pdl_trigger();

  // the shares in turn: `next` waits for share `k` and hands it out, `done` gives its slot back
  // (after the share, when the words that `next` loaded have all been used)
  auto next = [&](uint32_t k, Run& s) {
    if (!wait(&M.run_full[k % kRuns], (k / kRuns) & 1, fail)) return false;
    s = M.run[k % kRuns];
    return true;
  };
  auto done = [&](uint32_t k) { mbar_arrive(smem_u32(&M.run_empty[k % kRuns])); };

  if (warp == 2) {
    // ---------------------------------------------------------- shares
    // Every (row, KV head, query tile, 128-position tile) is a task; each block
    // owns an equal stretch of them. The rows' task counts are scanned, rows
    // in consecutive groups per lane.
    const Walk<Q4AttnArgs, TREE> walk{&a, a.n_q / a.n_kv, S::RT};
    // (by the lane that hands out the shares, so that its arrival orders these
    // stores before those of the warps that take a share)
    if (lane == 0) a.part_meta[2 * blockIdx.x] = a.part_meta[2 * blockIdx.x + 1] = make_int4(0, 0, 0, 0);
    const int per = (a.rows + 31) / 32, r0 = min(lane * per, a.rows), r1 = min(r0 + per, a.rows);
    long long sum = 0;
    int a0 = 0, n = 0, L = 0;
    long long ph = 0;
#pragma unroll 1
    for (int r = r0; r < r1; ++r) {
      walk.row(r, a0, n, L);
      if (blockIdx.x == 0 && L != a.len[r]) flag_status(a.status, MTP_ERR_BAD_ARG);
      if (TREE && blockIdx.x == 0 && min(a.start[r + 1], a.tokens) - a0 > kTreeMost) flag_status(a.status, MTP_ERR_BAD_ARG);
      ph = walk.per_head(n, L);
      sum += ph * a.n_kv;
    }
    long long inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xFFFFFFFFu, inc, o);
      if (lane >= o) inc += u;
    }
    const long long all = __shfl_sync(0xFFFFFFFFu, inc, 31);
    // equal stretches, the first ones a task longer; with fewer tasks than
    // blocks the first blocks take one each
    const int nb = (int)max(1LL, min((long long)gridDim.x, all)), b = blockIdx.x;
    long long q = 0;
    unsigned rem = 0;
    if (all >> 32 == 0) {
      q = (unsigned)all / (unsigned)nb;
      rem = (unsigned)all - (unsigned)q * nb;
    } else {
#pragma unroll 1
      for (int d = 48; d >= 0; d -= 16) {  // 16 bits a step (nb < 2^16)
        const unsigned part = rem << 16 | (unsigned)(all >> d & 0xFFFF), x = part / (unsigned)nb;
        q = q << 16 | x;
        rem = part - x * nb;
      }
    }
    const int more = (int)rem;
    const long long w0 = b < nb ? b * q + min(b, more) : all;
    long long left = b < nb ? q + (b < more) : 0;
    // the lane whose rows hold the first task
    const unsigned who = __ballot_sync(0xFFFFFFFFu, left > 0 && inc - sum <= w0 && w0 < inc);
    const int owner = who ? __ffs(who) - 1 : 0;
    long long at = __shfl_sync(0xFFFFFFFFu, inc - sum, owner);
    int r = __shfl_sync(0xFFFFFFFFu, r0, owner), g = 0, j = 0;
    long long o = 0;
    a0 = __shfl_sync(0xFFFFFFFFu, a0, owner);  // (the last row that the lane looked at: its only one, mostly)
    n = __shfl_sync(0xFFFFFFFFu, n, owner);
    L = __shfl_sync(0xFFFFFFFFu, L, owner);
    ph = __shfl_sync(0xFFFFFFFFu, ph, owner);
    if (left > 0) {
#pragma unroll 1
      for (;; ++r) {
        if (per > 1) {
          walk.row(r, a0, n, L);
          ph = walk.per_head(n, L);
        }
        if (w0 < at + ph * a.n_kv) {
          walk.find(w0 - at, ph, g, o);
          break;
        }
        at += ph * a.n_kv;
      }
    }
    bool found = false;
    uint32_t k = 0;
    if (left == 0 && lane == 0) {  // nothing: an empty last share
      M.run[0].nt = 0;
      M.run[0].flags = 4;
      mbar_arrive(smem_u32(&M.run_full[0]));
    }
#pragma unroll 1
    while (left > 0) {
      Run s;
      int cnt;
      walk.span(n, L, j, s.lo, s.end, s.first, cnt);
      if (!found && o >= cnt) {  // still before the first task
        o -= cnt;
        ++j;
        continue;
      }
      found = true;
      s.r = r;
      s.g = g;
      s.j = j;
      s.a0 = a0;
      s.n = n;
      s.pos = L - n;
      s.p0 = TREE ? s.pos - 1 : s.pos + j * S::RT / walk.G;
      s.p1 = TREE ? s.pos + n - 1 : s.pos + (min(n * walk.G, (j + 1) * S::RT) - 1) / walk.G;
      s.tile = s.first + (int)o;
      s.nt = (int)min(cnt - o, left);
      s.flags = (o == 0 ? 1 : 0) | (o + s.nt == cnt ? 2 : 0) | (s.nt == left ? 4 : 0);
      s.last = b;
#pragma unroll 1
      for (long long rest = cnt - o - s.nt; rest > 0; rest -= q + (s.last < more)) ++s.last;
      left -= s.nt;
      o = 0;
      if (k >= kRuns && !wait(&M.run_empty[k % kRuns], (k / kRuns - 1) & 1, fail)) break;
      if (lane == 0) {
        M.run[k % kRuns] = s;
        mbar_arrive(smem_u32(&M.run_full[k % kRuns]));
      }
      ++k;
      if (left > 0 && ++j == walk.tiles(n)) {
        j = 0;
        if (++g == a.n_kv) {
          g = 0;
#pragma unroll 1
          do walk.row(++r, a0, n, L);
          while (n == 0);
        }
      }
    }
  } else if (warp == 0 || warp == 3) {
    // ---------------------------------------------------------- copies: K, V
    const bool is_v = warp == 3;
    const int stages = is_v ? S::VS : S::KS;
    uint64_t *full = is_v ? M.rawv_full : M.rawk_full, *empty = is_v ? M.rawv_empty : M.rawk_empty;
    uint32_t *valid = is_v ? M.valid_v : M.valid_k, *copied = &M.copied[is_v];
    const uint8_t* cache = is_v ? a.vc : a.kc;
    const uint32_t ring = smem_u32(smem_raw) + (is_v ? S::oRawV : S::oRawK), bytes = ps * S::kRow;
    uint32_t it = 0, st = 0, round = 0;
    bool ok = true;
    Run s;
    s.flags = 0;
#pragma unroll 1
    for (uint32_t k = 0; ok && !(s.flags & 4); ++k) {
      ok = next(k, s);
      if (!ok) break;
      // lane 8 q + p holds the place of piece p of tile 4 g + q, a group of four
      // tiles ahead of the copies: the look-up would cost each tile an L2 trip
      const int32_t* tab = a.table + (long long)s.r * a.max_pages;
      auto places = [&](int g) {
        const int q = 4 * g + (lane >> 3), p0 = (lane & 7) * ps, t0 = (s.tile + q) * kT + p0;
        if (p0 >= kT || q >= s.nt || t0 >= s.end || t0 + ps <= s.lo) return -1LL;
        const int page = t0 / a.page, id = tab[page];
        if (id >= 0 && id < a.n_pages) return (((long long)id * a.n_kv + s.g) * a.page + (t0 - page * a.page)) * S::kRow;
        flag_status(a.status, MTP_ERR_BAD_ARG);
        return -1LL;
      };
      long long at = places(0), ahead = places(1);
#pragma unroll 1
      for (int i = 0; i < s.nt && ok; ++i, ++it) {
        if (i > 0 && (i & 3) == 0) {
          at = ahead;
          ahead = places((i >> 2) + 1);
        }
        long long src = __shfl_sync(0xFFFFFFFFu, at, (i & 3) * 8 + (lane & 7));
        if (lane >= 8) src = -1;
        const uint32_t mask = __ballot_sync(0xFFFFFFFFu, src >= 0);
        if (round > 0) ok = wait(&empty[st], (round - 1) & 1, fail);
        if (!ok) break;
        if (lane == 0) {
          valid[st] = mask;
          mbar_expect_tx(smem_u32(&full[st]), bytes * __popc(mask));
          *copied = it + 1;
        }
        __syncwarp();
        if (src >= 0) bulk_g2s(ring + st * S::kRaw + lane * bytes, cache + src, bytes, smem_u32(&full[st]));
        if (++st == stages) {
          st = 0;
          ++round;
        }
      }
      __syncwarp();
      if (lane == 0) done(k);
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMAs
    constexpr uint32_t idS = idesc_f16(128, N, false), idO = idesc_f16(128, N, true);
    // descriptors grow by their operand's offset / 16
    const uint32_t sm = smem_u32(smem_raw), tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
    const uint64_t dq = tc::sdesc(sm + S::oQ), dp = tc::sdesc(sm + S::oP);
    const uint64_t dv = sdesc_mn(sm + S::oV, DH == 64 ? 0 : 8192);
    auto issue_s = [&](uint32_t i) {
      const uint32_t b = i % S::SB;
#pragma unroll 1
      for (int c = 0; c < DH / 64; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          mma_f16_ts(tm + S::cS + b * N, tm + S::cK + b * S::KC + c * 32 + e * 8, dq + c * (N * 8) + e * 2, idS,
                     (c | e) > 0 ? 1u : 0u);
      mma_commit_elect(smem_u32(&M.k_empty[b]));
      mma_commit_elect(smem_u32(&M.s_full[b]));
    };
    auto issue_pv = [&](uint32_t i, bool first) {
      uint32_t acc = first ? 0u : 1u;
      const uint64_t dpb = dp + (i % S::SB) * (S::kP / 16);
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        const uint32_t vs = i % S::VB * 2 + h;
        if (!wait(&M.v_full[vs], i / S::VB & 1, fail)) return false;
        tc_fence_after();
        const uint64_t vh = dv + vs * (S::kV / 32), ph = dpb + h * (N * 8);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
#pragma unroll
          for (int mb = 0; mb < S::MB; ++mb)
            mma_f16_ss(tm + S::cO + mb * N, vh + mb * 1024 + k * 128, ph + k * 2, idO, acc);
          acc = 1u;
        }
        mma_commit_elect(smem_u32(&M.v_empty[(i & 1) * 2 + h]));
      }
      mma_commit_elect(smem_u32(&M.p_empty[i % S::SB]));
      return true;
    };
    uint32_t it = 0;  // tiles before the share
    bool ok = true;
    int flags = 0;
#pragma unroll 1
    for (uint32_t k = 0; ok && !(flags & 4); ++k) {
      ok = wait(&M.run_full[k % kRuns], (k / kRuns) & 1, fail);
      if (!ok) break;
      const int nt = __shfl_sync(0xFFFFFFFFu, M.run[k % kRuns].nt, 0);
      flags = __shfl_sync(0xFFFFFFFFu, M.run[k % kRuns].flags, 0);
      if (nt == 0) break;
      // With two buffers S runs two tiles ahead of P.V: a tile's softmax has
      // the other tile's products to hide behind. (The softmax that fills P of
      // tile i has read S of tile i, so S of tile i + 2 may follow P.V of tile
      // i without a wait of its own.) With one, S of tile i + 1 goes before
      // P.V of tile i, as soon as S of tile i has been read.
      const int ahead = min(S::SB, nt);
#pragma unroll 1
      for (int i = 0; i < ahead && ok; ++i) {
        const uint32_t t = it + i;
        ok = wait(&M.q_full, k & 1, fail) && wait(&M.k_full[t % S::SB], t / S::SB & 1, fail) &&
             (t < S::SB || wait(&M.s_empty[t % S::SB], (t / S::SB - 1) & 1, fail));
        tc_fence_after();
        if (ok) issue_s(t);
      }
#pragma unroll 1
      for (int i = 0; i < nt && ok; ++i) {
        const uint32_t t = it + i, n = t + S::SB;
        const bool more = i + S::SB < nt;
        if (S::SB == 1 && more) {
          ok = wait(&M.k_full[0], n & 1, fail) && wait(&M.s_empty[0], (n - 1) & 1, fail);
          tc_fence_after();
          if (!ok) break;
          issue_s(n);
        }
        ok = wait(&M.p_full[t % S::SB], t / S::SB & 1, fail) && issue_pv(t, i % S::kFar == 0);
        if (S::SB == 2 && more && ok) {
          ok = wait(&M.k_full[n % S::SB], n / S::SB & 1, fail);
          tc_fence_after();
          if (ok) issue_s(n);
        }
      }
      it += nt;
      if (lane == 0) done(k);
      __syncwarp();
    }
    if (!ok) {  // what was issued ends before its operands and tensor memory go
      mma_commit_elect(smem_u32(&M.drain));
      mbar_wait(smem_u32(&M.drain), 0, kAttnWaitLimit);
    }
    __syncwarp();
  } else if (warp >= 4 && warp < kSoftWarp) {
    // ---------------------------------------------------------- dequantisers
    // Two groups (one beside 128-column softmax) take the tiles in turn. Bound by
    // the ALU pipe (a conversion per two elements goes there, so all else is kept
    // off it: rows out of sight point at zeros, addresses are made once).
    const int quarter = warp & 3, tid = threadIdx.x & 127, group = (warp - 4) >> 2;
    const int psh = 31 - __clz(ps);
    constexpr int kKC = DH / 32;        // 32-element chunks of a K row
    constexpr int kD = DH / 2;          // elements of a thread's share of a V row
    const int tt = tid & 63, part = tid >> 6;
    uint32_t vdst[kD >= 64 ? 8 : 4];    // where its 8-element chunks go, in atoms of 64 dimensions
#pragma unroll
    for (int w = 0; w < (kD >= 64 ? 8 : 4); ++w)
      vdst[w] = smem_u32(smem_raw) + S::oV + part * kD / 64 * 8192 + tt * 128 +
                ((((part * kD & 63) / 8 + w) ^ (tt & 7)) << 4);

    // NC chunks of 32 elements and their scales, from one row
    auto load_row = [&](const uint8_t* codes, const uint8_t* scales, auto& code, auto& sc) {
      constexpr int NC = sizeof(code) / 16;
      load_words<4 * NC, S::kRow>(codes, code);
      if constexpr (NC >= 2) load_words<NC / 2, S::kRow>(scales, sc);
      else sc[0] = *reinterpret_cast<const uint16_t*>(scales);
    };
    // one chunk's 32 elements as f16 pairs: code x scale, exact
    auto expand = [](const uint32_t* code, uint32_t scales, uint32_t (&x)[16]) {
      const __half2 s2 = as_half2(e4m3x2_to_f16x2(scales));
      const __half2 lo = __low2half2(s2), hi = __high2half2(s2);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        uint32_t h[4];
        e2m1x8_to_f16(code[w], h);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[4 * w + e] = as_bits(__hmul2(as_half2(h[e]), w < 2 ? lo : hi));
      }
    };

    // position `tid` of tile `i` to tensor memory
    auto deq_k = [&](uint32_t i, const Run& sg, int tile) {
      const int st = i % S::KS;
      const uint32_t b = i % S::SB, round = i / S::SB;
      if (!wait(&M.rawk_full[st], (i / S::KS) & 1, fail)) return false;
      const int t = tile * kT + tid;
      const bool live = t >= sg.lo && t < sg.end && (M.valid_k[st] >> (tid >> psh) & 1);
      const uint8_t* row = live ? base + S::oRawK + st * S::kRaw + tid * S::kRow : M.zero;
      uint32_t code[4 * kKC], sc[(kKC + 1) / 2];
      load_row(row, row + DH / 2, code, sc);
      if (round > 0 && !wait(&M.k_empty[b], (round - 1) & 1, fail)) return false;
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < kKC; ++c) {
        uint32_t x[16];
        expand(code + 4 * c, sc[c / 2] >> (16 * (c & 1)), x);
        tmem_st_rows16(tmem + S::cK + b * S::KC + c * 16 + ((uint32_t)(32 * quarter) << 16), x);
      }
      // (the stage goes back once its words have been used: an arrival right behind
      // the loads does not wait for them, and a copy that hits L2 overtook them)
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&M.rawk_empty[st]));
      tc_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&M.k_full[b]));
      return true;
    };
    // tile `i`'s V in halves of 64 positions; a thread takes half a row
    auto deq_v = [&](uint32_t i, const Run& sg, int tile, uint32_t run) {
      const int st = i % S::VS;
      // 0 x NaN would reach rows that do not see the position: where a tile
      // has such rows, NaN is kept out of the product and noted for the end
      const bool edge = sg.edge(tile, a.window);
      if (!wait(&M.rawv_full[st], (i / S::VS) & 1, fail)) return false;
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        const int tr = h * 64 + tt, t = tile * kT + tr;
        const bool live = t >= sg.lo && t < sg.end && (M.valid_v[st] >> (tr >> psh) & 1);
        const uint8_t* row = live ? base + S::oRawV + st * S::kRaw + tr * S::kRow : M.zero;
        uint32_t code[kD / 8], sc[(kD / 32 + 1) / 2];
        load_row(row + part * (kD / 2), row + DH / 2 + part * (kD / 16), code, sc);
        const uint32_t vs = i % S::VB * 2 + h;
        if (i >= S::VB && !wait(&M.v_empty[(i - S::VB & 1) * 2 + h], (i - S::VB) / 2 & 1, fail)) return false;
        if (edge) {
          // (the words hold the notes of a share whose reader is done: see kNotes)
          const uint32_t set = run % Meta<DH>::kNotes;
          auto& notes = M.nan_bits[set][sg.edge_index(tile)];
          if (lane < kD / 16) notes[part * (kD / 16) + lane][tr >> 5] = 0;
          __syncwarp();
#pragma unroll
          for (int w = 0; w < (kD / 32 + 1) / 2; ++w) {
            uint32_t nan = __vcmpeq4(sc[w] & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
            sc[w] &= ~nan;
            while (nan) {
              const int q = (__ffs(nan) - 1) / 8;
              nan &= ~(0xFFu << (8 * q));
              atomicOr(&notes[part * (kD / 16) + 4 * w + q][tr >> 5], 1u << (tr & 31));
              M.nan_run[set] = run + 1;
            }
          }
        }
        const uint32_t to = vs * (S::kV / 2);
#pragma unroll
        for (int c = 0; c < kD / 32; ++c) {
          uint32_t x[16];
          expand(code + 4 * c, sc[c / 2] >> (16 * (c & 1)), x);
#pragma unroll
          for (int w = 0; w < 4; ++w)
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(vdst[(4 * c + w) & 7] + to + (4 * c + w) / 8 * 8192),
                         "r"(x[4 * w]), "r"(x[4 * w + 1]), "r"(x[4 * w + 2]), "r"(x[4 * w + 3])
                         : "memory");
        }
        if (h == 1) {  // (as K's: after the words' last use)
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&M.rawv_empty[st]));
        }
        fence_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&M.v_full[vs]));
      }
      return true;
    };
    uint32_t it = 0;
    bool ok = true;
    Run s, sv;         // V goes one of the group's tiles behind K
    int tv = -1;
    uint32_t rv = 0, iv = 0;
    s.flags = 0;
#pragma unroll 1
    for (uint32_t k = 0; ok && !(s.flags & 4); ++k) {
      ok = next(k, s);
      __syncwarp();
      if (!ok) break;
#pragma unroll 1
      for (int i = 0; i <= s.nt && ok; ++i) {
        const bool flush = i == s.nt;  // after the last tile, its V
        if (flush ? !(s.flags & 4) : kDq == 2 && (it & 1) != group) {
          it += !flush;
          continue;
        }
        if (!flush) ok = deq_k(it, s, s.tile + i);
        if (tv >= 0 && ok) ok = deq_v(iv, sv, tv, rv);
        sv = s;
        tv = s.tile + i;
        rv = k;
        iv = it;
        it += !flush;
      }
      if (lane == 0) done(k);
      __syncwarp();
    }
  } else if (warp >= kSoftWarp) {
    // ---------------------------------------------------------- softmax
    const int sg = (warp - kSoftWarp) >> 2, quarter = warp & 3, bar = 1 + sg;
    constexpr int NC = S::NC, NB = NC / 8;      // query rows and 8-row blocks of the group
    const int c0 = sg * NC;                     // its first query row (= column)
    const int pr = 2 * (lane & 3);              // the thread's column pair in a block
    const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
    const int G = a.n_q / a.n_kv;
    uint32_t it = 0, run = 0;
    bool ok = true;  // (a warp that fails leaves with its group, at a vote)
    Run s;
    s.flags = 0;
    uint4* const tree = reinterpret_cast<uint4*>(base + S::oTree);
    // whether a position is out of sight of the query of column `col`, whose place is `lim`
    const unsigned w = a.window > 0 ? (unsigned)a.window : 0x80000000u;
    auto hidden = [&](int t, int lim, int col) {
      if constexpr (TREE) {
        const int d = t - s.pos;
        if (d >= 0) return !((unsigned)d < (unsigned)kTreeMost && (reinterpret_cast<const uint32_t*>(&tree[col])[d >> 5] >> (d & 31) & 1));
      }
      return (unsigned)(lim - t) >= w;
    };
#pragma unroll 1
    for (; !(s.flags & 4); ++run) {
      ok = next(run, s);
      if (group_any(bar, !ok)) break;
      if (s.nt == 0) break;
      const int nt = s.nt;
      const bool begins = s.flags & 1, ends = s.flags & 2;
      // ---- queries: eight lanes per row, scaled by a power of two to [2^13, 2^14)
      const int kexp = head_exp(a.k_exp, s.g);
      // all rows' loads first: one trip to memory a share, not one for every 16 rows (one tree of 16 nodes 24.9 us, 25.4 with a trip each)
      constexpr int kTurns = (NC + 15) / 16, kWords = WIDE ? 8 : 4;
      uint32_t raw[kTurns][DH / 64][kWords];
#pragma unroll
      for (int turn = 0; turn < kTurns; ++turn) {
        const int j0 = 4 * quarter + 16 * turn + (lane >> 3), f = s.j * S::RT + c0 + j0, i = f / G, h = s.g * G + f % G;
        const bool real = j0 < NC && f < s.n * G;
        const long long at = (long long)(s.a0 + i) * a.ts + (long long)h * a.hs + (lane & 7) * 8;
#pragma unroll
        for (int k = 0; k < DH / 64; ++k) {
          uint32_t(&u)[kWords] = raw[turn][k];
#pragma unroll
          for (int e = 0; e < kWords; ++e) u[e] = 0u;
          if (real) {
            const uint8_t* p = static_cast<const uint8_t*>(a.q) + (at + 64 * k) * (WIDE ? 4 : 2);
            if (a.q_vec) {
#pragma unroll
              for (int e = 0; e < (WIDE ? 2 : 1); ++e) {
                const uint4 v = reinterpret_cast<const uint4*>(p)[e];
                u[4 * e] = v.x;
                u[4 * e + 1] = v.y;
                u[4 * e + 2] = v.z;
                u[4 * e + 3] = v.w;
              }
            } else if (WIDE) {
#pragma unroll
              for (int e = 0; e < 8; ++e) u[WIDE ? e : 0] = reinterpret_cast<const uint32_t*>(p)[e];
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                u[e] = (uint32_t)reinterpret_cast<const uint16_t*>(p)[2 * e] |
                       ((uint32_t)reinterpret_cast<const uint16_t*>(p)[2 * e + 1] << 16);
            }
          }
        }
      }
      if constexpr (TREE) {  // a thread per query row: its mask and its place
        const int me = threadIdx.x & 127, f = s.j * S::RT + c0 + me, n = s.n;
        if (me < NC) {
          uint4 m = make_uint4(0u, 0u, 0u, 0u);
          int lim = -1;
          if (f < n * G) {
            m = reinterpret_cast<const uint4*>(a.mask)[s.a0 + f / G];
            lim = a.place ? min(max(a.place[s.a0 + f / G], s.pos), s.pos + n - 1) : s.pos + n - 1;
            // bits of nodes that the row does not have
            m.x &= n >= 32 ? ~0u : (1u << n) - 1;
            m.y &= n >= 64 ? ~0u : (n > 32 ? (1u << (n - 32)) - 1 : 0u);
            m.z &= n >= 96 ? ~0u : (n > 64 ? (1u << (n - 64)) - 1 : 0u);
            m.w &= n >= 128 ? ~0u : (n > 96 ? (1u << (n - 96)) - 1 : 0u);
          }
          tree[c0 + me] = m;
          M.lim[c0 + me] = lim;
        }
      }
#pragma unroll
      for (int turn = 0; turn < kTurns; ++turn) {
        const int j0 = 4 * quarter + 16 * turn, j = c0 + j0 + (lane >> 3);
        const bool mine = j0 + (lane >> 3) < NC;
        const int f = s.j * S::RT + j, i = f / G, h = s.g * G + f % G;
        const bool real = mine && f < s.n * G;
        float x[DH / 8];
#pragma unroll
        for (int k = 0; k < DH / 64; ++k)
#pragma unroll
          for (int e = 0; e < 8; ++e)
            x[8 * k + e] = WIDE ? __uint_as_float(raw[turn][k][WIDE ? e : 0])
                                : ((e & 1) ? bf16hi(raw[turn][k][e / 2]) : bf16lo(raw[turn][k][e / 2]));
        float mx = 0.f;
#pragma unroll
        for (int e = 0; e < DH / 8; ++e) mx = fmaxf(mx, fabsf(x[e]));
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
        // the exponent of the largest; an infinity or a NaN stays one (and its
        // row's scores become NaN)
        const int ex = mx > 0.f && mx < INFINITY ? max((int)(__float_as_uint(mx) >> 23) - 127, -107) : 13;
        const float up = pow2i(13 - ex);
        if (mine) {
#pragma unroll
          for (int k = 0; k < DH / 64; ++k) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float y0 = x[8 * k + 2 * e] * up, y1 = x[8 * k + 2 * e + 1] * up;
              hi[e] = pack_f16(y0, y1);
              if (WIDE) {
                const float2 b = f16x2_to_f(hi[e]);
                lo[e] = pack_f16(y0 - b.x, y1 - b.y);
              }
            }
            uint8_t* p = base + S::oQ + k * N * 128 + (((lane & 7) ^ (j & 7)) << 4);
            *reinterpret_cast<uint4*>(p + j * 128) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            if (WIDE) *reinterpret_cast<uint4*>(p + (N / 2 + j) * 128) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          }
          if ((lane & 7) == 0) {
            M.cm[j][0] = ldexpf(a.scale * 1.44269504f, kexp - (13 - ex));
            M.cm[j][1] = kUnset;
            if (!TREE) M.lim[j] = real ? s.pos + i : -1;
            M.dst[j] = real ? (s.a0 + i) * a.n_q + h : -1;
          }
        }
      }
      fence_async();
      group_sync(bar);
      if (lane == 0) mbar_arrive(smem_u32(&M.q_full));

      float sum[2 * NB];
#pragma unroll
      for (int b = 0; b < 2 * NB; ++b) sum[b] = 0.f;

      bool broken = false;
      for (int i = 0; i < nt; ++i, ++it) {
        if (i > 0 && i % S::kFar == 0) {  // the tiles before: P.V of tile i starts O anew
          ok = wait(&M.p_empty[(it - 1) % S::SB], (it - 1) / S::SB & 1, fail) && ok;
          if (group_any(bar, !ok)) { broken = true; break; }
          tc_fence_after();
          add_far<DH, N, WIDE, TREE>(&a, &M, sg, i == S::kFar, false);
        }
        const uint32_t sb = it % S::SB;
        ok = wait(&M.s_full[sb], (it / S::SB) & 1, fail) && ok;
        tc_fence_after();
        const int t0 = (s.tile + i) * kT;
        const bool edge = s.edge(s.tile + i, a.window);
        uint32_t v[2][4 * NB];
        // y = c s - m, the vote, and where some y passes 15 a move of the maxima
        // and y once more (the code is there once: it has to stay in the
        // instruction cache beside the other roles')
#pragma unroll 1
        for (bool moved = false;; moved = true) {
#pragma unroll
          for (int hh = 0; hh < 2; ++hh)
            tmem_ld_frag<NB>(tmem + S::cS + sb * N + c0 + lanes + ((uint32_t)(16 * hh) << 16), v[hh]);
          if (WIDE) {
            uint32_t u[2][4 * NB];
#pragma unroll
            for (int hh = 0; hh < 2; ++hh)
              tmem_ld_frag<NB>(tmem + S::cS + sb * N + c0 + N / 2 + lanes + ((uint32_t)(16 * hh) << 16), u[hh]);
            tc_wait_ld();
#pragma unroll
            for (int hh = 0; hh < 2; ++hh)
#pragma unroll
              for (int e = 0; e < 4 * NB; ++e) {
                pin(v[hh][e]);
                pin(u[hh][e]);
                v[hh][e] = __float_as_uint(__uint_as_float(v[hh][e]) + __uint_as_float(u[hh][e]));
              }
          } else {
            tc_wait_ld();
#pragma unroll
            for (int hh = 0; hh < 2; ++hh)
#pragma unroll
              for (int e = 0; e < 4 * NB; ++e) pin(v[hh][e]);
          }
          float mx = -INFINITY;
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            const float4 cm = *reinterpret_cast<const float4*>(&M.cm[c0 + 8 * b + pr][0]);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t &x0 = v[k >> 1][4 * b + 2 * (k & 1)], &x1 = v[k >> 1][4 * b + 2 * (k & 1) + 1];
              x0 = __float_as_uint(fmaf(__uint_as_float(x0), cm.x, -cm.y));
              x1 = __float_as_uint(fmaf(__uint_as_float(x1), cm.z, -cm.w));
            }
            if (edge) {
              const int2 lim = *reinterpret_cast<const int2*>(&M.lim[c0 + 8 * b + pr]);
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const int t = t0 + 32 * quarter + 8 * k + (lane >> 2);
                uint32_t &x0 = v[k >> 1][4 * b + 2 * (k & 1)], &x1 = v[k >> 1][4 * b + 2 * (k & 1) + 1];
                if (hidden(t, lim.x, c0 + 8 * b + pr)) x0 = 0xFF800000u;  // -inf
                if (hidden(t, lim.y, c0 + 8 * b + pr + 1)) x1 = 0xFF800000u;
              }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mx = fmaxf(mx, fmaxf(__uint_as_float(v[k >> 1][4 * b + 2 * (k & 1)]),
                                   __uint_as_float(v[k >> 1][4 * b + 2 * (k & 1) + 1])));
          }
          if (moved || !group_any(bar, mx > 15.f || !ok)) break;
          if (group_any(bar, !ok)) { broken = true; break; }
          // column maxima of c s over the group's 128 positions
#pragma unroll 1
          for (int b = 0; b < NB; ++b) {
            const float4 cm = *reinterpret_cast<const float4*>(&M.cm[c0 + 8 * b + pr][0]);
            const int2 lim = *reinterpret_cast<const int2*>(&M.lim[c0 + 8 * b + pr]);
            float y0 = -INFINITY, y1 = -INFINITY;
            uint32_t r[2][4], u[2][4];
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
              const uint32_t t = tmem + S::cS + sb * N + c0 + 8 * b + lanes + ((uint32_t)(16 * hh) << 16);
              tmem_ld_frag<1>(t, r[hh]);
              if (WIDE) tmem_ld_frag<1>(t + N / 2, u[hh]);
            }
            tc_wait_ld();
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int t = t0 + 32 * quarter + 8 * k + (lane >> 2), e = 2 * (k & 1);
              pin(r[k >> 1][e]);
              pin(r[k >> 1][e + 1]);
              float z0 = __uint_as_float(r[k >> 1][e]), z1 = __uint_as_float(r[k >> 1][e + 1]);
              if (WIDE) {
                pin(u[k >> 1][e]);
                pin(u[k >> 1][e + 1]);
                z0 += __uint_as_float(u[k >> 1][e]);
                z1 += __uint_as_float(u[k >> 1][e + 1]);
              }
              if (!edge || !hidden(t, lim.x, c0 + 8 * b + pr)) y0 = fmaxf(y0, z0 * cm.x);
              if (!edge || !hidden(t, lim.y, c0 + 8 * b + pr + 1)) y1 = fmaxf(y1, z1 * cm.z);
            }
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
              y0 = fmaxf(y0, __shfl_xor_sync(0xFFFFFFFFu, y0, o));
              y1 = fmaxf(y1, __shfl_xor_sync(0xFFFFFFFFu, y1, o));
            }
            if (lane < 4) *reinterpret_cast<float2*>(&M.red[quarter][c0 + 8 * b + pr]) = make_float2(y0, y1);
          }
          group_sync(bar);
          const int me = threadIdx.x & 127;
          if (me < NC) {
            const int col = c0 + me;
            const float y = fmaxf(fmaxf(M.red[0][col], M.red[1][col]), fmaxf(M.red[2][col], M.red[3][col]));
            const float m = M.cm[col][1];
            float nm = m;
            if (y > -INFINITY && !(y - m <= 15.f)) nm = y - 7.f;
            M.f[col] = nm == m ? 1.f : (m == kUnset ? 0.f : ex2(m - nm));
            M.cm[col][1] = nm;
          }
          group_sync(bar);
          if (i == 0) continue;
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            const float2 f = *reinterpret_cast<const float2*>(&M.f[c0 + 8 * b + pr]);
            sum[2 * b] *= f.x;
            sum[2 * b + 1] *= f.y;
          }
          // O holds tiles before this one: rescale its columns once they are all in
          ok = wait(&M.p_empty[(it - 1) % S::SB], (it - 1) / S::SB & 1, fail);
          if (group_any(bar, !ok)) { broken = true; break; }
          tc_fence_after();
#pragma unroll 1
          for (int q = 0; q < (WIDE ? 2 : 1) * S::MB * NC / 8; ++q) {
            const int c = q % (NC / 8) * 8, mb = q / (NC / 8) % S::MB, part = q / (NC / 8 * S::MB);
            const uint32_t t = tmem + S::cO + mb * N + part * (N / 2) + c0 + c + lanes;
            float o[8];
            tc::tmem_ld8(t, o);
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] *= M.f[c0 + c + e];
            asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::"r"(__float_as_uint(o[0])),
                         "r"(__float_as_uint(o[1])), "r"(__float_as_uint(o[2])), "r"(__float_as_uint(o[3])),
                         "r"(__float_as_uint(o[4])), "r"(__float_as_uint(o[5])), "r"(__float_as_uint(o[6])),
                         "r"(__float_as_uint(o[7])), "r"(t));
          }
          tc_wait_st();
        }
        if (broken) break;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&M.s_empty[sb]));
        // weights, their sums, and P^T once the last tile's P has been read
        uint32_t w[NB][4], wl[WIDE ? NB : 1][4];
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int k = 0; k < 4; ++k) {  // k = 2 hh + e
            const float p0 = ex2(__uint_as_float(v[k >> 1][4 * b + 2 * (k & 1)]));
            const float p1 = ex2(__uint_as_float(v[k >> 1][4 * b + 2 * (k & 1) + 1]));
            sum[2 * b] += p0;
            sum[2 * b + 1] += p1;
            w[b][k] = pack_f16(p0, p1);
            if (WIDE) {
              const float2 h = f16x2_to_f(w[b][k]);
              wl[WIDE ? b : 0][k] = pack_f16(p0 - h.x, p1 - h.y);
            }
          }
        if (it >= S::SB) ok = wait(&M.p_empty[it % S::SB], (it / S::SB - 1) & 1, fail) && ok;
        {
          const int row = lane & 7, mi = lane >> 3;
          const uint32_t p = smem_u32(base + S::oP) + sb * S::kP + (quarter >> 1) * N * 128 + (c0 + row) * 128 +
                             (((4 * (quarter & 1) + mi) ^ row) << 4);
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            stmatrix_x4_t(p + b * 1024, w[b][0], w[b][1], w[b][2], w[b][3]);
            if (WIDE) {
              const int k = WIDE ? b : 0;
              stmatrix_x4_t(p + b * 1024 + N / 2 * 128, wl[k][0], wl[k][1], wl[k][2], wl[k][3]);
            }
          }
        }
        fence_async();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&M.p_full[sb]));
      }
      // ---- the run's share of this (row, head, query tile) is in O
      if (broken) break;
      ok = wait(&M.p_empty[(it - 1) % S::SB], (it - 1) / S::SB & 1, fail) && ok;
      if (group_any(bar, !ok)) break;
      tc_fence_after();
      if (nt > S::kFar) add_far<DH, N, WIDE, TREE>(&a, &M, sg, false, true);
#pragma unroll
      for (int b = 0; b < 2 * NB; ++b) {
        float y = sum[b];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) y += __shfl_xor_sync(0xFFFFFFFFu, y, o);
        if (lane < 4) M.red[quarter][c0 + 8 * (b >> 1) + pr + (b & 1)] = y;
      }
      group_sync(bar);
      const bool whole = begins && ends;
      const int slot = 2 * blockIdx.x + (begins ? 1 : 0);
      const int me = threadIdx.x & 127;
      if (me < NC) {
        const int col = c0 + me;
        const float l = M.red[0][col] + M.red[1][col] + M.red[2][col] + M.red[3][col];
        const float m = M.cm[col][1];
        if (whole) {
          M.f[col] = l != 0.f ? pow2i(head_exp(a.v_exp, s.g)) * __frcp_rn(l) : 0.f;
          if (a.lse && M.dst[col] >= 0) a.lse[M.dst[col]] = l != 0.f ? (m + __log2f(l)) * 0.693147181f : -INFINITY;
        } else {
          a.part_ml[(long long)slot * S::RT + col] = make_float2(m, l);
        }
      }
      if (!whole && sg == 0 && me == 0)
        a.part_meta[slot] = make_int4(s.r, s.g, s.j, begins ? s.last : -1);
      group_sync(bar);
      constexpr int kOut = NC < 16 ? 8 : 16;  // columns of O at a time
      auto load_o = [](uint32_t t, float* o) {
        if constexpr (kOut == 8) tc::tmem_ld8(t, o);
        else tc::tmem_ld16(t, o);
      };
      auto put = [](void* out, long long at, float y) {
        if (WIDE) static_cast<float*>(out)[at] = y;
        else static_cast<__nv_bfloat16*>(out)[at] = __float2bfloat16_rn(y);
      };
      if (DH > 64 || quarter < 2) {
#pragma unroll 1
        for (int mb = 0; mb < S::MB; ++mb)
#pragma unroll 1
          for (int c = 0; c < NC; c += kOut) {
            float o[kOut];
            load_o(tmem + S::cO + mb * N + c0 + c + lanes, o);
            if (WIDE) {
              float o2[kOut];
              load_o(tmem + S::cO + mb * N + N / 2 + c0 + c + lanes, o2);
#pragma unroll
              for (int e = 0; e < kOut; ++e) o[e] += o2[e];
            }
            const int d = mb * 128 + 32 * quarter + lane;
            const uint32_t set = run % Meta<DH>::kNotes;
            if (M.nan_run[set] == run + 1) {
              uint32_t nan = 0;
#pragma unroll 1
              for (int e = 0; e < kOut; ++e)
                nan |= (uint32_t)sees_nan<DH / 16, TREE>(s.first, s.tile, nt, s.p0, s.p1, M.nan_bits[set], d / 16,
                                                         M.lim[c0 + c + e], a.window,
                                                         TREE ? reinterpret_cast<const uint32_t*>(&tree[c0 + c + e]) : nullptr,
                                                         s.pos, s.n) << e;
#pragma unroll
              for (int e = 0; e < kOut; ++e)
                if (nan >> e & 1) o[e] = __int_as_float(0x7FC00000);
            }
            if (whole) {
#pragma unroll
              for (int e = 0; e < kOut; ++e) {
                const int dst = M.dst[c0 + c + e];
                if (dst >= 0) put(a.out, (long long)dst * DH + d, o[e] * M.f[c0 + c + e]);
              }
            } else {
              float* p = a.part_o + ((long long)slot * S::RT + c0 + c) * DH + d;
#pragma unroll
              for (int e = 0; e < kOut; ++e) p[e * DH] = o[e];
            }
          }
      }
      tc_fence_before();
      group_sync(bar);
      if (lane == 0) done(run);
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (threadIdx.x == 0) {
    if (M.fail) {
      flag_status(a.status, MTP_ERR_TIMEOUT);
      // let copies still in flight land before the shared memory is released
      for (uint32_t i = 0; i < (uint32_t)S::KS && i < M.copied[0]; ++i)
        mbar_wait(smem_u32(&M.rawk_full[i]), ((M.copied[0] - 1 - i) / S::KS) & 1, kAttnWaitLimit);
      for (uint32_t i = 0; i < (uint32_t)S::VS && i < M.copied[1]; ++i)
        mbar_wait(smem_u32(&M.rawv_full[i]), ((M.copied[1] - 1 - i) / S::VS) & 1, kAttnWaitLimit);
    }
  }
  __syncthreads();
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(S::kCols) : "memory");
}

template <int DH, int N, bool WIDE, bool TREE>
cudaError_t launch_q4_attn_t(const Q4AttnArgs& a, int blocks, cudaStream_t s) {
  using S = Shape<DH, N, WIDE, TREE>;
  auto k = k_q4_attn<DH, N, WIDE, TREE>;
  {
    // the dynamic shared memory limit, raised once per device
    static std::mutex mu;
    static bool set[kMaxDevices] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= kMaxDevices) dev = 0;
    std::lock_guard<std::mutex> lock(mu);
    if (!set[dev]) {
      const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
      if (e != cudaSuccess) {
        cudaGetLastError();
        return e;
      }
      set[dev] = true;
    }
  }
  count_launch();
  return launch_pdl(k, dim3(blocks), dim3(kAttnThreads), (size_t)S::kSmem, s, a);
}

template <int DH, bool TREE>
cudaError_t launch_q4_attn(const Q4AttnArgs& a, int n, bool wide, int blocks, cudaStream_t s) {
  if (wide) {
    if (n == 16) return launch_q4_attn_t<DH, 16, true, TREE>(a, blocks, s);
    if (n == 32) return launch_q4_attn_t<DH, 32, true, TREE>(a, blocks, s);
    return launch_q4_attn_t<DH, 64, true, TREE>(a, blocks, s);
  }
  if (n == 16) return launch_q4_attn_t<DH, 16, false, TREE>(a, blocks, s);
  if (n == 32) return launch_q4_attn_t<DH, 32, false, TREE>(a, blocks, s);
  if (n == 64) return launch_q4_attn_t<DH, 64, false, TREE>(a, blocks, s);
  return launch_q4_attn_t<DH, 128, false, TREE>(a, blocks, s);
}

// One head dimension's kernels each, blocks of positions and trees (their own translation units).
cudaError_t launch_q4_attn_64(const Q4AttnArgs& a, int n, bool wide, int blocks, cudaStream_t s);
cudaError_t launch_q4_attn_128(const Q4AttnArgs& a, int n, bool wide, int blocks, cudaStream_t s);
cudaError_t launch_q4_attn_256(const Q4AttnArgs& a, int n, bool wide, int blocks, cudaStream_t s);
cudaError_t launch_q4_tree_64(const Q4AttnArgs& a, int n, bool wide, int blocks, cudaStream_t s);
cudaError_t launch_q4_tree_128(const Q4AttnArgs& a, int n, bool wide, int blocks, cudaStream_t s);
cudaError_t launch_q4_tree_256(const Q4AttnArgs& a, int n, bool wide, int blocks, cudaStream_t s);

}  // namespace mtp
