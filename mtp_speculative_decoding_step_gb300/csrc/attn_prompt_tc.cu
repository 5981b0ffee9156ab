// kv_attend_prompt for bf16 on the 5th-generation tensor cores.
//
//   S[128 queries][128 keys] = Q . K^T       Q, K in shared memory
//   O[128 queries][DH]      += P . V         P = 2^(c s - m) in tensor memory, V in shared memory
//
// The query rows of one KV head are taken position-major (row f is position f / G,
// head f % G of the G that share the KV head), 256 of them to a unit, which reads
// its keys once: two query tiles of 128 in one block (DH <= 128), or one each in the
// two blocks of a cluster (DH = 256, where O takes half of tensor memory), which
// copy half of every tile each, to both. 12 warps:
//   warps 0-7   softmax: two groups of 128 threads, thread = query row. An item is a
//               query tile's 128 keys; items alternate between two places for S in
//               tensor memory, group s has place s. With two query tiles a group has
//               a tile of its own; with one, the groups take the keys in turn and
//               hand the running maximum on
//   warp 8      copies (TMA) K and V tiles through a ring in the order of their use
//   warp 9      issues the MMAs: S of item k + 2 behind P.V of item k
//   warps 10-11 clean V where some query of the unit does not see a position: 0
//               times what stands there has to be 0
// P is written as bf16 over its S (the tensor core reads it from there), off by at
// most 2^-8 of each weight; their sum is taken of the fp32 weights. The running maximum is
// lazy: O is rescaled only when a row's maximum has grown by 2^8, by the warp whose
// rows they are. Every wait is bounded: on expiry the block raises the status
// word, waits for its copies, frees its tensor memory and returns.
#include <algorithm>
#include <cfloat>
#include <mutex>

#include "attn_prompt.h"
#include "kernels.h"
#include "prompt_tiles.h"
#include "tc_attn.cuh"

namespace mtp {

namespace {

constexpr int kPromptThreads = 384;
constexpr int kUnit = 256;  // query rows that share their keys

// A warp's 32 rows (lane = row) of 32 columns.
__device__ __forceinline__ void tmem_ld_rows32(uint32_t t, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(t));
}

__device__ __forceinline__ void tmem_st_rows32(uint32_t t, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]),
      "r"(t)
      : "memory");
}

__device__ __forceinline__ void st_shared16(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// A box of a tensor (head dimension, head, position) to this block's shared memory, or to both blocks' of the cluster.
template <int CL>
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, int x, int head, int pos, uint32_t bar) {
  if constexpr (CL == 1) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"((uint64_t)map), "r"(x), "r"(head), "r"(pos), "r"(bar)
        : "memory");
  } else {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.multicast::cluster [%0], [%1, {%2, %3, %4}], [%5], "
        "%6;" ::"r"(dst),
        "l"((uint64_t)map), "r"(x), "r"(head), "r"(pos), "r"(bar), "h"((uint16_t)3)
        : "memory");
  }
}

// Arrives on the barrier at this place in this block, or in both blocks of the cluster, when the MMAs issued so far are done.
template <int CL>
__device__ __forceinline__ void commit_all(uint32_t bar) {
  if constexpr (CL == 1) {
    mma_commit_elect(bar);
  } else {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
  }
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// bf16 A and B, fp32 accumulators; `b_mn`: B is N-major
__host__ __device__ constexpr uint32_t idesc_bf(int m, int n, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

template <int DH>
struct PromptShape {
  static constexpr int QT = DH == 256 ? 1 : 2;    // query tiles of a block
  static constexpr int CL = DH == 256 ? 2 : 1;    // blocks of a unit
  static constexpr int CPT = DH == 256 ? 2 : 1;   // ring stages of a tile of K or V
  static constexpr int NS = DH == 64 ? 8 : 5;     // ring stages
  static constexpr int kQ = QT * 128 * DH * 2, kStage = 128 * DH * 2 / CPT;
  static constexpr int oRing = kQ, oMeta = oRing + NS * kStage;
  static constexpr int kMeta = 2048, kSmem = oMeta + kMeta;
  static constexpr uint32_t cS = 0, cO = 256;     // columns of tensor memory: S at 0 and 128, O from 256 on
  static_assert(kSmem <= 227 * 1024, "shared memory");
  // stages of K of tile j, and of V, in the order of their use: S of the first item(s), then P.V of item k and S of item k + 2
  __device__ static int k_at(int j) { return (DH == 256 ? j + max(0, j - 1) : 2 * j) * CPT; }
  __device__ static int v_at(int j, int nt) { return (DH == 256 ? min(j + 2, nt) + j : 2 * j + 1) * CPT; }
};

struct PromptMeta {
  uint64_t full[8], empty[8], s_full[2], p_full[2], pv_done[2], m_full[2][4], q_full, v_go, v_ok, drain;
  uint32_t tmem, copied;
  int fail, nan;
  int unit[4];   // first packed position of the row, its positions, the unit's first query row
  float m[128];  // one query tile: the running maxima
};
static_assert(sizeof(PromptMeta) <= 2048, "meta");

template <int DH>
__global__ void __launch_bounds__(kPromptThreads, 1)
    k_prompt_tc(const __grid_constant__ PromptArgs a, const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv) {
  using S = PromptShape<DH>;
  constexpr int CL = S::CL;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  auto& M = *reinterpret_cast<PromptMeta*>(smem_raw + S::oMeta);
  const uint32_t sm = smem_u32(smem_raw);
  const int warp = __shfl_sync(0xFFFFFFFFu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int G = a.n_q / a.n_kv, rank = CL == 1 ? 0 : (int)(blockIdx.x & 1), x = blockIdx.x / CL, g = x % a.n_kv;
  volatile int* fail = &M.fail;
  auto wait_all = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xFFFFFFFFu, wait(bar, parity, fail)) != 0; };

  if (threadIdx.x == 32) {
    for (int i = 0; i < 8; ++i) {
      mbar_init(smem_u32(&M.full[i]), 1);
      mbar_init(smem_u32(&M.empty[i]), CL);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&M.s_full[i]), 1);
      mbar_init(smem_u32(&M.p_full[i]), 4);
      mbar_init(smem_u32(&M.pv_done[i]), 1);
      for (int w = 0; w < 4; ++w) mbar_init(smem_u32(&M.m_full[i][w]), 1);
    }
    mbar_init(smem_u32(&M.q_full), 8);
    mbar_init(smem_u32(&M.v_go), 1);
    mbar_init(smem_u32(&M.v_ok), 2);
    mbar_init(smem_u32(&M.drain), 1);
    M.fail = M.nan = 0;
    M.copied = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  pdl_wait();
  if (warp == 0) {
    int a0 = 0, n = 0, j = 0;
    const bool some = find_tile(a, G, kUnit, x / a.n_kv, a0, n, j);
    if (lane == 0) {
      M.unit[0] = a0;
      M.unit[1] = some ? n : 0;
      M.unit[2] = j * kUnit;
    }
  }
  __syncthreads();
  const int a0 = M.unit[0], n = M.unit[1], f0 = M.unit[2];
  if (n == 0) return;  // (both blocks of a cluster)
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&M.tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  if (CL > 1) cluster_sync();  // the other block's barriers are there
  tc_fence_after();
  pdl_trigger();  // (with tensor memory in hand: a dependent kernel may take what is left of it before it waits for this one)
  const uint32_t tmem = M.tmem;
  // positions of the unit's first and last query row, and its tiles of 128 keys
  const int p0 = f0 / G, p1 = (min(n * G, f0 + kUnit) - 1) / G;
  const int t_first = a.window > 0 ? max(0, p0 - (a.window - 1)) / 128 : 0, nt = p1 / 128 + 1 - t_first;
  const int items = nt * S::QT;
  // whether some query of rows at positions q0 to q1 does not see some position of a tile
  auto edge = [&](int j, int q0, int q1) {
    const int t0 = (t_first + j) * 128;
    return t0 + 127 > q0 || (a.window > 0 && t0 <= q1 - a.window);
  };

  if (warp == 8) {
    // ---------------------------------------------------------- copies
    if (lane == 0) {
      int at = 0;
      bool ok = true;
      auto tile = [&](const CUtensorMap* map, int j, bool is_v) {
#pragma unroll 1
        for (int c = 0; c < S::CPT && ok; ++c, ++at) {
          const int st = at % S::NS, round = at / S::NS;
          if (round > 0 && !(ok = wait(&M.empty[st], (round - 1) & 1, fail))) return;
          const uint32_t bar = smem_u32(&M.full[st]), dst = sm + S::oRing + st * S::kStage;
          mbar_expect_tx(bar, S::kStage);
          M.copied = at + 1;
          const int pos = a0 + (t_first + j) * 128;
          if constexpr (DH == 256) {
            // K: 128 positions of half the dimensions; V: 64 positions of all. Half of it from each block
            if (!is_v) {
              tma_box<CL>(dst + rank * 16384, map, (2 * c + rank) * 64, g, pos, bar);
            } else {
              for (int b = 2 * rank; b < 2 * rank + 2; ++b) tma_box<CL>(dst + b * 8192, map, b * 64, g, pos + 64 * c, bar);
            }
          } else {
            for (int b = 0; b < DH / 64; ++b) tma_box<CL>(dst + b * 16384, map, b * 64, g, pos, bar);
          }
        }
      };
      if (DH == 256) {
        tile(&mk, 0, false);
        if (nt > 1) tile(&mk, 1, false);
        for (int j = 0; j < nt && ok; ++j) {
          tile(&mv, j, true);
          if (j + 2 < nt) tile(&mk, j + 2, false);
        }
      } else {
        for (int j = 0; j < nt && ok; ++j) {
          tile(&mk, j, false);
          tile(&mv, j, true);
        }
      }
      // the last arrivals on this block's barriers, the other block's among them
      for (int i = max(0, at - S::NS); i < at && ok; ++i) ok = wait(&M.empty[i % S::NS], i / S::NS & 1, fail);
    }
    __syncwarp();
  } else if (warp == 9) {
    // ---------------------------------------------------------- MMAs
    constexpr uint32_t idS = idesc_bf(128, 128, false), idO = idesc_bf(128, DH, true);
    const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
    const uint64_t dq = tc::sdesc(sm);
    int edges = 0;  // tiles whose V was cleaned
    bool ok = wait_all(&M.q_full, 0);
    auto issue_s = [&](int k) {
      const int j = S::QT == 2 ? k >> 1 : k, slot = k & 1, at = S::k_at(j);
#pragma unroll 1
      for (int c = 0; c < S::CPT; ++c) {
        const int st = (at + c) % S::NS;
        if (!wait_all(&M.full[st], (at + c) / S::NS & 1)) return false;
        tc_fence_after();
        const uint64_t dk = tc::sdesc(sm + S::oRing + st * S::kStage);
        const uint64_t da = dq + (S::QT == 2 ? slot * (128 * DH * 2 / 16) : 0) + c * (DH / S::CPT / 64) * 1024;
#pragma unroll
        for (int e = 0; e < DH / S::CPT / 16; ++e)
          mma_f16_ss(tm + S::cS + slot * 128, da + (e >> 2) * 1024 + (e & 3) * 2, dk + (e >> 2) * 1024 + (e & 3) * 2, idS,
                        (c | e) > 0 ? 1u : 0u);
        if (S::QT == 1 || slot == 1) commit_all<CL>(smem_u32(&M.empty[st]));
      }
      mma_commit_elect(smem_u32(&M.s_full[slot]));
      return true;
    };
    auto issue_pv = [&](int k) {
      const int j = S::QT == 2 ? k >> 1 : k, slot = k & 1, at = S::v_at(j, nt);
      const bool first = S::QT == 1 || slot == 0, clean = first && edge(j, p0, p1);
      if (first) {
#pragma unroll 1
        for (int c = 0; c < S::CPT; ++c)
          if (!wait_all(&M.full[(at + c) % S::NS], (at + c) / S::NS & 1)) return false;
        if (clean && lane == 0) mbar_arrive(smem_u32(&M.v_go));
        __syncwarp();
      }
      if (!wait_all(&M.p_full[slot], k >> 1 & 1)) return false;
      if (clean && !wait_all(&M.v_ok, edges++ & 1)) return false;
      tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < S::CPT; ++c) {
        const int st = (at + c) % S::NS;
        const uint64_t dv = sdesc_mn(sm + S::oRing + st * S::kStage, 16384 / S::CPT);
#pragma unroll
        for (int e = 0; e < 8 / S::CPT; ++e)
          mma_f16_ts(tm + S::cO + (S::QT == 2 ? slot * DH : 0), tm + S::cS + slot * 128 + (c * (8 / S::CPT) + e) * 8, dv + e * 128, idO,
                        k >= S::QT || (c | e) > 0 ? 1u : 0u);
        if (S::QT == 1 || slot == 1) commit_all<CL>(smem_u32(&M.empty[st]));
      }
      mma_commit_elect(smem_u32(&M.pv_done[slot]));
      return true;
    };
    ok = ok && issue_s(0);
    if (items > 1) ok = ok && issue_s(1);
#pragma unroll 1
    for (int k = 0; k < items && ok; ++k) {
      ok = issue_pv(k);
      if (ok && k + 2 < items) ok = issue_s(k + 2);
    }
    // what was issued ends before its operands and tensor memory go
    mma_commit_elect(smem_u32(&M.drain));
    mbar_wait(smem_u32(&M.drain), 0, kAttnWaitLimit);
    __syncwarp();
  } else if (warp >= 10) {
    // ---------------------------------------------------------- V of edge tiles
    const int me = threadIdx.x - 320;
    constexpr int kSegs = DH / 8;  // 16-byte pieces of a position
    int edges = 0;
#pragma unroll 1
    for (int j = 0; j < nt; ++j) {
      if (!edge(j, p0, p1)) continue;
      // (told by the MMA warp, which has seen all stages of the ring in turn)
      if (!wait_all(&M.v_go, edges++ & 1)) break;
      const int t0 = (t_first + j) * 128, at = S::v_at(j, nt);
#pragma unroll 1
      for (int c = 0; c < S::CPT; ++c) {
        const int st = (at + c) % S::NS;
        const uint32_t base = sm + S::oRing + st * S::kStage;
        constexpr int kRows = 128 / S::CPT;
        // positions that all queries of the unit see lie between those that some do not
        for (int i = me; i < kRows * kSegs; i += 64) {
          const int r = i / kSegs, e = i % kSegs, t = t0 + c * kRows + r;
          if (t <= p0 && (a.window == 0 || t > p1 - a.window)) continue;
          const uint32_t addr = base + (e >> 3) * (kRows * 128) + r * 128 + (e & 7) * 16;
          if (t > p1 || (a.window > 0 && t <= p0 - a.window)) {
            st_shared16(addr, make_uint4(0u, 0u, 0u, 0u));
            continue;
          }
          uint4 v;
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
          uint32_t w[4] = {v.x, v.y, v.z, v.w}, bad = 0;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint32_t lo = (w[q] & 0x7F80u) == 0x7F80u ? 0xFFFFu : 0u, hi = (w[q] & 0x7F800000u) == 0x7F800000u ? 0xFFFF0000u : 0u;
            bad |= lo | hi;
            w[q] &= ~(lo | hi);
          }
          if (bad) {
            M.nan = 1;
            st_shared16(addr, make_uint4(w[0], w[1], w[2], w[3]));
          }
        }
      }
      fence_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&M.v_ok));
    }
  } else {
    // ---------------------------------------------------------- softmax
    const int slot = warp >> 2, quarter = warp & 3, row = threadIdx.x & 127;
    const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
    const int fq = f0 + (CL == 2 ? rank : slot) * 128;  // the query tile's first row
    // ---- queries to swizzled shared memory, negated for a negative scale
    {
      constexpr int kPer = DH / 8;                       // 16-byte pieces of a row
      const uint32_t flip = a.scale < 0.f ? 0x80008000u : 0u;
      const int r0 = S::QT == 2 ? 32 * quarter : 16 * warp, rows = S::QT == 2 ? 32 : 16;
#pragma unroll 4
      for (int i = lane; i < rows * kPer; i += 32) {
        const int r = r0 + i / kPer, e = i % kPer, f = fq + r;
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (f < n * G) {
          const int p = f / G, h = g * G + f - p * G;
          v = ld_stream(static_cast<const uint16_t*>(a.q) + (long long)(a0 + p) * a.ts[0] + (long long)h * a.hs[0] + 8 * e);
          v.x ^= flip, v.y ^= flip, v.z ^= flip, v.w ^= flip;
        }
        st_shared16(sm + (S::QT == 2 ? slot * 128 * DH * 2 : 0) + (e >> 3) * 16384 + r * 128 + (((e & 7) ^ (r & 7)) << 4), v);
      }
      fence_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&M.q_full));
    }
    const int f = fq + row;
    const bool real = f < n * G;
    const int pos = real ? f / G : -1;
    const int q0 = fq / G, q1 = (min(n * G, fq + 128) - 1) / G;
    const unsigned win = a.window > 0 ? (unsigned)a.window : 0x80000000u;
    // (above 0: -inf times 0 would be no weight)
    const float c = fmaxf(fabsf(a.scale) * 1.44269504f, FLT_MIN);
    float m = -INFINITY, l = 0.f;
    bool ok = true;
#pragma unroll 1
    for (int k = slot; k < items; k += 2) {
      const int j = S::QT == 2 ? k >> 1 : k;
      ok = wait_all(&M.s_full[slot], k >> 1 & 1);
      if (!ok) break;
      tc_fence_after();
      uint32_t s[128];
#pragma unroll
      for (int q = 0; q < 4; ++q) tmem_ld_rows32(tmem + S::cS + slot * 128 + 32 * q + lanes, s + 32 * q);
      tc_wait_ld();
#pragma unroll
      for (int e = 0; e < 128; ++e) pin(s[e]);
      if (edge(j, q0, q1)) {
        const int rel = pos - (t_first + j) * 128;
#pragma unroll
        for (int e = 0; e < 128; ++e)
          if ((unsigned)(rel - e) >= win) s[e] = 0xFF800000u;  // -inf: out of sight
      }
      float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int e = 0; e < 128; e += 4)
#pragma unroll
        for (int q = 0; q < 4; ++q) mx[q] = fmaxf(mx[q], __uint_as_float(s[e + q]));
      const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
      // the maximum so far; one that moves takes O with it
      float was = m;
      if (S::QT == 1 && k > 0) {
        ok = wait_all(&M.m_full[slot ^ 1][quarter], (k - 1) >> 1 & 1);
        if (!ok) break;
        was = M.m[row];
      }
      const float now = top > was + 8.f || was == -INFINITY ? fmaxf(top, was) : was;
      if (S::QT == 1) {
        M.m[row] = now;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&M.m_full[slot][quarter]));
      }
      const bool moved = now != was && was != -INFINITY;
      if (now != m) l = m == -INFINITY ? 0.f : l * ex2(m - now);
      m = now;
      if (__any_sync(0xFFFFFFFFu, moved)) {
        if (S::QT == 1) {  // (with a tile of its own, S of this item came behind P.V of the last)
          ok = wait_all(&M.pv_done[slot ^ 1], (k - 1) >> 1 & 1);
          if (!ok) break;
          tc_fence_after();
        }
        const float fac = moved ? ex2(was - now) : 1.f;
#pragma unroll 1
        for (int d = 0; d < DH; d += 16) {
          const uint32_t t = tmem + S::cO + (S::QT == 2 ? slot * DH : 0) + d + lanes;
          float o[16];
          tc::tmem_ld16(t, o);
          uint32_t u[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) u[e] = __float_as_uint(o[e] * fac);
          tmem_st_rows16(t, u);
        }
      }
      const float base = m == -INFINITY ? 0.f : m;
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t w[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const float u = ex2(fmaf(__uint_as_float(s[64 * h + 2 * e]), c, -base)), v = ex2(fmaf(__uint_as_float(s[64 * h + 2 * e + 1]), c, -base));
          sum[e & 1] += u;
          sum[2 + (e & 1)] += v;
          w[e] = pack_bf16(u, v);
        }
        tmem_st_rows32(tmem + S::cS + slot * 128 + 32 * h + lanes, w);
      }
      l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
      tc_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&M.p_full[slot]));
    }
    // ---- O of this query tile
    int c0 = 0, cn = DH;
    if (ok) {
      const int last = S::QT == 2 ? items - 2 + slot : items - 1;
      // (in turn: a parity tells only neighbouring phases apart)
      ok = (last < 2 || wait_all(&M.pv_done[last & 1], ((last >> 1) - 1) & 1)) && wait_all(&M.pv_done[last & 1], last >> 1 & 1);
      tc_fence_after();
    }
    if (S::QT == 1) {  // the groups' sums, then half of the dimensions each
      float2* ml = reinterpret_cast<float2*>(smem_raw);  // (Q has been read)
      ml[slot * 128 + row] = make_float2(m, l);
      asm volatile("barrier.cta.sync.aligned 1, 256;" ::: "memory");
      const float2 o = ml[(slot ^ 1) * 128 + row];
      const float top = fmaxf(m, o.x);
      l = (m == -INFINITY ? l : l * ex2(m - top)) + (o.x == -INFINITY ? o.y : o.y * ex2(o.x - top));
      m = top;
      c0 = slot * (DH / 2);
      cn = DH / 2;
    }
    if (ok) {
      const float r = l != 0.f ? 1.f / l : 0.f;
      const long long dst = real ? (long long)(a0 + pos) * a.n_q + g * G + (f - pos * G) : 0;
      if (real && a.lse && c0 == 0) a.lse[dst] = l != 0.f ? (m + log2f(l)) * 0.693147181f : -INFINITY;
      const bool nan = *reinterpret_cast<volatile int*>(&M.nan) != 0;
#pragma unroll 1
      for (int d = c0; d < c0 + cn; d += 32) {
        uint32_t o[32];
        tmem_ld_rows32(tmem + S::cO + (S::QT == 2 ? slot * DH : 0) + d + lanes, o);
        tc_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          pin(o[e]);
          o[e] = l != 0.f ? __float_as_uint(__uint_as_float(o[e]) * r) : 0u;
        }
        if (nan && real) {  // what was cleaned out of V and this query sees
          const int lo = a.window > 0 ? max(0, pos - (a.window - 1)) : 0;
#pragma unroll 1
          for (int t = lo; t <= pos; ++t) {
            if (t <= p0 && (a.window == 0 || t > p1 - a.window)) {
              t = p0;  // (all queries of the unit see it and what follows up to here: V was left as it was)
              continue;
            }
            const uint16_t* v = static_cast<const uint16_t*>(a.v) + (long long)(a0 + t) * a.ts[2] + (long long)g * a.hs[2] + d;
#pragma unroll 1
            for (int q = 0; q < 32; ++q) {
              const float y = bf16_to_f(v[q]);
              if (isfinite(y)) continue;
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (e == q) o[e] = __float_as_uint(__uint_as_float(o[e]) + y);
            }
          }
        }
        if (real) {
          uint4* p = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + dst * DH + d);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t u[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) u[q] = pack_bf16(__uint_as_float(o[8 * e + 2 * q]), __uint_as_float(o[8 * e + 2 * q + 1]));
            p[e] = make_uint4(u[0], u[1], u[2], u[3]);
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && M.fail) {
    flag_status(a.status, MTP_ERR_TIMEOUT);
    // let copies still in flight land before the shared memory is released
    for (uint32_t i = 0; i < (uint32_t)S::NS && i < M.copied; ++i)
      mbar_wait(smem_u32(&M.full[(M.copied - 1 - i) % S::NS]), ((M.copied - 1 - i) / S::NS) & 1, kAttnWaitLimit);
  }
  __syncthreads();
  if (CL > 1) cluster_sync();  // the other block's copies and arrivals end here too
  tc_fence_after();
  if (warp == 0) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

// K or V as (head dimension, head, position), boxes of 64 x 1 x `rows`.
bool head_map(CUtensorMap* m, const void* p, int dh, int heads, int tokens, long long hs, long long ts, int rows) {
  auto enc = tc::get_encode();
  if (!enc) return false;
  cuuint64_t dims[3] = {(cuuint64_t)dh, (cuuint64_t)heads, (cuuint64_t)tokens};
  // (the stride of a dimension of one is any that the encoder takes)
  cuuint64_t strides[2] = {(cuuint64_t)(heads > 1 ? hs : dh) * 2, (cuuint64_t)(tokens > 1 ? ts : (long long)dh * heads) * 2};
  cuuint32_t box[3] = {64, 1, (cuuint32_t)rows}, one[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DH>
cudaError_t launch(const PromptArgs& a, cudaStream_t s) {
  using S = PromptShape<DH>;
  CUtensorMap mk, mv;
  if (!head_map(&mk, a.k, DH, a.n_kv, a.tokens, a.hs[1], a.ts[1], 128) ||
      !head_map(&mv, a.v, DH, a.n_kv, a.tokens, a.hs[2], a.ts[2], DH == 256 ? 64 : 128))
    return cudaErrorInvalidValue;
  static std::mutex mu;
  static bool set[kMaxDevices] = {};
  {
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= kMaxDevices) dev = 0;
    std::lock_guard<std::mutex> lock(mu);
    if (!set[dev]) {
      const cudaError_t e = cudaFuncSetAttribute(k_prompt_tc<DH>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
      if (e != cudaSuccess) {
        cudaGetLastError();
        return e;
      }
      set[dev] = true;
    }
  }
  const int G = a.n_q / a.n_kv;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(prompt_most_tiles(a.tokens, a.rows, G, kUnit) * a.n_kv * S::CL));
  cfg.blockDim = dim3(kPromptThreads);
  cfg.dynamicSmemBytes = S::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = S::CL;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = S::CL > 1 ? 2 : 1;
  count_launch();
  return cudaLaunchKernelEx(&cfg, k_prompt_tc<DH>, a, mk, mv);
}

}  // namespace

cudaError_t launch_prompt_tc(const PromptArgs& a, int head_dim, cudaStream_t s) {
  return head_dim == 64 ? launch<64>(a, s) : (head_dim == 128 ? launch<128>(a, s) : launch<256>(a, s));
}

}  // namespace mtp
