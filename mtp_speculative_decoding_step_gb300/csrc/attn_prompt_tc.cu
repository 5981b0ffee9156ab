// kv_attend_prompt for bf16 on the 5th-generation tensor cores.
//
//   S[128 queries][128 keys] = Q . K^T       Q, K in shared memory
//   O[128 queries][DH]      += P . V         P = 2^(c s - m) in tensor memory, V in shared memory
//
// The query rows of the heads that share a KV head are taken position-major, a
// query tile being as many whole positions as 128 rows hold. A block takes a unit of
// two query tiles, which reads its keys once, or of one (DH = 256, where O takes half
// of tensor memory). Blocks stay and take units in turn, the longest first. 12 warps:
//   warps 0-7   softmax: two groups of 128 threads, thread = query row. An item is a
//               query tile's 128 keys; items alternate between two places for S in
//               tensor memory, group s has place s. With two query tiles a group has
//               a tile of its own; with one, the groups take the keys in turn and
//               hand the running maximum on
//   warp 8      finds the units; copies (TMA) Q, and K and V through a ring in the order
//               of their use
//   warp 9      issues the MMAs: S of item k + 2 behind P.V of item k
//   warps 10-11 clean V of what is not finite where some query of the unit does not see
//               a position: 0 times it has to be 0. (What such queries do see of it is
//               added at the end.)
// P is written as bf16 over its S (the tensor core reads it from there), off by at
// most 2^-8 of each weight; their sum is taken of the fp32 weights. The running maximum is
// lazy: O is rescaled only when a row's maximum has grown by 2^8, by the warp whose
// rows they are. Every wait is bounded: on expiry the block raises the status
// word, waits for its copies, frees its tensor memory and returns.
//
// Each block copies its own tiles, from L2 where another has the same. Two blocks of 256 dimensions that shared a unit's
// keys, half of each tile copied by either to both, took 484 us where this takes 500 (24 heads on 4, 8192 positions), 330
// where it takes 361 (8 prompts of 2048), and 80 where it takes 72 (64 of 128); but such copies have to stay within one
// GPU's memory, which a call here says nothing about.
//
// What it measured: 8192 positions of 24 heads on 4 of 256 500 us, 1.65 PFLOP/s; of 32 on 8 of 128 311 us, 1.77 PFLOP/s; of
// 32 on 4 of 64 278 us, 0.99 PFLOP/s; seconds of such calls run at the power limit, 256 dimensions at 1760 MHz 545 us. The
// tensor pipe is active 77 % (256 dimensions), shared memory 79 % on its side: S reads 8 KB an MMA of 64 cycles and the
// copies write as much again; L2 55 %. With 64 dimensions the softmax is longer than the products. Short prompts wait on one
// query tile's chain: with 512 positions of 128 dimensions a unit is 18,500 cycles, of which the MMAs take 5300; the softmax
// of its 2.6 items 6700, waits for S between them 2500, the first S 1500, the last product 1000, O's way out 4000. 32 rows of
// those take 104 to 112 us (0.61 to 0.66 PFLOP/s), of 24 heads of 256 179 us (0.58), 32 rows of 1 to 2047 of 8 heads on 2 of
// 128 92 us (1.02).
#include <algorithm>
#include <cfloat>
#include <mutex>
#include <type_traits>

#include "attn_prompt.h"
#include "kernels.h"
#include "prompt_tiles.h"
#include "tc_attn.cuh"

namespace mtp {

namespace {

constexpr int kPromptThreads = 384;

// A warp's 32 rows (lane = row) of 32 columns.
__device__ __forceinline__ void tmem_ld_rows32(uint32_t t, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(t));
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ void fma2(float& x, float& y, float c, float d) {
  asm("{\n\t.reg .b64 s, t, u;\n\t"
      "mov.b64 s, {%0, %1};\n\t"
      "mov.b64 t, {%2, %2};\n\t"
      "mov.b64 u, {%3, %3};\n\t"
      "fma.rn.f32x2 s, s, t, u;\n\t"
      "mov.b64 {%0, %1}, s;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(c), "f"(d));
}
__device__ __forceinline__ void mul2(float& x, float& y, float c) {
  asm("{\n\t.reg .b64 s, t;\n\t"
      "mov.b64 s, {%0, %1};\n\t"
      "mov.b64 t, {%2, %2};\n\t"
      "mul.rn.f32x2 s, s, t;\n\t"
      "mov.b64 {%0, %1}, s;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(c));
}
__device__ __forceinline__ void add2(float& x, float& y, float u, float v) {
  asm("{\n\t.reg .b64 s, t;\n\t"
      "mov.b64 s, {%0, %1};\n\t"
      "mov.b64 t, {%2, %3};\n\t"
      "add.rn.f32x2 s, s, t;\n\t"
      "mov.b64 {%0, %1}, s;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(u), "f"(v));
}

// 32 bytes: one sector where they begin on one (`whole`: outputs at 32 bytes), else two halves. 32 prompts of 512 positions of
// 32 heads on 8 of 128 take 106 us with sectors, 111 with halves; 32 heads on 4 of 64 90 and 93.
__device__ __forceinline__ void st_global32(void* p, const uint32_t (&w)[8], bool whole) {
  if (!whole) {
    reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    return;
  }
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]),
               "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

__device__ __forceinline__ void st_shared16(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// A box of a tensor (head dimension, head, position) to shared memory.
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, int x, int head, int pos, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"((uint64_t)map), "r"(x), "r"(head), "r"(pos), "r"(bar)
      : "memory");
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

constexpr int kMeta = 3 << 10;  // bytes of PromptMeta, rounded up

template <int DH>
struct PromptShape {
  static constexpr int QT = DH == 256 ? 1 : 2;    // query tiles of a unit
  static constexpr int CPT = DH == 256 ? 2 : 1;   // ring stages of a tile of K or V
  static constexpr int NS = DH == 64 ? 8 : 5;     // ring stages
  static constexpr int kHalves = DH == 64 ? 1 : 2;  // P is given on in one piece or in two (64 dimensions' products are too short to wait twice)
  static constexpr int kQ = QT * 128 * DH * 2, kStage = 128 * DH * 2 / CPT;
  static constexpr int oRing = kQ, oMeta = oRing + NS * kStage;
  static constexpr int kSmem = oMeta + kMeta;
  static constexpr uint32_t cS = 0, cO = 256;     // columns of tensor memory: S at 0 and 128, O from 256 on
  static_assert(kSmem <= 227 * 1024, "shared memory");
  // a unit's stage of V of tile j, in the order of use: S of the first item(s), then P.V of item k and S of item k + 2
  __device__ static int v_at(int j, int nt) { return (DH == 256 ? min(j + 2, nt) + j : 2 * j + 1) * CPT; }
};

// A unit: a row's positions, a group of heads, and the unit's number in the row.
struct Unit {
  int a0, n, grp, j;
};

// Unit x of the order in which blocks take them (`per` positions each): a row's
// later units are its longest, so units go by their number in the row, the highest
// first, at each number all rows that have one, for each all groups of heads. False
// behind the last. By a whole warp. (The number is looked for by halving: F(j), the
// units with numbers from j on, falls as j rises.)
__device__ __forceinline__ bool find_unit(const PromptArgs& a, int per, long long x, Unit& u) {
  const int lane = threadIdx.x & 31, groups = a.n_q / a.group;
  const long long y = x / groups;
  u.grp = (int)(x - y * groups);
  constexpr int kOwn = 4;  // rows a lane keeps
  int own[kOwn], most = 0;
#pragma unroll
  for (int q = 0; q < kOwn; ++q) {
    const int r = lane + 32 * q;
    int a0, n = 0;
    if (r < a.rows) prompt_row(a.start, a.tokens, r, a0, n);
    own[q] = (n + per - 1) / per;
    most = max(most, own[q]);
  }
  auto units_of = [&](int r) {
    int a0, n;
    prompt_row(a.start, a.tokens, r, a0, n);
    return (n + per - 1) / per;
  };
  for (int r = lane + 32 * kOwn; r < a.rows; r += 32) most = max(most, units_of(r));
  most = __reduce_max_sync(0xFFFFFFFFu, most);
  auto from = [&](int j) {  // (units of a call: below 2^31)
    int sum = 0;
#pragma unroll
    for (int q = 0; q < kOwn; ++q) sum += max(0, own[q] - j);
    for (int r = lane + 32 * kOwn; r < a.rows; r += 32) sum += max(0, units_of(r) - j);
    return __reduce_add_sync(0xFFFFFFFFu, sum);
  };
  if (y >= from(0)) return false;
  int lo = 0, hi = most;  // F(lo) > y >= F(hi)
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (from(mid) > y) lo = mid;
    else hi = mid;
  }
  u.j = lo;
  int left = (int)y - from(lo + 1);  // the so manieth row with more than lo units
  for (int r0 = 0; r0 < a.rows; r0 += 32) {
    int a0 = 0, n = 0;
    if (r0 + lane < a.rows) prompt_row(a.start, a.tokens, r0 + lane, a0, n);
    const unsigned has = __ballot_sync(0xFFFFFFFFu, (n + per - 1) / per > lo);
    if (left < __popc(has)) {
      const int src = __fns(has, 0, left + 1);
      u.a0 = __shfl_sync(0xFFFFFFFFu, a0, src);
      u.n = __shfl_sync(0xFFFFFFFFu, n, src);
      return true;
    }
    left -= __popc(has);
  }
  return false;
}

constexpr int kUnits = 4;  // units handed out ahead

struct PromptMeta {
  uint64_t full[8], empty[8], s_full[2], p_full[2][2], pv_done[2], m_full[2][4], l_full[kMeets], q_full, q_empty, o_empty[2], v_go, v_ok, drain;
  uint64_t unit_full[kUnits], unit_empty[kUnits];
  Unit unit[kUnits];
  uint32_t tmem, copied;
  int fail;
  int nan[kUnits];     // 1 + the last unit of this slot that had something cleaned out of V that one of its queries may see
  float m[128];        // one query tile: the running maxima
  float l[2][128];     // the groups' sums
};
static_assert(sizeof(PromptMeta) <= kMeta, "meta");

// Eight words a lane that belong to one of four columns of two each: lane q of four neighbouring ones gets column q of
// all four (its words 2 j, 2 j + 1: lane j's).
__device__ __forceinline__ void transpose4(uint32_t (&w)[8], int lane) {
#pragma unroll
  for (int bit = 1; bit < 4; bit <<= 1) {
    const bool up = lane & bit;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (c & bit) continue;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        uint32_t &x = w[2 * c + e], &y = w[2 * (c | bit) + e];
        const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, up ? x : y, bit);
        if (up) x = got;
        else y = got;
      }
    }
  }
}

// x with what was cleaned out of V in dimension d and the query of row `dst` of the output sees. (Rare and slow.)
__device__ __noinline__ float add_cleaned(const PromptArgs& a, const Unit& u, int p0, int p1, long long dst, int d, float x) {
  if (dst < 0) return x;
  const int pos = (int)(dst / a.n_q) - u.a0, head = u.grp * a.group / (a.n_q / a.n_kv);
  const uint16_t* v = static_cast<const uint16_t*>(a.v) + (long long)u.a0 * a.ts[2] + (long long)head * a.hs[2] + d;
  for (int t = a.window > 0 ? max(0, pos - (a.window - 1)) : 0; t <= pos; ++t) {
    if (t <= p0 && (a.window == 0 || t > p1 - a.window)) {
      t = p0;  // (all queries of the unit see it and what follows up to here: V was left as it was)
      continue;
    }
    const float y = bf16_to_f(v[t * a.ts[2]]);
    if (!isfinite(y)) x += y;
  }
  return x;
}

template <int DH>
__global__ void __launch_bounds__(kPromptThreads, 1)
    k_prompt_tc(const __grid_constant__ PromptArgs a, const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                const __grid_constant__ CUtensorMap mv) {
  using S = PromptShape<DH>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  auto& M = *reinterpret_cast<PromptMeta*>(smem_raw + S::oMeta);
  const uint32_t sm = smem_u32(smem_raw);
  const int warp = __shfl_sync(0xFFFFFFFFu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int G = a.group;
  const int PT = 128 / G, per = S::QT * PT;  // positions of a query tile, of a unit
  volatile int* fail = &M.fail;
  auto ready = [&](uint64_t* bar, uint32_t parity) { return wait(bar, parity, fail); };

  if (threadIdx.x == 0) {
    for (int i = 0; i < 8; ++i) {
      mbar_init(smem_u32(&M.full[i]), 1);
      mbar_init(smem_u32(&M.empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&M.s_full[i]), 1);
      for (int h = 0; h < 2; ++h) mbar_init(smem_u32(&M.p_full[i][h]), 4);
      mbar_init(smem_u32(&M.pv_done[i]), 1);
      mbar_init(smem_u32(&M.o_empty[i]), 4);
      for (int w = 0; w < 4; ++w) mbar_init(smem_u32(&M.m_full[i][w]), 1);
    }
    for (int i = 0; i < kMeets; ++i) mbar_init(smem_u32(&M.l_full[i]), 1);
    mbar_init(smem_u32(&M.q_full), 1);
    mbar_init(smem_u32(&M.q_empty), 1);
    mbar_init(smem_u32(&M.v_go), 1);
    mbar_init(smem_u32(&M.v_ok), 2);
    mbar_init(smem_u32(&M.drain), 1);
    for (int i = 0; i < kUnits; ++i) {
      mbar_init(smem_u32(&M.unit_full[i]), 1);
      mbar_init(smem_u32(&M.unit_empty[i]), 11);  // the warps but the one that hands them out
      M.nan[i] = 0;
    }
    M.fail = 0;
    M.copied = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  // (tensor memory after the kernels before this one have given theirs back, and before a dependent kernel may take some)
  pdl_wait();
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&M.tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_trigger();
  const uint32_t tmem = M.tmem;

  // what a unit asks for: positions p0 to p1 of its queries, tiles of 128 keys from t_first on
  struct Span {
    int p0, p1, t_first, nt;
  };
  auto span = [&](const Unit& u) {
    Span s;
    s.p0 = u.j * per;
    s.p1 = min(u.n, s.p0 + per) - 1;
    s.t_first = a.window > 0 ? max(0, s.p0 - (a.window - 1)) / 128 : 0;
    s.nt = s.p1 / 128 + 1 - s.t_first;
    return s;
  };
  // whether some query at positions q0 to q1 does not see some position of the tile from t0 on
  auto edge = [&](int t0, int q0, int q1) { return t0 + 127 > q0 || (a.window > 0 && t0 <= q1 - a.window); };
  // steps of 16 keys of a tile that some query of the unit sees
  auto steps = [&](const Span& s, int t0, int& lo, int& hi) {
    hi = min(8, (s.p1 - t0) / 16 + 1);
    lo = a.window > 0 ? max(0, max(0, s.p0 - (a.window - 1)) - t0) / 16 : 0;
  };
  // unit number i of this block; false behind the last
  auto take = [&](int i, Unit& u) {
    if (!ready(&M.unit_full[i % kUnits], i / kUnits & 1)) return false;
    u = M.unit[i % kUnits];
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&M.unit_empty[i % kUnits]));
    return u.n > 0;
  };

  if (warp == 8) {
    // ---------------------------------------------------------- units, copies
    int at = 0;
    bool ok = true;
    Unit u;
    auto tile = [&](const CUtensorMap* map, int head, int pos, bool is_v) {
#pragma unroll 1
      for (int c = 0; c < S::CPT && ok; ++c, ++at) {
        const int st = at % S::NS, round = at / S::NS;
        if (round > 0 && !(ok = wait(&M.empty[st], (round - 1) & 1, fail))) return;
        const uint32_t bar = smem_u32(&M.full[st]), dst = sm + S::oRing + st * S::kStage;
        mbar_expect_tx(bar, S::kStage);
        M.copied = at + 1;
        if constexpr (DH == 256) {
          // K: 128 positions of half the dimensions; V: 64 positions of all
          if (!is_v) {
            for (int b = 0; b < 2; ++b) tma_box(dst + b * 16384, map, (2 * c + b) * 64, head, pos, bar);
          } else {
            for (int b = 0; b < 4; ++b) tma_box(dst + b * 8192, map, b * 64, head, pos + 64 * c, bar);
          }
        } else {
          for (int b = 0; b < DH / 64; ++b) tma_box(dst + b * 16384, map, b * 64, head, pos, bar);
        }
      }
    };
    // unit i of this block, found and handed out; false behind the last
    auto hand_out = [&](int i, Unit& u) {
      // there and back: who has the longest unit of one turn has the shortest of the next
      const int blocks = gridDim.x, b = blockIdx.x;
      if (!find_unit(a, per, (long long)i * blocks + (i & 1 ? blocks - 1 - b : b), u)) u.n = 0;
      if (i >= kUnits && !ready(&M.unit_empty[i % kUnits], (i / kUnits - 1) & 1)) return false;
      if (lane == 0) {
        M.unit[i % kUnits] = u;
        mbar_arrive(smem_u32(&M.unit_full[i % kUnits]));
      }
      return u.n > 0;
    };
    Unit ahead;
    bool some = hand_out(0, ahead);
#pragma unroll 1
    for (int i = 0; some; ++i) {
      u = ahead;
      some = hand_out(i + 1, ahead);  // (before the copies of this one, which wait for room)
      if (lane == 0) {
        const Span s = span(u);
        if (i > 0) ok = wait(&M.q_empty, (i - 1) & 1, fail);
        if (ok) {
          mbar_expect_tx(smem_u32(&M.q_full), S::QT * (DH / 64) * PT * G * 128);
          for (int q = 0; q < S::QT; ++q)
            for (int b = 0; b < DH / 64; ++b)
              tma_box(sm + q * 128 * DH * 2 + b * 16384, &mq, b * 64, u.grp * G, u.a0 + s.p0 + q * PT, smem_u32(&M.q_full));
        }
        const int head = u.grp * G / (a.n_q / a.n_kv), pos = u.a0 + s.t_first * 128;
        if (DH == 256) {
          if (ok) tile(&mk, head, pos, false);
          if (s.nt > 1 && ok) tile(&mk, head, pos + 128, false);
#pragma unroll 1
          for (int j = 0; j < s.nt && ok; ++j) {
            tile(&mv, head, pos + 128 * j, true);
            if (j + 2 < s.nt && ok) tile(&mk, head, pos + 128 * (j + 2), false);
          }
        } else {
#pragma unroll 1
          for (int j = 0; j < s.nt && ok; ++j) {
            tile(&mk, head, pos + 128 * j, false);
            if (ok) tile(&mv, head, pos + 128 * j, true);
          }
        }
      }
      ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
      if (!ok) break;
    }
    // the last arrivals on this block's barriers
    if (lane == 0)
      for (int i = max(0, at - S::NS); i < at && ok; ++i) ok = wait(&M.empty[i % S::NS], i / S::NS & 1, fail);
    __syncwarp();
  } else if (warp == 9) {
    // ---------------------------------------------------------- MMAs
    // By one warp in one order: while the tensor core has one item's products, the other's softmax runs. (Two warps, an
    // item each, fell into step with each other and took a quarter longer.) The waits between the products cost some 80
    // cycles each, so there are no more of them than the order needs, and no branch depends on how one ended: what the
    // compiler can see to be the same for the warp stays in uniform registers, where the MMAs take their operands from. A wait
    // that ran out ends the role at the next unit.
    constexpr uint32_t idS = idesc_bf(128, 128, false), idO = idesc_bf(128, DH, true);
    const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
    const uint64_t dq = tc::sdesc(sm);
    auto await = [&](uint64_t* bar, uint32_t parity) {
      const uint32_t b = smem_u32(bar);
#pragma unroll 1
      for (unsigned i = 0; !mbar_try(b, parity); ++i) {
        if (i == kAttnWaitLimit) *fail = 1;
        if (i == kAttnWaitLimit || ((i & 63) == 63 && *fail)) break;
      }
      __syncwarp();
    };
    struct Ring {
      int st, ph;
      __device__ void next() {
        if (++st == S::NS) {
          st = 0;
          ph ^= 1;
        }
      }
    };
    Ring ring = {0, 0};   // the next stage in the order of use
    int edges = 0;        // tiles whose V was cleaned
    int done[2] = {0, 0}; // items of each place so far
    auto full = [&](const Ring& r) {
      await(&M.full[r.st], r.ph);
      tc_fence_after();
    };
    // S in place `slot` of query tile q and one stage of K, the tile's c-th
    auto products_s = [&](int slot, int q, int c, int st) {
      const uint64_t dk = tc::sdesc(sm + S::oRing + st * S::kStage);
      const uint64_t da = dq + q * (128 * DH * 2 / 16) + c * (DH / S::CPT / 64) * 1024;
#pragma unroll
      for (int e = 0; e < DH / S::CPT / 16; ++e)
        mma_f16_ss(tm + S::cS + slot * 128, da + (e >> 2) * 1024 + (e & 3) * 2, dk + (e >> 2) * 1024 + (e & 3) * 2, idS, (c | e) > 0 ? 1u : 0u);
    };
    // P.V of the c-th 64 keys; st: their stage; [lo, hi): the tile's steps of 16 keys that count
    auto products_o = [&](int slot, int c, int st, int lo, int hi, uint32_t& acc) {
      const uint32_t d = tm + S::cO + (S::QT == 2 ? slot * DH : 0), p = tm + S::cS + slot * 128 + c * 32;
      const uint64_t dv = sdesc_mn(sm + S::oRing + st * S::kStage, 16384 / S::CPT) + (S::CPT == 2 ? 0 : c * 512);
      if (lo <= 4 * c && hi >= 4 * c + 4) {
#pragma unroll
        for (int e = 0; e < 4; ++e) mma_f16_ts(d, p + e * 8, dv + e * 128, idO, e > 0 ? 1u : acc);
        acc = 1u;
      } else {
#pragma unroll 1
        for (int e = max(0, lo - 4 * c); e < min(4, hi - 4 * c); ++e) {
          mma_f16_ts(d, p + e * 8, dv + e * 128, idO, acc);
          acc = 1u;
        }
      }
    };
    auto weights = [&](int slot, int c) {
      await(&M.p_full[slot][c], done[slot] & 1);
      tc_fence_after();
    };
#pragma unroll 1
    for (int i = 0;; ++i) {
      Unit u;
      const bool some = take(i, u) && !*fail;
      if (__shfl_sync(0xFFFFFFFFu, (int)some, 0) == 0) break;
      u.n = __shfl_sync(0xFFFFFFFFu, u.n, 0);
      u.j = __shfl_sync(0xFFFFFFFFu, u.j, 0);
      const Span sp = span(u);
      await(&M.q_full, i & 1);
      // one query tile: K of the first two tiles comes before V
      const int lead = S::QT == 2 ? 1 : min(2, sp.nt);
#pragma unroll 1
      for (int j = 0; j < lead; ++j) {
#pragma unroll 1
        for (int c = 0; c < S::CPT; ++c) {
          full(ring);
          products_s(j, 0, c, ring.st);
          if (S::QT == 2) {
            mma_commit_elect(smem_u32(&M.s_full[0]));
            products_s(1, 1, c, ring.st);
          }
          mma_commit_elect(smem_u32(&M.empty[ring.st]));
          ring.next();
        }
        mma_commit_elect(smem_u32(&M.s_full[S::QT == 2 ? 1 : j]));
      }
      if (lead == sp.nt) mma_commit_elect(smem_u32(&M.q_empty));
#pragma unroll 1
      for (int j = 0; j < sp.nt; ++j) {
        const int t0 = (sp.t_first + j) * 128;
        const bool clean = edge(t0, sp.p0, sp.p1);
        int lo = 0, hi = 8;
        const Ring v = ring;
        full(ring);
        ring.next();
        if (clean) {  // (all of V, then the cleaners)
          steps(sp, t0, lo, hi);
          if (S::CPT == 2) full(ring);
          if (lane == 0) mbar_arrive(smem_u32(&M.v_go));
          __syncwarp();
        }
        if (S::CPT == 2) ring.next();
        const bool more = j + lead < sp.nt;  // (a tile of K left for S)
        if constexpr (S::QT == 2) {
          const Ring k = ring;
#pragma unroll
          for (int slot = 0; slot < 2; ++slot) {
            if (i > 0 && j == 0) await(&M.o_empty[slot], (i - 1) & 1);  // O of the unit before has been read
            uint32_t acc = j > 0 ? 1u : 0u;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              if (c < S::kHalves) weights(slot, c);
              if (clean && slot == 0 && c == 0) await(&M.v_ok, edges++ & 1);
              products_o(slot, c, v.st, lo, hi, acc);
            }
            ++done[slot];
            if (slot == 1) mma_commit_elect(smem_u32(&M.empty[v.st]));
            if (j + 1 == sp.nt) mma_commit_elect(smem_u32(&M.pv_done[slot]));
            if (more) {
              if (slot == 0) full(k);
              products_s(slot, slot, 0, k.st);
              if (slot == 1) mma_commit_elect(smem_u32(&M.empty[k.st]));
              mma_commit_elect(smem_u32(&M.s_full[slot]));
            }
          }
          if (more) ring.next();
        } else {
          const int slot = j & 1;
          if (i > 0 && j == 0) {
            await(&M.o_empty[0], (i - 1) & 1);
            await(&M.o_empty[1], (i - 1) & 1);
          }
          uint32_t acc = j > 0 ? 1u : 0u;
          Ring r = v;
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            weights(slot, c);
            if (clean && c == 0) await(&M.v_ok, edges++ & 1);
            if (!clean && c == 1) full(r);
            products_o(slot, c, r.st, lo, hi, acc);
            mma_commit_elect(smem_u32(&M.empty[r.st]));
            r.next();
          }
          ++done[slot];
          mma_commit_elect(smem_u32(&M.pv_done[slot]));
          if (more) {
#pragma unroll 1
            for (int c = 0; c < S::CPT; ++c) {
              full(ring);
              products_s(slot, 0, c, ring.st);
              mma_commit_elect(smem_u32(&M.empty[ring.st]));
              ring.next();
            }
            mma_commit_elect(smem_u32(&M.s_full[slot]));
          }
        }
        if (more && j + lead + 1 == sp.nt) mma_commit_elect(smem_u32(&M.q_empty));
      }
    }
    // what was issued ends before its operands and tensor memory go
    mma_commit_elect(smem_u32(&M.drain));
    mbar_wait(smem_u32(&M.drain), 0, kAttnWaitLimit);
    __syncwarp();
  } else if (warp >= 10) {
    // ---------------------------------------------------------- V of edge tiles
    const int me = threadIdx.x - 320;
    constexpr int kSegs = DH / 8, kRows = 128 / S::CPT;  // 16-byte pieces of a position, positions of a stage
    int edges = 0, base = 0;
    bool ok = true;
    Unit u;
#pragma unroll 1
    for (int i = 0; ok && take(i, u); ++i) {
      const Span sp = span(u);
#pragma unroll 1
      for (int j = 0; j < sp.nt; ++j) {
        const int t0 = (sp.t_first + j) * 128, at = base + S::v_at(j, sp.nt);
        if (!edge(t0, sp.p0, sp.p1)) continue;
        // (told by the MMA warp, which has seen all stages of the ring in turn)
        if (!(ok = ready(&M.v_go, edges++ & 1))) break;
        int lo, hi;
        steps(sp, t0, lo, hi);
        bool found = false;
        // positions [r0, r1) of the tile without what is not finite
        auto clean = [&](int r0, int r1) {
          // a thread has a piece of every 64 / kSegs th position
          const int q = me % kSegs, step = 64 / kSegs;
#pragma unroll 1
          for (int c = 0; c < S::CPT; ++c) {
            const uint32_t to = sm + S::oRing + (at + c) % S::NS * S::kStage + (q >> 3) * (kRows * 128) + (q & 7) * 16;
            const int end = min(r1, (c + 1) * kRows) - c * kRows;
#pragma unroll 1
            for (int r = max(r0, c * kRows) - c * kRows + me / kSegs; r < end; r += 4 * step) {
              uint4 v[4];
#pragma unroll
              for (int x = 0; x < 4; ++x)
                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(v[x].x), "=r"(v[x].y), "=r"(v[x].z), "=r"(v[x].w)
                             : "r"(to + min(r + x * step, end - 1) * 128));
              // an exponent of all ones carries into its sign's place
              auto odd = [](uint32_t w) { return ((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u; };
#pragma unroll
              for (int x = 0; x < 4; ++x)
                if (odd(v[x].x) | odd(v[x].y) | odd(v[x].z) | odd(v[x].w)) {  // (a piece that two threads have: both store the same)
                  uint32_t w[4] = {v[x].x, v[x].y, v[x].z, v[x].w};
#pragma unroll
                  for (int y = 0; y < 4; ++y) w[y] &= ~((odd(w[y]) >> 15) * 0xFFFFu);
                  const int rx = min(r + x * step, end - 1), t = t0 + c * kRows + rx;
                  st_shared16(to + rx * 128, make_uint4(w[0], w[1], w[2], w[3]));
                  found |= t <= sp.p1 && !(a.window > 0 && t <= sp.p0 - a.window);
                }
            }
          }
        };
        const int low = a.window > 0 ? min(16 * hi, max(16 * lo, sp.p1 - a.window + 1 - t0)) : 16 * lo;
        clean(16 * lo, low);
        clean(max(low, max(16 * lo, sp.p0 + 1 - t0)), 16 * hi);
        if (found) M.nan[i % kUnits] = i + 1;
        fence_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&M.v_ok));
      }
      base += 2 * sp.nt * S::CPT;
    }
  } else {
    // ---------------------------------------------------------- softmax
    const int slot = warp >> 2, quarter = warp & 3, row = threadIdx.x & 127;
    const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
    const unsigned win = a.window > 0 ? (unsigned)a.window : 0x80000000u;
    // (above 0: -inf times 0 would be no weight)
    const float c = fmaxf(fabsf(a.scale) * 1.44269504f, FLT_MIN);
    const int in_pos = row / G, in_head = row - in_pos * G;  // the row's place in a query tile
    int done[2] = {0, 0};
    bool ok = true;
    Unit u;
#pragma unroll 1
    for (int i = 0; ok && take(i, u); ++i) {
      const Span sp = span(u);
      const int items = sp.nt * S::QT;
      const int q0 = sp.p0 + (S::QT == 2 ? slot * PT : 0), q1 = min(u.n, q0 + PT) - 1;  // the query tile's positions
      const bool real = in_pos < PT && q0 + in_pos < u.n;
      const int pos = real ? q0 + in_pos : -1;
      float m = -INFINITY, l = 0.f;
#pragma unroll 1
      for (int k = slot; k < items; k += 2) {
        const int t0 = (sp.t_first + (S::QT == 2 ? k >> 1 : k)) * 128;
        ok = ready(&M.s_full[slot], (done[slot] + (k >> 1)) & 1);
        if (!ok) break;
        tc_fence_after();
        uint32_t s[128];
#pragma unroll
        for (int q = 0; q < 4; ++q) tmem_ld_rows32(tmem + S::cS + slot * 128 + 32 * q + lanes, s + 32 * q);
        tc_wait_ld();
#pragma unroll
        for (int e = 0; e < 128; ++e) pin(s[e]);
        if (a.scale < 0.f) {
#pragma unroll
          for (int e = 0; e < 128; ++e) s[e] ^= 0x80000000u;
        }
        if (edge(t0, q0, q1)) {
          const int rel = pos - t0;
#pragma unroll
          for (int e = 0; e < 128; ++e)
            if ((unsigned)(rel - e) >= win) s[e] = 0xFF800000u;  // -inf: out of sight
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int e = 0; e < 128; e += 8)
#pragma unroll
          for (int q = 0; q < 4; ++q) mx[q] = max3(mx[q], __uint_as_float(s[e + 2 * q]), __uint_as_float(s[e + 2 * q + 1]));
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
        // the maximum so far; one that moves takes O with it
        float was = m;
        if (S::QT == 1 && k > 0) {
          ok = ready(&M.m_full[slot ^ 1][quarter], (done[slot ^ 1] + ((k - 1) >> 1)) & 1);
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
            ok = ready(&M.pv_done[slot ^ 1], (done[slot ^ 1] + ((k - 1) >> 1)) & 1);
            if (!ok) break;
            tc_fence_after();
          }
          const float fac = moved ? ex2(was - now) : 1.f;
#pragma unroll 1
          for (int d = 0; d < DH; d += 16) {
            const uint32_t t = tmem + S::cO + (S::QT == 2 ? slot * DH : 0) + d + lanes;
            float o[16];
            tc::tmem_ld16(t, o);
            uint32_t x[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = __float_as_uint(o[e] * fac);
            tmem_st_rows16(t, x);
          }
        }
        const float base = m == -INFINITY ? 0.f : m;
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          uint32_t w[16];
          if (h > 0)
#pragma unroll
            for (int e = 32 * h; e < 32 * h + 32; ++e) pin(s[e]);
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float x = __uint_as_float(s[32 * h + 2 * e]), y = __uint_as_float(s[32 * h + 2 * e + 1]);
            fma2(x, y, c, -base);
            x = ex2(x);
            y = ex2(y);
            add2(sum[2 * (e & 1)], sum[2 * (e & 1) + 1], x, y);
            w[e] = pack_bf16(x, y);
          }
          tmem_st_rows16(tmem + S::cS + slot * 128 + 16 * h + lanes, w);
          if ((h & 1) == 0 || (h == 1 && S::kHalves == 1)) continue;
          tc_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&M.p_full[slot][S::kHalves == 1 ? 0 : h >> 1]));
        }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
      }
      // ---- O of this query tile
      int c0 = 0;
      constexpr int kDims = S::QT == 2 ? DH : DH / 2;
      if (S::QT == 1) {  // the groups' sums, then half of the dimensions each
        // Two warps have the same rows. Each says twice a unit where it is: that its maxima are written, that its sums
        // are. (Not a barrier of the two groups: one that had left would keep the other for good.)
        auto meet = [&](int time) {
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&M.l_full[meet_barrier(time, slot, quarter)]));
          ok = ready(&M.l_full[meet_barrier(time, slot ^ 1, quarter)], meet_parity(time, i));
        };
        if (!ok) break;
        meet(0);
        if (!ok) break;
        const float top = M.m[row];
        l = m == -INFINITY ? l : l * ex2(m - top);
        M.l[slot][row] = l;
        meet(1);
        if (!ok) break;
        l += M.l[slot ^ 1][row];
        m = top;
        c0 = slot * kDims;
      }
      // (beside the last product: what the rows' sums give does not wait for it)
      const float r = l != 0.f ? 1.f / l : 0.f;
      const long long dst = real ? (long long)(u.a0 + pos) * a.n_q + u.grp * G + in_head : -1;
      if (real && a.lse && c0 == 0) a.lse[dst] = l != 0.f ? (m + log2f(l)) * 0.693147181f : -INFINITY;
      // rows to dimensions four lanes at a time: a store is eight whole lines
      float rr[4];
      long long to[4];  // the lane's rows: lane / 4 + 8 y of the warp's 32
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        rr[y] = __shfl_sync(0xFFFFFFFFu, r, (lane >> 2) + 8 * y);
        to[y] = __shfl_sync(0xFFFFFFFFu, dst, (lane >> 2) + 8 * y);
      }
      if (ok) {
        // (the phase before is over: S of the last item, which this group or the other one has seen, came behind that P.V)
        const int last = items - 1;
        ok = S::QT == 2 ? ready(&M.pv_done[slot], i & 1) : ready(&M.pv_done[last & 1], (done[last & 1] + (last >> 1)) & 1);
        tc_fence_after();
      }
      done[0] += (items + 1) / 2;
      done[1] += items / 2;
      if (!ok) break;
      // (or a row that nothing weighs in: its products may be 0 times NaN)
      const bool nan = *reinterpret_cast<volatile int*>(&M.nan[i % kUnits]) == i + 1 || __any_sync(0xFFFFFFFFu, r == 0.f && dst >= 0);
      auto put = [&](auto slow) {
#pragma unroll 1
        for (int d = c0; d < c0 + kDims; d += 64) {
          uint32_t o[2][2][16];  // 16 rows, 32 dimensions
#pragma unroll
          for (int hh = 0; hh < 2; ++hh)
#pragma unroll
            for (int q = 0; q < 2; ++q)
              tmem_ld_frag<4>(tmem + S::cO + (S::QT == 2 ? slot * DH : 0) + d + 32 * q + lanes + ((uint32_t)(16 * hh) << 16), o[hh][q]);
          tc_wait_ld();
#pragma unroll
          for (int hh = 0; hh < 2; ++hh)
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
              for (int e = 0; e < 16; ++e) pin(o[hh][q][e]);
          if (d + 64 >= c0 + kDims) {  // O may be written again
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&M.o_empty[slot]));
          }
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            uint32_t w[8];
#pragma unroll
            for (int b = 0; b < 8; ++b) {  // dimensions 8 b + 2 (lane % 4), + 1 of the row
              float x[2];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                x[e] = __uint_as_float(o[y >> 1][b >> 2][4 * (b & 3) + 2 * (y & 1) + e]);
                if (!decltype(slow)::value) continue;
                x[e] = rr[y] != 0.f ? x[e] * rr[y] : 0.f;
                x[e] = add_cleaned(a, u, sp.p0, sp.p1, to[y], d + 8 * b + 2 * (lane & 3) + e, x[e]);
              }
              if (!decltype(slow)::value) mul2(x[0], x[1], rr[y]);
              w[b] = pack_bf16(x[0], x[1]);
            }
            transpose4(w, lane);
            // words 2 j, 2 j + 1 are lane j's of blocks 2 (lane % 4), + 1
            const uint32_t v[8] = {w[0], w[2], w[4], w[6], w[1], w[3], w[5], w[7]};
            if (to[y] >= 0) st_global32(static_cast<uint16_t*>(a.out) + to[y] * DH + d + 16 * (lane & 3), v, a.out_whole);
          }
        }
      };
      if (nan) put(std::true_type{});
      else put(std::false_type{});
    }
  }

  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && M.fail) {
    flag_status(a.status, MTP_ERR_TIMEOUT);
    // let copies still in flight land before the shared memory is released
    for (uint32_t i = 0; i < (uint32_t)S::NS && i < M.copied; ++i)
      mbar_wait(smem_u32(&M.full[(M.copied - 1 - i) % S::NS]), ((M.copied - 1 - i) / S::NS) & 1, kAttnWaitLimit);
    mbar_wait(smem_u32(&M.q_full), 0, kAttnWaitLimit);
    mbar_wait(smem_u32(&M.q_full), 1, kAttnWaitLimit);
  }
  __syncthreads();
  tc_fence_after();
  if (warp == 0) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

// Q, K or V as (head dimension, head, position), boxes of 64 x `per` x `rows`.
bool head_map(CUtensorMap* m, const void* p, int dh, int heads, int tokens, long long hs, long long ts, int per, int rows) {
  auto enc = tc::get_encode();
  if (!enc) return false;
  cuuint64_t dims[3] = {(cuuint64_t)dh, (cuuint64_t)heads, (cuuint64_t)tokens};
  // (the stride of a dimension of one is any that the encoder takes)
  cuuint64_t strides[2] = {(cuuint64_t)(heads > 1 ? hs : dh) * 2, (cuuint64_t)(tokens > 1 ? ts : (long long)dh * heads) * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)per, (cuuint32_t)rows}, one[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DH>
cudaError_t launch(PromptArgs a, cudaStream_t s) {
  using S = PromptShape<DH>;
  CUtensorMap mq, mk, mv;
  if (!head_map(&mq, a.q, DH, a.n_q, a.tokens, a.hs[0], a.ts[0], a.group, 128 / a.group) ||
      !head_map(&mk, a.k, DH, a.n_kv, a.tokens, a.hs[1], a.ts[1], 1, 128) ||
      !head_map(&mv, a.v, DH, a.n_kv, a.tokens, a.hs[2], a.ts[2], 1, DH == 256 ? 64 : 128))
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
  const long long units = prompt_most_tiles(a.tokens, a.rows, 1, S::QT * (128 / a.group)) * (a.n_q / a.group);
  count_launch();
  return launch_pdl(k_prompt_tc<DH>, dim3((unsigned)std::min<long long>(units, device_sm_count())), dim3(kPromptThreads), S::kSmem, s, a,
                    mq, mk, mv);
}

}  // namespace

cudaError_t launch_prompt_tc(PromptArgs a, int head_dim, cudaStream_t s) {
  // heads to a query tile: all that share a KV head, or their largest divisor that fits
  const int G = a.n_q / a.n_kv;
  for (a.group = std::min(G, 128); G % a.group != 0;) --a.group;
  return head_dim == 64 ? launch<64>(a, s) : (head_dim == 128 ? launch<128>(a, s) : launch<256>(a, s));
}

}  // namespace mtp
