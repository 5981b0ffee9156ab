// Log probabilities of given tokens, ranks, entropy and alternatives
// (spec_logprobs), in one read of the logits.
//
// With m = max x:  S = sum e^(x-m),  T = sum (x-m) e^(x-m),
//   log p_t = x_t - m - log S,   H = log S - T / S,
//   rank = #{j : (x_j, j) before (x_t, t)},  and the first k of that order.
//
// k_lp_part: a row is cut into parts, one block each. A thread keeps its own
// running (m, S, T); when m grows by d, S and T become f S and f (T - d S) with
// f = e^-d. Alternatives: at least k elements reach the k-th largest of the
// maxima that groups of threads saw. A thread also keeps its maxima over eight
// stretches of the part, so that only stretches whose maximum reaches that
// bound are looked at again (from L2), a vector per lane: some 25 elements for
// k = 20. A collection that overflows is cut to its k best as it goes. Elements
// go by 64-bit keys (value descending, id ascending), so ties need no care
// anywhere.
// k_lp_join: a block per row adds up the parts and merges their lists.
//
// Bound by issue (70 % of its rate: 23 instructions an element, the
// alternatives' included, one an exponential at 16 a cycle and SM) and, at a
// part's end, by latency: some 8,000 cycles for the alternatives, which four
// blocks an SM hide only in part. 256 rows of 152,064
// fp32 logits with 20 alternatives: 42 us, 3.7 TB/s; without any 37 us; 1001
// rows of 32,769 bf16 logits with 8: 33 us; 3 rows of 152,064 with 5: 10 us.
// One block per SM slot for all its rows' parts (copies running on into the
// next part) was slower, 50 and 46 us: its loop needs registers that four
// blocks an SM do not have.
#include <algorithm>
#include <climits>

#include "common.cuh"
#include "kernels.h"

namespace mtp {

namespace {

constexpr int kLpThreads = 256;     // (and a warp more that copies)
constexpr int kLpBlocksPerSM = 4;
constexpr int kLpMaxTop = 64;
constexpr int kLpCap = 1024;        // collected keys of a block
constexpr int kLpList = 128;        // keys that a part hands on
constexpr int kLpMaxParts = 128;
constexpr int kLpCells = 8;
constexpr int kLpStages = 4;
constexpr int kLpStage = 8192;      // bytes: two 16-byte vectors a thread
constexpr unsigned kLpWaitLimit = 1u << 20;

struct LpArgs {
  const void* x;
  long long stride;
  const int32_t* tok;
  float *lp, *ent, *top_lp;
  int32_t *rank, *top_id, *status;
  int n, V, top, parts;
  float4* sums;                     // [n][parts] m, S, T, rank count (bits)
  uint4* heads;                     // [n][parts] a bound (key), keys handed on
  unsigned long long* keys;         // [n][parts][kLpList], in no order
};

// Order key: larger value first, then lower id; -0 counts as +0.
__device__ __forceinline__ uint32_t value_key(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ unsigned long long lp_key(float x, int id) {
  return (unsigned long long)value_key(x) << 32 | (0xFFFFFFFFu - (uint32_t)id);
}
__device__ __forceinline__ float key_value(unsigned long long k) {
  const uint32_t u = (uint32_t)(k >> 32);
  return __uint_as_float(u & 0x80000000u ? u & 0x7FFFFFFFu : ~u);
}

// max that keeps a NaN
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float kLog2e = 1.44269504f;
constexpr float kFloor = -110.f;    // e^-110 is zero in fp32

// (m, S, T) of two disjoint sets.
struct LpSum {
  float m, S, T;
  __device__ void raise(float to) {  // to >= m
    if (m == -INFINITY) {
      m = to;
      return;
    }
    const float d = to - m, f = exp2_fast(-d * kLog2e);
    T = f == 0.f ? 0.f : f * (T - d * S);
    S *= f;
    m = to;
  }
  __device__ void add(LpSum o) {
    if (o.m == -INFINITY && o.S == o.S) return;
    if (o.m > m) raise(o.m);
    else o.raise(m);
    S += o.S;
    T += o.T;
  }
};

// The sum over the first `lanes` lanes of a warp (a power of two; in lane 0):
// the largest m first, then plain sums.
__device__ __forceinline__ void lp_warp_add(LpSum& s, int& before, int lanes) {
  float m = s.m;
#pragma unroll
  for (int o = lanes / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  if (s.m < m) s.raise(m);
#pragma unroll
  for (int o = lanes / 2; o > 0; o >>= 1) {
    s.S += __shfl_xor_sync(0xFFFFFFFFu, s.S, o);
    s.T += __shfl_xor_sync(0xFFFFFFFFu, s.T, o);
    before += __shfl_xor_sync(0xFFFFFFFFu, before, o);
  }
}

// Two fp32 values side by side (one instruction for both).
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ void unpair(uint64_t d, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(d));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
// Moves paired sums into (m, S, T).
__device__ __forceinline__ void fold(LpSum& s, uint64_t& S2, uint64_t& T2) {
  float a, b;
  unpair(S2, a, b);
  s.S += a + b;
  unpair(T2, a, b);
  s.T += a + b;
  S2 = T2 = 0;
}

struct LpShared {
  union {
    alignas(128) uint8_t ring[kLpStages][kLpStage];
    unsigned long long key[2][kLpCap];  // collected keys, and those left of them (once the ring is done)
  };
  float cell[kLpCells][kLpThreads];   // the threads' maxima over stretches of the part
  int n_list[kLpThreads / 32];
  uint16_t list[kLpThreads / 32][32 * kLpCells];  // a warp's cells that may hold alternatives: cell * 32 + lane
  alignas(16) unsigned long long group[128];
  unsigned long long bound, kth;
  uint64_t full[kLpStages], empty[kLpStages];
  int n, n_live;
  float4 sums[kLpThreads / 32];
};

// Barrier of the 256 threads that compute.
__device__ __forceinline__ void lp_sync() { asm volatile("barrier.cta.sync.aligned 1, 256;" ::: "memory"); }
__device__ __forceinline__ bool lp_any(bool p) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\t"
      "barrier.cta.red.or.aligned.pred q, 1, 256, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(any)
      : "r"((uint32_t)p)
      : "memory");
  return any != 0;
}

// The k-th largest (k = top) of the block's group maxima of the threads' keys,
// into sh.kth: groups of 4 threads up to 24 alternatives, else of 2. (Whole
// keys, not values: where thousands of logits are equal, as a mask's are, the
// ids keep the bound sharp.)
__device__ __forceinline__ void kth_bound(LpShared& sh, unsigned long long v, int top) {
  const int tid = threadIdx.x, g = top <= 24 ? 4 : 2, ng = kLpThreads / g;
  v = max(v, __shfl_xor_sync(0xFFFFFFFFu, v, 1));
  if (g == 4) v = max(v, __shfl_xor_sync(0xFFFFFFFFu, v, 2));
  if (tid % g == 0) sh.group[tid / g] = v;
  if (tid == 0) sh.kth = 0;
  lp_sync();
  // a group's rank, counted by its g threads, every g-th pair each (side by side in the banks)
  const unsigned long long mine = sh.group[tid / g];
  int before = 0;
#pragma unroll 4
  for (int i = tid % g * 2; i < ng; i += 2 * g) {
    const ulonglong2 o = *reinterpret_cast<const ulonglong2*>(&sh.group[i]);
    before += (o.x > mine) + (o.y > mine);
  }
  before += __shfl_xor_sync(0xFFFFFFFFu, before, 1);
  if (g == 4) before += __shfl_xor_sync(0xFFFFFFFFu, before, 2);
  if (before == top - 1 && mine) sh.kth = mine;  // (keys differ; 0: the group saw nothing)
  lp_sync();
}

// Cuts sh.key[0][0, n) to its `top` best in descending order, sh.n of them; where
// there were that many, the last one is the new bound.
__device__ __noinline__ void cut(LpShared& sh, int top) {
  const int tid = threadIdx.x;
  lp_sync();
  const int n = min(sh.n, kLpCap);
  unsigned long long bound = 0;
  if (n > 64) {
    unsigned long long v = 0;
    for (int i = tid; i < n; i += kLpThreads) v = max(v, sh.key[0][i]);
    kth_bound(sh, v, top);
    bound = sh.kth;
  }
  if (tid == 0) sh.n_live = 0;
  lp_sync();
  for (int i = tid; i < n; i += kLpThreads) {
    const unsigned long long k = sh.key[0][i];
    if (k >= bound) sh.key[1][atomicAdd(&sh.n_live, 1)] = k;
  }
  lp_sync();
  const int live = sh.n_live;
  for (int i = tid; i < live; i += kLpThreads) {
    const unsigned long long k = sh.key[1][i];
    int before = 0;
#pragma unroll 4
    for (int j = 0; j < live; ++j) before += sh.key[1][j] > k;
    if (before < top) sh.key[0][before] = k;
    if (before == top - 1) sh.bound = k;
  }
  if (tid == 0) sh.n = min(live, top);
  lp_sync();
}

template <int DT>
__global__ void __launch_bounds__(kLpThreads + 32, kLpBlocksPerSM) k_lp_part(const __grid_constant__ LpArgs a) {
  constexpr int W = DT == MTP_DTYPE_BF16 ? 8 : 4;   // elements of a 16-byte vector
  constexpr int Q = kLpStage / 16 / kLpThreads;     // vectors of a thread and stage
  constexpr int kVecs = kLpStage / 16;              // vectors of a stage
  __shared__ LpShared sh;
  const int tid = threadIdx.x, part = blockIdx.x, r = blockIdx.y;
  const uint8_t* row = static_cast<const uint8_t*>(a.x) + (long long)r * a.stride * (16 / W);
  // whole vectors from the row's first 16-byte boundary on, and the elements
  // before and after them
  const int head = min((int)((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / (16 / W), a.V);
  const int n_vec = (a.V - head) / W, tail = (a.V - head) % W;
  const int v0 = (int)((long long)n_vec * part / a.parts), v1 = (int)((long long)n_vec * (part + 1) / a.parts);
  const uint8_t* body = row + head * (16 / W);
  if (tid == 0) {
    sh.n = 0;
    for (int i = 0; i < kLpThreads / 32; ++i) sh.n_list[i] = 0;
    for (int i = 0; i < kLpStages; ++i) {
      mbar_init(smem_u32(&sh.full[i]), 1);
      mbar_init(smem_u32(&sh.empty[i]), kLpThreads / 32);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  if (tid >= kLpThreads) {
    // the copying warp: the part in stages of contiguous bytes
    int st = 0, round = 0, last[kLpStages];
#pragma unroll
    for (int i = 0; i < kLpStages; ++i) last[i] = -1;
#pragma unroll 1
    for (int v = v0; v < v1; v += kVecs) {
      if (round > 0 && !mbar_wait(smem_u32(&sh.empty[st]), (round - 1) & 1, kLpWaitLimit)) break;
      if (tid == kLpThreads) {
        const uint32_t bytes = min(kVecs, v1 - v) * 16;
        mbar_expect_tx(smem_u32(&sh.full[st]), bytes);
        bulk_g2s(smem_u32(sh.ring[st]), body + 16LL * v, bytes, smem_u32(&sh.full[st]));
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < kLpStages; ++i)
        if (i == st) last[i] = round;
      if (++st == kLpStages) {
        st = 0;
        ++round;
      }
    }
    // (copies land before the block's shared memory goes, whatever the others do)
#pragma unroll
    for (int i = 0; i < kLpStages; ++i)
      if (last[i] >= 0) mbar_wait(smem_u32(&sh.full[i]), last[i] & 1, kLpWaitLimit);
    __syncwarp();
    asm volatile("barrier.cta.sync.aligned 2, 288;" ::: "memory");
    const float4 f = sh.sums[tid & 7];
    LpSum s{f.x, f.y, f.z};
    int before = __float_as_int(f.w);
    lp_warp_add(s, before, 8);
    if (tid == kLpThreads) a.sums[(long long)r * a.parts + part] = make_float4(s.m, s.S, s.T, __int_as_float(before));
    return;
  }
  const int t = a.tok[r];
  const bool given = t >= 0 && t < a.V;
  const float xt = given ? load_elem(row, DT, t) : INFINITY;
  const uint32_t xt_bits = __float_as_uint(xt);
  // before t an equal logit comes first too: x >= xt is x > the float below xt
  // (below -inf: a NaN, which nothing is at most)
  const float below = xt == 0.f ? -__uint_as_float(1) : __uint_as_float(xt_bits & 0x80000000u ? xt_bits + 1 : xt_bits - 1);

  LpSum s{-INFINITY, 0.f, 0.f};
  int before = 0;
  // thread t's share of the elements outside the vectors: one at most
  unsigned long long lone = 0, best = 0;  // its key; a key that some element of the thread reaches
  {
    int id = -1;
    if (part == 0 && tid < head) id = tid;
    if (part == a.parts - 1 && tid >= 8 && tid - 8 < tail) id = head + n_vec * W + tid - 8;
    if (id >= 0) {
      const float x = load_elem(row, DT, id);
      if (!(x == -INFINITY)) {
        s.m = x;
        s.S = x < INFINITY ? 1.f : x - x;  // (a NaN or +inf makes the sum NaN)
        lone = best = lp_key(x, id);
      }
      before += x > xt || (x == xt && id < t);
    }
  }

  float seen = -INFINITY;  // the largest of the vectors, and the first one that had it
  int seen_at = v0;
  const int cell_len = max(1, ((v1 - v0 + kVecs - 1) / kVecs + kLpCells - 1) / kLpCells);  // batches of a cell
  int cell_at = 0, n_cells = 0;
  float cell_max = -INFINITY;
  uint64_t S2 = 0, T2 = 0;  // even and odd elements' sums
  int st = 0, phase = 0;
  bool ok = true;
#pragma unroll 1
  for (int v = v0; v < v1; v += kVecs) {
    const bool whole = v + kVecs <= v1;
    ok = ok && mbar_wait(smem_u32(&sh.full[st]), phase, kLpWaitLimit);
    uint4 w[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) w[q] = reinterpret_cast<const uint4*>(sh.ring[st])[q * kLpThreads + tid];
    if (!whole) {
#pragma unroll
      for (int q = 0; q < Q; ++q)
        if (v + q * kLpThreads + tid >= v1) {  // -inf past the part's end
          const uint32_t none = W == 8 ? 0xFF80FF80u : 0xFF800000u;
          w[q] = make_uint4(none, none, none, none);
        }
    }
    // element e of vector q
    auto elem = [&](int q, int e) {
      const uint32_t u[4] = {w[q].x, w[q].y, w[q].z, w[q].w};
      return W == 8 ? ((e & 1) ? bf16hi(u[e / 2]) : bf16lo(u[e / 2])) : __uint_as_float(u[W == 8 ? 0 : e]);
    };
    float most[Q], top = -INFINITY;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      most[q] = elem(q, 0);
#pragma unroll
      for (int e = 1; e < W; ++e) most[q] = fmaxf(most[q], elem(q, e));
      top = fmaxf(top, most[q]);
    }
    // The stage goes back by the lane that the vote names: it hangs on every word
    // loaded. (An arrival right behind the loads does not wait for them, and the
    // next copy could overtake them.)
    const bool higher = top > seen;
    if ((tid & 31) == (__any_sync(0xFFFFFFFFu, higher) ? 0 : 1)) mbar_arrive(smem_u32(&sh.empty[st]));
    if (++st == kLpStages) {
      st = 0;
      phase ^= 1;
    }
    if (higher) {
      seen = top;
#pragma unroll
      for (int q = Q - 1; q >= 0; --q)
        if (most[q] == top) seen_at = v + q * kLpThreads + tid;
      if (top > s.m) {
        fold(s, S2, T2);
        s.raise(top);
      }
    }
    cell_max = fmaxf(cell_max, top);
    if (++cell_at == cell_len) {
      sh.cell[n_cells++][tid] = cell_max;
      cell_max = -INFINITY;
      cell_at = 0;
    }
    const int id0 = head + v * W, id1 = id0 + kVecs * W;
    const bool mixed = id0 <= t && t < id1;
    const float m = s.m == -INFINITY ? 0.f : s.m, over = mixed ? INFINITY : (id1 <= t ? below : xt);
    const uint64_t minus_m = pair(-m, -m), l2e = pair(kLog2e, kLog2e);
    int count = 0;
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
      for (int e = 0; e < W; e += 2) {
        const float x0 = elem(q, e), x1 = elem(q, e + 1);
        float d0, d1, p0, p1;
        unpair(add2(pair(x0, x1), minus_m), d0, d1);
        const uint64_t d = pair(max_nan(d0, kFloor), max_nan(d1, kFloor));
        unpair(mul2(d, l2e), p0, p1);
        const uint64_t p = pair(exp2_fast(p0), exp2_fast(p1));
        S2 = add2(S2, p);
        T2 = fma2(d, p, T2);
        count += !(x0 <= over);
        count += !(x1 <= over);
      }
    // (what was filled in past the part's end is -inf: over a NaN, not counted)
    if (!whole && over != over) {
      count = 0;
#pragma unroll
      for (int q = 0; q < Q; ++q) count += v + q * kLpThreads + tid < v1 ? W : 0;
    }
    before += count;
    if (mixed) {
#pragma unroll
      for (int q = 0; q < Q; ++q)
#pragma unroll
        for (int e = 0; e < W; ++e) {
          const int i = v + q * kLpThreads + tid, id = head + i * W + e;
          const float x = elem(q, e);
          before += i < v1 && (x > xt || (x == xt && id < t));
        }
    }
  }
  fold(s, S2, T2);
  if (cell_at > 0) sh.cell[n_cells++][tid] = cell_max;
  if (!ok) flag_status(a.status, MTP_ERR_TIMEOUT);

  // the warps' sums; the copying warp adds them up
  const int lane = tid & 31, warp = tid >> 5;
  lp_warp_add(s, before, 32);
  if (lane == 0) sh.sums[warp] = make_float4(s.m, s.S, s.T, __int_as_float(before));
  __syncwarp();
  asm volatile("barrier.cta.arrive.aligned 2, 288;" ::: "memory");
  const long long at = (long long)r * a.parts + part;
  if (a.top == 0) return;

  // the alternatives (`each` hands the thread's elements of batch v on)
  auto each = [&](int v, auto&& f) {
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int i = v + q * kLpThreads + tid;
      if (i >= v1) continue;
      const uint4 u4 = reinterpret_cast<const uint4*>(body)[i];
      const uint32_t u[4] = {u4.x, u4.y, u4.z, u4.w};
#pragma unroll
      for (int e = 0; e < W; ++e)
        f(W == 8 ? ((e & 1) ? bf16hi(u[e / 2]) : bf16lo(u[e / 2])) : __uint_as_float(u[W == 8 ? 0 : e]), head + i * W + e);
    }
  };
  // (the last id of the vector that has it: a key not above the element's own)
  if (seen > -INFINITY) best = max(best, lp_key(seen, head + seen_at * W + W - 1));
  kth_bound(sh, best, a.top);
  unsigned long long bound = sh.kth;  // 0 where fewer groups than alternatives saw anything
  unsigned long long known = bound;     // at least `top` of the part's keys reach it (if it is not 0)
  const float least = bound ? key_value(bound) : -INFINITY;
  auto push = [&](unsigned long long k) {
    const int at = atomicAdd(&sh.n, 1);
    if (at < kLpCap) sh.key[0][at] = k;
    return at < kLpCap;
  };
  if (lone >= bound && lone) push(lone);
  // cells that may hold some (where their maximum is the bound's value, some id
  // is before its), and then those cells' elements again, a vector per lane
  const float reach = fmaxf(least, -3.402823466e38f);
  uint16_t* list = sh.list[warp];
  if (best >= bound && seen >= reach) {
    const int last_id = bound ? (int)(0xFFFFFFFFu - (uint32_t)bound) : INT_MAX;
    unsigned in = 0;
    int id = head + (v0 + tid) * W;
#pragma unroll
    for (int c = 0; c < kLpCells; ++c, id += cell_len * kVecs * W) {
      const float x = c < n_cells ? sh.cell[c][tid] : -INFINITY;
      in |= (x > reach || (x == reach && id <= last_id)) << c;
    }
    int to = atomicAdd(&sh.n_list[warp], __popc(in));
    for (; in; in &= in - 1) list[to++] = (uint16_t)((__ffs(in) - 1) * 32 + lane);
  }
  __syncwarp();
  const unsigned per_cell = cell_len * Q, items = sh.n_list[warp] * per_cell;
  const unsigned inverse = 0xFFFFFFFFu / per_cell + 1;  // i / per_cell = the product's high half: i per_cell < 2^32
#pragma unroll 1
  for (unsigned i0 = lane; i0 < items; i0 += 128) {
    uint4 u4[4];
    int at[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const unsigned i = i0 + 32 * c, k = __umulhi(i, inverse);
      at[c] = v1;
      if (i < items) {
        const int e = list[k];
        at[c] = v0 + (e >> 5) * cell_len * kVecs + (int)(i - k * per_cell) * kLpThreads + (tid & ~31) + (e & 31);
      }
      if (at[c] < v1) u4[c] = reinterpret_cast<const uint4*>(body)[at[c]];
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (at[c] >= v1) continue;
      const uint32_t u[4] = {u4[c].x, u4[c].y, u4[c].z, u4[c].w};
#pragma unroll
      for (int e = 0; e < W; ++e) {
        const float x = W == 8 ? ((e & 1) ? bf16hi(u[e / 2]) : bf16lo(u[e / 2])) : __uint_as_float(u[W == 8 ? 0 : e]);
        if (x >= reach) {
          const unsigned long long k = lp_key(x, head + at[c] * W + e);
          if (k >= bound) push(k);
        }
      }
    }
  }
  lp_sync();
  if (sh.n > kLpCap) {
    // too many (a few threads hold the top of the row): again, batch by batch
    // with a cut and a sharper bound whenever the collection is full
    lp_sync();
    if (tid == 0) sh.n = 0;
    lp_sync();
    if (lone >= bound && lone) push(lone);
#pragma unroll 1
    for (int v = v0; v < v1; v += kVecs) {
      uint32_t bits = 0xFFFF;  // the thread's elements that are still to be looked at
      int e = 0;
      while (lp_any(bits != 0)) {
        e = 0;
        uint32_t left = 0;
        each(v, [&](float x, int id) {
          const unsigned long long k = lp_key(x, id);
          if ((bits >> e & 1) && x > -INFINITY && k >= bound && !push(k)) left |= 1u << e;
          ++e;
        });
        bits = left;
        if (lp_any(left != 0)) {
          cut(sh, a.top);
          known = sh.bound;
          bound = known + 1;
        }
      }
    }
  }
  // the part's bound and what reaches it: the row's join takes the sharpest of
  // the parts' bounds, so the list needs no order
  if (sh.n > kLpList || (!known && sh.n >= a.top)) {
    cut(sh, a.top);
    if (sh.n == a.top) known = sh.bound;
  }
  const int n = sh.n;
  if (tid < n) a.keys[at * kLpList + tid] = sh.key[0][tid];
  if (tid == 0) a.heads[at] = make_uint4((uint32_t)known, (uint32_t)(known >> 32), (uint32_t)n, 0u);
}

constexpr int kLpJoinThreads = 256;
constexpr int kLpLive = 1024;

__global__ void __launch_bounds__(kLpJoinThreads) k_lp_join(const __grid_constant__ LpArgs a, int dt) {
  __shared__ unsigned long long s_live[kLpLive], s_bound;
  __shared__ int s_n, s_cnt[kLpMaxParts];
  __shared__ float s_red[4][kLpJoinThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, r = blockIdx.x, P = a.parts, top = a.top;
  if (tid == 0) {
    s_bound = 1ull;
    s_n = 0;
  }
  pdl_wait();  // (no early trigger: the next call's blocks, four to an SM, would find less room beside these)
  __syncthreads();
  LpSum s{-INFINITY, 0.f, 0.f};
  int before = 0;
  unsigned long long bound = 0;
  for (int p = tid; p < P; p += kLpJoinThreads) {
    const float4 f = a.sums[(long long)r * P + p];
    if (top > 0) {
      const uint4 h = a.heads[(long long)r * P + p];
      bound = max(bound, (unsigned long long)h.y << 32 | h.x);
      s_cnt[p] = min((int)h.z, kLpList);
    }
    s.add(LpSum{f.x, f.y, f.z});
    before += __float_as_int(f.w);
  }
  const int t = a.tok[r];
  const bool given = t >= 0 && t < a.V;
  const float xt = given && tid == 0 ? load_elem(a.x, dt, (long long)r * a.stride + t) : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    LpSum x;
    x.m = __shfl_xor_sync(0xFFFFFFFFu, s.m, o);
    x.S = __shfl_xor_sync(0xFFFFFFFFu, s.S, o);
    x.T = __shfl_xor_sync(0xFFFFFFFFu, s.T, o);
    s.add(x);
    before += __shfl_xor_sync(0xFFFFFFFFu, before, o);
    bound = max(bound, __shfl_xor_sync(0xFFFFFFFFu, bound, o));
  }
  if (lane == 0) {
    s_red[0][warp] = s.m;
    s_red[1][warp] = s.S;
    s_red[2][warp] = s.T;
    s_red[3][warp] = __int_as_float(before);
    if (bound > 1) atomicMax(&s_bound, bound);
  }
  __syncthreads();
  s = LpSum{-INFINITY, 0.f, 0.f};
  before = 0;
#pragma unroll
  for (int i = 0; i < kLpJoinThreads / 32; ++i) {
    s.add(LpSum{s_red[0][i], s_red[1][i], s_red[2][i]});
    before += __float_as_int(s_red[3][i]);
  }
  const bool none = s.m == -INFINITY && s.S == s.S;  // every logit is -inf
  const float ls = none ? 0.f : logf(s.S);
  if (tid == 0) {
    if (!(s.S == s.S)) flag_status(a.status, MTP_ERR_NONFINITE);
    if (!given && t != -1) flag_status(a.status, MTP_ERR_BAD_ARG);
    a.lp[r] = given ? (none ? -INFINITY : (xt - s.m) - ls) : 0.f;
    if (a.rank) a.rank[r] = given ? before : -1;
    if (a.ent) a.ent[r] = none ? 0.f : ls - s.T / s.S;
  }
  if (top == 0) return;
  // what reaches the sharpest bound, ranked by counting
  auto put = [&](unsigned long long k, int rank) {
    a.top_id[(long long)r * top + rank] = (int32_t)(0xFFFFFFFFu - (uint32_t)k);
    a.top_lp[(long long)r * top + rank] = (key_value(k) - s.m) - ls;
  };
  auto keys = [&](auto&& f) {  // eight threads per part's list, four keys each in flight
#pragma unroll 1
    for (int p = tid >> 3; p < P; p += kLpJoinThreads / 8) {
      const unsigned long long* list = a.keys + ((long long)r * P + p) * kLpList;
      const int n = s_cnt[p];
#pragma unroll 1
      for (int i = tid & 7; i < n; i += 32) {
        unsigned long long k[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) k[c] = i + 8 * c < n ? list[i + 8 * c] : 0ull;
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (k[c]) f(k[c]);
      }
    }
  };
  auto collect = [&]() {
    keys([&](unsigned long long k) {
      if (k >= bound) {
        const int i = atomicAdd(&s_n, 1);
        if (i < kLpLive) s_live[i] = k;
      }
    });
    __syncthreads();
  };
  bound = s_bound;
  collect();
  if (s_n > kLpJoinThreads) {
    // many are left, where parts have fewer tokens than alternatives: the
    // top-th largest of the threads' own maxima is a bound again
    unsigned long long mine = 0;
    keys([&](unsigned long long k) { mine = max(mine, k); });
    __syncthreads();
    s_live[tid] = mine;
    if (tid == 0) s_n = 0;
    __syncthreads();
    int rank = 0;
#pragma unroll 4
    for (int i = 0; i < kLpJoinThreads; ++i) rank += s_live[i] > mine || (s_live[i] == mine && i < tid);
    if (rank == top - 1 && mine > bound) s_bound = mine;
    __syncthreads();
    bound = s_bound;
    collect();
  }
  const int n = s_n;
  if (n <= kLpLive) {
    for (int i = tid; i < n; i += kLpJoinThreads) {
      const unsigned long long k = s_live[i];
      int rank = 0;
#pragma unroll 4
      for (int j = 0; j < n; ++j) rank += s_live[j] > k;
      if (rank < top) put(k, rank);
    }
  } else {
    // (long lists of many parts without a bound: each key against all)
    keys([&](unsigned long long k) {
      int rank = 0;
      for (int p = 0; p < P; ++p) {
        for (int i = 0; i < s_cnt[p]; ++i) rank += a.keys[((long long)r * P + p) * kLpList + i] > k;
      }
      if (rank < top) put(k, rank);
    });
  }
  for (int i = min(n, top) + tid; i < top; i += kLpJoinThreads) {  // past the last token that is possible
    a.top_id[(long long)r * top + i] = -1;
    a.top_lp[(long long)r * top + i] = -INFINITY;
  }
}

// Parts per row: the count with the least (waves of resident blocks) x (a
// part's elements + a block's fixed cost, counted in elements), the join's cost
// per part added. Many rows: whole waves; few rows: short parts. (The constants
// were tried at one size alone (256 rows of 152,064: 8000 gives 2 parts
// and 43 us, 1000 to 4000 give 7 parts and 54; the 110 was not varied.)
int lp_parts(int n, int V) {
  const long long slots = (long long)kLpBlocksPerSM * device_sm_count();
  const int most = std::min(kLpMaxParts, std::max(1, V / 2048));
  int best = 1;
  double least = 0;
  for (int p = 1; p <= most; ++p) {
    const double cost = (double)(((long long)n * p + slots - 1) / slots) * ((double)V / p + 8000.0) + 110.0 * p;
    if (p == 1 || cost < least) {
      least = cost;
      best = p;
    }
  }
  return best;
}

}  // namespace
}  // namespace mtp

using namespace mtp;

extern "C" {

size_t spec_logprobs_workspace_bytes(int32_t n, int32_t vocab, int32_t top) {
  if (n < 1 || vocab < 1 || top < 0 || top > kLpMaxTop) return 0;
  const size_t parts = (size_t)n * lp_parts(n, vocab);
  return parts * (sizeof(float4) + (top > 0 ? sizeof(uint4) + sizeof(unsigned long long) * kLpList : 0));
}

mtp_status spec_logprobs(mtp_stream stream, int32_t n, int32_t vocab, const void* d_logits, int64_t row_stride,
                         int32_t dtype, const int32_t* d_tok, int32_t top, float* d_logprob, int32_t* d_rank,
                         float* d_entropy, int32_t* d_top_id, float* d_top_lp, int32_t* d_status, void* d_workspace) {
  if (n < 0 || n > 65535 || vocab < 1 || vocab > (1 << 20) || top < 0 || top > kLpMaxTop ||
      (dtype != MTP_DTYPE_BF16 && dtype != MTP_DTYPE_F32))
    return MTP_ERR_BAD_ARG;
  if (n == 0) return MTP_OK;
  const int es = dtype == MTP_DTYPE_BF16 ? 2 : 4;
  if (!d_logits || !d_tok || !d_logprob || !d_workspace || (top > 0 && (!d_top_id || !d_top_lp)) ||
      (n > 1 && row_stride < vocab) || (reinterpret_cast<uintptr_t>(d_logits) & (es - 1)) != 0 ||
      (reinterpret_cast<uintptr_t>(d_workspace) & 15) != 0)
    return MTP_ERR_BAD_ARG;
  LpArgs a{d_logits, row_stride, d_tok, d_logprob, d_entropy, d_top_lp, d_rank, d_top_id, d_status, n, vocab, top,
           lp_parts(n, vocab), static_cast<float4*>(d_workspace), nullptr, nullptr};
  a.heads = reinterpret_cast<uint4*>(a.sums + (size_t)n * a.parts);
  a.keys = reinterpret_cast<unsigned long long*>(a.heads + (size_t)n * a.parts);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = launch_pdl(dtype == MTP_DTYPE_BF16 ? k_lp_part<MTP_DTYPE_BF16> : k_lp_part<MTP_DTYPE_F32>,
                             dim3(a.parts, n), dim3(kLpThreads + 32), 0, s, a);
  if (e == cudaSuccess) e = launch_pdl(k_lp_join, dim3(n), dim3(kLpJoinThreads), 0, s, a, dtype);
  count_launch(2);
  return e == cudaSuccess ? MTP_OK : MTP_ERR_CUDA;
}

}  // extern "C"
