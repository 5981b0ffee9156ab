// Page plans of the paged 4-bit cache: block tables, free pages and slot maps
// from device-side row lengths, in one launch (kv_page_plan).
//
// With held = ceil(cover / page) and want = ceil((keep + new) / page) the row
// gives rel = max(0, held - want) pages back or takes take = max(0, want -
// held). Three exclusive prefix sums over the rows (of rel, take and new) place
// everything: the k-th page given back (rows and table positions ascending)
// stands at F[top - 1 - k] with top = n_free + sum rel, and the k-th page taken
// is what stands at F[top - 1 - k], so page k of the takers is page k of the
// givers while k < sum rel and a stack entry after that. No entry that a plan
// reads is one that it writes:
//   table  reads positions below held, writes positions from held on
//   stack  reads F[top-1-k] for k in [sum rel, sum take), writes it for
//          k in [sum take, sum rel): one of the two ranges is empty
// so the blocks need no order among them. Each block redoes the row scan (12
// bytes per row from L2) rather than wait for another block or launch.
//
// Few rows are bound by latency: the scan, one binary search and two dependent
// loads; a block's lengths, its table rows and its stack entries are one load
// each. 8 rows of 4 positions: 4.3 us in a graph of such calls, of which a launch
// is about 2. Many rows with prompts are bound by instructions (5.7 M a call,
// the issue slots 62 % busy): the 64-bit scans that each block repeats, and the
// divisions and selects of each position. 512 rows and 512,000 positions: 9.0 us
// (8.4 MB, 0.9 TB/s).
#include <algorithm>
#include <mutex>

#include "common.cuh"
#include "kernels.h"

namespace mtp {

namespace {

constexpr int kPlanThreads = 512;
constexpr int kPlanMaxRows = 4096;
constexpr int kNo = 1 << 30;   // (pages of a row stay below 2^27)
constexpr int kPlanTokens = 4 * kPlanThreads;  // packed positions per block and turn

struct PlanArgs {
  int rows, page, max_pages, n_pages, max_tokens;
  const int32_t *cover, *keep, *fresh;
  int32_t *table, *free_pages, *cover_out, *start, *slot, *pos, *status;
};

// One row's lengths, checked. (32-bit throughout: a row's capacity is below
// 2^31, and two counts below that add up below 2^32.)
struct PlanRow {
  int held, want, fresh;  // fresh: appended positions that the packing counts
  int fault;              // 0, or 1 << status
  int keep, total;
};

__device__ __forceinline__ PlanRow plan_row(const PlanArgs& a, int r) {
  PlanRow p;
  const unsigned cap = (unsigned)a.page * a.max_pages, page = a.page;
  const int c = a.cover[r], k = a.keep[r], n = a.fresh[r];
  const unsigned cc = min((unsigned)max(c, 0), cap), total = (unsigned)k + (unsigned)n;
  p.held = (int)((cc + page - 1) / page);
  p.keep = k;
  p.total = (int)total;
  p.fresh = max(n, 0);
  p.fault = c != (int)cc || k < 0 || k > c || n < 0 ? 1 << MTP_ERR_BAD_ARG : (total > cap ? 1 << MTP_ERR_KV_CAPACITY : 0);
  p.want = p.fault ? p.held : (int)((total + page - 1) / page);
  return p;
}

// Last index i of [0, n) with v[i] <= x (v ascending, v[0] <= x).
__device__ __forceinline__ int last_le(const int* v, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (v[mid] <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Exclusive prefix over the block's threads of N sums, and their totals.
template <int N>
__device__ __forceinline__ void block_scan(long long (&v)[N], long long (&tot)[N], long long (*s_w)[kPlanThreads / 32]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long inc[N];
#pragma unroll
  for (int j = 0; j < N; ++j) {
    inc[j] = v[j];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xFFFFFFFFu, inc[j], o);
      if (lane >= o) inc[j] += u;
    }
    if (lane == 31) s_w[j][warp] = inc[j];
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < N; ++j) {
    long long before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kPlanThreads / 32; ++w) {
      const long long x = s_w[j][w];
      if (w < warp) before += x;
      all += x;
    }
    v[j] = before + inc[j] - v[j];
    tot[j] = all;
  }
}

__global__ void __launch_bounds__(kPlanThreads) k_page_plan(const PlanArgs a) {
  extern __shared__ int s_dyn[];
  int* s_start = s_dyn;               // [rows] first packed position
  int* s_take = s_start + a.rows;     // [rows] pages taken before the row
  int* s_rel = s_take + a.rows;       // [rows] pages given back before the row
  int* s_keep = s_rel + a.rows;       // [rows] positions kept
  int* s_held = s_keep + a.rows;      // [rows] pages held, bit 30: refused
  __shared__ long long s_w[2][2][kPlanThreads / 32];
  __shared__ int s_fault, s_granted;
  const int t = threadIdx.x;
  if (t == 0) s_fault = s_granted = 0;
  pdl_wait();
  pdl_trigger();

  // the row scans, consecutive rows per thread: packed positions and pages
  // held, then pages given back and taken by the rows that are in order
  const int per = (a.rows + kPlanThreads - 1) / kPlanThreads;
  const int r0 = min(t * per, a.rows), r1 = min(r0 + per, a.rows);
  long long v[2] = {0, 0}, tot[2];
  PlanRow p;  // (with a row a thread at most, made once)
  for (int r = r0; r < r1; ++r) {
    p = plan_row(a, r);
    v[0] += p.fresh;
    v[1] += p.held;
  }
  block_scan(v, tot, s_w[0]);
  const int n_tok = (int)min(tot[0], (long long)a.max_tokens);
  const long long n_free = a.n_pages - tot[1];
  const bool broken = n_free < 0;  // the lengths hold more pages than there are
  long long at = v[0];
  int fault = 0;
  v[0] = v[1] = 0;
  bool no = false;
  for (int r = r0; r < r1; ++r) {
    if (per > 1) p = plan_row(a, r);
    s_start[r] = (int)min(at, (long long)a.max_tokens);
    at += p.fresh;
    const bool fits = at <= a.max_tokens;
    no = p.fault || broken || !fits;
    s_keep[r] = p.keep;
    s_held[r] = p.held | (no ? kNo : 0);
    fault |= p.fault | (broken || !fits ? 1 << MTP_ERR_BAD_ARG : 0);
    if (!no) {
      v[0] += max(0, p.want - p.held);
      v[1] += max(0, p.held - p.want);
    }
  }
  block_scan(v, tot, s_w[1]);
  const int sum_rel = (int)tot[1];
  const int top = broken ? 0 : (int)n_free + sum_rel;
  long long tk = v[0], rl = v[1];
  int granted = 0;
  for (int r = r0; r < r1; ++r) {
    if (per > 1) {
      p = plan_row(a, r);
      no = s_held[r] & kNo;
    }
    s_take[r] = (int)tk;
    s_rel[r] = (int)rl;
    if (!no) {
      const int take = max(0, p.want - p.held);
      rl += max(0, p.held - p.want);
      tk += take;
      if (take && tk > top) {  // as is every later taker
        no = true;
        s_held[r] = p.held | kNo;
        fault |= 1 << MTP_ERR_KV_CAPACITY;
      } else if (take) {
        granted = (int)tk;
      }
    }
    if (blockIdx.x == 0) {
      a.start[r] = s_start[r];
      a.cover_out[r] = no ? min(max(a.cover[r], 0), a.page * a.max_pages) : p.total;
    }
  }
  if (blockIdx.x == 0 && t == 0) a.start[a.rows] = n_tok;
  if (fault) atomicOr(&s_fault, fault);
  if (granted) atomicMax(&s_granted, granted);
  __syncthreads();
  if (blockIdx.x == 0 && t == 0 && s_fault && a.status) atomicOr(a.status, s_fault);
  const int n_take = s_granted;

  auto checked = [&](int id) {
    if (id >= 0 && id < a.n_pages) return id;
    flag_status(a.status, MTP_ERR_BAD_ARG);
    return -1;
  };
  // the k-th page taken
  auto taken = [&](int k) {
    if (k < sum_rel) {
      const int r = last_le(s_rel, a.rows, k);
      // (a row that gives pages back is not refused)
      const int want = (s_keep[r] + a.fresh[r] + a.page - 1) / a.page;
      return checked(a.table[(long long)r * a.max_pages + want + (k - s_rel[r])]);
    }
    return checked(a.free_pages[top - 1 - k]);
  };
  const long long gt = (long long)blockIdx.x * kPlanThreads + t, nt = (long long)gridDim.x * kPlanThreads;

  // pages taken go into the tables; pages given back and not taken again go
  // onto the stack
  for (long long k = gt; k < n_take; k += nt) {
    const int r = last_le(s_take, a.rows, (int)k);
    a.table[(long long)r * a.max_pages + s_held[r] + ((int)k - s_take[r])] = taken((int)k);
  }
  for (long long k = n_take + gt; k < sum_rel; k += nt) a.free_pages[top - 1 - k] = taken((int)k);

  // slots and positions, four packed positions per thread and turn
  for (long long b = 4 * gt; b < a.max_tokens; b += 4 * nt) {
    int slot[4], pos[4];
    int r = b < n_tok ? last_le(s_start, a.rows, (int)b) : 0;
    int r_have = -1, at_have = -1, id_have = -1, keep = 0, held = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = (int)b + j;
      slot[j] = pos[j] = -1;
      if (i >= n_tok) continue;
      while (r + 1 < a.rows && s_start[r + 1] <= i) ++r;
      if (r != r_have) {
        keep = s_keep[r];
        held = s_held[r];
        r_have = r;
        at_have = -1;
      }
      pos[j] = keep + (i - s_start[r]);
      if (held & kNo) continue;
      const int at = pos[j] / a.page;
      if (at != at_have) {
        id_have = at < held ? checked(a.table[(long long)r * a.max_pages + at]) : taken(s_take[r] + (at - held));
        at_have = at;
      }
      if (id_have >= 0) slot[j] = id_have * a.page + (pos[j] - at * a.page);
    }
    const bool whole = b + 4 <= a.max_tokens && ((reinterpret_cast<uintptr_t>(a.slot) | reinterpret_cast<uintptr_t>(a.pos)) & 15) == 0;
    if (whole) {
      *reinterpret_cast<int4*>(a.slot + b) = make_int4(slot[0], slot[1], slot[2], slot[3]);
      *reinterpret_cast<int4*>(a.pos + b) = make_int4(pos[0], pos[1], pos[2], pos[3]);
    } else {
      for (int j = 0; j < 4 && b + j < a.max_tokens; ++j) {
        a.slot[b + j] = slot[j];
        a.pos[b + j] = pos[j];
      }
    }
  }
}

}  // namespace
}  // namespace mtp

using namespace mtp;

extern "C" mtp_status kv_page_plan(mtp_stream stream, int32_t rows, int32_t page, int32_t max_pages, int32_t n_pages,
                                   int32_t max_tokens, const int32_t* d_cover, const int32_t* d_keep,
                                   const int32_t* d_new, int32_t* d_table, int32_t* d_free, int32_t* d_cover_out,
                                   int32_t* d_start, int32_t* d_slot, int32_t* d_pos, int32_t* d_status) {
  if (rows < 1 || rows > kPlanMaxRows || page < 16 || page % 16 != 0 || max_pages < 1 || n_pages < 1 ||
      max_tokens < 0 || (long long)rows * max_pages >= (1LL << 31) || (long long)n_pages * page >= (1LL << 31) ||
      (long long)max_pages * page >= (1LL << 31))
    return MTP_ERR_BAD_ARG;
  if (!d_cover || !d_keep || !d_new || !d_table || !d_free || !d_cover_out || !d_start ||
      (max_tokens > 0 && (!d_slot || !d_pos)))
    return MTP_ERR_BAD_ARG;
  // blocks read the lengths to the end while others write
  const struct { const int32_t* p; long long n; } written[] = {
      {d_table, (long long)rows * max_pages}, {d_free, n_pages}, {d_cover_out, rows}, {d_start, rows + 1},
      {d_slot, max_tokens}, {d_pos, max_tokens}};
  for (const int32_t* in : {d_cover, d_keep, d_new})
    for (const auto& w : written)
      if (w.p < in + rows && in < w.p + w.n) return MTP_ERR_BAD_ARG;
  PlanArgs a{rows, page, max_pages, n_pages, max_tokens, d_cover, d_keep, d_new, d_table, d_free, d_cover_out,
             d_start, d_slot, d_pos, d_status};
  const int smem = 20 * rows;  // at 4096 rows more than the default limit
  {
    static std::mutex mu;
    static bool set[kMaxDevices] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= kMaxDevices) dev = 0;
    std::lock_guard<std::mutex> lock(mu);
    if (!set[dev]) {
      if (cudaFuncSetAttribute(k_page_plan, cudaFuncAttributeMaxDynamicSharedMemorySize, 20 * kPlanMaxRows) != cudaSuccess) {
        cudaGetLastError();
        return MTP_ERR_CUDA;
      }
      set[dev] = true;
    }
  }
  // one block up to kPlanTokens packed positions (the scan is the whole cost
  // there), then one per kPlanTokens, at most two per SM
  const int blocks = (int)std::min((long long)2 * device_sm_count(), ((long long)max_tokens + kPlanTokens - 1) / kPlanTokens);
  const cudaError_t e = launch_pdl(k_page_plan, dim3(std::max(1, blocks)), dim3(kPlanThreads), (size_t)smem,
                                   reinterpret_cast<cudaStream_t>(stream), a);
  count_launch();
  return e == cudaSuccess ? MTP_OK : MTP_ERR_CUDA;
}
