// What a target's attention layer does between its projection and its
// attention, in one pass (kv_q4_append_rope): norms of queries and keys per
// head, the rotation by position, queries (and on request keys) out, K and V
// into the paged 4-bit cache.
//
//   y = x rsqrt(mean(x^2) + eps) w                     (w: optional, with the norm)
//   (z_i, z_{i+h}) = (y_i c - y_{i+h} s, y_{i+h} c + y_i s),  h = rot / 2, i < h
//   c, s = cos, sin (pos f_i); dimensions from rot on pass through
//
// Angles. f_i is held as a fraction of a turn in units of 2^-64, so pos f_i
// modulo a turn is one wrapping 64-bit product, exact but for f_i's own rounding
// (2^-53 of it): at position 2^20 that is 2^-33 radians of the fastest pair. The nearest 64th of
// a turn comes off and is looked up, the rest (0.05 radians at most) goes through
// the first terms of the sine's and cosine's series; the two are joined by the
// addition theorems. Everything is held in two floats, good to 2^-32.
//
// What is kept of a key is discrete: with results off by 2^-22 some of a few million
// elements fall on the other side of a 4-bit border than the exact ones. So a
// row of keys that comes so near a border, of a code or of a scale, that fp32 cannot
// tell the side (one of 30) is taken again in two floats per value, and rounded to
// odd before it is compared, so that no value that is not on a border is taken for
// one that is. Queries, which are only rounded, are fp32.
//
// Layout. A row of dh elements is dh / 8 lanes' work. A lane holds two runs of
// four elements, A and B, such that a rotated pair is in one lane: A at 4 l and
// B at h + 4 l for the first h / 4 lanes, the halves of what is not rotated in
// the same way for the others. The sum of squares and the maxima of 16 elements
// (four neighbouring lanes) are the only exchanges. That needs rot % 32 == 0 and
// 4-element alignment; every other call takes the general kernel, which stages
// a row in shared memory.
//
// V is what kv_q4_append makes of it, bit for bit.
//
// What it measured, 24 query heads and 4 KV heads of 256, a quarter of each rotated: 16,383 positions 140 us for 522 MB,
// 3.7 TB/s; with the whole head rotated 179 us, from fp32 192 us (5.3 TB/s); 48 query heads 209 us (4.4 TB/s); 8 and 2
// heads of 128 37 us; 32 positions 4.4 us. The issue slots are 60 % busy (106 M instructions): four rows of queries are some
// 350 of a warp's, a row of keys with its values 700, and the block's warps wait for one another once in two positions. The
// general kernel takes 370 us where this one takes 179.
#include <algorithm>
#include <cfloat>
#include <cmath>

#include "common.cuh"
#include "kernels.h"
#include "ranges.h"
#include "q4.cuh"

namespace mtp {

namespace {

constexpr int kRopeThreads = 256;  // of the general kernel
constexpr int kMostWarps = 10;     // of a block of the other
constexpr int kBatch = 4;          // rows of queries a group of lanes takes, loaded together

struct RopeArgs {
  const void* x[3];            // Q, K, V
  long long ts[3], hs[3];      // strides in elements
  void *q_out, *k_out;
  const float* norm[2];        // of Q, K
  uint8_t* cache[2];
  const int32_t* exp[2];
  const int32_t *pos, *slot;
  int32_t* status;
  int tokens, n_q, n_kv, page, n_slots;
  int q_parts, parts;          // warps per position: those of its queries, all
  float eps;
  float2 quarter[17];          // cos of the 64ths of a turn up to a quarter, in two floats
  mtp_rope rope;
};

// ------------------------------------------------------------ two floats

// A value as hi + lo.
struct Two {
  float hi, lo;
};

__device__ __forceinline__ Two two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}

// a b, plus c (small beside it), with hi the nearest float.
__device__ __forceinline__ Two two_prod(float a, float b, float c) {
  const float p = __fmul_rn(a, b);
  return {p, __fadd_rn(__fmaf_rn(a, b, -p), c)};
}

// a c - b s; the low parts' products of low parts are left out (2^-48).
__device__ __forceinline__ Two turn_one(Two a, Two b, float ch, float cl, float sh, float sl) {
  const Two p = two_prod(a.hi, ch, __fmaf_rn(a.hi, cl, a.lo * ch)), q = two_prod(b.hi, sh, __fmaf_rn(b.hi, sl, b.lo * sh));
  const Two r = two_sum(p.hi, -q.hi);
  return {r.hi, __fadd_rn(r.lo, __fsub_rn(p.lo, q.lo))};
}

// The nearest float. (Where an infinity made the low part a NaN, the high one.)
__device__ __forceinline__ float nearest(Two z) {
  const float y = z.hi + z.lo;
  return y == y ? y : z.hi;
}

// The value rounded to odd in 12 bits: cut off, with its last bit set where
// something was. So it lies on the same side of any number of 11 bits or fewer as
// the value, or on it as the value does.
__device__ __forceinline__ float to_odd(Two z) {
  const float y = nearest(z), rest = __fadd_rn(__fsub_rn(z.hi, y), z.lo);
  // (a rest that points to 0 takes a step of y off before the cut; not finite: as it is)
  const uint32_t u = __float_as_uint(y) - (rest * y < 0.f ? 1u : 0u);
  return __uint_as_float((u & 0xFFFFF000u) | ((u & 0xFFFu) != 0 || (rest != 0.f && y != 0.f) ? 0x1000u : 0u));
}

struct CosSin {
  float ch, cl, sh, sl;
};

// cos and sin of pos x turn.
__device__ __forceinline__ CosSin turn_cs(int pos, uint64_t turn, const float2* quarter) {
  const uint64_t p = (uint64_t)(uint32_t)pos * turn;
  const uint32_t k = (uint32_t)((p + (1ull << 57)) >> 58) & 63;
  const int64_t r = (int64_t)(p - ((uint64_t)k << 58));  // a 128th of a turn at most
  // in radians: 2 pi = 6.28318548 - 1.74845553e-7 in two floats
  const float rh = (float)r * 0x1p-64f, rl = (float)(r - (int64_t)(float)r) * 0x1p-64f;
  const Two d = two_prod(rh, 6.28318548f, __fmaf_rn(rh, -1.74845553e-7f, rl * 6.28318548f));
  const float d2 = d.hi * d.hi;
  const float cc = d2 * __fmaf_rn(d2, -1.f / 24, 0.5f);                                     // 1 - cos
  const float sl = __fmaf_rn(d.hi * d2, __fmaf_rn(d2, 1.f / 120, -1.f / 6), d.lo);          // sin - d.hi
  const float2 C = quarter[k & 15], S = quarter[16 - (k & 15)];
  const Two t = two_prod(S.x, d.hi, __fmaf_rn(S.x, sl, S.y * d.hi)), u = two_prod(C.x, d.hi, __fmaf_rn(C.x, sl, C.y * d.hi));
  const Two a = two_sum(C.x, -t.hi), b = two_sum(S.x, u.hi);
  const float al = a.lo + (C.y - t.lo - C.x * cc), bl = b.lo + (S.y + u.lo - S.x * cc);
  const float ch = a.hi + al, cl = al - (ch - a.hi), sh = b.hi + bl, sl2 = bl - (sh - b.hi);
  switch (k >> 4) {
    case 0: return {ch, cl, sh, sl2};
    case 1: return {-sh, -sl2, ch, cl};
    case 2: return {-ch, -cl, -sh, -sl2};
    default: return {sh, sl2, -ch, -cl};
  }
}

// 1 / sqrt(sum / dh + eps): one Newton step on the instruction's result.
__device__ __forceinline__ Two root(Two sum, float inv_dh, float eps) {
  Two m = two_sum(sum.hi * inv_dh, eps);  // (inv_dh: a power of two)
  m.lo = fmaf(sum.lo, inv_dh, m.lo);
  const float r = rsqrtf(m.hi + m.lo);
  const Two t = two_prod(r, r, 0.f);
  const float e = __fmaf_rn(-m.hi, t.hi, 1.f) - m.hi * t.lo - m.lo * t.hi, c = 0.5f * r * e;
  return {r, isfinite(c) ? c : 0.f};
}

// x r w, w optional.
__device__ __forceinline__ Two scaled(float x, Two r, float w) {
  const Two p = two_prod(r.hi, w, r.lo * w);
  return two_prod(x, p.hi, x * p.lo);
}

// The e4m3 scale of 16 elements whose largest magnitude is amax, and its value.
// (The correctly rounded quotient by 6: one correction of the product.)
__device__ __forceinline__ uint32_t scale4(float amax, float& s) {
  constexpr float kSixth = 1.f / 6.f;
  const float q0 = amax * kSixth, q = fmaf(fmaf(-q0, 6.f, amax), kSixth, q0);
  uint16_t sc;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(sc) : "f"(0.f), "f"(q));
  s = f16x2_to_f(e4m3x2_to_f16x2(sc)).x;
  return sc & 0xFFu;
}

// The correctly rounded quotient of y by the block scale s, rs near 1 / s. A y of 12
// bits or fewer is on a border between two codes (3 bits times the scale's 4) or 2^-12
// of it away, so the quotient is on a border exactly where y is.
__device__ __forceinline__ float over(float y, float s, float rs) {
  const float m = fminf(fabsf(y), 8.f * s), q = m * rs;  // (the largest code is 6; a quotient past fp32's range has none)
  return copysignf(fmaf(fmaf(-q, s, m), rs, q), y);      // (-0 stays -0)
}

__device__ __forceinline__ uint32_t codes4(const float (&q)[4]) {
  uint16_t c;
  asm("{\n\t.reg .b8 b0, b1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "mov.b16 %0, {b0, b1};\n\t}"
      : "=h"(c)
      : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]));
  return c;
}

// Four elements as they are in memory, and as fp32.
template <int DT>
struct Raw4 {
  uint32_t w[DT == MTP_DTYPE_BF16 ? 2 : 4];
};

template <int DT>
__device__ __forceinline__ Raw4<DT> load4(const void* src, long long at) {
  Raw4<DT> r;
  if constexpr (DT == MTP_DTYPE_BF16) {
    asm volatile("ld.global.L1::no_allocate.v2.u32 {%0,%1}, [%2];"
                 : "=r"(r.w[0]), "=r"(r.w[1])
                 : "l"(static_cast<const uint16_t*>(src) + at));
  } else {
    const uint4 u = ld_stream(static_cast<const float*>(src) + at);
    r.w[0] = u.x, r.w[1] = u.y, r.w[2] = u.z, r.w[3] = u.w;
  }
  return r;
}

template <int DT>
__device__ __forceinline__ void widen4(const Raw4<DT>& r, float (&x)[4]) {
  if constexpr (DT == MTP_DTYPE_BF16) {
    x[0] = bf16lo(r.w[0]), x[1] = bf16hi(r.w[0]), x[2] = bf16lo(r.w[1]), x[3] = bf16hi(r.w[1]);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = __uint_as_float(r.w[e]);
  }
}

template <int DT>
__device__ __forceinline__ void store4(void* dst, long long at, const float (&x)[4]) {
  if (DT == MTP_DTYPE_BF16) {
    uint2 w;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.x) : "f"(x[1]), "f"(x[0]));
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.y) : "f"(x[3]), "f"(x[2]));
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(dst) + at) = w;
  } else {
    *reinterpret_cast<float4*>(static_cast<float*>(dst) + at) = make_float4(x[0], x[1], x[2], x[3]);
  }
}

// Where a head's row goes in the cache, in rows.
__device__ __forceinline__ long long cache_row(const RopeArgs& a, int head, int slot) {
  const int pg = slot / a.page;
  return ((long long)pg * a.n_kv + head) * a.page + (slot - pg * a.page);
}

// The slot of a position that is appended, -1 else.
__device__ __forceinline__ int slot_of(const RopeArgs& a, int t, int pos, bool tell) {
  const int slot = a.slot[t];
  if (slot == -1 || (slot >= 0 && slot < a.n_slots && pos >= 0)) return slot;
  if (tell) flag_status(a.status, MTP_ERR_BAD_ARG);
  return -1;
}

// Codes and scale of 16 elements, a group of four lanes, 4 each, at their head's exponent: `mx` is the largest
// magnitude's bits (0x7F, NaN, where one of the elements is not finite: the row shows what it was given).
struct Block4 {
  float s, rs;  // the scale at the elements' size and its inverse
  uint32_t sc;
};

__device__ __forceinline__ uint32_t most4(const float (&y)[4]) {
  uint32_t mx = 0;  // (magnitudes as whole numbers: an infinity or a NaN is the largest)
#pragma unroll
  for (int e = 0; e < 4; ++e) mx = max(mx, __float_as_uint(y[e]) & 0x7FFFFFFFu);
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
  return mx;
}

__device__ __forceinline__ Block4 block4(uint32_t mx, float down, float up) {
  Block4 b;
  b.sc = scale4(fminf(__uint_as_float(mx) * down, FLT_MAX), b.s);
  b.s *= up;  // exact
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(b.rs) : "f"(b.s));
  if (mx >= 0x7F800000u) b.sc = 0x7F;
  return b;
}

// Elements of 12 bits at most. By whole warps.
__device__ __forceinline__ uint32_t quantize4(const float (&y)[4], float down, float up, uint32_t& sc) {
  const Block4 b = block4(most4(y), down, up);
  float q[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) q[e] = over(y[e], b.s, b.rs);
  const uint32_t code = codes4(q);
  sc = b.sc;
  return sc == 0 || sc == 0x7F ? 0u : code;
}

// fp32 elements off by at most err each: `near` where a code's border or the scale's may lie between them and the exact
// ones. Borders between codes are at 1, 3, 5, 7, 10, 14 and 20 quarters of the scale. By whole warps.
// `exact`: they are what they are.
__device__ __forceinline__ uint32_t quantize4_near(const float (&y)[4], const float (&err)[4], float down, float up, bool exact, uint32_t& sc,
                                                   bool& near) {
  float off = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) off = fmaxf(off, err[e]);
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) off = fmaxf(off, __shfl_xor_sync(0xFFFFFFFFu, off, o));
  const uint32_t mx = most4(y);
  const Block4 b = block4(mx, down, up);
  float other;
  const float top = __uint_as_float(mx);
  near = scale4(fminf((top + off) * down, FLT_MAX), other) != scale4(fminf(fmaxf(top - off, 0.f) * down, FLT_MAX), other);
  float q[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    q[e] = y[e] * b.rs;
    const float t = fabsf(q[e]) * 4.f, whole = rintf(t);
    // (the quotient itself is off by 2^-22 of at most 24 quarters; what is not finite has no side)
    near |= fabsf(t - whole) <= fmaf(err[e] * b.rs, 4.f, 0x1p-17f) && t < 24.f && !exact;
    if (exact) q[e] = over(to_odd({y[e], 0.f}), b.s, b.rs);
  }
  const uint32_t code = codes4(q);
  sc = b.sc;
  near = near && sc != 0x7F;
  return sc == 0 || sc == 0x7F ? 0u : code;
}

// A warp's keys in two floats: A and B of row `u` as they came, at the factors' place `cs`; codes of both runs (low and high
// half) and scales (a byte each). Out of line: few rows come here, and the others need the registers.
template <int DH>
__device__ __noinline__ uint2 exact_keys(float4 A4, float4 B4, const float* w, int ea, int eb, float eps, const CosSin* cs, bool mine, int exp) {
  constexpr int kLanes = DH / 8;
  const float A[4] = {A4.x, A4.y, A4.z, A4.w}, B[4] = {B4.x, B4.y, B4.z, B4.w};
  Two ka[4], kb[4];
  if (w) {
    Two sum = {0.f, 0.f};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float x = e < 4 ? A[e & 3] : B[e & 3];
      const Two p = two_prod(x, x, 0.f), n = two_sum(sum.hi, p.hi);
      sum = {n.hi, n.lo + (sum.lo + p.lo)};
    }
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) {
      const float hi = __shfl_xor_sync(0xFFFFFFFFu, sum.hi, o), lo = __shfl_xor_sync(0xFFFFFFFFu, sum.lo, o);
      const Two n = two_sum(sum.hi, hi);
      sum = {n.hi, n.lo + (sum.lo + lo)};
    }
    const Two r = root(sum, 1.f / DH, eps);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      ka[e] = scaled(A[e], r, w[ea + e]);
      kb[e] = scaled(B[e], r, w[eb + e]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      ka[e] = {A[e], 0.f};
      kb[e] = {B[e], 0.f};
    }
  }
  if (mine) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const CosSin c = cs[e];
      const Two x = ka[e], y = kb[e];
      ka[e] = turn_one(x, y, c.ch, c.cl, c.sh, c.sl);
      kb[e] = turn_one(y, x, c.ch, c.cl, -c.sh, -c.sl);
    }
  }
  __syncwarp();
  float ya[4], yb[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    ya[e] = to_odd(ka[e]);
    yb[e] = to_odd(kb[e]);
  }
  uint32_t sa, sb;
  const uint32_t ca = quantize4(ya, pow2i(-exp), pow2i(exp), sa), cb = quantize4(yb, pow2i(-exp), pow2i(exp), sb);
  return make_uint2(ca | cb << 16, sa | sb << 8);
}

// Codes of two runs and their scales to the cache row at byte `to`.
template <int DH>
__device__ __forceinline__ void store_codes(const RopeArgs& a, int side, long long to, int ea, int eb, uint32_t ca, uint32_t cb, uint32_t sa, uint32_t sb) {
  uint8_t* row = a.cache[side] + to;
  *reinterpret_cast<uint16_t*>(row + ea / 2) = (uint16_t)ca;
  *reinterpret_cast<uint16_t*>(row + eb / 2) = (uint16_t)cb;
  if ((ea & 15) == 0) row[DH / 2 + ea / 16] = (uint8_t)sa;
  if ((eb & 15) == 0) row[DH / 2 + eb / 16] = (uint8_t)sb;
  if (sa == 0x7F || sb == 0x7F) flag_status(a.status, MTP_ERR_NONFINITE);
}

// Two fp32 values for one instruction.
struct Pair {
  unsigned long long v;
};
__device__ __forceinline__ Pair pair(float x, float y) {
  Pair p;
  asm("mov.b64 %0, {%1, %2};" : "=l"(p.v) : "f"(x), "f"(y));
  return p;
}
__device__ __forceinline__ float2 both(Pair p) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(p.v));
  return f;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
  Pair p;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(p.v) : "l"(a.v), "l"(b.v));
  return p;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
  Pair p;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(p.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return p;
}

// Sums of four rows over kLanes lanes: a lane gets that of row 2 (lane & 1) + (lane >> 1 & 1).
template <int kLanes>
__device__ __forceinline__ float sum_rows(const float (&s)[4], int lane) {
  const bool b0 = lane & 1, b1 = lane & 2;
  float u = b0 ? s[2] : s[0], v = b0 ? s[3] : s[1];
  u += __shfl_xor_sync(0xFFFFFFFFu, b0 ? s[0] : s[2], 1);
  v += __shfl_xor_sync(0xFFFFFFFFu, b0 ? s[1] : s[3], 1);
  float w = b1 ? v : u;
  w += __shfl_xor_sync(0xFFFFFFFFu, b1 ? u : v, 2);
#pragma unroll
  for (int o = 4; o < kLanes; o <<= 1) w += __shfl_xor_sync(0xFFFFFFFFu, w, o);
  return w;
}

// A row's two runs as pairs.
template <int DT>
__device__ __forceinline__ void runs(const Raw4<DT>& x, const Raw4<DT>& y, Pair (&A)[2], Pair (&B)[2]) {
  float u[4], v[4];
  widen4<DT>(x, u);
  widen4<DT>(y, v);
  A[0] = pair(u[0], u[1]), A[1] = pair(u[2], u[3]);
  B[0] = pair(v[0], v[1]), B[1] = pair(v[2], v[3]);
}

__device__ __forceinline__ float square(const Pair (&A)[2], const Pair (&B)[2]) {
  const float2 s = both(fma2(A[0], A[0], fma2(A[1], A[1], fma2(B[0], B[0], mul2(B[1], B[1])))));
  return s.x + s.y;
}

// z = r (x w c - x' w' s): the weights go into the factors, once for all heads of an item.
struct Factors {
  Pair fa[2], fb[2], ga[2], gb[2];
  __device__ __forceinline__ Factors(float4 wa, float4 wb, const CosSin* cs, bool mine) {
    const float va[4] = {wa.x, wa.y, wa.z, wa.w}, vb[4] = {wb.x, wb.y, wb.z, wb.w};
    float c[4], s[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      c[e] = mine ? cs[e].ch : 1.f;
      s[e] = mine ? cs[e].sh : 0.f;
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      fa[e] = pair(va[2 * e] * c[2 * e], va[2 * e + 1] * c[2 * e + 1]);
      fb[e] = pair(vb[2 * e] * c[2 * e], vb[2 * e + 1] * c[2 * e + 1]);
      ga[e] = pair(-vb[2 * e] * s[2 * e], -vb[2 * e + 1] * s[2 * e + 1]);
      gb[e] = pair(va[2 * e] * s[2 * e], va[2 * e + 1] * s[2 * e + 1]);
    }
  }
  // what run x brings to the other one (nothing where nothing is turned: an infinity times 0 would show)
  __device__ __forceinline__ static void cross(const Pair (&x)[2], const Pair (&g)[2], bool mine, Pair (&y)[2]) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      y[e] = mul2(x[e], g[e]);
      y[e].v = mine ? y[e].v : 0ull;
    }
  }
  __device__ __forceinline__ static void turn(const Pair (&x)[2], const Pair (&f)[2], const Pair (&y)[2], float r, float (&z)[4]) {
    const Pair r2 = pair(r, r);
    const float2 u = both(mul2(fma2(x[0], f[0], y[0]), r2)), v = both(mul2(fma2(x[1], f[1], y[1]), r2));
    z[0] = u.x, z[1] = u.y, z[2] = v.x, z[3] = v.y;
  }
};

// Queries of up to kBatch x (32 / kLanes) heads.
template <int DH, int DT>
__device__ __forceinline__ void rope_queries(const RopeArgs& a, const Raw4<DT> (&ra)[kBatch], const Raw4<DT> (&rb)[kBatch], const Factors& F, bool norm,
                                             bool mine, int t, int pos, int h0, int ea, int eb, int lane) {
  constexpr int kLanes = DH / 8, kGroups = 32 / kLanes;
  const long long at = ((long long)t * a.n_q + h0) * DH;
  if (pos < 0) {  // padding
    const float none[4] = {0.f, 0.f, 0.f, 0.f};
    for (int u = 0; u < kBatch && h0 + u * kGroups < a.n_q; ++u) {
      store4<DT>(a.q_out, at + u * kGroups * DH + ea, none);
      store4<DT>(a.q_out, at + u * kGroups * DH + eb, none);
    }
    return;
  }
  Pair A[kBatch][2], B[kBatch][2];
  float sq[kBatch], r = 1.f;
#pragma unroll
  for (int u = 0; u < kBatch; ++u) {
    runs<DT>(ra[u], rb[u], A[u], B[u]);
    sq[u] = square(A[u], B[u]);
  }
  if (norm) r = rsqrtf(fmaf(sum_rows<kLanes>(sq, lane), 1.f / DH, a.eps));
#pragma unroll
  for (int u = 0; u < kBatch; ++u) {
    const float ru = norm ? __shfl_sync(0xFFFFFFFFu, r, (lane & ~3) | (u >> 1) | ((u & 1) << 1)) : 1.f;
    Pair x[2], y[2];
    float ya[4], yb[4];
    Factors::cross(B[u], F.ga, mine, x);
    Factors::cross(A[u], F.gb, mine, y);
    Factors::turn(A[u], F.fa, x, ru, ya);
    Factors::turn(B[u], F.fb, y, ru, yb);
    if (h0 + u * kGroups < a.n_q) {
      store4<DT>(a.q_out, at + u * kGroups * DH + ea, ya);
      store4<DT>(a.q_out, at + u * kGroups * DH + eb, yb);
    }
  }
}

// Keys and values of 32 / kLanes heads.
template <int DH, int DT>
__device__ __forceinline__ void rope_keys(const RopeArgs& a, const Raw4<DT> (&ra)[kBatch], const Raw4<DT> (&rb)[kBatch], const Factors& F, const float* w,
                                          const CosSin* cs, bool mine, int t, int pos, int h0, int ea, int eb, bool tell) {
  constexpr int kLanes = DH / 8;
  const bool head = h0 < a.n_kv;
  const int slot = slot_of(a, t, pos, tell);
  Pair A[2], B[2], x[2], y[2];
  runs<DT>(ra[0], rb[0], A, B);
  float r = 1.f;
  if (w) {
    float sum = square(A, B);
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    r = rsqrtf(fmaf(sum, 1.f / DH, a.eps));
  }
  float ya[4], yb[4];
  Factors::cross(B, F.ga, mine, x);
  Factors::cross(A, F.gb, mine, y);
  Factors::turn(A, F.fa, x, r, ya);
  Factors::turn(B, F.fb, y, r, yb);
  if (slot >= 0) {  // (the same for the warp)
    // off by 2^-19 of (|x w c| + |x' w' s|) r at most: the sum's 13 roundings, half of which reach its root, the root's two
    // steps, and a step or two each of the factors, products and their sum
    const float step = r * 0x1p-19f;
    float da[4], db[4];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float2 p = both(mul2(A[e], F.fa[e])), q = both(x[e]), v = both(mul2(B[e], F.fb[e])), z = both(y[e]);
      da[2 * e] = step * (fabsf(p.x) + fabsf(q.x)), da[2 * e + 1] = step * (fabsf(p.y) + fabsf(q.y));
      db[2 * e] = step * (fabsf(v.x) + fabsf(z.x)), db[2 * e + 1] = step * (fabsf(v.y) + fabsf(z.y));
    }
    const int exp = head ? head_exp(a.exp[0], h0) : 0;
    const bool exact = !w && !mine;  // neither scaled nor turned
    if (exact) {
#pragma unroll
      for (int e = 0; e < 4; ++e) da[e] = db[e] = 0.f;
    }
    uint32_t sa, sb;
    bool na, nb;
    uint32_t ca = quantize4_near(ya, da, pow2i(-exp), pow2i(exp), exact, sa, na), cb = quantize4_near(yb, db, pow2i(-exp), pow2i(exp), exact, sb, nb);
    if (__any_sync(0xFFFFFFFFu, (na || nb) && head)) {
      const float2 p = both(A[0]), q = both(A[1]), v = both(B[0]), z = both(B[1]);
      const uint2 again = exact_keys<DH>(make_float4(p.x, p.y, q.x, q.y), make_float4(v.x, v.y, z.x, z.y), w, ea, eb, a.eps, cs, mine, exp);
      ca = again.x & 0xFFFFu;
      cb = again.x >> 16;
      sa = again.y & 0xFFu;
      sb = again.y >> 8;
    }
    const long long to = head ? cache_row(a, h0, slot) * q4_row_bytes(DH) : 0;
    if (head) store_codes<DH>(a, 0, to, ea, eb, ca, cb, sa, sb);
    float va[4], vb[4];
    widen4<DT>(ra[1], va);
    widen4<DT>(rb[1], vb);
    if (DT != MTP_DTYPE_BF16) {  // (bf16 has 8 bits)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        va[e] = to_odd({va[e], 0.f});
        vb[e] = to_odd({vb[e], 0.f});
      }
    }
    const int vexp = head ? head_exp(a.exp[1], h0) : 0;
    ca = quantize4(va, pow2i(-vexp), pow2i(vexp), sa);
    cb = quantize4(vb, pow2i(-vexp), pow2i(vexp), sb);
    if (head) store_codes<DH>(a, 1, to, ea, eb, ca, cb, sa, sb);
  }
  if (a.k_out && head) {
    if (pos < 0) {
#pragma unroll
      for (int e = 0; e < 4; ++e) ya[e] = yb[e] = 0.f;
    }
    const long long at = ((long long)t * a.n_kv + h0) * DH;
    store4<DT>(a.k_out, at + ea, ya);
    store4<DT>(a.k_out, at + eb, yb);
  }
}

// Blocks stay and take two positions at a time, whose angles were made while the two before were worked on. An item is
// kBatch x (32 / kLanes) heads of the queries, or 32 / kLanes heads of the keys and values, which take longer: a warp that
// has those at one position has queries at the other. Its next rows are on their way while it works on those it has.
template <int DH, int DT>
__global__ void __launch_bounds__(32 * kMostWarps, 2) k_rope_rows(const __grid_constant__ RopeArgs a) {
  constexpr int kLanes = DH / 8, kGroups = 32 / kLanes;
  __shared__ CosSin s_cs[4][DH / 2];
  __shared__ uint64_t s_turn[DH / 2];
  __shared__ float2 s_quarter[17];
  const int lane = threadIdx.x & 31, l = lane % kLanes, grp = lane / kLanes;
  const int warp = __shfl_sync(0xFFFFFFFFu, (int)threadIdx.x >> 5, 0), warps = blockDim.x >> 5;
  const int half = a.rope.rot_dim / 2, turned = half / 4, rest = (DH - a.rope.rot_dim) / 2;
  const bool mine = l < turned;
  const int ea = mine ? 4 * l : 2 * half + 4 * (l - turned), eb = mine ? half + 4 * l : ea + rest;
  if (threadIdx.x < 17) s_quarter[threadIdx.x] = a.quarter[threadIdx.x];
  for (int i = threadIdx.x; i < half; i += blockDim.x) s_turn[i] = a.rope.turn[i];
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  const int step = gridDim.x, parts = a.parts;
  // of the block's positions k and k + 1
  auto angles = [&](int k) {
    for (int i = threadIdx.x; i < 2 * half; i += blockDim.x) {
      const int y = i >= half, t = blockIdx.x + (k + y) * step;
      if (t < a.tokens) s_cs[(k + y) & 3][i - y * half] = turn_cs(max(a.pos[t], 0), s_turn[i - y * half], s_quarter);
    }
  };
  // a warp's i-th item of position k
  auto part_of = [&](int k, int i) {
    const int p = i + (k & 1 ? parts / 2 : 0);
    return p < parts ? p : p - parts;
  };
  Raw4<DT> ra[kBatch], rb[kBatch];
  auto fetch = [&](int k, int i) {
    const int t = blockIdx.x + k * step;
    if (t >= a.tokens || i >= parts) return;
    const int part = part_of(k, i);
    const bool is_q = part < a.q_parts;
    const int h0 = is_q ? part * kBatch * kGroups + grp : (part - a.q_parts) * kGroups + grp, heads = is_q ? a.n_q : a.n_kv;
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int side = is_q ? 0 : 1 + u, h = is_q ? h0 + u * kGroups : h0;
      if (h < heads && (is_q || u < 2)) {
        const long long at = (long long)t * a.ts[side] + (long long)h * a.hs[side];
        ra[u] = load4<DT>(a.x[side], at + ea);
        rb[u] = load4<DT>(a.x[side], at + eb);
      }
    }
  };
  fetch(0, warp);
  angles(0);
#pragma unroll 1
  for (int k = 0;; ++k) {
    const int t = blockIdx.x + k * step;
    if (t >= a.tokens) break;
    if ((k & 1) == 0) __syncthreads();
    const int pos = a.pos[t];
    const CosSin* cs = s_cs[k & 3] + 4 * l;
#pragma unroll 1
    for (int i = warp; i < parts; i += warps) {
      const int part = part_of(k, i);
      const bool is_q = part < a.q_parts;
      const int h0 = is_q ? part * kBatch * kGroups + grp : (part - a.q_parts) * kGroups + grp;
      Raw4<DT> xa[kBatch], xb[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        xa[u] = ra[u];
        xb[u] = rb[u];
      }
      if (i + warps < parts) fetch(k, i + warps);
      else fetch(k + 1, warp);
      const float* w = a.norm[is_q ? 0 : 1];
      float4 wa = make_float4(1.f, 1.f, 1.f, 1.f), wb = wa;
      if (w) {
        wa = *reinterpret_cast<const float4*>(w + ea);
        wb = *reinterpret_cast<const float4*>(w + eb);
      }
      const Factors F(wa, wb, cs, mine);
      if (is_q) rope_queries<DH, DT>(a, xa, xb, F, w != nullptr, mine, t, pos, h0, ea, eb, lane);
      else rope_keys<DH, DT>(a, xa, xb, F, w, cs, mine, t, pos, h0, ea, eb, part == a.q_parts && lane == 0);
    }
    if (k & 1) angles(k + 1);
  }
}

// Any rotated width and any strides: a block per position, whose angles it makes once, a warp per head, the row in shared
// memory. Lane l has elements l, l + 32, ... of the row, so neighbouring lanes read neighbouring elements; 16 of them are
// half a warp. Keys in two floats, all of them.
template <int DH, int DT>
__global__ void __launch_bounds__(kRopeThreads) k_rope_any(const __grid_constant__ RopeArgs a) {
  constexpr int kRow = q4_row_bytes(DH), kN = DH / 32;
  __shared__ Two s_row[kRopeThreads / 32][DH];
  __shared__ CosSin s_cs[DH / 2];
  __shared__ float2 s_quarter[17];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, heads = a.n_q + 2 * a.n_kv, t = blockIdx.x, half = a.rope.rot_dim / 2;
  const int pos = a.pos[t];
  if (threadIdx.x < 17) s_quarter[threadIdx.x] = a.quarter[threadIdx.x];
  __syncthreads();
  for (int i = threadIdx.x; i < half; i += kRopeThreads) s_cs[i] = turn_cs(max(pos, 0), a.rope.turn[i], s_quarter);
  __syncthreads();
  const int slot = slot_of(a, t, pos, threadIdx.x == 0);
  Two* row_s = s_row[warp];
  float* flat = reinterpret_cast<float*>(row_s);
#pragma unroll 1
  for (int h = warp; h < heads; h += kRopeThreads / 32) {
    const int side = h < a.n_q ? 0 : (h < a.n_q + a.n_kv ? 1 : 2), g = h - (side == 0 ? 0 : (side == 1 ? a.n_q : a.n_q + a.n_kv));
    const long long from = (long long)t * a.ts[side] + (long long)g * a.hs[side];
    const float* w = side < 2 ? a.norm[side] : nullptr;
    float x[kN];
#pragma unroll
    for (int i = 0; i < kN; ++i) x[i] = load_elem(a.x[side], DT, from + 32 * i + lane);
    __syncwarp();
    if (side == 1) {
      Two sum = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const Two p = two_prod(x[i], x[i], 0.f), n = two_sum(sum.hi, p.hi);
        sum = {n.hi, n.lo + (sum.lo + p.lo)};
      }
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const float hi = __shfl_xor_sync(0xFFFFFFFFu, sum.hi, o), lo = __shfl_xor_sync(0xFFFFFFFFu, sum.lo, o);
        const Two n = two_sum(sum.hi, hi);
        sum = {n.hi, n.lo + (sum.lo + lo)};
      }
      const Two r = root(sum, 1.f / DH, a.eps);
#pragma unroll
      for (int i = 0; i < kN; ++i) row_s[32 * i + lane] = w ? scaled(x[i], r, w[32 * i + lane]) : Two{x[i], 0.f};
      __syncwarp();
      for (int i = lane; i < half; i += 32) {
        const CosSin c = s_cs[i];
        const Two u = row_s[i], v = row_s[half + i];
        row_s[i] = turn_one(u, v, c.ch, c.cl, c.sh, c.sl);
        row_s[half + i] = turn_one(v, u, c.ch, c.cl, -c.sh, -c.sl);
      }
      __syncwarp();
    } else if (side == 0) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < kN; ++i) sum = fmaf(x[i], x[i], sum);
      const float r = w ? rsqrtf(fmaf(warp_sum(sum), 1.f / DH, a.eps)) : 1.f;
#pragma unroll
      for (int i = 0; i < kN; ++i) flat[32 * i + lane] = w ? x[i] * (r * w[32 * i + lane]) : x[i];
      __syncwarp();
      for (int i = lane; i < half; i += 32) {
        const float c = s_cs[i].ch, s = s_cs[i].sh, u = flat[i], v = flat[half + i];
        flat[i] = fmaf(u, c, -(v * s));
        flat[half + i] = fmaf(v, c, u * s);
      }
      __syncwarp();
    }
    void* out = side == 0 ? a.q_out : (side == 1 ? a.k_out : nullptr);
    const long long to = ((long long)t * (side == 0 ? a.n_q : a.n_kv) + g) * DH;
    const int exp = side > 0 ? head_exp(a.exp[side - 1], g) : 0;
    const long long row_at = side > 0 && slot >= 0 ? cache_row(a, g, slot) * kRow : 0;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const Two z = side == 1 ? row_s[32 * i + lane] : Two{side == 0 ? flat[32 * i + lane] : x[i], 0.f};
      if (out) store_elem(out, DT, to + 32 * i + lane, pos >= 0 ? nearest(z) : 0.f);
      if (side == 0 || slot < 0) continue;  // (the same for the warp)
      const float y = to_odd(z);
      uint32_t mx = __float_as_uint(y) & 0x7FFFFFFFu;
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
      const Block4 b = block4(mx, pow2i(-exp), pow2i(exp));
      const float q[4] = {over(y, b.s, b.rs), 0.f, 0.f, 0.f};
      uint32_t code = b.sc == 0 || b.sc == 0x7F ? 0u : codes4(q);
      if (b.sc == 0x7F && (lane & 15) == 0) flag_status(a.status, MTP_ERR_NONFINITE);
      code |= __shfl_down_sync(0xFFFFFFFFu, code, 1) << 4;
      uint8_t* row = a.cache[side - 1] + row_at;
      if ((lane & 1) == 0) row[16 * i + lane / 2] = (uint8_t)code;
      if ((lane & 15) == 0) row[DH / 2 + 2 * i + lane / 16] = (uint8_t)b.sc;
    }
  }
}

// cos(2 pi i / 64) in two floats, made once.
struct Quarter {
  float2 c[17];
  Quarter() {
    for (int i = 0; i <= 16; ++i) {
      const double x = i < 16 ? std::cos(i * (6.283185307179586476925286766559 / 64)) : 0.0;
      c[i].x = (float)x;
      c[i].y = (float)(x - c[i].x);
    }
  }
};

}  // namespace
}  // namespace mtp

using namespace mtp;

extern "C" {

mtp_status mtp_rope_init(int32_t rot_dim, double theta, const double* h_freq, mtp_rope* out) {
  if (!out || rot_dim < 0 || rot_dim > 2 * MTP_ROPE_MAX || rot_dim % 2 != 0) return MTP_ERR_BAD_ARG;
  if (!h_freq && !(theta > 0.0 && std::isfinite(theta))) return MTP_ERR_BAD_ARG;
  mtp_rope r = {};
  r.rot_dim = rot_dim;
  for (int i = 0; i < rot_dim / 2; ++i) {
    const double f = h_freq ? h_freq[i] : std::pow(theta, -2.0 * i / rot_dim);
    if (!std::isfinite(f)) return MTP_ERR_BAD_ARG;
    double turn = f / 6.283185307179586476925286766559;
    turn -= std::floor(turn);  // in [0, 1]; 1 where a tiny negative one rounds up
    r.turn[i] = turn < 1.0 ? (uint64_t)std::ldexp(turn, 64) : 0;  // (a double below 1 times 2^64 fits)
  }
  *out = r;
  return MTP_OK;
}

mtp_status kv_q4_append_rope(mtp_stream stream, const kv_q4_cache* c, int32_t tokens, int32_t n_q, const void* d_q,
                             int64_t q_tok_stride, int64_t q_head_stride, const void* d_k, int64_t k_tok_stride,
                             int64_t k_head_stride, const void* d_v, int64_t v_tok_stride, int64_t v_head_stride,
                             int32_t dtype, const float* d_q_norm, const float* d_k_norm, float eps,
                             const mtp_rope* rope, const int32_t* d_pos, const int32_t* d_slot, void* d_q_out,
                             void* d_k_out, int32_t* d_status) {
  if (!q4_cache_ok(c) || tokens < 0 || n_q < 1 || n_q > 1024 || (dtype != MTP_DTYPE_BF16 && dtype != MTP_DTYPE_F32) ||
      (long long)tokens * (n_q + 2 * c->n_kv) >= (1LL << 31) - kRopeThreads || !rope || rope->rot_dim < 0 || rope->rot_dim > c->head_dim || rope->rot_dim % 2 != 0 || !(eps >= 0.f) || !std::isfinite(eps))
    return MTP_ERR_BAD_ARG;
  if (tokens == 0) return MTP_OK;
  if (!d_q || !d_k || !d_v || !d_pos || !d_slot || !d_q_out) return MTP_ERR_BAD_ARG;
  const int es = dtype == MTP_DTYPE_BF16 ? 2 : 4, dh = c->head_dim;
  auto bits = [](const void* p) { return reinterpret_cast<uintptr_t>(p); };
  if (((bits(d_q) | bits(d_k) | bits(d_v)) & (es - 1)) != 0 || ((bits(d_q_out) | bits(d_k_out) | bits(d_q_norm) | bits(d_k_norm)) & 15) != 0)
    return MTP_ERR_BAD_ARG;
  RopeArgs a{{d_q, d_k, d_v}, {q_tok_stride, k_tok_stride, v_tok_stride}, {q_head_stride, k_head_stride, v_head_stride},
             d_q_out, d_k_out, {d_q_norm, d_k_norm}, {static_cast<uint8_t*>(c->k), static_cast<uint8_t*>(c->v)},
             {c->k_exp, c->v_exp}, d_pos, d_slot, d_status, tokens, n_q, c->n_kv, c->page, c->n_pages * c->page, 1, 1, eps, {},
             *rope};
  static const Quarter quarter;
  std::copy(quarter.c, quarter.c + 17, a.quarter);
  // an output may be its own input, laid out the same; any other overlap would be read after it is written
  const void* in[3] = {d_q, d_k, d_v};
  const int heads[3] = {n_q, c->n_kv, c->n_kv};
  const void* out[2] = {d_q_out, d_k_out};
  for (int o = 0; o < 2; ++o) {
    const size_t bytes = (size_t)tokens * heads[o] * dh * es, index = (size_t)tokens * 4, norm = (size_t)dh * 4;
    if (cross(out[o], bytes, d_pos, index) || cross(out[o], bytes, d_slot, index) || cross(out[o], bytes, d_q_norm, norm) ||
        cross(out[o], bytes, d_k_norm, norm))
      return MTP_ERR_BAD_ARG;
    for (int i = 0; i < 3; ++i) {
      if (!out[o] || (i == o && in[i] == out[o] && (tokens == 1 || a.ts[i] == (long long)heads[i] * dh) && (heads[i] == 1 || a.hs[i] == dh))) continue;
      Bytes x;
      if (!rows_range(in[i], tokens, a.ts[i], heads[i], a.hs[i], dh, es, x) || cross(out[o], bytes, x.at, x.size)) return MTP_ERR_BAD_ARG;
    }
  }
  if (cross(d_q_out, (size_t)tokens * n_q * dh * es, d_k_out, d_k_out ? (size_t)tokens * c->n_kv * dh * es : 0)) return MTP_ERR_BAD_ARG;
  uintptr_t align = bits(d_q) | bits(d_k) | bits(d_v);
  for (int i = 0; i < 3; ++i) align |= (uintptr_t)a.ts[i] * es | (uintptr_t)a.hs[i] * es;
  const bool fast = rope->rot_dim % 32 == 0 && (align & (4 * es - 1)) == 0;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  void (*k)(RopeArgs);
  long long blocks;
  int threads = kRopeThreads;
  if (fast) {
    const int groups = 256 / dh;
    a.q_parts = (n_q + kBatch * groups - 1) / (kBatch * groups);
    a.parts = a.q_parts + (c->n_kv + groups - 1) / groups;
    const int warps = std::min(a.parts, kMostWarps);
    threads = 32 * warps;
    blocks = std::min<long long>(tokens, (long long)device_sm_count() * (2 * kMostWarps / warps));
    k = dtype == MTP_DTYPE_BF16
            ? (dh == 64 ? k_rope_rows<64, MTP_DTYPE_BF16> : (dh == 128 ? k_rope_rows<128, MTP_DTYPE_BF16> : k_rope_rows<256, MTP_DTYPE_BF16>))
            : (dh == 64 ? k_rope_rows<64, MTP_DTYPE_F32> : (dh == 128 ? k_rope_rows<128, MTP_DTYPE_F32> : k_rope_rows<256, MTP_DTYPE_F32>));
  } else {
    blocks = tokens;
    k = dtype == MTP_DTYPE_BF16
            ? (dh == 64 ? k_rope_any<64, MTP_DTYPE_BF16> : (dh == 128 ? k_rope_any<128, MTP_DTYPE_BF16> : k_rope_any<256, MTP_DTYPE_BF16>))
            : (dh == 64 ? k_rope_any<64, MTP_DTYPE_F32> : (dh == 128 ? k_rope_any<128, MTP_DTYPE_F32> : k_rope_any<256, MTP_DTYPE_F32>));
  }
  count_launch();
  const cudaError_t e = launch_pdl(k, dim3((unsigned)blocks), dim3(threads), 0, s, a);
  return e == cudaSuccess ? MTP_OK : MTP_ERR_CUDA;
}

}  // extern "C"
