// Append to and read from the paged 4-bit KV cache (kv_q4_append, kv_q4_read).
//
// Rounding of 16 elements y = x 2^-exp: scale = e4m3(max|y| / 6), code = the
// e2m1 value nearest to |y| / scale, ties to the even code. The seven borders
// between neighbouring values, times the scale, are exact in fp32 (three
// significant bits times four).
//   fp32 input: |y| is compared with them, which is exact; a quotient could
//     round onto a border that |y| only comes near.
//   bf16 input: |y| (8 bits) is either on a border or 2^-9 of it away, so the
//     correctly rounded quotient q = y r + (y - (y r) b) r, r = 1 / b (one
//     Newton step on the product) is on a border exactly where y is, and the
//     conversion instruction's rounding to nearest even is the definition's.
//     (By comparisons as fp32, the prompt below took 63 us instead of 39.)
//
// One thread per 16 elements: its loads are one or two sectors, its eight code
// bytes and one scale byte lie next to its neighbours'. A bf16 value is 2 bytes
// in and 9/16 out. 16,383 positions of 4 heads of 256, K and V: append and read
// together 39 us for 172 MB, 4.4 TB/s; the append is at three quarters of the
// issue rate (19.5 M instructions for 33.6 M values, the divisions that find a
// block's row among them), the read is HBM-bound. From fp32 and to it: 75 us for
// 306 MB, 4.1 TB/s.
#include <algorithm>
#include <cfloat>

#include "common.cuh"
#include "kernels.h"
#include "q4.cuh"

namespace mtp {

namespace {

constexpr int kQ4Threads = 256;

struct Q4AppendArgs {
  const void* x[2];            // K, V
  long long ts[2], hs[2];      // strides in elements
  uint8_t* cache[2];
  const int32_t* exp[2];
  const int32_t* slot;
  int32_t* status;
  int tokens, n_kv, page, n_slots;
  int vec;                     // 16-byte loads are aligned
};

// 16 elements from p as fp32.
template <int DT>
__device__ __forceinline__ void load16(const void* src, long long at, bool vec, float (&x)[16]) {
  if (DT == MTP_DTYPE_BF16) {
    const uint16_t* p = static_cast<const uint16_t*>(src) + at;
    if (vec) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint4 w = ld_stream(p + 8 * i);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x[8 * i + 2 * j] = bf16lo(u[j]);
          x[8 * i + 2 * j + 1] = bf16hi(u[j]);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = bf16_to_f(p[i]);
    }
  } else {
    const float* p = static_cast<const float*>(src) + at;
    if (vec) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 w = ld_stream(p + 4 * i);
        x[4 * i] = __uint_as_float(w.x);
        x[4 * i + 1] = __uint_as_float(w.y);
        x[4 * i + 2] = __uint_as_float(w.z);
        x[4 * i + 3] = __uint_as_float(w.w);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = p[i];
    }
  }
}

template <int DH, int DT>
__global__ void __launch_bounds__(kQ4Threads) k_q4_append(const __grid_constant__ Q4AppendArgs a) {
  constexpr int kB = DH / 16, kRow = q4_row_bytes(DH);
  pdl_wait();
  pdl_trigger();
  const int kv = blockIdx.y;
  const long long id = (long long)blockIdx.x * kQ4Threads + threadIdx.x;
  const int b = (int)(id % kB);
  const long long th = id / kB;
  const int head = (int)(th % a.n_kv);
  const long long t = th / a.n_kv;
  if (t >= a.tokens) return;
  const int slot = a.slot[t];
  if (slot < 0 || slot >= a.n_slots) {
    if (slot != -1) flag_status(a.status, MTP_ERR_BAD_ARG);
    return;
  }
  float x[16];
  load16<DT>(a.x[kv], t * a.ts[kv] + head * a.hs[kv] + 16 * b, a.vec, x);
  const float down = pow2i(-head_exp(a.exp[kv], head));
  float amax = 0.f;
  bool finite = true;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    finite &= isfinite(x[i]);
    x[i] *= down;
    amax = fmaxf(amax, fabsf(x[i]));
  }
  if (finite && amax == INFINITY) {  // past fp32's range by the exponent alone: as large as it gets, 6 x 448
    amax = FLT_MAX;
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = fminf(fmaxf(x[i], -FLT_MAX), FLT_MAX);
  }
  uint16_t sc;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(sc) : "f"(0.f), "f"(amax / 6.f));
  const float s = f16x2_to_f(e4m3x2_to_f16x2(sc)).x;
  uint32_t code[2] = {0, 0};
  if (DT == MTP_DTYPE_BF16) {
    const float rs = __frcp_rn(s);
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      float q[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float y = x[8 * w + i], q0 = y * rs;
        q[i] = copysignf(fmaf(fmaf(-q0, s, y), rs, q0), y);  // (-0 stays -0)
      }
      asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
          "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
          "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
          "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
          "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
          "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
          : "=r"(code[w])
          : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]), "f"(q[7]));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float m = fabsf(x[i]);
      // borders .25 .75 1.25 1.75 2.5 3.5 5; on a border the even code
      uint32_t c = (m > 0.25f * s) + (m >= 0.75f * s) + (m > 1.25f * s) + (m >= 1.75f * s) + (m > 2.5f * s) +
                   (m >= 3.5f * s) + (m > 5.f * s);
      c |= (__float_as_uint(x[i]) >> 31) << 3;
      code[i >> 3] |= c << (4 * (i & 7));
    }
  }
  uint8_t scale = (uint8_t)sc;
  if (!finite) {
    scale = 0x7F;  // NaN: the row shows what it was given
    code[0] = code[1] = 0;
    flag_status(a.status, MTP_ERR_NONFINITE);
  } else if (scale == 0) {
    code[0] = code[1] = 0;
  }
  uint8_t* row = a.cache[kv] + (((long long)(slot / a.page) * a.n_kv + head) * a.page + slot % a.page) * kRow;
  // rows start on multiples of 36, 72 or 144 bytes
  if (DH == 64) {
    reinterpret_cast<uint32_t*>(row + 8 * b)[0] = code[0];
    reinterpret_cast<uint32_t*>(row + 8 * b)[1] = code[1];
  } else {
    *reinterpret_cast<uint2*>(row + 8 * b) = make_uint2(code[0], code[1]);
  }
  row[DH / 2 + b] = scale;
}

struct Q4ReadArgs {
  const uint8_t* cache[2];
  const int32_t* exp[2];
  void* out[2];
  const int32_t* slot;
  int32_t* status;
  int tokens, n_kv, page, n_slots;
};

template <int DH, int DT>
__global__ void __launch_bounds__(kQ4Threads) k_q4_read(const __grid_constant__ Q4ReadArgs a) {
  constexpr int kB = DH / 16, kRow = q4_row_bytes(DH);
  pdl_wait();
  pdl_trigger();
  const int kv = blockIdx.y;
  const long long id = (long long)blockIdx.x * kQ4Threads + threadIdx.x;
  const int b = (int)(id % kB);
  const long long th = id / kB;
  const int head = (int)(th % a.n_kv);
  const long long t = th / a.n_kv;
  if (t >= a.tokens) return;
  const int slot = a.slot[t];
  float v[16];
  if (slot < 0 || slot >= a.n_slots) {
    if (slot != -1) flag_status(a.status, MTP_ERR_BAD_ARG);
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = 0.f;
  } else {
    const uint8_t* row = a.cache[kv] + (((long long)(slot / a.page) * a.n_kv + head) * a.page + slot % a.page) * kRow;
    const uint32_t* c = reinterpret_cast<const uint32_t*>(row + 8 * b);
    const uint32_t sc = row[DH / 2 + b];
    const uint32_t s2 = e4m3x2_to_f16x2(sc * 0x0101u);
    const float up = pow2i(head_exp(a.exp[kv], head));
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      uint32_t h[4];
      e2m1x8_to_f16(c[w], h);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = f16x2_to_f(hmul2_bits(h[j], s2));
        v[8 * w + 2 * j] = f.x * up;
        v[8 * w + 2 * j + 1] = f.y * up;
      }
    }
  }
  // six significant bits: exact in either type
  const long long at = (th * kB + b) * 16;
  if (DT == MTP_DTYPE_BF16) {
    uint4* o = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out[kv]) + at);
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      uint32_t u[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u[j]) : "f"(v[8 * w + 2 * j + 1]), "f"(v[8 * w + 2 * j]));
      o[w] = make_uint4(u[0], u[1], u[2], u[3]);
    }
  } else {
    float4* o = reinterpret_cast<float4*>(static_cast<float*>(a.out[kv]) + at);
#pragma unroll
    for (int w = 0; w < 4; ++w) o[w] = make_float4(v[4 * w], v[4 * w + 1], v[4 * w + 2], v[4 * w + 3]);
  }
}

template <typename A>
cudaError_t launch_dh(void (*k64)(A), void (*k128)(A), void (*k256)(A), int dh, long long items, const A& a,
                      cudaStream_t s) {
  const dim3 grid((unsigned)((items + kQ4Threads - 1) / kQ4Threads), 2);
  count_launch();
  return launch_pdl(dh == 64 ? k64 : (dh == 128 ? k128 : k256), grid, dim3(kQ4Threads), 0, s, a);
}

}  // namespace

bool q4_cache_ok(const kv_q4_cache* c) {
  return c && c->k && c->v && ((reinterpret_cast<uintptr_t>(c->k) | reinterpret_cast<uintptr_t>(c->v)) & 15) == 0 &&
         kv_q4_row_bytes(c->head_dim) != 0 && c->n_kv >= 1 && c->n_kv <= 1024 && c->page >= 16 && c->page % 16 == 0 &&
         c->n_pages >= 1 && (long long)c->n_pages * c->page < (1LL << 31);
}

}  // namespace mtp

using namespace mtp;

extern "C" {

size_t kv_q4_row_bytes(int32_t head_dim) {
  return head_dim == 64 || head_dim == 128 || head_dim == 256 ? (size_t)q4_row_bytes(head_dim) : 0;
}

mtp_status kv_q4_append(mtp_stream stream, const kv_q4_cache* c, int32_t tokens, const void* d_k,
                        int64_t k_tok_stride, int64_t k_head_stride, const void* d_v, int64_t v_tok_stride,
                        int64_t v_head_stride, int32_t dtype, const int32_t* d_slot, int32_t* d_status) {
  if (!q4_cache_ok(c) || tokens < 0 || (dtype != MTP_DTYPE_BF16 && dtype != MTP_DTYPE_F32)) return MTP_ERR_BAD_ARG;
  if (tokens == 0) return MTP_OK;
  if (!d_k || !d_v || !d_slot) return MTP_ERR_BAD_ARG;
  Q4AppendArgs a{{d_k, d_v}, {k_tok_stride, v_tok_stride}, {k_head_stride, v_head_stride},
                 {static_cast<uint8_t*>(c->k), static_cast<uint8_t*>(c->v)}, {c->k_exp, c->v_exp}, d_slot, d_status,
                 tokens, c->n_kv, c->page, c->n_pages * c->page, 0};
  const int es = dtype == MTP_DTYPE_BF16 ? 2 : 4;
  if (((reinterpret_cast<uintptr_t>(d_k) | reinterpret_cast<uintptr_t>(d_v)) & (es - 1)) != 0) return MTP_ERR_BAD_ARG;
  uintptr_t bits = reinterpret_cast<uintptr_t>(d_k) | reinterpret_cast<uintptr_t>(d_v);
  for (int i = 0; i < 2; ++i) bits |= (uintptr_t)(a.ts[i] * es) | (uintptr_t)(a.hs[i] * es);
  a.vec = (bits & 15) == 0;
  const long long items = (long long)tokens * c->n_kv * (c->head_dim / 16);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e =
      dtype == MTP_DTYPE_BF16
          ? launch_dh(k_q4_append<64, MTP_DTYPE_BF16>, k_q4_append<128, MTP_DTYPE_BF16>,
                         k_q4_append<256, MTP_DTYPE_BF16>, c->head_dim, items, a, s)
          : launch_dh(k_q4_append<64, MTP_DTYPE_F32>, k_q4_append<128, MTP_DTYPE_F32>,
                         k_q4_append<256, MTP_DTYPE_F32>, c->head_dim, items, a, s);
  return e == cudaSuccess ? MTP_OK : MTP_ERR_CUDA;
}

mtp_status kv_q4_read(mtp_stream stream, const kv_q4_cache* c, int32_t tokens, const int32_t* d_slot, void* d_k,
                      void* d_v, int32_t dtype, int32_t* d_status) {
  if (!q4_cache_ok(c) || tokens < 0 || (dtype != MTP_DTYPE_BF16 && dtype != MTP_DTYPE_F32)) return MTP_ERR_BAD_ARG;
  if (tokens == 0) return MTP_OK;
  if (!d_k || !d_v || !d_slot ||
      ((reinterpret_cast<uintptr_t>(d_k) | reinterpret_cast<uintptr_t>(d_v)) & 15) != 0)
    return MTP_ERR_BAD_ARG;
  Q4ReadArgs a{{static_cast<const uint8_t*>(c->k), static_cast<const uint8_t*>(c->v)}, {c->k_exp, c->v_exp}, {d_k, d_v},
               d_slot, d_status, tokens, c->n_kv, c->page, c->n_pages * c->page};
  const long long items = (long long)tokens * c->n_kv * (c->head_dim / 16);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e =
      dtype == MTP_DTYPE_BF16
          ? launch_dh(k_q4_read<64, MTP_DTYPE_BF16>, k_q4_read<128, MTP_DTYPE_BF16>, k_q4_read<256, MTP_DTYPE_BF16>,
                         c->head_dim, items, a, s)
          : launch_dh(k_q4_read<64, MTP_DTYPE_F32>, k_q4_read<128, MTP_DTYPE_F32>, k_q4_read<256, MTP_DTYPE_F32>,
                         c->head_dim, items, a, s);
  return e == cudaSuccess ? MTP_OK : MTP_ERR_CUDA;
}

}  // extern "C"
