// The 4-bit rows of the paged KV cache: 16 e2m1 codes (8 bytes) per e4m3
// scale; a row holds dh/2 code bytes, then dh/16 scale bytes.
#pragma once
#include "common.cuh"

namespace mtp {

__host__ __device__ constexpr int q4_row_bytes(int dh) { return dh / 2 + dh / 16; }

// Two e4m3 bytes (low half of w) as two halves: exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t w) {
  uint32_t d;
  asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(d) : "r"(w));
  return d;
}

// The eight e2m1 codes of a word as halves, low nibble first: exact.
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

__device__ __forceinline__ uint32_t hmul2_bits(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

__device__ __forceinline__ float2 f16x2_to_f(uint32_t h) {
  float2 f;
  asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, u;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}

// 2^e for e in [-126, 127]: exact.
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }

// The exponent of a head, held to [-64, 64] (NULL = 0).
__device__ __forceinline__ int head_exp(const int32_t* e, int h) { return e ? min(max(e[h], -64), 64) : 0; }

}  // namespace mtp
