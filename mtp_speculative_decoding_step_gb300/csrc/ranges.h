// Host checks of the memory that an entry point is given.
#pragma once
#include <cstddef>
#include <cstdint>

namespace mtp {

// Whether two ranges of bytes meet. Neither does where one is not given or empty.
inline bool cross(const void* a, size_t na, const void* b, size_t nb) {
  const uint8_t *p = static_cast<const uint8_t*>(a), *q = static_cast<const uint8_t*>(b);
  return p && q && na > 0 && nb > 0 && p < q + nb && q < p + na;
}

// The bytes of rows of `n` elements of `es` bytes, `tokens` by `heads` of them, whose strides in elements may be negative.
// False where no memory is that large.
struct Bytes {
  const uint8_t* at;
  size_t size;
};
inline bool rows_range(const void* base, long long tokens, long long tok_stride, long long heads, long long head_stride, int n, int es,
                       Bytes& out) {
  constexpr long long kMost = 1LL << 56;
  long long lo = 0, hi = n;
  const long long count[2] = {tokens, heads}, stride[2] = {tok_stride, head_stride};
  for (int i = 0; i < 2; ++i) {
    long long far = 0;
    if (count[i] > 1 && (__builtin_mul_overflow(count[i] - 1, stride[i], &far) || far > kMost || far < -kMost)) return false;
    (far < 0 ? lo : hi) += far;
  }
  out = {static_cast<const uint8_t*>(base) + lo * es, (size_t)(hi - lo) * es};
  return true;
}

}  // namespace mtp
