// batch.h -- host-side argument checks shared by the batched-decoding
// operators (slots.cu, rope.cu, prefix_attn.cu).
#pragma once
#include "host_util.h"

namespace mk {

inline bool misaligned(const void* p, uintptr_t bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0;
}

// Whether two byte ranges share a byte (empty and null ranges share none).
inline bool overlap(const void* a, int64_t na, const void* b, int64_t nb) {
  if (!a || !b || na <= 0 || nb <= 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + static_cast<uint64_t>(nb) && y < x + static_cast<uint64_t>(na);
}

// Bytes from the first to behind the last value of `rows` rows of `width`
// values that start `stride` values apart.
inline int64_t span_bytes(int64_t rows, int64_t width, int64_t stride, int64_t elem) {
  return rows <= 0 || width <= 0 ? 0 : ((rows - 1) * stride + width) * elem;
}

// MK_OK if `p` is device or managed memory that the current device can use and
// that device is a compute-capability 10.3 GPU; its number and SM count.
mk_status check_device(const void* p, int* device, int* sm_count);

// Quotients of numbers below 2^31 by a fixed divisor: with 2^(s-1) < d <= 2^s and
// m = floor(2^(31+s) / d) + 1, floor(x m / 2^(31+s)) = floor(x / d), since the error
// x (m - 2^(31+s) / d) / 2^(31+s) <= x / 2^(31+s) < 1 / d.
struct Divisor {
  uint32_t d, m, shift;
};
inline Divisor make_divisor(uint32_t d) {
  uint32_t s = 0;
  while ((uint64_t{1} << s) < d) ++s;
  return Divisor{d, static_cast<uint32_t>((uint64_t{1} << (31 + s)) / d + 1), 31 + s};
}
__device__ __forceinline__ uint32_t quotient(uint32_t x, const Divisor& v) {
  return static_cast<uint32_t>((static_cast<uint64_t>(x) * v.m) >> v.shift);
}

}  // namespace mk
