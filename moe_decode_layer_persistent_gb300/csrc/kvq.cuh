// kvq.cuh -- the paged cache in 4 bits: its addresses, its checks, and the
// conversions between codes and values.
//
// Code n of a group with the E4M3 scale s stands for (n - 8) s, times the head's
// 2^e.  Uniform steps and not E2M1's: a pair of codes masked into the mantissas
// of two fp16 1024s is a pair of values after one fused multiply-add with the
// scale, (1024 + n) s - 1032 s, while E2M1 codes have to have sign and magnitude
// moved apart first.  (n - 8) s has at most 7 bits, so that bf16 and fp16 hold it
// exactly.
#pragma once
#include <cuda_fp16.h>

#include "batch.h"
#include "ptx.cuh"

namespace mk {

MK_DEV int clamp_exp(int e) { return min(max(e, -64), 64); }
// 2^e, |e| <= 64.
MK_DEV float pow2(int e) { return __int_as_float((127 + e) << 23); }

// Two E4M3 bytes (low byte first) as fp16 values.
MK_DEV uint32_t e4m3x2_to_half2(uint32_t b) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(b)));
  return h;
}
// lo in the low byte, hi in the high one: E4M3, to nearest even, at most 448.
MK_DEV uint32_t floats_to_e4m3x2(float lo, float hi) {
  uint16_t b;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(b) : "f"(hi), "f"(lo));
  return b;
}

// Host checks shared by the calls that take a cache in 4 bits.
inline mk_status check_kvq(const mk_kvq_cache& c, bool pools) {
  const int64_t P = c.page_size;
  if (c.n_kv_heads < 1 || c.n_pages < 0) return MK_ERR_INVALID_ARG;
  if (c.n_kv_heads > 4096) return MK_ERR_UNSUPPORTED;
  if (c.head_dim < 16 || c.head_dim > 256 || c.head_dim % 16) return MK_ERR_UNSUPPORTED;
  if (P < 16 || P > 65536 || (P & (P - 1))) return MK_ERR_UNSUPPORTED;
  if (c.n_pages * P > INT32_MAX) return MK_ERR_INVALID_ARG;
  if (!pools) return MK_OK;
  if (c.n_pages && (!c.k_codes || !c.k_scales || !c.v_codes || !c.v_scales)) return MK_ERR_INVALID_ARG;
  if (misaligned(c.k_codes, 16) || misaligned(c.k_scales, 16) || misaligned(c.v_codes, 16) ||
      misaligned(c.v_scales, 16) || misaligned(c.k_exp, 4) || misaligned(c.v_exp, 4))
    return MK_ERR_INVALID_ARG;
  return MK_OK;
}

}  // namespace mk
