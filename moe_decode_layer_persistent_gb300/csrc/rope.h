// rope.h -- what the calls that rotate share (rope.cu, qkv_append.cu).
#pragma once
#include <cuda_fp16.h>

#include "batch.h"
#include "ptx.cuh"

struct mk_rope {
  mk_rope_config cfg;
  uint64_t turns[128];  // F_i: turns per position, in units of 2^-64
  double m64;
  float m;
};

namespace mk {

template <class T> struct Pack;  // two 16-bit values in a word
template <> struct Pack<__nv_bfloat16> {
  static MK_DEV float2 get(uint32_t w) {
    return __bfloat1622float2(*reinterpret_cast<__nv_bfloat162*>(&w));
  }
  static MK_DEV uint32_t put(float a, float b) {
    __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&v);
  }
};
template <> struct Pack<__half> {
  static MK_DEV float2 get(uint32_t w) { return __half22float2(*reinterpret_cast<__half2*>(&w)); }
  static MK_DEV uint32_t put(float a, float b) {
    __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&v);
  }
};

}  // namespace mk
