// rope.cu -- rotary positions with the K/V write (mk_rope_create,
// mk_rope_apply).
//
// Pair (a, b) of a head at position p turns by the angle p f_i:
//   y_a = m (x_a cos - x_b sin),  y_b = m (x_b cos + x_a sin).
// The angle is held in 64-bit fixed point as a fraction of a turn: F_i =
// floor(f_i / 2 pi 2^64), and p F_i modulo 2^64 drops the whole turns exactly,
// so that a position of 2^20 is as exact as one of 16 (in 32-bit floating
// point its angle would be off by 0.03 rad).  The top 32 bits, as a signed
// number of half turns, go to sincospif.
#include <algorithm>
#include <cmath>
#include <cuda_fp16.h>
#include <new>

#include "batch.h"
#include "ptx.cuh"

struct mk_rope {
  mk_rope_config cfg;
  uint64_t turns[128];  // F_i
  float m;
};

namespace mk {

namespace {

struct RopeParams {
  mk_rope_io io;
  int32_t d, rot;
  float m;
  uint64_t turns[128];
};

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

// A piece of work: 16 bytes of a head that turn with 16 others (half layout) or
// among themselves (interleaved), or that pass.
struct Piece {
  uint4 a, b;
};

// Turns piece j of a head: for the half layout the 8 pairs whose first values are
// a and second ones b, for the interleaved one the 4 pairs of a.  cs: cos and sin
// of the row's pairs.
template <class T, int LAYOUT>
MK_DEV void turn_piece(Piece& x, int j, const float2* cs) {
  uint32_t* wa = reinterpret_cast<uint32_t*>(&x.a);
  uint32_t* wb = reinterpret_cast<uint32_t*>(&x.b);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (LAYOUT == MK_ROPE_HALF) {
      const float2 u = Pack<T>::get(wa[i]), v = Pack<T>::get(wb[i]);
      const float2 c0 = cs[8 * j + 2 * i], c1 = cs[8 * j + 2 * i + 1];
      wa[i] = Pack<T>::put(u.x * c0.x - v.x * c0.y, u.y * c1.x - v.y * c1.y);
      wb[i] = Pack<T>::put(v.x * c0.x + u.x * c0.y, v.y * c1.x + u.y * c1.y);
    } else {
      const float2 u = Pack<T>::get(wa[i]), c = cs[4 * j + i];
      wa[i] = Pack<T>::put(u.x * c.x - u.y * c.y, u.y * c.x + u.x * c.y);
    }
  }
}

// One row per CTA: the row's cosines and sines once, in shared memory, then every
// head's pieces, one per thread at a time.  The first ones are on their way while
// the angles are being made, so that a CTA's life is one trip to memory and back.
// HBM bounds it with many rows: 128 threads per CTA and 32 registers leave room for
// 16 rows per SM (403 MB of a 16,384-row prompt, half layout, 32 + 2 x 8 heads of
// 128: 63.5 us, 6.3 TB/s; with 256 threads and two pieces at a time 72 us).  With
// few rows the launch does: there 256 threads take each (16 such rows: 2.7 us; with
// 128 threads 3.4 us).
template <class T, int LAYOUT, int THREADS>
__global__ void __launch_bounds__(THREADS, 2048 / THREADS)
    k_rope(const __grid_constant__ RopeParams P) {
  const mk_rope_io& io = P.io;
  __shared__ float2 cs[128];
  const int64_t row = blockIdx.x;
  const int d = P.d, rot = P.rot;
  const int32_t pos = io.positions[row];
  int64_t slot = -1;
  if (io.k) {
    slot = io.slots[row];
    if (slot >= io.n_slots) slot = -1;
  }
  const uint32_t turned = LAYOUT == MK_ROPE_HALF ? rot / 16 : rot / 8;  // pieces that turn
  const uint32_t pieces = turned + (d - rot) / 8;
  const uint32_t nq = io.n_q_heads * pieces, nk = io.n_kv_heads * pieces;
  const uint32_t n = nq + nk + (io.v ? io.n_kv_heads * (d / 8) : 0);
  const int64_t cache_row = slot * (static_cast<int64_t>(io.n_kv_heads) * d);
  for (uint32_t t = threadIdx.x; t == threadIdx.x || t < n; t += THREADS) {
    Piece x;
    T* dst = nullptr;
    int j = -1;  // piece that turns; -1: passes
    if (t < n) {
      const T* src;
      if (t < nq + nk) {
        const bool q = t < nq;
        const uint32_t u = q ? t : t - nq, head = u / pieces, p = u - head * pieces;
        src = q ? static_cast<const T*>(io.q) + row * io.q_stride
                : static_cast<const T*>(io.k) + row * io.k_stride;
        T* to = q ? static_cast<T*>(io.q_out) + row * io.q_out_stride
                  : static_cast<T*>(io.k_cache) + cache_row;
        const uint32_t at = head * d + (p < turned ? p * 8 : rot + (p - turned) * 8);
        src += at;
        if (q || slot >= 0) dst = to + at;
        if (p < turned) j = static_cast<int>(p);
      } else {
        const uint32_t at = (t - nq - nk) * 8;
        src = static_cast<const T*>(io.v) + row * io.v_stride + at;
        if (slot >= 0) dst = static_cast<T*>(io.v_cache) + cache_row + at;
      }
      x.a = __ldcs(reinterpret_cast<const uint4*>(src));
      if (LAYOUT == MK_ROPE_HALF && j >= 0) x.b = __ldcs(reinterpret_cast<const uint4*>(src + rot / 2));
    }
    if (t == threadIdx.x) {
      for (int i = threadIdx.x; i < rot / 2; i += THREADS) {
        const uint64_t phase = static_cast<uint64_t>(static_cast<int64_t>(pos)) * P.turns[i];
        const float half_turns = static_cast<float>(static_cast<int32_t>(phase >> 32)) * 0x1p-31f;
        float s, c;
        sincospif(half_turns, &s, &c);
        cs[i] = make_float2(c * P.m, s * P.m);
      }
      __syncthreads();
    }
    if (!dst) continue;
    if (j >= 0) {
      turn_piece<T, LAYOUT>(x, j, cs);
      if (LAYOUT == MK_ROPE_HALF) *reinterpret_cast<uint4*>(dst + rot / 2) = x.b;
    }
    *reinterpret_cast<uint4*>(dst) = x.a;
  }
}

template <class T, int LAYOUT>
void launch_rope(const RopeParams& P, int sms, cudaStream_t s) {
  if (P.io.n_rows < 4 * sms) k_rope<T, LAYOUT, 256><<<P.io.n_rows, 256, 0, s>>>(P);
  else k_rope<T, LAYOUT, 128><<<P.io.n_rows, 128, 0, s>>>(P);
}

}  // namespace

}  // namespace mk

using namespace mk;

extern "C" {

mk_status mk_rope_create(const mk_rope_config* cfg, mk_rope** out) {
  if (!out) return MK_ERR_INVALID_ARG;
  *out = nullptr;
  if (!cfg) return MK_ERR_INVALID_ARG;
  mk_rope_config c = *cfg;
  if (c.head_dim < 8 || c.head_dim > 256 || c.head_dim % 8) return MK_ERR_UNSUPPORTED;
  if (c.layout != MK_ROPE_HALF && c.layout != MK_ROPE_INTERLEAVED) return MK_ERR_INVALID_ARG;
  if (c.rot_dim < 8 || c.rot_dim > c.head_dim) return MK_ERR_INVALID_ARG;
  if (c.rot_dim % (c.layout == MK_ROPE_HALF ? 16 : 8)) return MK_ERR_UNSUPPORTED;
  if (c.scaling < MK_ROPE_SCALE_NONE || c.scaling > MK_ROPE_SCALE_PARTS) return MK_ERR_INVALID_ARG;
  // (the comparisons are false for NaN)
  if (!(c.theta >= 1.0 && c.theta <= 1e30) || !(c.factor >= 1.0 && c.factor <= 1e9))
    return MK_ERR_INVALID_ARG;
  if (c.scaling == MK_ROPE_SCALE_NONE && c.factor != 1.0) return MK_ERR_INVALID_ARG;
  if (!(c.attn_factor >= 0.0 && c.attn_factor <= 1e9)) return MK_ERR_INVALID_ARG;
  if (c.scaling == MK_ROPE_SCALE_PARTS) {
    if (c.beta_fast == 0.0 && c.beta_slow == 0.0) c.beta_fast = 32.0, c.beta_slow = 1.0;
    if (c.orig_ctx < 1 || !(c.beta_slow >= 0.0 && c.beta_fast > c.beta_slow && c.beta_fast <= 1e9))
      return MK_ERR_INVALID_ARG;
  }
  mk_rope* r = new (std::nothrow) mk_rope();
  if (!r) return MK_ERR_OOM;
  r->cfg = c;
  const double two_pi = 6.283185307179586476925;
  double theta = c.theta;
  if (c.scaling == MK_ROPE_SCALE_BASE)
    theta *= std::pow(c.factor, c.rot_dim / (c.rot_dim - 2.0));
  for (int i = 0; i < c.rot_dim / 2; ++i) {
    double f = std::pow(theta, -2.0 * i / c.rot_dim);
    if (c.scaling == MK_ROPE_SCALE_LINEAR) f /= c.factor;
    if (c.scaling == MK_ROPE_SCALE_PARTS) {
      const double g = std::min(
          1.0, std::max(0.0, (c.orig_ctx * f / two_pi - c.beta_slow) / (c.beta_fast - c.beta_slow)));
      f *= g + (1.0 - g) / c.factor;
    }
    // f <= 1 rad, less than a sixth of a turn
    r->turns[i] = static_cast<uint64_t>(std::ldexp(f / two_pi, 64));
  }
  r->m = static_cast<float>(c.attn_factor != 0.0                ? c.attn_factor
                            : c.scaling == MK_ROPE_SCALE_PARTS ? 0.1 * std::log(c.factor) + 1.0
                                                               : 1.0);
  *out = r;
  return MK_OK;
}

void mk_rope_destroy(mk_rope* rope) { delete rope; }

mk_status mk_rope_apply(const mk_rope* rope, const mk_rope_io* io, void* stream) {
  if (!rope || !io) return MK_ERR_INVALID_ARG;
  const int64_t d = rope->cfg.head_dim, n = io->n_rows;
  if (io->dtype != MK_BF16 && io->dtype != MK_FP16) return MK_ERR_UNSUPPORTED;
  if (io->head_dim != d) return MK_ERR_INVALID_ARG;
  if (n < 0 || io->n_q_heads < 0 || io->n_kv_heads < 0) return MK_ERR_INVALID_ARG;
  if (io->n_q_heads > 4096 || io->n_kv_heads > 4096) return MK_ERR_UNSUPPORTED;
  if (n == 0) return MK_OK;  // (tensors without rows may have no address)
  if ((io->q != nullptr) != (io->n_q_heads > 0) || (io->k != nullptr) != (io->n_kv_heads > 0))
    return MK_ERR_INVALID_ARG;
  if (!io->q && !io->k) return MK_ERR_INVALID_ARG;
  if (io->q && !io->q_out) return MK_ERR_INVALID_ARG;
  if (io->k && (!io->slots || !io->k_cache || io->n_slots < 0)) return MK_ERR_INVALID_ARG;
  if (io->v && (!io->k || !io->v_cache)) return MK_ERR_INVALID_ARG;
  if (!io->positions) return MK_ERR_INVALID_ARG;
  const void* ptrs[] = {io->q, io->q_out, io->k, io->v, io->k_cache, io->v_cache};
  for (const void* p : ptrs)
    if (misaligned(p, 16)) return MK_ERR_INVALID_ARG;
  if (misaligned(io->positions, 4) || misaligned(io->slots, 8)) return MK_ERR_INVALID_ARG;
  const int64_t qw = io->n_q_heads * d, kw = io->n_kv_heads * d;
  if (io->q && (io->q_stride % 8 || io->q_out_stride % 8 || io->q_stride < qw || io->q_out_stride < qw))
    return MK_ERR_INVALID_ARG;
  if (io->k && (io->k_stride % 8 || io->k_stride < kw)) return MK_ERR_INVALID_ARG;
  if (io->v && (io->v_stride % 8 || io->v_stride < kw)) return MK_ERR_INVALID_ARG;
  if (io->q) {
    const int64_t out = span_bytes(n, qw, io->q_out_stride, 2);
    const bool in_place = io->q == io->q_out && io->q_stride == io->q_out_stride;
    if (!in_place && overlap(io->q, span_bytes(n, qw, io->q_stride, 2), io->q_out, out))
      return MK_ERR_INVALID_ARG;
    if (overlap(io->positions, n * 4, io->q_out, out) ||
        (io->k && overlap(io->slots, n * 8, io->q_out, out)))
      return MK_ERR_INVALID_ARG;
  }
  int sms = 0;
  mk_status st = check_device(io->positions, nullptr, &sms);
  if (st != MK_OK) return st;
  RopeParams P;
  P.io = *io;
  P.d = rope->cfg.head_dim;
  P.rot = rope->cfg.rot_dim;
  P.m = rope->m;
  std::copy(rope->turns, rope->turns + 128, P.turns);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool half = rope->cfg.layout == MK_ROPE_HALF;
  if (io->dtype == MK_BF16) {
    if (half) launch_rope<__nv_bfloat16, MK_ROPE_HALF>(P, sms, s);
    else launch_rope<__nv_bfloat16, MK_ROPE_INTERLEAVED>(P, sms, s);
  } else {
    if (half) launch_rope<__half, MK_ROPE_HALF>(P, sms, s);
    else launch_rope<__half, MK_ROPE_INTERLEAVED>(P, sms, s);
  }
  MK_CUDA_TRY(cudaGetLastError());
  return MK_OK;
}

}  // extern "C"
