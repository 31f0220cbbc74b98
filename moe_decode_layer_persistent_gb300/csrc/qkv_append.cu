// qkv_append.cu -- norms of q and k, rotary positions and the write into a paged
// cache of 16 or 4 bits in one pass (mk_qkv_append), and rows of a cache in 4 bits
// as values again (mk_kvq_read).
//
// Of a head x, with r = 1 / sqrt(mean x^2 + eps), weights w and the angle t of a
// pair (a, b):
//   y_a = r (x_a (w_a m cos t) - x_b (w_b m sin t)),
//   y_b = r (x_b (w_b m cos t) + x_a (w_a m sin t)).
// A team of lanes holds a head, 8 values each, so that the brackets are the same
// for every head of a row that a thread works on: they are made once per row.
//
// What bounds it: of 8192 rows (32 + 2 x 8 heads of 128, norms, into 4 bits) the
// instructions, 4290 per row at 2.6 a cycle and SM, of which 4 could issue: 53 us for 177
// MB, where HBM would take 26 (into 16 bits 47 us for 30).  Few rows: the launch, and groups
// near a border one after the other in 64 bits (64 rows: 4 us more than into 16 bits).
// Reading those rows' values back, 12 us for 6.4: a word of codes and a scale per thread
// and turn, four turns one after the other.
#include <algorithm>
#include <climits>
#include <math_constants.h>

#include "attn_ptx.cuh"
#include "kvq.cuh"
#include "rope.h"

namespace mk {

namespace {

struct AppendParams {
  mk_qkv_append_io io;
  int32_t d, rot;     // rot 0: no rotation
  int32_t team;       // lanes per head: the power of two from d / 8 on
  int32_t team_shift;
  int32_t page_shift;
  float m, by_d;  // by_d: 1 / d
  double m64;
  uint64_t turns[128];
};

// Cosine and sine of phase / 2^64 turns.  The nearest quarter turn is taken off
// first: what is left is at most 2^-25 rad off in 32 bits.
MK_DEV float2 cos_sin(uint64_t phase) {
  const uint32_t u = static_cast<uint32_t>(phase >> 32);
  const uint32_t quarter = (u + (1u << 29)) >> 30;
  const float half_turns = static_cast<float>(static_cast<int32_t>(u - (quarter << 30))) * 0x1p-31f;
  float s, c;
  sincospif(half_turns, &s, &c);
  const float x = quarter & 1 ? s : c, y = quarter & 1 ? c : s;
  return make_float2((quarter + 1) & 2 ? -x : x, quarter & 2 ? -y : y);
}

// A parameter at a place of each thread's own: as constants, 32 places are read one by
// one.
MK_DEV uint64_t load_param(const uint64_t* p) {
  uint64_t x;
  asm("ld.u64 %0, [%1];" : "=l"(x) : "l"(p));
  return x;
}

template <class T>
MK_DEV void unpack8(const uint4& raw, float (&x)[8]) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = Pack<T>::get(w[i]);
    x[2 * i] = v.x;
    x[2 * i + 1] = v.y;
  }
}
template <class T>
MK_DEV uint4 pack8(const float (&y)[8]) {
  return make_uint4(Pack<T>::put(y[0], y[1]), Pack<T>::put(y[2], y[3]), Pack<T>::put(y[4], y[5]),
                    Pack<T>::put(y[6], y[7]));
}

// What 8 values of every q head, or of every k head, of a row are multiplied with:
// themselves by a, their partners by b.
struct Turn {
  float2 a[4], b[4];
};

// A thread's 8 norm weights and those of its values' partners with the sign that these
// have in the rotation.
struct Weights {
  uint4 own, partner;
};
template <class T, int LAYOUT>
MK_DEV Weights load_weights(const AppendParams& P, const void* w, int l, int from) {
  const uint32_t one = Pack<T>::put(1.f, 1.f);
  Weights x;
  x.own = x.partner = make_uint4(one, one, one, one);
  if (w && l * 8 < P.d) {
    x.own = reinterpret_cast<const uint4*>(w)[l];
    if (LAYOUT == MK_ROPE_HALF) x.partner = reinterpret_cast<const uint4*>(w)[from];
  }
  if (LAYOUT == MK_ROPE_HALF) {
    const uint32_t sign = l < P.rot / 16 ? 0x80008000u : 0u;
    x.partner.x ^= sign, x.partner.y ^= sign, x.partner.z ^= sign, x.partner.w ^= sign;
  } else {  // neighbours: the first of a pair takes away
    const uint32_t* o = reinterpret_cast<const uint32_t*>(&x.own);
    uint32_t* p = reinterpret_cast<uint32_t*>(&x.partner);
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = __byte_perm(o[i], 0, 0x1032) ^ 0x8000u;
  }
  return x;
}
// cosines, sines: of the thread's pairs (8 or, of neighbours, 4).
template <class T, int LAYOUT>
MK_DEV Turn make_turn(const Weights& w, const float* cosines, const float* sines) {
  const uint32_t own[4] = {w.own.x, w.own.y, w.own.z, w.own.w};
  const uint32_t partner[4] = {w.partner.x, w.partner.y, w.partner.z, w.partner.w};
  Turn t;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 c = LAYOUT == MK_ROPE_HALF ? make_float2(cosines[2 * i], cosines[2 * i + 1]) : make_float2(cosines[i], cosines[i]);
    const float2 s = LAYOUT == MK_ROPE_HALF ? make_float2(sines[2 * i], sines[2 * i + 1]) : make_float2(sines[i], sines[i]);
    t.a[i] = mul2(Pack<T>::get(own[i]), c);
    t.b[i] = mul2(Pack<T>::get(partner[i]), s);
  }
  return t;
}

// Value i = lane % 16 of a group in 64 bits (z, and the codes' unit); the lanes of a
// warp share out the sum of squares.  x, w: the head's values and weights (or null).
template <class T, int LAYOUT>
MK_DEV double exact_value(const AppendParams& P, const T* x, const T* w, int32_t pos, int group, int e) {
  double r = 1.0;
  if (w) {
    double sum = 0.0;
    for (int i = lane_id(); i < P.d; i += 32) {
      const double v = static_cast<float>(x[i]);
      sum += v * v;
    }
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    r = 1.0 / sqrt(sum / P.d + static_cast<double>(P.io.eps));
  }
  const double unit = r * static_cast<double>(pow2(-e));
  const int at = group * 16 + (lane_id() & 15);
  const double own = static_cast<double>(static_cast<float>(x[at])) * (w ? static_cast<double>(static_cast<float>(w[at])) : 1.0);
  if (at >= P.rot) return own * unit;
  const bool half = LAYOUT == MK_ROPE_HALF;
  const bool second = half ? at >= P.rot / 2 : at & 1;
  const int to = half ? (second ? at - P.rot / 2 : at + P.rot / 2) : at ^ 1;
  const int pair = half ? min(at, to) : at / 2;
  const double other = static_cast<double>(static_cast<float>(x[to])) * (w ? static_cast<double>(static_cast<float>(w[to])) : 1.0);
  const int64_t phase = static_cast<int64_t>(static_cast<uint64_t>(static_cast<int64_t>(pos)) * P.turns[pair]);
  double s, c;
  sincospi(static_cast<double>(phase) * 0x1p-63, &s, &c);
  return (own * c + (second ? other : -other) * s) * P.m64 * unit;
}

// A double to the E4M3 scale nearest to a seventh of it: through a float that is
// odd where it is not exact, so that it is rounded once.
MK_DEV uint32_t exact_scale(double top) {
  const double q = top / 7.0;
  float f = __double2float_rz(q);
  if (static_cast<double>(f) != q) f = __uint_as_float(__float_as_uint(f) | 1u);
  return floats_to_e4m3x2(f, 0.f) & 0xFFu;
}

// One group's codes (value i in bits 4 i of 64) and scale, in 64 bits, by a whole warp.
template <class T, int LAYOUT>
__device__ __noinline__ uint3 exact_group(const AppendParams& P, const T* x, const T* w, int32_t pos, int group, int e) {
  const double z = exact_value<T, LAYOUT>(P, x, w, pos, group, e);
  double top = fabs(z);
  for (int o = 8; o; o >>= 1) top = fmax(top, __shfl_xor_sync(0xffffffffu, top, o));
  const uint32_t scale = exact_scale(top);
  const double u = e4m3_to_float(scale);
  const double n = u > 0.0 ? rint(z / u) : 0.0;
  const uint32_t code = static_cast<uint32_t>(static_cast<int>(fmin(fmax(n, -8.0), 7.0)) + 8);
  const int i = lane_id() & 15;
  const uint32_t lo = __reduce_or_sync(0xffffffffu, i < 8 ? code << (4 * i) : 0u);
  const uint32_t hi = __reduce_or_sync(0xffffffffu, i >= 8 ? code << (4 * i - 32) : 0u);
  return make_uint3(lo, hi, scale);
}

// Codes of 8 values (value i in bits 4 i) and the scale of their group; the lane's
// neighbour has the group's other 8.  MADE: the values were computed, and are off by
// `off` at most; near_border: this could tell.  Else they are given, in at most 11
// bits, and ties between codes or scales are frequent among them: quotients come by
// way of a reciprocal, whose error of 2^-20 would break the ties, and are rounded to
// more than that and less than what lies between a tie and its neighbours first.
template <bool MADE>
MK_DEV uint2 quantise(const float (&z)[8], float top, float off, bool* near_border) {
  top = max_or_nan(top, __shfl_xor_sync(0xffffffffu, top, 1));
  const bool nan = top != top;
  float seventh = top * (1.f / 7.f);
  bool near = false;
  if (MADE) {
    off = fmaxf(off, __shfl_xor_sync(0xffffffffu, off, 1));
    // (the product is off by 2^-23)
    const float room = off + seventh * 0x1p-22f;
    const uint32_t both = floats_to_e4m3x2(seventh - room, seventh + room);
    near = (both & 0xFFu) != (both >> 8);
  } else if (seventh < 1e30f) {
    const float c = __fmul_rn(seventh, 4097.f);  // to 12 bits
    seventh = __fsub_rn(c, __fsub_rn(c, seventh));
  }
  const uint32_t scale = floats_to_e4m3x2(seventh, 0.f) & 0xFFu;
  const float s = e4m3_to_float(scale), inv = s > 0.f ? __frcp_rn(s) : 0.f;
  float dev = 0.f;
  uint32_t word = 0;
  constexpr float kWhole = 12582912.f;  // 1.5 2^23: what is added to it is rounded to a whole number
#pragma unroll
  for (int i = 7; i >= 0; --i) {
    float t = fminf(fmaxf(z[i] * inv, -8.25f), 7.25f);  // (what lies beyond are codes 0 and 15)
    if (!MADE) t = __fsub_rn(__fadd_rn(t, 48.f), 48.f);  // to 2^-18
    const float n = __fadd_rn(t, kWhole);
    if (MADE) dev = fmaxf(dev, fabsf(t - __fsub_rn(n, kWhole)));
    word = word * 16 + __float_as_uint(n);
  }
  // of the eight 0x4B400000 + n (mod 2^32) to codes n + 8
  word += 0x88888888u - 0x4B400000u * 0x11111111u;
  if (MADE) {
    near = (near || dev > 0.5f - off * inv - 0x1p-19f) && !nan;
    *near_border = __shfl_xor_sync(0xffffffffu, static_cast<int>(near), 1) || near;
  }
  if (nan) return make_uint2(0x88888888u, 0x7Fu);
  return make_uint2(word, scale);
}

MK_DEV float largest(const float (&z)[8]) {
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max_or_nan(top, fabsf(z[i]));
  return top;
}

// Where the slot's row of a kv head starts in the pools of codes and scales, in rows.
MK_DEV int64_t kvq_row(const mk_kvq_cache& c, int page_shift, int64_t slot, int head) {
  return (((slot >> page_shift) * c.n_kv_heads + head) << page_shift) + (slot & (c.page_size - 1));
}

// A row per CTA (gridDim.y 3: a CTA each for its q, k and v heads).
template <class T, int LAYOUT, int BITS, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) k_append(const __grid_constant__ AppendParams P) {
  const mk_qkv_append_io& io = P.io;
  // of the row's pairs, and behind them those of values that pass: cosine 1, sine 0
  __shared__ __align__(16) float cosines[128 + 8], sines[128 + 8];
  const int d = P.d, team = P.team;
  const int l = threadIdx.x & (team - 1), first = threadIdx.x >> P.team_shift, teams = THREADS >> P.team_shift;
  const int warp_first = (threadIdx.x & ~31) >> P.team_shift;
  const bool some = l * 8 < d;
  const int parts = gridDim.y == 3 ? 1 << blockIdx.y : 7;
  // lane of the partners, and where this thread's pairs lie
  const int h16 = P.rot / 16;
  const bool turns = l < P.rot / 8;
  const int from = LAYOUT == MK_ROPE_HALF && turns ? (l < h16 ? l + h16 : l - h16) : l;
  const int at_pairs = !turns ? 128 : LAYOUT == MK_ROPE_HALF ? (l < h16 ? l : l - h16) * 8 : l * 4;
  const uint32_t passes = turns ? ~0u : 0u;  // (a partner that is none is 0: infinity times the sine 0 is NaN)
  if (threadIdx.x < 8) cosines[128 + threadIdx.x] = 1.f, sines[128 + threadIdx.x] = 0.f;

  // The normed and rotated values of a head.  For a cache in 4 bits: they are off by
  // the angle's and the sine's rounding (2^-23.4 of the pair), those of the brackets
  // and products (3 x 2^-24) and of r (2^-21.4 of the value), together less than 2^-20.5
  // (|n_a| + |n_b|) m, which is at most sqrt 2 (|y_a| + |y_b|).
  auto turned = [&](const uint4& raw, const Turn& t, bool norm, float (&y)[8]) {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    float2 x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = Pack<T>::get(w[i]);
    float r = 1.f;
    if (norm) {
      const float2 ss = add2(fma2(x[1], x[1], mul2(x[0], x[0])), fma2(x[3], x[3], mul2(x[2], x[2])));
      float sum = ss.x + ss.y;
#pragma unroll
      for (int o = 16; o; o >>= 1)
        if (o < team) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      r = rsqrtf(sum * P.by_d + io.eps);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 p;
      if (LAYOUT == MK_ROPE_HALF) p = Pack<T>::get(__shfl_sync(0xffffffffu, w[i], from, team) & passes);
      else p = Pack<T>::get(__byte_perm(w[i], 0, 0x1032) & passes);
      const float2 v = mul2(fma2(x[i], t.a[i], mul2(p, t.b[i])), make_float2(r, r));
      y[2 * i] = v.x;
      y[2 * i + 1] = v.y;
    }
  };

  const int64_t row = blockIdx.x;
  int64_t slot = -1;
  if (io.k && (parts & 6)) {
    slot = io.slots[row];
    const int64_t most = BITS == 4 ? static_cast<int64_t>(io.kvq.n_pages) << P.page_shift : io.n_slots;
    if (slot >= most) slot = -1;
  }
  const int32_t pos = P.rot ? io.positions[row] : 0;
  constexpr int kAhead = 4;
  uint4 raw4[kAhead];
  // the first loads are on their way while the angles are made
  const T* q = static_cast<const T*>(io.q) + row * io.q_stride + l * 8;
  if (parts & 1)
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (some && first + u * teams < io.n_q_heads) raw4[u] = __ldcs(reinterpret_cast<const uint4*>(q + (first + u * teams) * d));
  for (int i = threadIdx.x; i < P.rot / 2 && (parts & 3); i += THREADS) {
    const float2 c = cos_sin(static_cast<uint64_t>(static_cast<int64_t>(pos)) * load_param(&P.turns[i]));
    cosines[i] = c.x * P.m;
    sines[i] = c.y * P.m;
  }
  __syncthreads();

  if (parts & 1) {
    T* out = static_cast<T*>(io.q_out) + row * io.q_out_stride + l * 8;
    const Turn t = make_turn<T, LAYOUT>(load_weights<T, LAYOUT>(P, io.q_norm, l, from), cosines + at_pairs, sines + at_pairs);
    // (the loop is the same for a whole warp: its teams meet in the shuffles)
    for (int at = 0; warp_first + at < io.n_q_heads; at += kAhead * teams) {
      if (at)
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
          if (some && first + at + u * teams < io.n_q_heads) raw4[u] = __ldcs(reinterpret_cast<const uint4*>(q + (first + at + u * teams) * d));
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int h = first + at + u * teams;
        if (!some || h >= io.n_q_heads) raw4[u] = make_uint4(0, 0, 0, 0);
        if (warp_first + at + u * teams >= io.n_q_heads) break;
        float y[8];
        turned(raw4[u], t, io.q_norm != nullptr, y);
        if (some && h < io.n_q_heads) *reinterpret_cast<uint4*>(out + h * d) = pack8<T>(y);
      }
    }
  }
#pragma unroll 1
  for (int part = 1; part < 3; ++part) {
    const bool is_k = part == 1;
    const T* src = static_cast<const T*>(is_k ? io.k : io.v);
    if (!(parts >> part & 1) || !src || slot < 0) continue;
    src += row * (is_k ? io.k_stride : io.v_stride);
    Turn t;
    if (is_k) t = make_turn<T, LAYOUT>(load_weights<T, LAYOUT>(P, io.k_norm, l, from), cosines + at_pairs, sines + at_pairs);
    for (int at = 0; warp_first + at < io.n_kv_heads; at += teams) {
      const int h = first + at;
      const bool mine = some && h < io.n_kv_heads;
      uint4 raw = make_uint4(0, 0, 0, 0);
      if (mine) raw = __ldcs(reinterpret_cast<const uint4*>(src + h * d + l * 8));
      if (BITS == 16) {
        if (is_k) {
          float y[8];
          turned(raw, t, io.k_norm != nullptr, y);
          raw = pack8<T>(y);
        }
        if (mine)
          *reinterpret_cast<uint4*>(static_cast<T*>(is_k ? io.k_cache : io.v_cache) +
                                    (slot * io.n_kv_heads + h) * d + l * 8) = raw;
        continue;
      }
      const int32_t* exps = is_k ? io.kvq.k_exp : io.kvq.v_exp;
      const int e = exps && mine ? clamp_exp(exps[h]) : 0;
      const float unit = pow2(-e);
      float z[8];
      uint2 code;
      if (is_k) turned(raw, t, io.k_norm != nullptr, z);
      else unpack8<T>(raw, z);
#pragma unroll
      for (int i = 0; i < 8; ++i) z[i] *= unit;
      const float top = largest(z);
      if (is_k && (P.rot || io.k_norm)) {
        bool near = false;
        const float other = LAYOUT == MK_ROPE_HALF ? __shfl_sync(0xffffffffu, top, from, team) : top;
        code = quantise<true>(z, top, 0x1p-20f * (top + other), &near);
        // Without norms, groups that pass and those of position 0 are as they were given,
        // ties among them (worked out in 64 bits they took 3826 rows, 32 of 128 values
        // rotated, from 27 to 75 us).
        const bool passed = pos == 0 && P.m == 1.f;
        if (!io.k_norm && (P.rot < d || passed)) {
          const uint2 given = quantise<false>(z, top, 0.f, nullptr);
          if (passed || (l & ~1) * 8 >= P.rot) code = given, near = false;
        }
        // groups near a border, one after the other (about one row of 40 has one)
        uint32_t todo = __ballot_sync(0xffffffffu, near && mine && !(l & 1));
        while (todo) {
          const int from_lane = __ffs(todo) - 1;
          todo &= todo - 1;
          const int gh = __shfl_sync(0xffffffffu, h, from_lane), gl = __shfl_sync(0xffffffffu, l, from_lane);
          const int ge = __shfl_sync(0xffffffffu, e, from_lane);
          const uint3 x = exact_group<T, LAYOUT>(P, src + gh * d, static_cast<const T*>(io.k_norm), pos, gl / 2, ge);
          const int mine_too = static_cast<int>(lane_id()) - from_lane;
          if (mine_too == 0) code = make_uint2(x.x, x.z);
          if (mine_too == 1) code = make_uint2(x.y, x.z);
        }
      } else {
        code = quantise<false>(z, top, 0.f, nullptr);
      }
      if (!mine) continue;
      const int64_t to = kvq_row(io.kvq, P.page_shift, slot, h);
      uint8_t* codes = static_cast<uint8_t*>(is_k ? io.kvq.k_codes : io.kvq.v_codes);
      uint8_t* scales = static_cast<uint8_t*>(is_k ? io.kvq.k_scales : io.kvq.v_scales);
      *reinterpret_cast<uint32_t*>(codes + to * (d / 2) + l * 4) = code.x;
      if (!(l & 1)) scales[to * (d / 16) + l / 2] = static_cast<uint8_t>(code.y);
    }
  }
}

// ------------------------------------------------------------------ values again

struct ReadParams {
  mk_kvq_read_io io;
  int32_t page_shift;
  int32_t group;   // rows of a CTA's piece of work
  int64_t pieces;  // groups of rows by kv heads
  Divisor per;     // of 8 values in a head
};

// A CTA per group of rows and kv head, a thread per 8 values: in the order of the pools
// where every slot is read.
template <class T>
__global__ void __launch_bounds__(256) k_read(const __grid_constant__ ReadParams P) {
  const mk_kvq_read_io& io = P.io;
  const mk_kvq_cache& c = io.kvq;
  const bool is_k = blockIdx.y == 0;
  T* out = static_cast<T*>(is_k ? io.k_out : io.v_out);
  if (!out) return;
  const uint8_t* codes = static_cast<const uint8_t*>(is_k ? c.k_codes : c.v_codes);
  const uint8_t* scales = static_cast<const uint8_t*>(is_k ? c.k_scales : c.v_scales);
  const int32_t* exps = is_k ? c.k_exp : c.v_exp;
  const int64_t slots = static_cast<int64_t>(c.n_pages) << P.page_shift;
  for (int64_t piece = blockIdx.x; piece < P.pieces; piece += gridDim.x) {
    const int64_t row0 = piece / c.n_kv_heads * P.group;
    const int h = static_cast<int>(piece % c.n_kv_heads);
    const float unit = pow2(exps ? clamp_exp(exps[h]) : 0);
    for (uint32_t i = threadIdx.x; i < P.group * P.per.d; i += 256) {
      const uint32_t r = quotient(i, P.per), g = i - r * P.per.d;
      const int64_t row = row0 + r;
      const bool there = row < io.n_rows;
      const int64_t slot = !there ? -1 : io.slots ? io.slots[row] : row;
      uint32_t word = 0x88888888u;
      float s = 0.f;
      if (slot >= 0 && slot < slots) {
        const int64_t at = kvq_row(c, P.page_shift, slot, h);
        word = *reinterpret_cast<const uint32_t*>(codes + at * (c.head_dim / 2) + g * 4);
        s = e4m3_to_float(scales[at * (c.head_dim / 16) + g / 2]) * unit;
      }
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)  // (2^23 + n, less 2^23 + 8)
        v[j] = (__uint_as_float(0x4B000000u | (word >> (4 * j) & 15u)) - 8388616.f) * s;
      if (there) *reinterpret_cast<uint4*>(out + (row * c.n_kv_heads + h) * c.head_dim + g * 8) = pack8<T>(v);
    }
  }
}

template <class T, int LAYOUT, int BITS>
void launch_append(const AppendParams& P, int sms, cudaStream_t s) {
  const unsigned n = static_cast<unsigned>(P.io.n_rows);
  // Few rows: many threads for each, with q, k and v apart.  Many: a warp for each, as
  // what a row's threads wait for in turn is hidden by other rows only, and a warp does
  // least of what is the same for all heads (with the values read back, 32 + 2 x 8 heads
  // of 128 into 4 bits: 8192 rows 67 us, with 64 threads for each part 68, with 128 for a
  // row 75; 1024 rows 29 and 18 us).
  if (P.io.n_rows < 2 * sms) k_append<T, LAYOUT, BITS, 256><<<dim3(n, 3), 256, 0, s>>>(P);
  else if (P.io.n_rows < 24 * sms) k_append<T, LAYOUT, BITS, 64><<<dim3(n, 3), 64, 0, s>>>(P);
  else k_append<T, LAYOUT, BITS, 32><<<n, 32, 0, s>>>(P);
}
template <class T>
void launch_append(const AppendParams& P, bool half, int sms, cudaStream_t s) {
  if (P.io.bits == 16) {
    if (half) launch_append<T, MK_ROPE_HALF, 16>(P, sms, s);
    else launch_append<T, MK_ROPE_INTERLEAVED, 16>(P, sms, s);
  } else {
    if (half) launch_append<T, MK_ROPE_HALF, 4>(P, sms, s);
    else launch_append<T, MK_ROPE_INTERLEAVED, 4>(P, sms, s);
  }
}

// Whether n rows of `wa` 16-bit values, `sa` apart, and n of `wb`, `sb` apart, have a value
// in common.  Rows of different strides count as having one where their stretches meet.
bool rows_meet(const void* a, int64_t wa, int64_t sa, const void* b, int64_t wb, int64_t sb, int64_t n) {
  if (!a || !b || !overlap(a, span_bytes(n, wa, sa, 2), b, span_bytes(n, wb, sb, 2))) return false;
  if (n == 1 || sa != sb) return true;
  // b's row j starts away - m s behind a's row j + m: within that row for m = q, or less than
  // a row in front of it for m = q + 1
  const int64_t s = sa * 2;
  const int64_t away = static_cast<int64_t>(reinterpret_cast<uintptr_t>(b) - reinterpret_cast<uintptr_t>(a));
  const int64_t q = (away >= 0 ? away : away - s + 1) / s, r = away - q * s;
  return (r < wa * 2 && q > -n && q < n) || (s - r < wb * 2 && q + 1 > -n && q + 1 < n);
}

}  // namespace

}  // namespace mk

using namespace mk;

extern "C" {

mk_status mk_qkv_append(const mk_rope* rope, const mk_qkv_append_io* io, void* stream) {
  if (!io) return MK_ERR_INVALID_ARG;
  const int64_t d = io->head_dim, n = io->n_rows;
  if (io->dtype != MK_BF16 && io->dtype != MK_FP16) return MK_ERR_UNSUPPORTED;
  if (io->bits != 16 && io->bits != 4) return MK_ERR_UNSUPPORTED;
  if (n < 0 || io->n_q_heads < 0 || io->n_kv_heads < 0) return MK_ERR_INVALID_ARG;
  if (d < 8 || d > 256 || d % 8) return MK_ERR_UNSUPPORTED;
  if (rope && rope->cfg.head_dim != d) return MK_ERR_INVALID_ARG;
  if (io->n_q_heads > 4096 || io->n_kv_heads > 4096) return MK_ERR_UNSUPPORTED;
  if ((io->q_norm || io->k_norm) && !(io->eps >= 0.f && io->eps <= 1e30f)) return MK_ERR_INVALID_ARG;
  if (io->bits == 4 && io->n_kv_heads) {
    const mk_status st = check_kvq(io->kvq, true);
    if (st != MK_OK) return st;
    if (io->kvq.head_dim != d || io->kvq.n_kv_heads != io->n_kv_heads) return MK_ERR_INVALID_ARG;
  }
  if (n == 0) return MK_OK;  // (tensors without rows may have no address)
  if ((io->q != nullptr) != (io->n_q_heads > 0) || (io->k != nullptr) != (io->n_kv_heads > 0))
    return MK_ERR_INVALID_ARG;
  if (!io->q && !io->k) return MK_ERR_INVALID_ARG;
  if (io->q && !io->q_out) return MK_ERR_INVALID_ARG;
  if (io->k && !io->slots) return MK_ERR_INVALID_ARG;
  if (io->v && !io->k) return MK_ERR_INVALID_ARG;
  if (io->k && io->bits == 16 && (!io->k_cache || (io->v && !io->v_cache) || io->n_slots < 0))
    return MK_ERR_INVALID_ARG;
  if (rope && !io->positions) return MK_ERR_INVALID_ARG;
  const void* ptrs[] = {io->q, io->q_out, io->k, io->v, io->k_cache, io->v_cache, io->q_norm, io->k_norm};
  for (const void* p : ptrs)
    if (misaligned(p, 16)) return MK_ERR_INVALID_ARG;
  if (misaligned(io->positions, 4) || misaligned(io->slots, 8)) return MK_ERR_INVALID_ARG;
  const int64_t qw = io->n_q_heads * d, kw = io->n_kv_heads * d;
  if (io->q && (io->q_stride % 8 || io->q_out_stride % 8 || io->q_stride < qw || io->q_out_stride < qw))
    return MK_ERR_INVALID_ARG;
  if (io->k && (io->k_stride % 8 || io->k_stride < kw)) return MK_ERR_INVALID_ARG;
  if (io->v && (io->v_stride % 8 || io->v_stride < kw)) return MK_ERR_INVALID_ARG;
  // What is written against what is read and against one another, each as the stretch from
  // its first value to its last; but q_out may lie between the rows of k and v, and k and
  // v in the rows of the 16-bit caches that they go to.
  struct Range { const void* p; int64_t n; };
  const Range q = {io->q, io->q ? span_bytes(n, qw, io->q_stride, 2) : 0};
  const Range q_out = {io->q_out, io->q ? span_bytes(n, qw, io->q_out_stride, 2) : 0};
  const Range k = {io->k, io->k ? span_bytes(n, kw, io->k_stride, 2) : 0};
  const Range v = {io->v, io->v ? span_bytes(n, kw, io->v_stride, 2) : 0};
  const bool in_place = io->q == io->q_out && (n == 1 || io->q_stride == io->q_out_stride);
  const bool four = io->bits == 4;
  const Range in[] = {{rope ? io->positions : nullptr, n * 4}, {io->k ? io->slots : nullptr, n * 8},
                      {io->q_norm, d * 2}, {io->k ? io->k_norm : nullptr, d * 2},
                      {io->k && four ? io->kvq.k_exp : nullptr, io->n_kv_heads * 4ll},
                      {io->k && four ? io->kvq.v_exp : nullptr, io->n_kv_heads * 4ll}};
  Range pools[4] = {};  // codes and scales, or the cache, of k and of v
  if (io->k && four) {
    const int64_t rows = static_cast<int64_t>(io->kvq.n_pages) * io->kvq.page_size * io->n_kv_heads;
    pools[0] = {io->kvq.k_codes, rows * (d / 2)};
    pools[1] = {io->kvq.k_scales, rows * (d / 16)};
    if (io->v) {
      pools[2] = {io->kvq.v_codes, rows * (d / 2)};
      pools[3] = {io->kvq.v_scales, rows * (d / 16)};
    }
  } else if (io->k) {
    if (io->n_slots > INT64_MAX / 2 / kw) return MK_ERR_INVALID_ARG;
    pools[0] = {io->k_cache, io->n_slots * kw * 2};
    if (io->v) pools[2] = {io->v_cache, io->n_slots * kw * 2};
  }
  auto meet = [](const Range& a, const Range& b) { return overlap(a.p, a.n, b.p, b.n); };
  for (const Range& r : in) {
    if (meet(r, q_out)) return MK_ERR_INVALID_ARG;
    for (const Range& w : pools)
      if (meet(r, w)) return MK_ERR_INVALID_ARG;
  }
  for (int a = 0; a < 4; ++a) {
    if (meet(q, pools[a]) || meet(q_out, pools[a])) return MK_ERR_INVALID_ARG;
    if ((four || a >= 2) && meet(k, pools[a])) return MK_ERR_INVALID_ARG;
    if ((four || a < 2) && meet(v, pools[a])) return MK_ERR_INVALID_ARG;
    for (int b = a + 1; b < 4; ++b)
      if (meet(pools[a], pools[b])) return MK_ERR_INVALID_ARG;
  }
  if (!in_place && meet(q, q_out)) return MK_ERR_INVALID_ARG;
  if (io->q && (rows_meet(io->q_out, qw, io->q_out_stride, io->k, kw, io->k_stride, n) ||
                rows_meet(io->q_out, qw, io->q_out_stride, io->v, kw, io->v_stride, n)))
    return MK_ERR_INVALID_ARG;
  int sms = 0;
  const mk_status st = check_device(io->q ? io->q_out : io->slots, nullptr, &sms);
  if (st != MK_OK) return st;
  AppendParams P;
  P.io = *io;
  P.d = static_cast<int32_t>(d);
  P.by_d = 1.f / static_cast<float>(d);
  P.rot = rope ? rope->cfg.rot_dim : 0;
  P.team = 1;
  while (P.team * 8 < d) P.team *= 2;
  if (io->bits == 4) P.team = std::max(P.team, 2);
  P.team_shift = __builtin_ctz(static_cast<uint32_t>(P.team));
  P.page_shift = io->bits == 4 && io->n_kv_heads ? __builtin_ctz(static_cast<uint32_t>(io->kvq.page_size)) : 0;
  P.m = rope ? rope->m : 1.f;
  P.m64 = rope ? rope->m64 : 1.0;
  std::fill(P.turns, P.turns + 128, 0);
  if (rope) std::copy(rope->turns, rope->turns + 128, P.turns);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool half = !rope || rope->cfg.layout == MK_ROPE_HALF;
  if (io->dtype == MK_BF16) launch_append<__nv_bfloat16>(P, half, sms, s);
  else launch_append<__half>(P, half, sms, s);
  MK_CUDA_TRY(cudaGetLastError());
  return MK_OK;
}

mk_status mk_kvq_read(const mk_kvq_read_io* io, void* stream) {
  if (!io) return MK_ERR_INVALID_ARG;
  if (io->dtype != MK_BF16 && io->dtype != MK_FP16) return MK_ERR_UNSUPPORTED;
  mk_status st = check_kvq(io->kvq, true);
  if (st != MK_OK) return st;
  const mk_kvq_cache& c = io->kvq;
  const int64_t slots = static_cast<int64_t>(c.n_pages) * c.page_size, n = io->n_rows;
  if (n < 0 || (!io->slots && n > slots)) return MK_ERR_INVALID_ARG;
  if (n == 0) return MK_OK;
  if (!io->k_out && !io->v_out) return MK_ERR_INVALID_ARG;
  if (misaligned(io->k_out, 16) || misaligned(io->v_out, 16) || misaligned(io->slots, 8)) return MK_ERR_INVALID_ARG;
  const int64_t out = n * c.n_kv_heads * c.head_dim * 2, rows = slots * c.n_kv_heads;
  if (overlap(io->k_out, out, io->v_out, out)) return MK_ERR_INVALID_ARG;
  for (const void* p : {io->k_out, io->v_out})
    if (overlap(p, out, io->slots, n * 8) || overlap(p, out, c.k_codes, rows * (c.head_dim / 2)) ||
        overlap(p, out, c.v_codes, rows * (c.head_dim / 2)) || overlap(p, out, c.k_scales, rows * (c.head_dim / 16)) ||
        overlap(p, out, c.v_scales, rows * (c.head_dim / 16)) || overlap(p, out, c.k_exp, c.n_kv_heads * 4ll) ||
        overlap(p, out, c.v_exp, c.n_kv_heads * 4ll))
      return MK_ERR_INVALID_ARG;
  int sms = 0;
  st = check_device(io->k_out ? io->k_out : io->v_out, nullptr, &sms);
  if (st != MK_OK) return st;
  ReadParams P;
  P.io = *io;
  P.page_shift = __builtin_ctz(static_cast<uint32_t>(c.page_size));
  P.group = std::min(64, c.page_size);
  P.pieces = (n + P.group - 1) / P.group * c.n_kv_heads;
  P.per = make_divisor(static_cast<uint32_t>(c.head_dim / 8));
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>(P.pieces, 16ll * sms)), 2);
  if (io->dtype == MK_BF16) k_read<__nv_bfloat16><<<grid, 256, 0, static_cast<cudaStream_t>(stream)>>>(P);
  else k_read<__half><<<grid, 256, 0, static_cast<cudaStream_t>(stream)>>>(P);
  MK_CUDA_TRY(cudaGetLastError());
  return MK_OK;
}

}  // extern "C"
