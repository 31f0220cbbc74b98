// kvq_attn.cuh -- what the kernels of attention over a cache in 4 bits share
// (kvq_attn.cu, kvq_wide.cu).
#pragma once
#include <cfloat>
#include <climits>

#include "attn_ptx.cuh"
#include "kvq.cuh"
#include "rope.h"

namespace mk {

// Weights are 2^(score - r) in fp16: r is set so that a row's largest is 2^6 and
// moves when one passes 2^15; those below 2^-25 of the type vanish, 2^-31 of the
// largest at most.
constexpr float kRefBelow = 6.f, kRefMost = 15.f;
constexpr float kNoRef = -1e30f;
// What an item takes on top of its key tiles, in key tiles (of 32 keys and of 128).
// 200 requests of one token over up to 2000 keys: 69 us with 1, 60 with 2, 58 with 3, 59
// with 4; token trees of 60 requests over up to 4000 keys: 139, 121, 114, 104 and 108 us
// with 3, 5, 7, 9 and 14 (of 16 over up to 16384 keys 100, 89, 88, 88 and 93).
constexpr int kLead = 3, kWideLead = 9;

// An item whose stretches lie in several workers, as the one with its first key tile
// says.
struct Split {
  int32_t parts;     // 0: none
  int32_t folded;    // row r lies in rows r and r + kWideRows / 2 of each part
  int32_t cu, rows;  // first row of the request, its rows of this kv head
  int32_t first;     // first of these in the tile
  int32_t h;
};

constexpr uint64_t kKvqWaitNs = 2000ull * 1000 * 1000;
// Hand-offs of the kernel for row tiles of up to 128 rows that a self-test withholds, so
// that waits run out: a tile's scores, its weights, its keys, its values, their buffers
// after use, a row tile, the second half's results, its place after the first has them.
enum KvqWithhold {
  kKvqNothing, kKvqScores, kKvqWeights, kKvqKeys, kKvqValues, kKvqKeysUsed, kKvqValuesUsed, kKvqRowTile, kKvqHalf, kKvqTaken
};

struct KvqParams {
  mk_kvq_attn_io io;
  float scale_log2;  // scale * log2(e)
  int32_t group;
  int32_t page_shift;
  uint32_t page_bytes;  // of codes
  int32_t workers;
  Divisor by_group;
  uint32_t* status;
  Split* split;      // [workers]
  float2* stat;      // (r, l) of the rows of part 2 w (begins inside an item), 2 w + 1
  float* o;          // [2 workers][rows][D]
  // of a self-test: limit of a wait; which hand-off to withhold, and the how manieth
  uint64_t wait_ns;
  int32_t withhold, withhold_at;
  bool test;
};

// The bits that any lane has.
MK_DEV uint64_t bits_of_all(uint64_t x) {
  const uint32_t lo = __reduce_or_sync(0xffffffffu, static_cast<uint32_t>(x));
  const uint32_t hi = __reduce_or_sync(0xffffffffu, static_cast<uint32_t>(x >> 32));
  return static_cast<uint64_t>(hi) << 32 | lo;
}
MK_DEV int clampi(int64_t v, int lo, int hi) { return v < lo ? lo : v > hi ? hi : static_cast<int>(v); }

// What a row's products are multiplied with to become scores in units of log2; factor: what
// its q was divided by.  (The 8: see Scales.)  Neither 0, which a masked score, -infinity,
// must not meet, nor infinity, which a score of 0 must not.
MK_DEV float score_factor(const KvqParams& P, float factor, int h) {
  const mk_kvq_cache& c = P.io.kvq;
  return fminf(fmaxf(P.scale_log2 * factor * (8.f * pow2(c.k_exp ? clamp_exp(c.k_exp[h]) : 0)), FLT_MIN), FLT_MAX);
}

// One request's lengths, made safe, and its place on the line: for each kv head and
// row tile an item of its key tiles, in front of them `lead` units for what an item
// takes on top (Q, the first copies, the results).
struct Req {
  int32_t cu, n, len, base;
  int32_t tile0, tiles;  // first key tile of its items and how many they have
  int32_t row_tiles;
  int32_t lead;
  MK_DEV int64_t cost(int heads) const { return static_cast<int64_t>(tiles + lead) * row_tiles * heads; }
};
// The part of an item that lies between two places of it: key tiles [a, b).
struct Piece {
  int32_t a, b;
};
MK_DEV Piece piece_of(const Req& r, int64_t from, int64_t to) {
  return {static_cast<int32_t>(max(from - r.lead, static_cast<int64_t>(0))),
          static_cast<int32_t>(max(min(to - r.lead, static_cast<int64_t>(r.tiles)), static_cast<int64_t>(0)))};
}
// How many workers share the key tiles of an item that starts at a place of the line.
MK_DEV int parts_of(const Req& r, int64_t start, int64_t share) {
  return static_cast<int>((start + r.lead + r.tiles - 1) / share - (start + r.lead) / share + 1);
}
template <int R, int KEYS>
MK_DEV Req read_req(const KvqParams& P, int b) {
  const mk_kvq_attn_io& io = P.io;
  Req r;
  r.cu = clampi(io.cu_rows[b], 0, io.n_rows);
  r.n = clampi(io.cu_rows[b + 1], r.cu, io.n_rows) - r.cu;
  r.len = clampi(io.lens[b], 0, io.max_pages << P.page_shift);
  r.base = max(0, r.len - r.n);
  // (a row with an empty tree word is at base - 1)
  const int low = io.window ? max(0, r.base - io.window + (io.tree_mask ? 0 : 1)) : 0;
  r.tile0 = low / KEYS;
  r.lead = KEYS == 32 ? kLead : kWideLead;
  // (at least one, so that rows without keys are written)
  r.tiles = max(1, (r.len + KEYS - 1) / KEYS - r.tile0);
  r.row_tiles = static_cast<int>((static_cast<int64_t>(r.n) * P.group + R - 1) / R);
  return r;
}

MK_DEV void cp_async16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0)
               : "memory");
}
MK_DEV void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
MK_DEV void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// D += A B, 16 x 8 by 16.
MK_DEV void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
MK_DEV uint32_t transposed8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
MK_DEV uint32_t half2_bits(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
MK_DEV __half2 as_half2(uint32_t x) { return *reinterpret_cast<const __half2*>(&x); }
MK_DEV uint32_t and_or(uint32_t a, uint32_t mask, uint32_t c) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(a), "r"(mask), "r"(c));
  return d;
}

// Factors for a pair of scales s: of codes in the low nibbles, 1024 + n, and the
// high ones, 1024 + 16 n.  All in eighths, so that 1032 times the largest scale is
// still an fp16; every factor and every result is exact.
struct Scales {
  __half2 lo, hi, lo_off, hi_off;
  MK_DEV Scales first() const { return {__low2half2(lo), __low2half2(hi), __low2half2(lo_off), __low2half2(hi_off)}; }
  MK_DEV Scales second() const { return {__high2half2(lo), __high2half2(hi), __high2half2(lo_off), __high2half2(hi_off)}; }
};
MK_DEV Scales make_scales(uint32_t pair) {  // two E4M3 bytes
  const __half2 s = as_half2(e4m3x2_to_half2(pair));
  return {__hmul2(s, as_half2(0x30003000u)), __hmul2(s, as_half2(0x20002000u)), __hmul2(s, as_half2(0xD808D808u)),
          __hmul2(s, as_half2(0xC880C880u))};
}
// Eight codes, as four pairs (x, x + 4).
MK_DEV void values(uint32_t word, const Scales& f, uint32_t (&y)[4]) {
  const uint32_t up = word >> 8;
  const __half2 v[4] = {__hfma2(as_half2(and_or(word, 0x000F000Fu, 0x64006400u)), f.lo, f.lo_off),
                        __hfma2(as_half2(and_or(word, 0x00F000F0u, 0x64006400u)), f.hi, f.hi_off),
                        __hfma2(as_half2(and_or(up, 0x000F000Fu, 0x64006400u)), f.lo, f.lo_off),
                        __hfma2(as_half2(and_or(up, 0x00F000F0u, 0x64006400u)), f.hi, f.hi_off)};
#pragma unroll
  for (int i = 0; i < 4; ++i) y[i] = *reinterpret_cast<const uint32_t*>(&v[i]);
}

// Row tiles of up to 128 rows on tcgen05 (kvq_wide.cu): one worker per CTA.
constexpr int kWideRows = 128;
mk_status launch_kvq_wide(const KvqParams& P, int device, int sms, cudaStream_t s);

}  // namespace mk
