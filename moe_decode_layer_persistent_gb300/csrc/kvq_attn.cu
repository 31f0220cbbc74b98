// kvq_attn.cu -- attention over a paged cache in 4 bits (mk_kvq_attn).
//
// Of a request's rows (token, q head of the group) those of one kv head form row
// tiles of 8 or 16.  With a row tile's Q and 32 keys a step is
//   S^T = K Q^T,  P = 2^(S - r),  l += P,  O^T += V^T P^T
// in units of log2, r a reference near the maximum of each row so far.  K and V are
// the products' first operands, 16 keys or 16 dimensions by 8 rows: with 4 rows per
// kv head, as in plain decoding, half of the tensor core's work counts and not a
// quarter or less, and the codes become operands in the registers of the thread
// that needs them, without a second trip through shared memory.
//
// A key takes 144 bytes and 256 conversions per kv head (d = 128), so that the
// conversions cost as much as HBM does.  What keeps them cheap: the dimensions of a
// head may be summed over in any order, so each thread takes 32 neighbouring ones of
// a key (16 bytes) and Q is laid out to match; a mask turns two codes into two fp16
// 1024 + n, a fused multiply-add with the scale into values, exactly; for V, two
// keys' words are interleaved by halves first, so that the pairs are pairs of keys.
//
// All key tiles of all items (request, kv head, row tile) lie on one line, of which
// every warp takes an equal stretch, whatever the lengths are; each warp works by
// itself, its copies in flight in a ring of its own.  A stretch that holds a whole
// item writes its result, the others (O, r, l), which a second kernel, chained with
// programmatic dependent launch, joins in the order of the line.
//
// What bounds it: 64 requests of one row and up to 8192 keys (32 heads over 8, d 128,
// 304 MB) take 66 us with the join; what more keys add comes at 6.1 TB/s, and 17 us are
// start, join and ends (twice the keys 116 us, four times 215).  2.1 instructions per cycle
// and SM: the conversions issue while HBM is waited for, but not freely.
//
// A call takes one kernel, by its requests' rows on average: single tokens beside a long
// chunk go the way of many rows (64 of those above, 66 us, and 512 rows over 8192 keys,
// 102 us by themselves, take 267 us in one call), and a request of many rows among single
// tokens is read once per 8 or 16 rows (60 rows in place of the 512: 31 us, in one call
// 113).  Calls of their own take less there.
#include <algorithm>
#include <atomic>
#include <cfloat>
#include <climits>
#include <cmath>
#include <type_traits>

#include "../../include/mk_selftest.h"
#include "kvq_attn.cuh"

namespace mk {

namespace {

constexpr int kKeys = 32;   // of a key tile: a step of a warp, and the unit of the line
constexpr int kStages = 3;  // key tiles of a warp's ring

// A stage of a warp's ring: two blocks of 16 keys, each K's codes, V's codes, K's
// scales, V's scales (a page may hold no more than 16 keys).
template <int D>
struct Layout {
  static constexpr int kCodes = 16 * D / 2, kScales = 16 * D / 16;
  static constexpr int kK = 0, kV = kCodes, kKs = 2 * kCodes, kVs = 2 * kCodes + kScales;
  static constexpr int kBlock = 2 * (kCodes + kScales);
  static constexpr int kStage = 2 * kBlock;
  // Key of row 2 t + 1 (the even rows' are t): chosen so that neither K's rows nor
  // V's pairs of keys meet in a bank.
  static constexpr int kFlip = D == 128 ? 1 : 2;
};

// What a warp knows of its stretch, out of its registers while it works: they are
// what bounds the number of warps.
template <int R>
struct Stretch {
  int64_t pos, begin, part;
  uint64_t tree;  // bits of all rows' tree words
  int32_t b, h, cu, rows, first, base, whole, klo, khi;
  int32_t lo[R], hi[R];  // keys that each row sees (of a tree: those before its own)
};
template <int WARPS, int R>
struct PlanSmem {
  int64_t sum[WARPS];
  int64_t first_at[WARPS];
  int32_t first[WARPS];
  Stretch<R> at[WARPS];
};

// Warps per CTA (one CTA per SM).  With 16 of 128 registers each and with 8 the same
// work takes 5 to 7 % longer (64 requests, one token, up to 8192 keys: 91 and 91 us, 12: 85).
template <int NT>
constexpr int kWarps = 12;

template <class T, int D, int NT>
__global__ void __launch_bounds__(kWarps<NT> * 32, 1) k_kvq_attn(const __grid_constant__ KvqParams P) {
  constexpr int R = 8 * NT, W = kWarps<NT>, TH = W * 32;
  constexpr int KS = D / 16;   // products per 16 keys for the scores
  constexpr int MT = D / 16;   // and for the values
  using L = Layout<D>;
  const mk_kvq_attn_io& io = P.io;
  const mk_kvq_cache& c = io.kvq;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ PlanSmem<W, R> plan;
  const int lane = lane_id(), warp = threadIdx.x / 32, Hk = c.n_kv_heads;
  const int worker = warp * gridDim.x + blockIdx.x;
  pdl_launch_dependents();
  pdl_wait();
  if (blockIdx.x == 0 && threadIdx.x == 0) *P.status = 0;

  // The line: each thread adds up the requests of a stretch of the batch.
  const int per = (io.n_requests + TH - 1) / TH;
  const int b0 = min(io.n_requests, static_cast<int>(threadIdx.x) * per), b1 = min(io.n_requests, b0 + per);
  int64_t mine = 0;
  for (int b = b0; b < b1; ++b) mine += read_req<R, kKeys>(P, b).cost(Hk);
  int64_t upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += x;
  }
  if (lane == 31) plan.sum[warp] = upto;
  __syncthreads();
  int64_t total = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    if (w == warp) upto += total;
    total += plan.sum[w];
  }
  const int64_t share = max(static_cast<int64_t>(1), (total + P.workers - 1) / P.workers);
  if (mine) {
    for (int w = 0; w < W; ++w) {
      const int64_t at = (static_cast<int64_t>(w) * gridDim.x + blockIdx.x) * share;
      if (at < upto - mine || at >= upto) continue;
      int64_t begin = upto - mine;
      int b = b0;
      for (; b < b1 - 1; ++b) {
        const int64_t cost = read_req<R, kKeys>(P, b).cost(Hk);
        if (at < begin + cost) break;
        begin += cost;
      }
      plan.first[w] = b;
      plan.first_at[w] = begin;
    }
  }
  __syncthreads();
  {
    const int64_t pos = worker * share;
    if (lane == 0) P.split[worker].parts = 0;
    if (pos >= total) return;
    if (lane == 0) {
      plan.at[warp].pos = pos;
      plan.at[warp].begin = plan.first_at[warp];
      plan.at[warp].b = plan.first[warp];
    }
    __syncwarp();
  }
  volatile Stretch<R>& at = plan.at[warp];

  uint8_t* ring = smem + warp * (kStages * L::kStage);
  const uint32_t ring32 = smem_u32(ring);
  // this lane's 16 bytes of each copy: of 16 keys' codes, and of their scales
  constexpr int kScaleLanes = L::kScales / 16;
  const uint8_t* k_lane = static_cast<const uint8_t*>(c.k_codes) + lane * 16;
  const uint8_t* v_lane = static_cast<const uint8_t*>(c.v_codes) + lane * 16;
  const uint8_t* s_lane = static_cast<const uint8_t*>(lane < kScaleLanes ? c.k_scales : c.v_scales) + (lane & (kScaleLanes - 1)) * 16;
  const int g = lane >> 2, t = lane & 3;
  const int key_even = g >> 1, key_g = g & 1 ? 4 + (key_even ^ L::kFlip) : key_even;  // of row g of K
  const int key_0 = t, key_1 = 4 + (t ^ L::kFlip);                                    // of V's pair
  while (true) {
    uint32_t qf[NT][KS][2];    // Q of this thread's column of the second operand: row g of each 8
    float c_row[NT][2];        // factor on the scores of rows 2 t, 2 t + 1
    int full_lo = 0, full_hi = INT_MAX;  // keys that every row sees
    int tile, tile_end, h;
    const int32_t* table;
    {
      int64_t pos = at.pos, begin = at.begin;
      const int64_t end = min(total, static_cast<int64_t>(worker + 1) * share);
      if (pos >= end) return;
      int b = at.b;
      Req rq = read_req<R, kKeys>(P, b);
      for (int64_t cost; pos >= begin + (cost = rq.cost(Hk)); rq = read_req<R, kKeys>(P, b)) {
        begin += cost;
        ++b;
      }
      const int64_t off = pos - begin, item = off / (rq.tiles + rq.lead);
      h = static_cast<int>(item / rq.row_tiles);
      const int rt = static_cast<int>(item - static_cast<int64_t>(h) * rq.row_tiles);
      const int64_t start = begin + item * (rq.tiles + rq.lead), to = min(end, start + rq.tiles + rq.lead);
      const Piece piece = piece_of(rq, pos - start, to - start);
      const int ta = piece.a, tb = piece.b;
      if (ta >= tb) {  // (what an item takes on top of its key tiles)
        __syncwarp();
        if (lane == 0) at.pos = to, at.begin = begin, at.b = b;
        __syncwarp();
        continue;
      }
      const int rows = rq.n * P.group;  // (checked by the host to be an int)
      int klo = INT_MAX, khi = 0;
      uint64_t tree = 0;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int f = rt * R + nt * 8 + g;
        const bool valid = f < rows;
        const int i = quotient(valid ? f : 0, P.by_group), hq = h * P.group + (valid ? f - i * P.group : 0);
        const int64_t row = rq.cu + i;
        // dimensions 32 t .. (64: 16 t ..), 8 at a time: two words of pairs (x, x + 4)
        float factor = 1.f;
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const T*>(io.q) + row * io.q_stride + hq * D + t * (D / 4));
        uint4 raw[D / 32];
#pragma unroll
        for (int j = 0; j < D / 32; ++j) raw[j] = valid ? src[j] : make_uint4(0, 0, 0, 0);
        if (!std::is_same<T, __half>::value) {
          // bf16 into fp16, relative to the row's largest value
          uint32_t top = 0;
#pragma unroll
          for (int j = 0; j < D / 32; ++j)
            top = __vmaxu2(top, __vmaxu2(__vmaxu2(raw[j].x & 0x7FFF7FFFu, raw[j].y & 0x7FFF7FFFu),
                                         __vmaxu2(raw[j].z & 0x7FFF7FFFu, raw[j].w & 0x7FFF7FFFu)));
          top = max(top & 0xFFFFu, top >> 16);
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
          const int e = min(max(static_cast<int>(top >> 7), 1), 253);  // biased; up to 2 * 2^e
          factor = top < 0x7F80u ? __int_as_float(e << 23) : 1.f;
          const float inv = top < 0x7F80u ? __int_as_float((254 - e) << 23) : 1.f;
#pragma unroll
          for (int j = 0; j < D / 32; ++j) {
            uint32_t* w = reinterpret_cast<uint32_t*>(&raw[j]);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 x = Pack<T>::get(w[k]);
              w[k] = half2_bits(x.x * inv, x.y * inv);
            }
          }
        }
        // words (0,1)(2,3)(4,5)(6,7) into (0,4)(1,5)(2,6)(3,7)
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
          qf[nt][2 * j][0] = __byte_perm(raw[j].x, raw[j].z, 0x5410);
          qf[nt][2 * j][1] = __byte_perm(raw[j].x, raw[j].z, 0x7632);
          qf[nt][2 * j + 1][0] = __byte_perm(raw[j].y, raw[j].w, 0x5410);
          qf[nt][2 * j + 1][1] = __byte_perm(raw[j].y, raw[j].w, 0x7632);
        }
        int my_lo = 0, my_hi = 0;
        if (valid) {
          const uint64_t word = io.tree_mask ? io.tree_mask[row] : 0;
          tree |= word;
          const int p = rq.base + (io.tree_mask ? __popcll(word) - 1 : i);
          my_lo = io.window ? max(0, p - io.window + 1) : 0;
          my_hi = io.tree_mask ? min(rq.len, rq.base) : min(rq.len, rq.base + i + 1);
          klo = min(klo, my_lo);
          khi = max(khi, io.tree_mask ? min(rq.len, rq.base + 64) : my_hi);
          full_lo = max(full_lo, my_lo);
          full_hi = min(full_hi, my_hi);
        }
        if (t == 0) at.lo[nt * 8 + g] = my_lo, at.hi[nt * 8 + g] = my_hi;
#pragma unroll
        for (int k = 0; k < 2; ++k) c_row[nt][k] = score_factor(P, __shfl_sync(0xffffffffu, factor, 8 * t + 4 * k), h);
      }
      klo = __reduce_min_sync(0xffffffffu, klo);
      khi = __reduce_max_sync(0xffffffffu, khi);
      tree = bits_of_all(tree);
      full_lo = __reduce_max_sync(0xffffffffu, full_lo);
      full_hi = __reduce_min_sync(0xffffffffu, full_hi);
      tile = max(rq.tile0 + ta, min(klo, khi) / kKeys);
      tile_end = min(rq.tile0 + tb, (khi + kKeys - 1) / kKeys);
      table = io.block_table + b * io.table_stride;
      if (lane == 0) {
        const bool whole = ta == 0 && tb == rq.tiles;
        at.pos = to;
        at.begin = begin;
        at.b = b, at.h = h, at.cu = rq.cu, at.rows = rows, at.first = rt * R, at.base = rq.base;
        at.whole = whole, at.klo = klo, at.khi = khi, at.tree = tree;
        at.part = 2ll * worker + (ta == 0);
        if (ta == 0 && !whole) P.split[worker] = {parts_of(rq, start, share), 0, rq.cu, rows, rt * R, h};
      }
      __syncwarp();
    }

    float o[NT][MT][4];
    float ref[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      ref[nt][0] = ref[nt][1] = kNoRef;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[nt][i][k] = 0.f;
    }

    // Pages of 32 blocks of 16 keys, one per lane, and those of the next 32.
    const uint32_t head_bytes = static_cast<uint32_t>(h << P.page_shift) * (D / 2);
    const int blocks_end = 2 * tile_end;
    int block = 2 * tile, pages_at = block;
    auto page_of = [&](int x) { return x < blocks_end && x * 16 < at.khi ? table[x * 16 >> P.page_shift] : -1; };
    int pages = page_of(block + lane), pages_next = page_of(block + 32 + lane);
    auto issue = [&](uint32_t to) {
      if (block < blocks_end) {
        if (block - pages_at == 32) {
          pages_at = block;
          pages = pages_next;
          pages_next = page_of(block + 32 + lane);
        }
#pragma unroll
        for (int half = 0; half < 2; ++half, ++block) {
          const int page = __shfl_sync(0xffffffffu, pages, block - pages_at);
          const bool there = static_cast<uint32_t>(page) < static_cast<uint32_t>(c.n_pages);
          // (a page's codes are less than 2^31 bytes)
          const int64_t off = there ? static_cast<int64_t>(static_cast<uint64_t>(static_cast<uint32_t>(page)) * P.page_bytes +
                                                           (head_bytes + ((block * 16) & (c.page_size - 1)) * (D / 2)))
                                    : 0;
          const uint32_t st = to + half * L::kBlock + lane * 16;
          const uint8_t *k = k_lane + off, *v = v_lane + off;
          cp_async16(st + L::kK, k, there);
          if (D == 128) {
            const uint32_t turned = st ^ ((lane >> 3 & 1) << 5);  // see the loads of V
            cp_async16(st + L::kK + 512, k + 512, there);
            cp_async16(turned + L::kV, v, there);
            cp_async16(turned + L::kV + 512, v + 512, there);
          } else {
            cp_async16(st + L::kV, v, there);
          }
          if (lane < 2 * kScaleLanes) cp_async16(st + L::kKs, s_lane + (off >> 3), there);
        }
      }
      cp_async_commit();
    };
    uint32_t stage = 0, stage_in = 0;  // offsets in the ring: of the tile at hand, of the next copy
    auto next_stage = [](uint32_t x) { return x == (kStages - 1) * L::kStage ? 0u : x + L::kStage; };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
      issue(ring32 + stage_in);
      stage_in = next_stage(stage_in);
    }
#pragma unroll 1
    for (; tile < tile_end; ++tile) {
      cp_async_wait<kStages - 2>();
      __syncwarp();
      issue(ring32 + stage_in);
      stage_in = next_stage(stage_in);
      uint8_t* st = ring + stage;
      stage = next_stage(stage);
      float sc[2][NT][4];
      // scores: of each block rows g and g + 8 are the keys key_g and key_g + 8
#pragma unroll
      for (int blk = 0; blk < 2; ++blk) {
        constexpr int WORDS = D / 32;  // of 8 codes, of this thread's dimensions of a key
        const uint8_t* sb = st + blk * L::kBlock;
        uint32_t w[2][WORDS];
        Scales f[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int key = key_g + 8 * k;
          if (D == 128) {
            const uint4 x = *reinterpret_cast<const uint4*>(sb + L::kK + key * 64 + t * 16);
            w[k][0] = x.x, w[k][1] = x.y, w[k][2 % WORDS] = x.z, w[k][3 % WORDS] = x.w;
            f[k] = make_scales(*reinterpret_cast<const uint16_t*>(sb + L::kKs + key * 8 + t * 2));
          } else {
            const uint2 x = *reinterpret_cast<const uint2*>(sb + L::kK + key * 32 + t * 8);
            w[k][0] = x.x, w[k][1] = x.y;
            const uint32_t one = sb[L::kKs + key * 4 + t];
            f[k] = make_scales(one | one << 8);
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 4; ++k) sc[blk][nt][k] = 0.f;
#pragma unroll
        for (int j = 0; j < WORDS; ++j) {
          uint32_t a[2][4];
#pragma unroll
          for (int k = 0; k < 2; ++k)  // (d 128: words 0, 1 are of the first group of 16, 2, 3 of the second)
            values(w[k][j], D == 64 || j < 2 ? f[k].first() : f[k].second(), a[k]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma16816(sc[blk][nt], a[0][0], a[1][0], a[0][1], a[1][1], qf[nt][2 * j][0], qf[nt][2 * j][1]);
            mma16816(sc[blk][nt], a[0][2], a[1][2], a[0][3], a[1][3], qf[nt][2 * j + 1][0], qf[nt][2 * j + 1][1]);
          }
        }
      }
      const bool edge = tile * kKeys < full_lo || tile * kKeys + kKeys > full_hi;
      if (edge) {
        // keys that no row sees may hold anything: a weight of 0 must meet a number
        const int j = tile * kKeys + lane;
        if (j < at.klo || j >= at.khi || (io.tree_mask && j >= at.base && !(at.tree >> (j - at.base) & 1))) {
          uint8_t* scales = st + (lane >> 4) * L::kBlock + L::kVs + (lane & 15) * (D / 16);
          if (D == 128) *reinterpret_cast<uint2*>(scales) = make_uint2(0, 0);
          else *reinterpret_cast<uint32_t*>(scales) = 0;
        }
        __syncwarp();
#pragma unroll 1
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int x = 0; x < 8; ++x) {
            const int k = x & 3, j = tile * kKeys + (x >> 2) * 16 + key_g + (k & 2) * 4, r = nt * 8 + 2 * t + (k & 1);
            bool see = j >= at.lo[r] && j < at.hi[r];
            if (io.tree_mask && j >= at.base && j < at.khi) {
              const int fr = at.first + r;
              see = fr < at.rows && (io.tree_mask[at.cu + quotient(fr, P.by_group)] >> (j - at.base) & 1);
            }
#pragma unroll
            for (int m = 0; m < NT; ++m)
              if (m == nt && !see) sc[x >> 2][m][k] = -INFINITY;
          }
      }
      bool over = false;
      float top[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          top[nt][k] = fmaxf(fmaxf(sc[0][nt][k], sc[0][nt][k + 2]), fmaxf(sc[1][nt][k], sc[1][nt][k + 2]));
          over |= fmaf(top[nt][k], c_row[nt][k], -ref[nt][k]) > kRefMost;
        }
      if (__any_sync(0xffffffffu, over)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float x = top[nt][k];
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
            x *= c_row[nt][k];
            const float next = x - ref[nt][k] > kRefMost ? x - kRefBelow : ref[nt][k];
            const float old = exp2_approx(ref[nt][k] - next);
            ref[nt][k] = next;
            l[nt][k] *= old;
#pragma unroll
            for (int i = 0; i < MT; ++i) {
              o[nt][i][k] *= old;
              o[nt][i][k + 2] *= old;
            }
          }
      }
      uint32_t pf[2][NT][2];
#pragma unroll
      for (int blk = 0; blk < 2; ++blk)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float p[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) p[k] = exp2_approx(fmaf(sc[blk][nt][k], c_row[nt][k & 1], -ref[nt][k & 1]));
          l[nt][0] += p[0] + p[2];
          l[nt][1] += p[1] + p[3];
          pf[blk][nt][0] = transposed8x8(half2_bits(p[0], p[1]));
          pf[blk][nt][1] = transposed8x8(half2_bits(p[2], p[3]));
        }
      // values: of each block the pairs of keys (key_0, key_1) and 8 further on
#pragma unroll
      for (int blk = 0; blk < 2; ++blk) {
        constexpr int WORDS = D / 64;  // of this thread's dimensions of a key
        const uint8_t* sb = st + blk * L::kBlock;
        uint32_t w[4][WORDS];
        Scales f[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int ka = key_0 + 8 * k, kb = key_1 + 8 * k;
          uint32_t sa, sb8;
          if (D == 128) {
            const uint2 x = *reinterpret_cast<const uint2*>(sb + L::kV + ((ka * 64 + g * 8) ^ ((ka >> 1 & 1) << 5)));
            const uint2 y = *reinterpret_cast<const uint2*>(sb + L::kV + ((kb * 64 + g * 8) ^ ((kb >> 1 & 1) << 5)));
            w[2 * k][0] = x.x, w[2 * k][1 % WORDS] = x.y;
            w[2 * k + 1][0] = y.x, w[2 * k + 1][1 % WORDS] = y.y;
            sa = sb[L::kVs + ka * 8 + g], sb8 = sb[L::kVs + kb * 8 + g];
          } else {
            w[2 * k][0] = *reinterpret_cast<const uint32_t*>(sb + L::kV + ka * 32 + g * 4);
            w[2 * k + 1][0] = *reinterpret_cast<const uint32_t*>(sb + L::kV + kb * 32 + g * 4);
            sa = sb[L::kVs + ka * 4 + g / 2], sb8 = sb[L::kVs + kb * 4 + g / 2];
          }
          f[k] = make_scales(sa | sb8 << 8);
        }
#pragma unroll
        for (int j = 0; j < WORDS; ++j)
#pragma unroll
          for (int half = 0; half < 2; ++half) {  // dimensions 8 j + 4 half ..
            uint32_t a[2][4];
#pragma unroll
            for (int k = 0; k < 2; ++k)
              values(__byte_perm(w[2 * k][j], w[2 * k + 1][j], half ? 0x7632 : 0x5410), f[k], a[k]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma16816(o[nt][4 * j + 2 * half], a[0][0], a[0][1], a[1][0], a[1][1], pf[blk][nt][0], pf[blk][nt][1]);
              mma16816(o[nt][4 * j + 2 * half + 1], a[0][2], a[0][3], a[1][2], a[1][3], pf[blk][nt][0], pf[blk][nt][1]);
            }
          }
      }
    }
    cp_async_wait<0>();
    __syncwarp();

    // this thread's: rows 2 t and 2 t + 1, dimensions D / 8 g .. (o[i][k]: 2 i, o[i][k + 2]: 2 i + 1)
    h = at.h;
    const float unit_v = 8.f * pow2(c.v_exp ? clamp_exp(c.v_exp[h]) : 0);
    const int64_t part = at.part;
    const int rows = at.rows, first = at.first, cu = at.cu;
    const bool whole = at.whole;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float sum = l[nt][k];
        sum += __shfl_xor_sync(0xffffffffu, sum, 4);
        sum += __shfl_xor_sync(0xffffffffu, sum, 8);
        sum += __shfl_xor_sync(0xffffffffu, sum, 16);
        const int r = nt * 8 + 2 * t + k, fr = first + r;
        if (fr >= rows) continue;
        if (!whole) {
          float* to = P.o + (part * R + r) * D + g * (D / 8);
#pragma unroll
          for (int i = 0; i < MT; i += 2)
            *reinterpret_cast<float4*>(to + 2 * i) = make_float4(o[nt][i][k] * unit_v, o[nt][i][k + 2] * unit_v, o[nt][i + 1][k] * unit_v, o[nt][i + 1][k + 2] * unit_v);
          if (g == 0) P.stat[part * R + r] = make_float2(ref[nt][k], sum);
          continue;
        }
        const int i = quotient(fr, P.by_group), hq = h * P.group + fr - i * P.group;
        const int64_t row = cu + i;
        const float inv = sum != 0.f ? unit_v / sum : 0.f;
        uint32_t y[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) y[m] = Pack<T>::put(o[nt][m][k] * inv, o[nt][m][k + 2] * inv);
        uint4* to = reinterpret_cast<uint4*>(static_cast<T*>(io.out) + row * io.out_stride + hq * D + g * (D / 8));
#pragma unroll
        for (int m = 0; m < MT / 4; ++m) to[m] = make_uint4(y[4 * m], y[4 * m + 1], y[4 * m + 2], y[4 * m + 3]);
        if (g == 0 && io.lse)
          io.lse[row * io.n_q_heads + hq] = sum != 0.f ? (ref[nt][k] + log2f(sum)) * 0.6931471805599453f : -INFINITY;
      }
    __syncwarp();
  }
}

// Joins the parts of items: part 2 w + 1 of the worker with the first and parts
// 2 (w + 1), ... of those behind it.  A CTA takes R / gridDim.y rows of the items of
// every gridDim.x-th worker (most have none: a CTA for each takes 7 us longer): a row
// per warp, or where there are many parts all warps one row after the other, the parts
// shared out among them.
constexpr int kFewParts = 12;
template <class T, int D, int R, int kJoinWarps>
__global__ void __launch_bounds__(kJoinWarps * 32) k_kvq_join(const __grid_constant__ KvqParams P) {
  constexpr int V = D / 32;
  __shared__ float sum_o[kJoinWarps][D];
  __shared__ float2 sum_l[kJoinWarps];
  const mk_kvq_attn_io& io = P.io;
  const int lane = lane_id(), warp = threadIdx.x / 32;
  pdl_wait();
  const int mine = blockIdx.x + lane * gridDim.x;  // (the host sees to it that 32 are enough)
  uint32_t todo = __ballot_sync(0xffffffffu, mine < P.workers && P.split[mine].parts != 0);
  const int rows = R / gridDim.y, r0 = blockIdx.y * rows;
  for (; todo; todo &= todo - 1) {
    const int worker = blockIdx.x + (__ffs(todo) - 1) * gridDim.x;
    const Split sp = P.split[worker];
    const int n = sp.parts << sp.folded;
    // adds up parts from, from + step, ...
    auto add = [&](int r, int from, int step, float& top, float& all, float (&acc)[V]) {
      top = kNoRef, all = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] = 0.f;
#pragma unroll 4
      for (int k = from; k < n; k += step) {
        const int p = k >> sp.folded;
        const int64_t at = (p ? 2ll * (worker + p) : 2ll * worker + 1) * R + r + (sp.folded & k) * (R / 2);
        const float2 x = P.stat[at];
        const float* o = P.o + at * D + lane * V;
        float y[V];
        if (V == 4) *reinterpret_cast<float4*>(y) = __ldcs(reinterpret_cast<const float4*>(o));
        else *reinterpret_cast<float2*>(y) = __ldcs(reinterpret_cast<const float2*>(o));
        const float next = fmaxf(top, x.x), old = exp2f(top - next), f = exp2f(x.x - next);
        top = next;
        all = all * old + x.y * f;
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] = acc[v] * old + y[v] * f;
      }
    };
    auto write = [&](int fr, float top, float all, const float (&acc)[V]) {
      const float inv = all != 0.f ? 1.f / all : 0.f;
      const int i = quotient(fr, P.by_group), hq = sp.h * P.group + fr - i * P.group;
      const int64_t row = sp.cu + i;
      uint32_t y[V / 2];
#pragma unroll
      for (int v = 0; v < V; v += 2) y[v / 2] = Pack<T>::put(acc[v] * inv, acc[v + 1] * inv);
      uint32_t* to = reinterpret_cast<uint32_t*>(static_cast<T*>(io.out) + row * io.out_stride + hq * D + lane * V);
#pragma unroll
      for (int v = 0; v < V / 2; ++v) to[v] = y[v];
      if (lane == 0 && io.lse)
        io.lse[row * io.n_q_heads + hq] = all != 0.f ? (top + log2f(all)) * 0.6931471805599453f : -INFINITY;
    };
    float acc[V], top, all;
    if (n <= kFewParts) {
      for (int r = r0 + warp; r < r0 + rows && sp.first + r < sp.rows; r += kJoinWarps) {
        add(r, 0, 1, top, all, acc);
        write(sp.first + r, top, all, acc);
      }
      continue;
    }
    for (int r = r0; r < r0 + rows && sp.first + r < sp.rows; ++r) {
      add(r, warp, kJoinWarps, top, all, acc);
#pragma unroll
      for (int v = 0; v < V; ++v) sum_o[warp][lane * V + v] = acc[v];
      if (lane == 0) sum_l[warp] = make_float2(top, all);
      __syncthreads();
      if (warp == 0) {
        float m = kNoRef, s = 0.f, out[V] = {};
        for (int w = 0; w < kJoinWarps; ++w) m = fmaxf(m, sum_l[w].x);
        for (int w = 0; w < kJoinWarps; ++w) {
          const float f = exp2f(sum_l[w].x - m);
          s += sum_l[w].y * f;
#pragma unroll
          for (int v = 0; v < V; ++v) out[v] += sum_o[w][lane * V + v] * f;
        }
        write(sp.first + r, m, s, out);
      }
      __syncthreads();
    }
  }
}

int64_t align256(int64_t v) { return (v + 255) & ~static_cast<int64_t>(255); }

// Lays the workspace out for `workers` over `base`; returns its size.
int64_t lay_out(int workers, int rows, int d, uint8_t* base, KvqParams* P) {
  int64_t at = 256;
  P->status = reinterpret_cast<uint32_t*>(base);
  P->split = reinterpret_cast<Split*>(base + at);
  at = align256(at + workers * static_cast<int64_t>(sizeof(Split)));
  P->stat = reinterpret_cast<float2*>(base + at);
  at = align256(at + 2ll * workers * rows * 8);
  P->o = reinterpret_cast<float*>(base + at);
  return align256(at + 2ll * workers * rows * d * 4);
}

// Rows per tile, by what the requests' rows of a kv head are on average (see above).
int rows_of_tile(const mk_kvq_attn_io* io) {
  const int64_t group = io->n_q_heads / io->kvq.n_kv_heads, rows = io->n_rows * group;
  return rows > 16ll * io->n_requests ? kWideRows : rows > 8ll * io->n_requests ? 16 : 8;
}
int workers_of(int rows, int sms) { return rows == kWideRows ? sms : sms * (rows == 8 ? kWarps<1> : kWarps<2>); }

template <class T, int D, int R>
mk_status launch(const KvqParams& P, int device, int sms, cudaStream_t s) {
  cudaLaunchConfig_t lc = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = attr;
  lc.numAttrs = 1;
  lc.stream = s;
  if (R == kWideRows) {
    const mk_status st = launch_kvq_wide(P, device, sms, s);
    if (st != MK_OK) return st;
  } else {
    constexpr int NT = R == 16 ? 2 : 1, smem = kWarps<NT> * kStages * Layout<D>::kStage;
    static std::atomic<uint64_t> ready{0};  // (once per device: it takes as long as a launch)
    const uint64_t bit = device < 64 ? uint64_t{1} << device : 0;
    if (!(ready.load(std::memory_order_relaxed) & bit)) {
      MK_CUDA_TRY(cudaFuncSetAttribute(k_kvq_attn<T, D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
      ready.fetch_or(bit, std::memory_order_relaxed);
    }
    lc.gridDim = dim3(sms);
    lc.blockDim = dim3(kWarps<NT> * 32);
    lc.dynamicSmemBytes = smem;
    MK_CUDA_TRY(cudaLaunchKernelEx(&lc, k_kvq_attn<T, D, NT>, P));
  }
  // few items, many parts each: rows on CTAs of their own
  const int64_t items = (static_cast<int64_t>(P.io.n_rows) * P.group / R + P.io.n_requests) * P.io.kvq.n_kv_heads;
  const bool few = items * 16 < P.workers;
  lc.gridDim = dim3(std::min(P.workers, (few ? 1 : 12) * sms), few ? R : R == kWideRows ? R / 8 : 1);
  lc.dynamicSmemBytes = 0;
  if (few) {
    lc.blockDim = dim3(8 * 32);
    MK_CUDA_TRY(cudaLaunchKernelEx(&lc, k_kvq_join<T, D, R, 8>, P));
  } else {
    lc.blockDim = dim3(4 * 32);
    MK_CUDA_TRY(cudaLaunchKernelEx(&lc, k_kvq_join<T, D, R, 4>, P));
  }
  return MK_OK;
}
template <class T, int D>
mk_status launch(const KvqParams& P, int rows, int device, int sms, cudaStream_t s) {
  return rows == 8    ? launch<T, D, 8>(P, device, sms, s)
         : rows == 16 ? launch<T, D, 16>(P, device, sms, s)
                      : launch<T, D, kWideRows>(P, device, sms, s);
}

mk_status check_shapes(const mk_kvq_attn_io* io) {
  if (!io) return MK_ERR_INVALID_ARG;
  const mk_status st = check_kvq(io->kvq, false);
  if (st != MK_OK) return st;
  if (io->n_requests < 1 || io->n_requests > 65536 || io->n_rows < 0) return MK_ERR_INVALID_ARG;
  if (io->n_q_heads < 1 || io->n_q_heads % io->kvq.n_kv_heads) return MK_ERR_INVALID_ARG;
  if (io->n_q_heads / io->kvq.n_kv_heads > 64 || io->n_q_heads > 4096) return MK_ERR_UNSUPPORTED;
  if (io->kvq.head_dim != 64 && io->kvq.head_dim != 128) return MK_ERR_UNSUPPORTED;
  if (io->dtype != MK_BF16 && io->dtype != MK_FP16) return MK_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(io->n_rows) * io->n_q_heads > INT32_MAX - 4096) return MK_ERR_UNSUPPORTED;
  return MK_OK;
}

// What a self-test sets about the waits.
struct Waits {
  uint64_t ns;
  int32_t withhold, which;
};

mk_status call_attn(const mk_kvq_attn_io* io, void* workspace, int64_t workspace_bytes, void* stream,
                    const Waits* test) {
  mk_status st = check_shapes(io);
  if (st != MK_OK) return st;
  st = check_kvq(io->kvq, true);
  if (st != MK_OK) return st;
  const mk_kvq_cache& c = io->kvq;
  const int64_t d = c.head_dim, n = io->n_rows, slots = static_cast<int64_t>(c.n_pages) * c.page_size;
  const int64_t page_bytes = static_cast<int64_t>(c.n_kv_heads) * c.page_size * (d / 2);
  if (page_bytes > INT32_MAX) return MK_ERR_UNSUPPORTED;
  if (io->max_pages < 0 || io->table_stride < io->max_pages || io->window < 0) return MK_ERR_INVALID_ARG;
  if (static_cast<int64_t>(io->max_pages) * c.page_size > INT32_MAX - 256) return MK_ERR_INVALID_ARG;
  if (!(io->scale >= 0.f && io->scale <= FLT_MAX / 2)) return MK_ERR_INVALID_ARG;
  if (io->tree_mask && io->window > 0 && io->window < 64) return MK_ERR_UNSUPPORTED;
  if (!io->lens || !io->cu_rows || !workspace) return MK_ERR_INVALID_ARG;
  if (io->max_pages && !io->block_table) return MK_ERR_INVALID_ARG;
  if (n && (!io->q || !io->out)) return MK_ERR_INVALID_ARG;
  const int64_t width = io->n_q_heads * d;
  if (io->q_stride % 8 || io->out_stride % 8 || io->q_stride < width || io->out_stride < width)
    return MK_ERR_INVALID_ARG;
  if (misaligned(io->q, 16) || misaligned(io->out, 16) || misaligned(workspace, 256) || misaligned(io->lens, 4) ||
      misaligned(io->cu_rows, 4) || misaligned(io->block_table, 4) || misaligned(io->tree_mask, 8) ||
      misaligned(io->lse, 4))
    return MK_ERR_INVALID_ARG;
  // what is written, against what is read
  struct Range { const void* p; int64_t n; };
  const int64_t rows = slots * c.n_kv_heads;
  const Range out[] = {{io->out, span_bytes(n, width, io->out_stride, 2)}, {io->lse, n * io->n_q_heads * 4},
                       {workspace, workspace_bytes}};
  const Range in[] = {{io->q, span_bytes(n, width, io->q_stride, 2)},
                      {io->block_table, span_bytes(io->n_requests, io->max_pages, io->table_stride, 4)},
                      {io->lens, io->n_requests * 4ll}, {io->cu_rows, io->n_requests * 4ll + 4},
                      {io->tree_mask, n * 8}, {c.k_codes, rows * (d / 2)}, {c.v_codes, rows * (d / 2)},
                      {c.k_scales, rows * (d / 16)}, {c.v_scales, rows * (d / 16)},
                      {c.k_exp, c.n_kv_heads * 4ll}, {c.v_exp, c.n_kv_heads * 4ll}};
  for (int a = 0; a < 3; ++a) {
    for (const Range& r : in)
      if (overlap(r.p, r.n, out[a].p, out[a].n)) return MK_ERR_INVALID_ARG;
    for (int b = a + 1; b < 3; ++b)
      if (overlap(out[a].p, out[a].n, out[b].p, out[b].n)) return MK_ERR_INVALID_ARG;
  }
  int device = 0, sms = 0;
  st = check_device(workspace, &device, &sms);
  if (st != MK_OK) return st;
  const int tile = rows_of_tile(io);
  KvqParams P;
  P.workers = workers_of(tile, sms);
  if (workspace_bytes < lay_out(P.workers, tile, static_cast<int>(d), static_cast<uint8_t*>(workspace), &P))
    return MK_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (n == 0) {
    MK_CUDA_TRY(cudaMemsetAsync(workspace, 0, sizeof(uint32_t), s));
    return MK_OK;
  }
  P.io = *io;
  if (!c.n_pages)  // (a pool without pages is never read)
    P.io.kvq.k_codes = P.io.kvq.v_codes = P.io.kvq.k_scales = P.io.kvq.v_scales = const_cast<void*>(io->q);
  P.scale_log2 = (io->scale != 0.f ? io->scale : 1.f / std::sqrt(static_cast<float>(d))) * 1.4426950408889634f;
  P.group = io->n_q_heads / c.n_kv_heads;
  P.by_group = make_divisor(P.group);
  P.page_shift = __builtin_ctz(static_cast<uint32_t>(c.page_size));
  P.page_bytes = static_cast<uint32_t>(page_bytes);
  P.test = test != nullptr;
  P.wait_ns = test ? test->ns : kKvqWaitNs;
  P.withhold = test ? test->withhold : kKvqNothing;
  P.withhold_at = test ? test->which : 0;
  if (io->dtype == MK_BF16)
    return d == 128 ? launch<__nv_bfloat16, 128>(P, tile, device, sms, s) : launch<__nv_bfloat16, 64>(P, tile, device, sms, s);
  return d == 128 ? launch<__half, 128>(P, tile, device, sms, s) : launch<__half, 64>(P, tile, device, sms, s);
}

}  // namespace

}  // namespace mk

using namespace mk;

extern "C" {

mk_status mk_kvq_attn_workspace(const mk_kvq_attn_io* io, int64_t* bytes) {
  if (!bytes) return MK_ERR_INVALID_ARG;
  *bytes = 0;
  const mk_status st = check_shapes(io);
  if (st != MK_OK) return st;
  int dev = -1, sms = 0;
  MK_CUDA_TRY(cudaGetDevice(&dev));
  MK_CUDA_TRY(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
  KvqParams P;
  const int rows = rows_of_tile(io);
  *bytes = lay_out(workers_of(rows, sms), rows, io->kvq.head_dim, nullptr, &P);
  return MK_OK;
}

mk_status mk_kvq_attn(const mk_kvq_attn_io* io, void* workspace, int64_t workspace_bytes, void* stream) {
  return call_attn(io, workspace, workspace_bytes, stream, nullptr);
}

mk_status mk_selftest_kvq_waits(const mk_kvq_attn_io* io, void* workspace, int64_t workspace_bytes,
                                uint64_t wait_ns, int32_t withhold, int32_t which, void* stream) {
  if (!wait_ns || wait_ns > kKvqWaitNs || withhold < kKvqNothing || withhold > kKvqTaken || which < 0)
    return MK_ERR_INVALID_ARG;
  mk_status st = check_shapes(io);
  if (st != MK_OK) return st;
  if (io->dtype != MK_BF16 || io->kvq.head_dim != 64 || rows_of_tile(io) != kWideRows) return MK_ERR_UNSUPPORTED;
  const Waits w{wait_ns, withhold, which};
  st = call_attn(io, workspace, workspace_bytes, stream, &w);
  if (st != MK_OK) return st;
  MK_CUDA_TRY(cudaStreamSynchronize(static_cast<cudaStream_t>(stream)));
  return mk_kvq_attn_status(workspace);
}

mk_status mk_kvq_attn_status(const void* workspace) {
  if (!workspace) return MK_ERR_INVALID_ARG;
  uint32_t s = 0;
  MK_CUDA_TRY(cudaMemcpy(&s, workspace, sizeof(s), cudaMemcpyDeviceToHost));
  return s == 0 ? MK_OK : MK_ERR_TIMEOUT;
}

}  // extern "C"
