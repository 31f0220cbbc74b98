// kvq_wide.cu -- attention over a paged cache in 4 bits for row tiles of up to 128
// rows, on the 5th-generation tensor cores.
//
// The steps of kvq_attn.cu with the rows as operand A: S = Q K^T (128 rows by 128
// keys), P = 2^(S - r) over S's place in tensor memory, O += P V.  With 16 rows the
// conversions of the codes cost more than the products; here every key is converted
// once for all of a tile's rows:
//   8 warps  bring 16 keys of each tile into a ring of their own, turn their codes
//            into fp16 and store them as operand B (K along the dimensions, V along
//            the keys: both are rows of a key's dimensions in shared memory);
//   4 warps  keep a row per thread: they bring Q, turn scores into weights, and write
//            the results;
//   1 warp   (of a fourth warpgroup) issues the products, the scores of the next tile before P V.
// Two tiles of K and of S and three of V keep them busy at the same time; Q, S, P and
// O are in tensor memory (two tiles of S: with three the time was the same).  Key tiles
// of all items lie on one line, of which each CTA (one per SM) takes an equal stretch;
// k_kvq_join joins what lies in several.
//
// What bounds it: a key tile takes the converting warps about 2400 cycles (issue of the
// copies 430, K and V 500 each and 200 each until their buffers are free, fence and
// hand-off 420), the chain from S (920) by way of the weights (1630) to P V 3500 for two
// tiles at a time, the tensor cores 1024 (by time stamps, which slow the kernel by a
// seventh).  16 requests of up to 16 rows (32 heads over 8) and 16384 keys of d 128: 89 us,
// 157 MB, the tensor pipe active 33 % of the time; on row tiles of 16 without tcgen05 143 us.
// Copies by warps of their own (bulk or cp.async) take 110 us, twelve converting warps 93.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "kvq_attn.cuh"

namespace mk {

namespace {

constexpr int kKeys = 128;       // of a key tile
constexpr int kRows = kWideRows;
constexpr int kConvert = 8;      // warps that convert: 16 keys of a tile each
constexpr int kThreads = 512;    // four warpgroups: rows, two that convert, products
constexpr int kStages = 3;       // tiles of a converting warp's ring
constexpr int kValues = 3;       // tiles of V
constexpr float kMost = 32768.f; // a row's sum of weights over a tile
constexpr uint64_t kWaitNs = kKvqWaitNs;
constexpr uint32_t kTimeout = 1;
// columns of tensor memory: two tiles of scores and weights, O, Q
constexpr uint32_t kOutAt = 256, kQAt = 384;

template <int D>
struct alignas(1024) WideSmem {
  static constexpr int kTile = kKeys * D * 2;
  static constexpr int kCodes = 16 * D / 2, kScales = 16 * D / 16, kStage = 2 * (kCodes + kScales);
  uint8_t k[2][kTile], v[kValues][kTile];
  uint8_t raw[kConvert][kStages][kStage];  // of each 16 keys: K's codes, V's, K's scales, V's
  uint64_t k_full[2], k_empty[2], v_full[kValues], v_empty[kValues], s_full[2], p_full[2], q_full, halves, taken, drained;
  int64_t sum[kThreads / 32];
  int64_t first_at;
  int32_t first;
  uint32_t tmem, abort;
};

// fp16 operands, f32 sums, M 128; b_along_n: operand B runs along N.
__host__ __device__ constexpr uint32_t idesc_fp16(int N, bool b_along_n) {
  return (1u << 4) | (b_along_n ? 1u << 16 : 0u) | (static_cast<uint32_t>(N >> 3) << 17) | (8u << 24);
}

// Whether a self-test withholds this hand-off.
template <bool kTest>
MK_DEV bool withheld(const KvqParams& P, KvqWithhold what, int at) {
  return kTest && P.withhold == what && P.withhold_at == at;
}

// Bounded waits of whole warps: false once any wait of the CTA has run out.
template <bool kTest, int D>
MK_DEV bool wait_warp(const KvqParams& P, WideSmem<D>& S, uint64_t* bar, uint32_t parity) {
  bool ok = mbar_try_wait(bar, parity);
  if (!ok) {
    const uint64_t t0 = globaltimer();
    while (true) {
#pragma unroll 1
      for (int i = 0; i < 64 && !ok; ++i) ok = mbar_try_wait(bar, parity);
      if (ok || *const_cast<volatile uint32_t*>(&S.abort)) break;
      if (globaltimer() - t0 > (kTest ? P.wait_ns : kWaitNs)) {
        *const_cast<volatile uint32_t*>(&S.abort) = 1;
        atomicExch(P.status, kTimeout);
        break;
      }
    }
  }
  return __all_sync(0xffffffffu, ok);
}

// A stretch of one item's key tiles, as every warp works it out.
struct Item {
  int32_t b, h, cu, n, base, len, rows, first;  // rows of the kv head, the tile's first
  int32_t tile, tile_end;                       // key tiles to go through
  int32_t klo, khi;                             // keys that some row sees
  int32_t parts;                                // workers that share it
  bool starts;                                  // this one has its first key tile
  // No more than half of the tile's rows: they are there twice, and the first half of
  // the threads takes the even key tiles, the second the odd ones (the other half's
  // weights are zeros), so that the weights of two tiles are made at the same time.
  bool folded;
};
struct Walk {
  int64_t pos, end, begin, share;
  int32_t b;
  // The next stretch (for whole warps); false if there is none.
  MK_DEV bool next(const KvqParams& P, Item& it) {
    const mk_kvq_attn_io& io = P.io;
    const int Hk = io.kvq.n_kv_heads;
    Req rq;
    Piece piece;
    int64_t item, start;
    do {
      if (pos >= end) return false;
      rq = read_req<kRows, kKeys>(P, b);
      for (int64_t cost; pos >= begin + (cost = rq.cost(Hk)); rq = read_req<kRows, kKeys>(P, b)) {
        begin += cost;
        ++b;
      }
      item = (pos - begin) / (rq.tiles + rq.lead);
      start = begin + item * (rq.tiles + rq.lead);
      const int64_t to = min(end, start + rq.tiles + rq.lead);
      piece = piece_of(rq, pos - start, to - start);
      pos = to;
    } while (piece.a >= piece.b);  // (what an item takes on top of its key tiles)
    it.h = static_cast<int>(item / rq.row_tiles);
    const int rt = static_cast<int>(item - static_cast<int64_t>(it.h) * rq.row_tiles);
    const int ta = piece.a, tb = piece.b;
    it.b = b, it.cu = rq.cu, it.n = rq.n, it.base = rq.base, it.len = rq.len;
    it.rows = rq.n * P.group;
    it.first = rt * kRows;
    it.starts = ta == 0;
    it.parts = parts_of(rq, start, share);
    it.folded = it.rows - it.first <= kRows / 2;
    const int i0 = quotient(it.first, P.by_group), i1 = quotient(min(it.rows, it.first + kRows) - 1, P.by_group);
    int depth = i0;
    it.khi = min(rq.len, rq.base + i1 + 1);
    if (io.tree_mask) {
      // (a row sees its own key and no row the 65th; the lowest window is that of the
      // row with the fewest bits)
      it.khi = min(rq.len, rq.base + 64);
      depth = 0;
      if (io.window) {
        int least = 63;
        for (int i = i0 + static_cast<int>(lane_id()); i <= i1; i += 32) least = min(least, __popcll(io.tree_mask[rq.cu + i]) - 1);
        depth = __reduce_min_sync(0xffffffffu, least);
      }
    }
    it.klo = io.window ? max(0, rq.base + depth - io.window + 1) : 0;
    it.tile = max(rq.tile0 + ta, min(it.klo, it.khi) / kKeys);
    it.tile_end = min(rq.tile0 + tb, (it.khi + kKeys - 1) / kKeys);
    return true;
  }
};

// ---- converting warps
template <int D, bool kTest>
MK_DEV void convert(const KvqParams& P, WideSmem<D>& S, Walk walk, int w) {
  using L = WideSmem<D>;
  const mk_kvq_attn_io& io = P.io;
  const mk_kvq_cache& c = io.kvq;
  constexpr int kChunks = D / 32;           // of 32 codes (16 bytes) of a key
  constexpr int kPer = 16 * kChunks / 32;   // of a lane
  const int lane = lane_id(), key = lane & 15, row = w * 16 + key;
  const uint32_t ring = smem_u32(S.raw[w]);
  constexpr int kScaleLanes = L::kScales / 16;
  // this lane's 16 bytes of each copy, and their place: the chunks of a key are turned
  // so that eight keys' meet no bank twice when they are read
  const int ck = lane / kChunks, cc = lane % kChunks;
  const uint32_t place = ck * (D / 2) + ((cc ^ (D == 128 ? ck >> 1 & 3 : ck >> 2 & 1)) << 4);
  const uint8_t* k_lane = static_cast<const uint8_t*>(c.k_codes) + lane * 16;
  const uint8_t* v_lane = static_cast<const uint8_t*>(c.v_codes) + lane * 16;
  const uint8_t* s_lane = static_cast<const uint8_t*>(lane < kScaleLanes ? c.k_scales : c.v_scales) + (lane & (kScaleLanes - 1)) * 16;
  int done = 0;  // tiles of this CTA
  Item it;
  while (walk.next(P, it)) {
    const int32_t* table = io.block_table + it.b * io.table_stride;
    const uint32_t head_bytes = static_cast<uint32_t>(it.h << P.page_shift) * (D / 2);
    // pages of this warp's keys of 32 tiles, one per lane, and those of the next 32
    auto page_of = [&](int tile) {
      const int j = tile * kKeys + w * 16;
      return tile < it.tile_end && j < it.khi ? table[j >> P.page_shift] : -1;
    };
    int load = it.tile, pages_at = load;
    int pages = page_of(load + lane), pages_next = page_of(load + 32 + lane);
    auto issue = [&](int stage) {
      if (load < it.tile_end) {
        if (load - pages_at == 32) {
          pages_at = load;
          pages = pages_next;
          pages_next = page_of(load + 32 + lane);
        }
        const int page = __shfl_sync(0xffffffffu, pages, load - pages_at);
        const bool there = static_cast<uint32_t>(page) < static_cast<uint32_t>(c.n_pages);
        const int64_t off = there ? static_cast<int64_t>(static_cast<uint64_t>(static_cast<uint32_t>(page)) * P.page_bytes +
                                                         (head_bytes + ((load * kKeys + w * 16) & (c.page_size - 1)) * (D / 2)))
                                  : 0;
        const uint32_t st = ring + stage * L::kStage;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          cp_async16(st + place + i * 512, k_lane + off + i * 512, there);
          cp_async16(st + L::kCodes + place + i * 512, v_lane + off + i * 512, there);
        }
        if (lane < 2 * kScaleLanes) cp_async16(st + 2 * L::kCodes + lane * 16, s_lane + (off >> 3), there);
        ++load;
      }
      cp_async_commit();
    };
    int stage = 0, stage_in = 0;
    auto after = [](int x) { return x == kStages - 1 ? 0 : x + 1; };
    for (int i = 0; i < kStages - 1; ++i, stage_in = after(stage_in)) issue(stage_in);
    for (int tile = it.tile; tile < it.tile_end; ++tile, ++done, stage = after(stage)) {
      cp_async_wait<kStages - 2>();
      __syncwarp();
      issue(stage_in);
      stage_in = after(stage_in);
      const uint8_t* st = S.raw[w][stage];
      const int j = tile * kKeys + row;
      const bool seen = j >= it.klo && j < it.khi;
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const int of = kv ? kValues : 2, buf = done % of, round = done / of;
        if (round && !wait_warp<kTest>(P, S, kv ? &S.v_empty[buf] : &S.k_empty[buf], (round - 1) & 1)) {
          cp_async_wait<0>();
          return;
        }
        uint8_t* to = (kv ? S.v[buf] : S.k[buf]) + row * 128;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int chunk = (lane >> 4) + 2 * i;
          const uint4 x = *reinterpret_cast<const uint4*>(st + kv * L::kCodes + key * (D / 2) + ((chunk ^ (D == 128 ? key >> 1 & 3 : key >> 2 & 1)) << 4));
          uint32_t pair = *reinterpret_cast<const uint16_t*>(st + 2 * L::kCodes + kv * L::kScales + key * (D / 16) + chunk * 2);
          // keys that no row sees may hold anything: a weight of 0 must meet a number (those
          // between a tree's keys: see issue_mmas)
          if (kv && !seen) pair = 0;
          const Scales f = make_scales(pair);
          const uint32_t words[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            uint32_t y[4];
            values(words[n], n < 2 ? f.first() : f.second(), y);
            const int unit = chunk * 4 + n;  // of 8 dimensions; 8 of them to a panel
            *reinterpret_cast<uint4*>(to + (unit >> 3) * (kKeys * 128) + (((unit & 7) ^ (row & 7)) << 4)) = make_uint4(y[0], y[1], y[2], y[3]);
          }
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        if (!withheld<kTest>(P, kKvqKeys, done)) mbar_arrive(&S.k_full[done & 1]);
        if (!withheld<kTest>(P, kKvqValues, done)) mbar_arrive(&S.v_full[done % kValues]);
      }
      __syncwarp();
    }
    cp_async_wait<0>();
    __syncwarp();
  }
}

// ---- the products' issuer
template <int D, bool kTest>
MK_DEV bool issue_mmas(const KvqParams& P, WideSmem<D>& S, Walk walk) {
  constexpr uint32_t kIdS = idesc_fp16(kKeys, false), kIdO = idesc_fp16(D, true);
  const uint32_t tmem = S.tmem, to = tmem + kOutAt, tq = tmem + kQAt;
  const mk_kvq_attn_io& io = P.io;
  int done = 0, items = 0;
  Item it;
  uint64_t hidden = 0;  // keys from it.base on that no row's tree word has
  int hidden_from = INT_MAX;  // first key tile with such
  // O += P V of a tile
  auto pv = [&](int at, int tile) {
    const int buf = at & 1, vb = at % kValues;
    const bool first = tile == it.tile;
    if (!wait_warp<kTest>(P, S, &S.v_full[vb], (at / kValues) & 1)) return false;
    if (tile >= hidden_from) {
      // They may hold anything, and a weight of 0 must meet a number.  (Here 16 trees over
      // 16384 keys take 89 us, 88 without; by the warps that convert, 92 to 97.)
      const int j0 = tile * kKeys;
      for (int j = max(j0, it.base); j < min(j0 + kKeys, it.khi); ++j)
        if (hidden >> (j - it.base) & 1 && lane_id() < D / 8)
          *reinterpret_cast<uint4*>(S.v[vb] + (lane_id() >> 3) * (kKeys * 128) + (j - j0) * 128 + (lane_id() & 7) * 16) = make_uint4(0, 0, 0, 0);
      fence_proxy_async_smem();
      __syncwarp();
    }
    if (!wait_warp<kTest>(P, S, &S.p_full[buf], (at >> 1) & 1)) return false;
    tc_fence_after();
    if (elect_one()) {
      const uint64_t vd = sdesc_mnmajor_sw128(smem_u32(S.v[vb]), kKeys * 128);
#pragma unroll
      for (int k = 0; k < kKeys / 16; ++k)
        mma_ts(to, tmem + buf * 128 + 8 * k, vd + k * (16 * 128 >> 4), kIdO, !first || k > 0);
      if (!withheld<kTest>(P, kKvqValuesUsed, at)) mma_commit(&S.v_empty[vb]);
    }
    __syncwarp();
    return true;
  };
  while (walk.next(P, it)) {
    const int n = it.tile_end - it.tile;
    if (n <= 0) continue;
    if (!wait_warp<kTest>(P, S, &S.q_full, items++ & 1)) return false;
    for (int t = 0; t < n; ++t, ++done) {
      const int buf = done & 1;
      if (!wait_warp<kTest>(P, S, &S.k_full[buf], (done >> 1) & 1)) return false;
      // (its scores go over weights that the product two tiles back reads; products with
      // other sums need not run in order)
      if (done >= 2 && !wait_warp<kTest>(P, S, &S.v_empty[(done - 2) % kValues], ((done - 2) / kValues) & 1)) return false;
      tc_fence_after();
      if (elect_one()) {
        const uint64_t kd = sdesc_kmajor_sw128(smem_u32(S.k[buf]));
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint64_t at = (k >> 2) * (kKeys * 128 >> 4) + (k & 3) * 2;
          mma_ts(tmem + buf * 128, tq + 8 * k, kd + at, kIdS, k);
        }
        if (!withheld<kTest>(P, kKvqScores, done)) mma_commit(&S.s_full[buf]);
        if (!withheld<kTest>(P, kKvqKeysUsed, done)) mma_commit(&S.k_empty[buf]);
      }
      __syncwarp();
      // (while the scores are on their way)
      if (t == 0 && io.tree_mask) {
        uint64_t tree = 0;
        const int i1 = quotient(min(it.rows, it.first + kRows) - 1, P.by_group);
        for (int i = quotient(it.first, P.by_group) + static_cast<int>(lane_id()); i <= i1; i += 32) tree |= io.tree_mask[it.cu + i];
        hidden = ~bits_of_all(tree);
        hidden_from = it.base / kKeys;
      }
      if (t && !pv(done - 1, it.tile + t - 1)) return false;
    }
    if (!pv(done - 1, it.tile_end - 1)) return false;
  }
  return true;
}

// ---- a row per thread
// What a thread knows of its row of an item.
struct Row {
  Item it;
  int64_t at;     // row of q
  uint64_t tree;  // bits of the keys from it.base on
  int32_t hq, lo, hi;
  float c;        // factor on its scores
  bool valid;
};

// Brings the row's Q (the CTA's row tile number `taken`) into tensor memory, in fp16 relative to its largest value, the
// pairs in the order of the codes'.
template <class T, int D, bool kTest>
MK_DEV void take_row(const KvqParams& P, WideSmem<D>& S, Row& r, int taken) {
  const mk_kvq_attn_io& io = P.io;
  const Item& it = r.it;
  const int row = threadIdx.x, f = it.first + (it.folded ? row & (kRows / 2 - 1) : row);
  r.valid = f < it.rows;
  const int i = quotient(r.valid ? f : 0, P.by_group);
  r.hq = it.h * P.group + (r.valid ? f - i * P.group : 0);
  r.at = it.cu + i;
  r.lo = r.hi = 0;
  r.tree = 0;
  if (r.valid) {
    if (io.tree_mask) r.tree = io.tree_mask[r.at];
    const int p = it.base + (io.tree_mask ? __popcll(r.tree) - 1 : i);
    r.lo = io.window ? max(0, p - io.window + 1) : 0;
    r.hi = io.tree_mask ? min(it.len, it.base) : min(it.len, it.base + i + 1);
  }
  if (it.tile >= it.tile_end) return;
  float factor = 1.f;
  const uint4* src = reinterpret_cast<const uint4*>(static_cast<const T*>(io.q) + r.at * io.q_stride + r.hq * D);
  uint4 raw[D / 8];
#pragma unroll
  for (int j = 0; j < D / 8; ++j) raw[j] = r.valid ? src[j] : make_uint4(0, 0, 0, 0);
  if (!std::is_same<T, __half>::value) {
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < D / 8; ++j)
      top = __vmaxu2(top, __vmaxu2(__vmaxu2(raw[j].x & 0x7FFF7FFFu, raw[j].y & 0x7FFF7FFFu),
                                   __vmaxu2(raw[j].z & 0x7FFF7FFFu, raw[j].w & 0x7FFF7FFFu)));
    top = max(top & 0xFFFFu, top >> 16);
    const int e = min(max(static_cast<int>(top >> 7), 1), 253);
    const float inv = top < 0x7F80u ? __int_as_float((254 - e) << 23) : 1.f;
    factor = top < 0x7F80u ? __int_as_float(e << 23) : 1.f;
#pragma unroll
    for (int j = 0; j < D / 8; ++j) {
      uint32_t* x = reinterpret_cast<uint32_t*>(&raw[j]);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 y = Pack<T>::get(x[k]);
        x[k] = half2_bits(y.x * inv, y.y * inv);
      }
    }
  }
  r.c = score_factor(P, factor, it.h);
#pragma unroll
  for (int j = 0; j < D / 8; ++j)
    raw[j] = make_uint4(__byte_perm(raw[j].x, raw[j].z, 0x5410), __byte_perm(raw[j].x, raw[j].z, 0x7632),
                        __byte_perm(raw[j].y, raw[j].w, 0x5410), __byte_perm(raw[j].y, raw[j].w, 0x7632));
  const uint32_t to = S.tmem + (static_cast<uint32_t>(row & ~31) << 16) + kQAt;
#pragma unroll
  for (int j = 0; j < D / 64; ++j) tmem_st32(to + 32 * j, reinterpret_cast<const uint32_t*>(raw + 8 * j));
  tmem_st_wait();
  tc_fence_before();
  __syncwarp();
  if (lane_id() == 0 && !withheld<kTest>(P, kKvqRowTile, taken)) mbar_arrive(&S.q_full);
  __syncwarp();
}

template <class T, int D, bool kTest>
MK_DEV void rows(const KvqParams& P, WideSmem<D>& S, Walk walk) {
  const mk_kvq_attn_io& io = P.io;
  const int lane = lane_id(), warp = threadIdx.x / 32, row = threadIdx.x;
  const uint32_t lanes = S.tmem + (static_cast<uint32_t>(warp * 32) << 16), to = lanes + kOutAt;
  int done = 0, joined = 0, items = 0;
  Row r;
  bool more = walk.next(P, r.it);
  if (more) take_row<T, D, kTest>(P, S, r, items++);
  while (more) {
    const bool warp_valid = __any_sync(0xffffffffu, r.valid);
    const int n = r.it.tile_end - r.it.tile;
    float ref = kNoRef, l = 0.f;
    for (int t = 0; t < n; ++t, ++done) {
      const int buf = done & 1, k0 = (r.it.tile + t) * kKeys;
      if (!wait_warp<kTest>(P, S, &S.s_full[buf], (done >> 1) & 1)) return;
      tc_fence_after();
      const uint32_t ts = lanes + buf * 128;
      if (warp_valid && r.it.folded && (t & 1) != warp >> 1) {
        uint32_t p[32];
#pragma unroll
        for (int x = 0; x < 32; ++x) p[x] = 0;
        tmem_st32(ts, p);
        tmem_st32(ts + 32, p);
        tmem_st_wait();
      } else if (warp_valid) {
        const bool edge = __any_sync(0xffffffffu, r.valid && (k0 < r.lo || k0 + kKeys > r.hi));
        auto scores = [&](int half, float (&s)[64]) {
          tmem_ld32(ts + half * 64, s);
          tmem_ld32(ts + half * 64 + 32, s + 32);
          tmem_ld_wait();
          if (!edge) return;
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const int at = k0 + half * 64 + q * 32;
            uint32_t see = below(r.hi - at) & ~below(r.lo - at);
            if (io.tree_mask) {
              // bit x: key at + x, of which those from base on follow the row's word
              const int off = r.it.base - at;
              see |= (off >= 32    ? 0u
                      : off >= 0   ? static_cast<uint32_t>(r.tree) << off
                      : off > -64 ? static_cast<uint32_t>(r.tree >> -off)
                                   : 0u) &
                     below(r.it.khi - at);
            }
#pragma unroll
            for (int x = 0; x < 32; ++x)
              if (!(see >> x & 1)) s[32 * q + x] = -INFINITY;
          }
        };
        uint32_t p[64];
        float total;
        bool look = __any_sync(0xffffffffu, r.valid && ref == kNoRef);
#pragma unroll 1
        while (true) {
          if (look) {
            // the row's largest score: the reference moves if it is far above it
            float top = -INFINITY;
#pragma unroll 1
            for (int half = 0; half < 2; ++half) {
              float s[64];
              scores(half, s);
#pragma unroll
              for (int x = 0; x < 64; x += 2) top = max3(top, s[x], s[x + 1]);
            }
            top *= r.c;
            const float next = r.valid && top - ref > kRefBelow ? top - kRefBelow : ref;
            const float old = exp2_approx(ref - next);
            l *= old;
            ref = next;
            if (t && __any_sync(0xffffffffu, old != 1.f)) {
              // (the tile before is in O when its V is free)
              if (!wait_warp<kTest>(P, S, &S.v_empty[(done - 1) % kValues], ((done - 1) / kValues) & 1)) return;
              tc_fence_after();
#pragma unroll 1
              for (int q = 0; q < D / 32; ++q) {
                float o[32];
                tmem_ld32(to + 32 * q, o);
                tmem_ld_wait();
#pragma unroll
                for (int y = 0; y < 32; ++y) o[y] *= old;
                tmem_st32(to + 32 * q, reinterpret_cast<uint32_t*>(o));
              }
              tmem_st_wait();
            }
          }
          float2 sum = make_float2(0.f, 0.f);
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            float s[64];
            scores(half, s);
#pragma unroll
            for (int x = 0; x < 64; x += 2) {
              float2 y = fma2(make_float2(s[x], s[x + 1]), make_float2(r.c, r.c), make_float2(-ref, -ref));
              y.x = exp2_approx(y.x);
              y.y = exp2_approx(y.y);
              sum = add2(sum, y);
              p[half * 32 + x / 2] = half2_bits(y.x, y.y);
            }
          }
          total = sum.x + sum.y;
          // (the comparison is false for NaN)
          if (look || !__any_sync(0xffffffffu, r.valid && total > kMost)) break;
          look = true;
        }
        l += total;
        tmem_st32(ts, p);
        tmem_st32(ts + 32, p + 32);
        tmem_st_wait();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0 && !withheld<kTest>(P, kKvqWeights, done)) mbar_arrive(&S.p_full[buf]);
      __syncwarp();
    }

    // The next item's Q goes its way before this one's results: Q's last products, the
    // last tile's scores, are there.
    const Row mine = r;
    more = walk.next(P, r.it);
    if (more) take_row<T, D, kTest>(P, S, r, items++);
    if (n > 0) {
      if (!wait_warp<kTest>(P, S, &S.v_empty[(done - 1) % kValues], ((done - 1) / kValues) & 1)) return;
      tc_fence_after();
    }
    // An item that this CTA has whole is written from here.  If it is folded, the second
    // half of the threads leaves its results in the CTA's own place of the workspace,
    // where the first half takes them before the second writes there again.
    const bool whole = mine.it.parts == 1, twice = whole && mine.it.folded && n > 0, second = twice && warp >= 2;
    const float unit_v = 8.f * pow2(io.kvq.v_exp ? clamp_exp(io.kvq.v_exp[mine.it.h]) : 0);
    const int64_t part = (2ll * blockIdx.x + mine.it.starts) * kRows;
    float f1 = 1.f, f2 = 0.f;  // what this half's and the other one's O are multiplied with
    if (warp >= 2 && joined && !wait_warp<kTest>(P, S, &S.taken, (joined - 1) & 1)) return;
    joined += twice;
    if (twice && !second) {
      if (!wait_warp<kTest>(P, S, &S.halves, (joined - 1) & 1)) return;
      if (mine.valid) {
        const float2 other = P.stat[part + row + kRows / 2];
        const float top = fmaxf(ref, other.x);
        f1 = exp2_approx(ref - top);
        f2 = exp2_approx(other.x - top);
        l = l * f1 + other.y * f2;
        ref = top;
      }
    }
    if (whole && !second) {
      const float inv = l != 0.f ? unit_v / l : 0.f;
      f1 *= inv;
      f2 = l != 0.f ? f2 / l : 0.f;  // (the other half's are in the values' units)
    } else {
      f1 = unit_v;
    }
    if (warp_valid && !(whole && mine.it.folded && n <= 0 && warp >= 2)) {
#pragma unroll 1
      for (int q = 0; q < D / 32; ++q) {
        float o[32];
        if (n > 0) {
          tmem_ld32(to + 32 * q, o);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int x = 0; x < 32; ++x) o[x] = 0.f;
        }
        if (mine.valid) {
          // eight columns are the dimensions 0 4 1 5 2 6 3 7
          float y[32];
#pragma unroll
          for (int x = 0; x < 32; ++x) y[x] = o[(x & ~7) + (x & 3) * 2 + (x >> 2 & 1)] * f1;
          if (whole && !second) {
            if (twice) {
              const float4* from = reinterpret_cast<const float4*>(P.o + (part + row + kRows / 2) * D + 32 * q);
#pragma unroll
              for (int x = 0; x < 8; ++x) {
                const float4 v = from[x];
                y[4 * x] += v.x * f2, y[4 * x + 1] += v.y * f2, y[4 * x + 2] += v.z * f2, y[4 * x + 3] += v.w * f2;
              }
            }
            uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(io.out) + mine.at * io.out_stride + mine.hq * D + 32 * q);
#pragma unroll
            for (int x = 0; x < 4; ++x)
              dst[x] = make_uint4(Pack<T>::put(y[8 * x], y[8 * x + 1]), Pack<T>::put(y[8 * x + 2], y[8 * x + 3]),
                                  Pack<T>::put(y[8 * x + 4], y[8 * x + 5]), Pack<T>::put(y[8 * x + 6], y[8 * x + 7]));
          } else {
            float4* dst = reinterpret_cast<float4*>(P.o + (part + row) * D + 32 * q);
#pragma unroll
            for (int x = 0; x < 8; ++x) dst[x] = make_float4(y[4 * x], y[4 * x + 1], y[4 * x + 2], y[4 * x + 3]);
          }
        }
        __syncwarp();
      }
      if (mine.valid && (!whole || second)) P.stat[part + row] = make_float2(ref, l);
      if (mine.valid && whole && !second && io.lse)
        io.lse[mine.at * io.n_q_heads + mine.hq] = l != 0.f ? (ref + log2f(l)) * 0.6931471805599453f : -INFINITY;
    }
    tc_fence_before();
    __syncwarp();
    if (twice && lane == 0 && !withheld<kTest>(P, second ? kKvqHalf : kKvqTaken, joined - 1))
      mbar_arrive(second ? &S.halves : &S.taken);
    __syncwarp();
  }
}

template <class T, int D, bool kTest>
__global__ void __launch_bounds__(kThreads, 1) k_kvq_wide(const __grid_constant__ KvqParams P) {
  extern __shared__ uint8_t raw_smem[];
  WideSmem<D>& S = *reinterpret_cast<WideSmem<D>*>((reinterpret_cast<uintptr_t>(raw_smem) + 1023) & ~uintptr_t{1023});
  const mk_kvq_attn_io& io = P.io;
  const int warp = threadIdx.x / 32, lane = lane_id(), Hk = io.kvq.n_kv_heads;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&S.k_full[i], kConvert);
      mbar_init(&S.k_empty[i], 1);
      mbar_init(&S.s_full[i], 1);
      mbar_init(&S.p_full[i], 4);
    }
    for (int i = 0; i < kValues; ++i) {
      mbar_init(&S.v_full[i], kConvert);
      mbar_init(&S.v_empty[i], 1);
    }
    mbar_init(&S.q_full, 4);
    mbar_init(&S.halves, 2);
    mbar_init(&S.taken, 2);
    mbar_init(&S.drained, 1);
    S.abort = 0;
    fence_mbar_init();
  }
  if (warp == 12) {
    __syncwarp();
    tmem_alloc(&S.tmem, 512);
    tmem_relinquish();
    // (not before: a dependent grid that took the columns first would wait for this one,
    // which would wait for the columns)
    pdl_launch_dependents();
  }
  pdl_wait();
  if (blockIdx.x == 0 && threadIdx.x == 0) *P.status = 0;

  // The line: each thread adds up the requests of a stretch of the batch.
  const int per = (io.n_requests + kThreads - 1) / kThreads;
  const int b0 = min(io.n_requests, static_cast<int>(threadIdx.x) * per), b1 = min(io.n_requests, b0 + per);
  int64_t mine = 0;
  for (int b = b0; b < b1; ++b) mine += read_req<kRows, kKeys>(P, b).cost(Hk);
  int64_t upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += x;
  }
  if (lane == 31) S.sum[warp] = upto;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  int64_t total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w == warp) upto += total;
    total += S.sum[w];
  }
  Walk walk;
  walk.share = max(static_cast<int64_t>(1), (total + P.workers - 1) / P.workers);
  walk.pos = blockIdx.x * walk.share;
  walk.end = min(total, walk.pos + walk.share);
  if (walk.pos >= upto - mine && walk.pos < upto) {
    int64_t begin = upto - mine;
    int b = b0;
    for (; b < b1 - 1; ++b) {
      const int64_t cost = read_req<kRows, kKeys>(P, b).cost(Hk);
      if (walk.pos < begin + cost) break;
      begin += cost;
    }
    S.first = b;
    S.first_at = begin;
  }
  if (threadIdx.x == 0) P.split[blockIdx.x].parts = 0;
  __syncthreads();
  walk.b = S.first;
  walk.begin = S.first_at;

  if (walk.pos < walk.end) {
    if (warp < 4) {
      reg_alloc<208>();
      rows<T, D, kTest>(P, S, walk);
    } else if (warp < 4 + kConvert) {
      reg_dealloc<120>();
      convert<D, kTest>(P, S, walk, warp - 4);
    } else {
      reg_dealloc<64>();
      if (warp == 12 && issue_mmas<D, kTest>(P, S, walk)) {
        // an item to join
        Item it;
        while (walk.next(P, it)) {
          if (it.starts && it.parts > 1 && lane == 0)
            P.split[blockIdx.x] = {it.parts, it.folded, it.cu, it.rows, it.first, it.h};
        }
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 12) {
    // A wait has run out (every warp is through: none writes the word any more).
    // Whichever it was: no product may run on when the CTA leaves.  (The converting warps
    // have waited for their own copies.)
    if (*const_cast<volatile uint32_t*>(&S.abort)) {
      if (elect_one()) mma_commit(&S.drained);
      __syncwarp();
      mbar_wait_bounded(&S.drained, 0, kWaitNs);
      __syncwarp();
    }
    tmem_dealloc(S.tmem, 512);
  }
}

template <class T, int D, bool kTest = false>
mk_status launch(const KvqParams& P, int device, int sms, cudaStream_t s) {
  constexpr int smem = sizeof(WideSmem<D>) + 1024;
  static std::atomic<uint64_t> ready{0};  // (once per device: it takes as long as a launch)
  const uint64_t bit = device < 64 ? uint64_t{1} << device : 0;
  if (!(ready.load(std::memory_order_relaxed) & bit)) {
    MK_CUDA_TRY(cudaFuncSetAttribute(k_kvq_wide<T, D, kTest>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
    ready.fetch_or(bit, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t lc = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = attr;
  lc.numAttrs = 1;
  lc.stream = s;
  lc.gridDim = dim3(sms);
  lc.blockDim = dim3(kThreads);
  lc.dynamicSmemBytes = smem;
  MK_CUDA_TRY(cudaLaunchKernelEx(&lc, k_kvq_wide<T, D, kTest>, P));
  return MK_OK;
}

}  // namespace

mk_status launch_kvq_wide(const KvqParams& P, int device, int sms, cudaStream_t s) {
  const bool d128 = P.io.kvq.head_dim == 128;
  if (P.test) return launch<__nv_bfloat16, 64, true>(P, device, sms, s);
  if (P.io.dtype == MK_BF16)
    return d128 ? launch<__nv_bfloat16, 128>(P, device, sms, s) : launch<__nv_bfloat16, 64>(P, device, sms, s);
  return d128 ? launch<__half, 128>(P, device, sms, s) : launch<__half, 64>(P, device, sms, s);
}

}  // namespace mk
