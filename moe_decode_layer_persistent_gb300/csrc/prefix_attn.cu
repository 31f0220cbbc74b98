// prefix_attn.cu -- attention of a batch whose requests share a prefix
// (mk_prefix_attn), on the 5th-generation tensor cores.
//
// For one KV head, the rows (token, q head of the group) of ALL requests form
// one matrix Q against the prefix, and each request's rows one against its own
// keys.  Both are the same computation on a row tile (up to 128 rows) and a
// range of 128-key tiles, with running maximum m and sum l (log2 units):
//   S = Q K^T,  m' = max(m, rowmax S),  P = 2^(S - m'),
//   l' = l 2^(m - m') + rowsum P,  O' = O 2^(m - m') + P V.
// Each stretch of key tiles leaves (O, m, l); the second kernel joins a row's
// stretches: out = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i.
//
// Two launches, the second one chained with programmatic dependent launch:
//   k_attn_tiles  lays all work out on one line (cost units) from the lengths,
//                 which only the GPU knows; one CTA per SM takes an equal
//                 stretch of it, whatever heads, requests and key ranges it
//                 crosses;
//   k_attn_merge  joins the partial results of each row.
#include <algorithm>
#include <cfloat>
#include <climits>
#include <cmath>
#include <cstring>
#include <cuda_fp16.h>

#include "batch.h"
#include "ptx.cuh"

namespace mk {

namespace {

// Cost units of a step, in which both softmax warpgroups take one tile each:
// two row tiles on one key tile (kPairCost), or one row tile on two key tiles
// (kAltCost), which loads twice the bytes.
constexpr int kPairCost = 2;
constexpr int kAltCost = 3;

constexpr int kTileKeys = 128;
constexpr int kStages = 5;          // K and V tiles in flight
constexpr int kFifo = 4;            // pieces handed out ahead
constexpr int kTileThreads = 384;
constexpr float kGrow = 8.f;        // the maximum may lag by 2^8 before O is rescaled
constexpr uint64_t kWaitNs = 2000ull * 1000 * 1000;

// How the line is laid out (every CTA of k_attn_tiles works it out for itself,
// the first leaves it for k_attn_merge).
struct Plan {
  int64_t total, share;     // cost of everything, of one CTA
  int64_t prefix_cost;      // the prefix items come first
  int32_t n_used;           // rows in use
  int32_t tiles;            // row tiles of the prefix
  int32_t kt0, kt1;         // key tiles of the prefix that some row sees
  int32_t lo;               // first prefix key that some row sees
};

// Workspace layout.
struct Space {
  uint32_t* status;
  Plan* plan;
  int64_t* cost;    // [B + 1]: where request b's items start on the line
  float2* ml;       // (m, l) per partial row
  float* o;         // D values per partial row
  // first partial row of each region: the prefix's first (or only) slot by row
  // and head; its second slot (only the last row tile has one) by head; the
  // requests' own first and second slots by row and head; stretches that start
  // in the middle of an item, by CTA and slot
  int64_t pre0, pre1, own0, own1, carry;
};

struct AttnParams {
  mk_prefix_attn_io io;
  float scale_log2;  // scale * log2(e)
  int32_t group;     // G: q heads per KV head
  int32_t tile_tok;  // tokens per row tile: floor(128 / G)
  int32_t box;       // keys per TMA box: min(page_size, 128)
  int32_t page_shift;
  int32_t ctas;
  Space ws;
};

MK_DEV int clampi(int64_t v, int lo, int hi) {
  return v < lo ? lo : v > hi ? hi : static_cast<int>(v);
}
MK_DEV int ceil_div(int a, int b) { return (a + b - 1) / b; }

// One request's lengths, made safe.
struct Req {
  int32_t cu, n, len, base;
  int32_t kt0, kt1;  // key tiles of its own that some row of it sees
};
MK_DEV Req make_req(const AttnParams& P, int64_t cu0, int64_t cu1, int64_t len) {
  const mk_prefix_attn_io& io = P.io;
  Req r;
  r.cu = clampi(cu0, 0, io.n_rows);
  r.n = clampi(cu1, r.cu, io.n_rows) - r.cu;
  r.len = clampi(len, 0, io.max_pages * io.page_size);
  r.base = max(0, r.len - r.n);
  const int64_t low = io.window ? static_cast<int64_t>(r.base) - io.window + 1 : 0;
  r.kt0 = low > 0 ? static_cast<int>(low) / kTileKeys : 0;
  r.kt1 = r.n ? max(r.kt0, ceil_div(r.len, kTileKeys)) : r.kt0;
  return r;
}
MK_DEV Req read_req(const AttnParams& P, int b) {
  return make_req(P, P.io.cu_rows[b], P.io.cu_rows[b + 1], P.io.lens[b]);
}

// Cost of the items of one head: `tiles` row tiles against `kt` key tiles.
MK_DEV int64_t head_cost(int tiles, int kt) {
  return static_cast<int64_t>(tiles >> 1) * kt * kPairCost + (tiles & 1) * ((kt + 1) >> 1) * kAltCost;
}

// ------------------------------------------------------------------ tiles

// A stretch of key tiles of one item, as the scheduler warp hands it out.
struct Piece {
  int32_t kind;      // 0 prefix, 1 a request's own keys, -1 no more
  int32_t alt;       // 1: one row tile, its key tiles by turns to the two slots
  int32_t h, b;
  int32_t tok0;      // first token (row of q) of slot 0's row tile
  int32_t tok_end;   // behind the last token of the prefix rows / the request
  int32_t kt_a, kt_b;
  int32_t klo, khi;  // keys that some row sees
  int32_t first;     // starts its item: leaves its result by row, else by CTA
  int32_t cu, base;
};

template <int D>
struct alignas(1024) TileSmem {
  uint8_t q[2][128 * D * 2];
  uint8_t kv[kStages][128 * D * 2];
  uint64_t kv_full[kStages], kv_empty[kStages];
  uint64_t q_full[2], q_empty[2];
  uint64_t s_full[2], p_full[2], o_done[2];
  uint64_t drained;
  uint64_t fifo_full[kFifo], fifo_empty[kFifo];
  Piece fifo[kFifo];
  Plan plan;
  int64_t sum[kTileThreads / 32];
  int32_t low[kTileThreads / 32];
  int64_t first_at;   // where request `first` starts on the line
  int32_t first;      // the first request with work for this CTA
  uint32_t tmem;
  uint32_t abort;
};

struct Ctx {
  volatile uint32_t* abort;
  uint32_t* status;
};

// Bounded wait: false once any wait of the CTA has run out.
MK_DEV bool wait_bar(const Ctx& c, uint64_t* bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer();
  while (!mbar_try_wait(bar, parity)) {
    if (*c.abort) return false;
    if (globaltimer() - t0 > kWaitNs) {
      *c.abort = 1;
      atomicExch(c.status, 1u);
      return false;
    }
  }
  return true;
}
MK_DEV bool wait_warp(const Ctx& c, uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, wait_bar(c, bar, parity));
}

MK_DEV void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// 32 lanes x 32 columns of 32-bit, this thread's lane (wait with tmem_ld_wait).
MK_DEV void tmem_ld32(uint32_t taddr, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32"
      " {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
MK_DEV void tmem_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32],"
      " {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]),
      "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]),
      "r"(r[30]), "r"(r[31]), "r"(taddr)
      : "memory");
}
MK_DEV void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// D[tmem] (+)= A[tmem] B[smem].
MK_DEV void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                   uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Descriptor of V [keys][64 values of D] as operand B with N = the values: N
// runs along the 128-byte rows (64 values), the next 64 values `lbo` bytes
// on, the next 8 keys 1024 bytes on.
MK_DEV uint64_t sdesc_mnmajor_sw128(uint32_t saddr, uint32_t lbo) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(lbo >> 4) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}

template <class T> struct Types;
template <> struct Types<__nv_bfloat16> {
  static constexpr uint32_t kFormat = 1;
  static MK_DEV uint32_t pack(float a, float b) {
    __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&v);
  }
};
template <> struct Types<__half> {
  static constexpr uint32_t kFormat = 0;
  static MK_DEV uint32_t pack(float a, float b) {
    __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&v);
  }
};
// f32 accumulators, A and B of one 16-bit type, M = 128; bit 16: B runs along N.
template <class T>
__host__ __device__ constexpr uint32_t idesc_of(int N, bool b_along_n) {
  return (1u << 4) | (Types<T>::kFormat << 7) | (Types<T>::kFormat << 10) |
         (b_along_n ? 1u << 16 : 0u) | (static_cast<uint32_t>(N >> 3) << 17) | (8u << 24);
}

MK_DEV float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

MK_DEV void st_global_8(float* p, const float* v) {
  asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "f"(v[0]), "f"(v[1]),
               "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}

// The lowest n bits, n clamped to 0 .. 32.
MK_DEV uint32_t below(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }

// Tile count of a slot in a piece of `tiles` key tiles.
MK_DEV int slot_tiles(const Piece& w, int slot) {
  const int t = w.kt_b - w.kt_a;
  return !w.alt ? t : (t + 1 - slot) >> 1;
}

// ---- the line of work, worked out by the whole CTA
// kReqs consecutive requests per thread and turn: one turn up to 1,536 requests.
constexpr int kReqs = 4;

template <int D>
MK_DEV void lay_out_work(const AttnParams& P, TileSmem<D>& S) {
  const mk_prefix_attn_io& io = P.io;
  const int B = io.n_requests, lane = lane_id(), warp = threadIdx.x >> 5;
  constexpr int kTurn = kTileThreads * kReqs;
  int64_t cost[kReqs], mine = 0;
  int low = INT_MAX;
  auto read_costs = [&](int turn) {
    const int b0 = turn * kTurn + threadIdx.x * kReqs;
    int32_t cu[kReqs + 1], len[kReqs];
#pragma unroll
    for (int i = 0; i <= kReqs; ++i) cu[i] = b0 + i <= B ? io.cu_rows[b0 + i] : 0;
#pragma unroll
    for (int i = 0; i < kReqs; ++i) len[i] = b0 + i < B ? io.lens[b0 + i] : 0;
    int64_t sum = 0;
#pragma unroll
    for (int i = 0; i < kReqs; ++i) {
      cost[i] = 0;
      if (b0 + i < B) {
        const Req r = make_req(P, cu[i], cu[i + 1], len[i]);
        cost[i] = head_cost(ceil_div(r.n, P.tile_tok), r.kt1 - r.kt0) * io.n_kv_heads;
        if (r.n) low = min(low, r.base);
      }
      sum += cost[i];
    }
    return sum;
  };
  const int turns = ceil_div(B, kTurn);
  int64_t all = 0;
  for (int t = 0; t < turns; ++t) all += mine = read_costs(t);
  // the sum of all costs, and the lowest position of any row, which decides
  // where the prefix starts to be seen
#pragma unroll
  for (int o = 16; o; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
  low = __reduce_min_sync(0xffffffffu, low);
  if (lane == 0) S.sum[warp] = all, S.low[warp] = low;
  const int n_used = clampi(io.cu_rows[B], 0, io.n_rows);
  __syncthreads();
  all = 0;
#pragma unroll
  for (int w = 0; w < kTileThreads / 32; ++w) all += S.sum[w], low = min(low, S.low[w]);
  Plan p;
  const int64_t lo64 =
      io.window && low != INT_MAX ? static_cast<int64_t>(io.prefix_len) + low - io.window + 1 : 0;
  p.n_used = n_used;
  p.tiles = ceil_div(n_used, P.tile_tok);
  p.lo = clampi(lo64, 0, io.prefix_len);
  p.kt1 = ceil_div(io.prefix_len, kTileKeys);
  p.kt0 = p.lo >= io.prefix_len ? p.kt1 : p.lo / kTileKeys;
  p.prefix_cost = head_cost(p.tiles, p.kt1 - p.kt0) * io.n_kv_heads;
  p.total = p.prefix_cost + all;
  // at least one step each, so that every CTA inside an item has a piece of it
  p.share = max((p.total + P.ctas - 1) / P.ctas, static_cast<int64_t>(max(kPairCost, kAltCost)));
  const int64_t begin = static_cast<int64_t>(blockIdx.x) * p.share;
  if (threadIdx.x == 0) {
    S.plan = p;
    if (begin < p.prefix_cost) S.first = 0, S.first_at = p.prefix_cost;
    if (blockIdx.x == 0) *P.ws.plan = p;
  }
  // where each request starts: the request of this CTA's beginning, and from
  // the first CTA all of them
  if (blockIdx.x != 0 && (begin < p.prefix_cost || begin >= p.total)) return;
  int64_t at = p.prefix_cost;
  for (int t = 0; t < turns; ++t) {
    if (turns > 1) mine = read_costs(t);
    int64_t v = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    __syncthreads();
    if (lane == 31) S.sum[warp] = v;
    __syncthreads();
    int64_t here = at + v - mine;
#pragma unroll
    for (int w = 0; w < kTileThreads / 32; ++w) {
      if (w < warp) here += S.sum[w];
      at += S.sum[w];
    }
#pragma unroll
    for (int i = 0; i < kReqs; ++i) {
      const int b = t * kTurn + threadIdx.x * kReqs + i;
      if (b < B) {
        if (blockIdx.x == 0) P.ws.cost[b] = here;
        if (begin >= here && begin < here + cost[i]) S.first = b, S.first_at = here;
      }
      here += cost[i];
    }
  }
}

// ---- scheduler: the CTA's stretch of the line, item by item
template <int D>
MK_DEV void run_scheduler(const AttnParams& P, TileSmem<D>& S, const Ctx& c) {
  const mk_prefix_attn_io& io = P.io;
  const Plan plan = S.plan;
  const int Hk = io.n_kv_heads, lane = lane_id();
  const int64_t begin = static_cast<int64_t>(blockIdx.x) * plan.share;
  const int64_t end = min(plan.total, begin + plan.share);
  int n_out = 0;
  auto push = [&](const Piece& w) -> bool {
    const int k = n_out % kFifo;
    if (n_out >= kFifo && !wait_warp(c, &S.fifo_empty[k], ((n_out / kFifo) - 1) & 1)) return false;
    if (lane == 0) {
      S.fifo[k] = w;
      mbar_arrive(&S.fifo_full[k]);
    }
    ++n_out;
    return true;
  };
  // all items of one row set: `tiles` row tiles against key tiles [kt0, kt1) for
  // every head, the first at cost `at` of the line, in the order head by head
  // (the prefix, whose row tiles then share its keys in L2) or row tile by row
  // tile (a request's own keys)
  auto items = [&](Piece w, int64_t at, int tok, int tiles, int kt0, int kt1, bool heads_outer) -> bool {
    const int kt = kt1 - kt0;
    if (kt <= 0 || tiles <= 0) return true;
    const int pairs = tiles >> 1, n_items = pairs + (tiles & 1);
    const int64_t pair_cost = static_cast<int64_t>(kt) * kPairCost;
    const int64_t alt_cost = static_cast<int64_t>((kt + 1) >> 1) * kAltCost;
    // the first item that ends behind `begin`
    int h = 0, p = 0;
    int64_t s = at;
    if (begin > at) {
      const int64_t off = begin - at;
      if (heads_outer) {
        const int64_t hc = head_cost(tiles, kt);
        h = static_cast<int>(off / hc);
        p = static_cast<int>(min((off - h * hc) / pair_cost, static_cast<int64_t>(pairs)));
        s = at + h * hc + p * pair_cost;
      } else {
        p = static_cast<int>(min(off / (pair_cost * Hk), static_cast<int64_t>(pairs)));
        const int64_t hc = p < pairs ? pair_cost : alt_cost;
        h = static_cast<int>((off - p * pair_cost * Hk) / hc);
        s = at + p * pair_cost * Hk + h * hc;
      }
    }
    while (h < Hk && p < n_items && s < end) {
      const bool alt = p == pairs;
      const int step = alt ? kAltCost : kPairCost, steps = alt ? (kt + 1) >> 1 : kt;
      const int s0 = s >= begin ? 0 : (static_cast<int>(begin - s) + step - 1) / step;
      const int64_t room = (end - s + step - 1);
      const int s1 = room >= static_cast<int64_t>(steps) * step ? steps : static_cast<int>(room) / step;
      if (s0 < s1) {
        w.alt = alt;
        w.h = h;
        w.tok0 = tok + 2 * p * P.tile_tok;
        w.kt_a = kt0 + (alt ? 2 * s0 : s0);
        w.kt_b = alt ? min(kt1, kt0 + 2 * s1) : kt0 + s1;
        w.first = s0 == 0;
        if (!push(w)) return false;
      }
      s += alt ? alt_cost : pair_cost;
      if (heads_outer) {
        if (++p == n_items) p = 0, ++h;
      } else {
        if (++h == Hk) h = 0, ++p;
      }
    }
    return true;
  };
  Piece w;
  std::memset(&w, 0, sizeof(w));
  bool ok = true;
  if (begin < plan.prefix_cost) {
    w.kind = 0;
    w.tok_end = plan.n_used;
    w.klo = plan.lo;
    w.khi = io.prefix_len;
    ok = items(w, 0, 0, plan.tiles, plan.kt0, plan.kt1, true);
  }
  if (ok && end > plan.prefix_cost && begin < end) {
    w.kind = 1;
    int64_t at = S.first_at;
    for (int b0 = S.first; ok && at < end && b0 < io.n_requests; b0 += 32) {
      // 32 requests' lengths at a time
      Req mine{0, 0, 0, 0, 0, 0};
      if (b0 + lane < io.n_requests) mine = read_req(P, b0 + lane);
      for (int i = 0; ok && at < end && i < 32 && b0 + i < io.n_requests; ++i) {
        Req r;
        r.cu = __shfl_sync(0xffffffffu, mine.cu, i);
        r.n = __shfl_sync(0xffffffffu, mine.n, i);
        r.len = __shfl_sync(0xffffffffu, mine.len, i);
        r.base = max(0, r.len - r.n);
        r.kt0 = __shfl_sync(0xffffffffu, mine.kt0, i);
        r.kt1 = __shfl_sync(0xffffffffu, mine.kt1, i);
        const int tiles = ceil_div(r.n, P.tile_tok);
        w.b = b0 + i;
        w.cu = r.cu;
        w.base = r.base;
        w.tok_end = r.cu + r.n;
        w.klo = io.window ? clampi(static_cast<int64_t>(r.base) - io.window + 1, 0, r.len) : 0;
        w.khi = r.len;
        ok = items(w, at, r.cu, tiles, r.kt0, r.kt1, false);
        at += head_cost(tiles, r.kt1 - r.kt0) * Hk;
      }
    }
  }
  if (ok) {
    w.kind = -1;
    push(w);
  }
}

// ---- producer: Q tiles and the ring of K and V tiles
template <int D>
MK_DEV void run_tile_producer(const AttnParams& P, TileSmem<D>& S, const Ctx& c,
                              const CUtensorMap* tm_q, const CUtensorMap* tm_k,
                              const CUtensorMap* tm_v) {
  const mk_prefix_attn_io& io = P.io;
  constexpr int kHalves = D / 64;
  const int lane = lane_id();
  const int boxes = kTileKeys / P.box;  // per tile and half
  const int group_tiles = 32 / boxes;   // key tiles whose pages one lane each holds
  int seq = 0;       // loads into the ring
  int q_seq = 0;     // loads of row tiles
  int piece = 0;
  bool ok = true;
  auto next_piece = [&](Piece& w) -> bool {
    const int k = piece % kFifo;
    if (!wait_warp(c, &S.fifo_full[k], (piece / kFifo) & 1)) return false;
    w = S.fifo[k];
    __syncwarp();
    if (lane == 0) mbar_arrive(&S.fifo_empty[k]);
    ++piece;
    return true;
  };
  // First slot of box number 32 g + lane of a piece; -1: no row sees its keys.
  // A page outside the pool: behind the end, where the copy fills in zeros.
  auto fetch = [&](const Piece& w, int g) -> int {
    const int box = 32 * g + lane, key = w.kt_a * kTileKeys + box * P.box;
    if (w.kind < 0 || box >= (w.kt_b - w.kt_a) * boxes || key >= w.khi || key + P.box <= w.klo)
      return -1;
    const int page = key >> P.page_shift;
    const int id = w.kind == 0 ? io.prefix_pages[page] : io.block_table[w.b * io.table_stride + page];
    return id >= 0 && id < io.n_pages ? (id << P.page_shift) + (key & (io.page_size - 1))
                                      : max(1, io.n_pages << P.page_shift);
  };
  Piece w;
  ok = next_piece(w);
  int pages_next = ok ? fetch(w, 0) : -1;
  while (ok && w.kind >= 0) {
    // the page numbers are read one group ahead, those of the next piece too:
    // each read is a round trip to L2 or HBM
    const Piece me = w;
    const int t_all = me.kt_b - me.kt_a;
    int pages = pages_next, pages_ahead = -1, group = 0;
    if (!(ok = next_piece(w))) break;
    pages_next = fetch(w, 0);
    if (t_all > group_tiles) pages_ahead = fetch(me, 1);
    int pages_old = -1;  // the group before: V follows K by up to two tiles
    auto load = [&](const CUtensorMap* map, int x) -> bool {
      const int st = seq % kStages, g = x / group_tiles;
      if (g > group) {
        pages_old = pages;
        pages = pages_ahead;
        group = g;
        if (t_all > (g + 1) * group_tiles) pages_ahead = fetch(me, g + 1);
      }
      // lane = half * boxes + box
      const int box = lane % boxes, half = lane / boxes;
      const int slot = __shfl_sync(0xffffffffu, g == group ? pages : pages_old,
                                   (x % group_tiles) * boxes + box);
      const bool mine = lane < boxes * kHalves && slot >= 0;
      const uint32_t n = __popc(__ballot_sync(0xffffffffu, mine));
      if (seq >= kStages && !wait_warp(c, &S.kv_empty[st], ((seq / kStages) - 1) & 1)) return false;
      if (lane == 0) mbar_arrive_expect_tx(&S.kv_full[st], n * P.box * 128);
      __syncwarp();
      if (mine)
        tma_load_3d(S.kv[st] + half * 128 * 128 + box * P.box * 128, map, &S.kv_full[st],
                    half * 64, me.h, slot);
      ++seq;
      return true;
    };
    ok = load(tm_k, 0);
    if (ok && me.alt && t_all > 1) ok = load(tm_k, 1);
    for (int t = 0; ok && t < (me.alt ? 1 : 2); ++t, ++q_seq) {
      const int q = q_seq & 1;
      if (q_seq >= 2 && !(ok = wait_warp(c, &S.q_empty[q], ((q_seq >> 1) - 1) & 1))) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(&S.q_full[q], kHalves * P.group * P.tile_tok * 128);
        for (int f = 0; f < kHalves; ++f)
          tma_load_3d(S.q[q] + f * 128 * 128, tm_q, &S.q_full[q], f * 64, me.h * P.group,
                      me.tok0 + t * P.tile_tok);
      }
      __syncwarp();
    }
    const int lead = me.alt ? 2 : 1;
    for (int x = 0; ok && x < t_all; ++x) {
      ok = load(tm_v, x);
      if (ok && x + lead < t_all) ok = load(tm_k, x + lead);
    }
  }
  if (!ok) {
    // give up: no copy may land after the CTA has left
    uint32_t none = 0;
    const Ctx drain{&none, c.status};
    for (int s = max(0, seq - kStages); s < seq; ++s)
      wait_warp(drain, &S.kv_full[s % kStages], (s / kStages) & 1);
    for (int s = max(0, q_seq - 2); s < q_seq; ++s)
      wait_warp(drain, &S.q_full[s & 1], (s >> 1) & 1);
  }
}

// ---- MMA issuer: the whole warp walks the pieces, one elected lane issues, so
// that descriptors and addresses are warp-uniform; false once a wait has run out
template <class T, int D>
MK_DEV bool issue_mmas(const AttnParams& P, TileSmem<D>& S, const Ctx& c) {
  constexpr uint32_t kIdS = idesc_of<T>(kTileKeys, false), kIdO = idesc_of<T>(D, true);
  const uint32_t tm = S.tmem;
  int seq = 0, q_seq = 0, piece = 0;
  uint32_t p_par[2] = {0, 0};
  auto commit = [&](uint64_t* bar) {
    if (elect_one()) mma_commit(bar);
    __syncwarp();
  };
  auto wait_stage = [&](int s) { return wait_warp(c, &S.kv_full[s % kStages], (s / kStages) & 1); };
  auto qk = [&](int slot, int q_tile, int s) {
    const uint64_t qd = sdesc_kmajor_sw128(smem_u32(S.q[q_tile]));
    const uint64_t kd = sdesc_kmajor_sw128(smem_u32(S.kv[s % kStages]));
    if (elect_one()) {
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const uint64_t off = ((k >> 2) * 128 * 128 + (k & 3) * 32) >> 4;
        mma_bf16(tm + slot * 128, qd + off, kd + off, kIdS, k);
      }
      mma_commit(&S.s_full[slot]);
    }
    __syncwarp();
  };
  auto pv = [&](int slot, int s, bool first) {
    const uint64_t vd = sdesc_mnmajor_sw128(smem_u32(S.kv[s % kStages]), 128 * 128);
    if (elect_one()) {
#pragma unroll
      for (int k = 0; k < kTileKeys / 16; ++k)
        mma_ts(tm + 256 + slot * 128, tm + slot * 128 + 8 * k, vd + k * (16 * 128 >> 4), kIdO,
               !(first && k == 0));
    }
    __syncwarp();
  };
  while (true) {
    const int k = piece % kFifo;
    if (!wait_warp(c, &S.fifo_full[k], (piece / kFifo) & 1)) return false;
    const Piece w = S.fifo[k];
    __syncwarp();
    if (elect_one()) mbar_arrive(&S.fifo_empty[k]);
    if (w.kind < 0) return true;
    const int n[2] = {slot_tiles(w, 0), slot_tiles(w, 1)};
    // row tile of each slot
    const int q_tiles = w.alt ? 1 : 2, q0 = q_seq & 1, q1 = w.alt ? q0 : q0 ^ 1;
    for (int t = 0; t < q_tiles; ++t)
      if (!wait_warp(c, &S.q_full[(q_seq + t) & 1], ((q_seq + t) >> 1) & 1)) return false;
    q_seq += q_tiles;
    auto free_q = [&] {
      commit(&S.q_empty[q0]);
      if (q1 != q0) commit(&S.q_empty[q1]);
    };
    // scores of the first tiles
    if (!wait_stage(seq)) return false;
    tc_fence_after();
    qk(0, q0, seq);
    if (!w.alt) qk(1, q1, seq);
    commit(&S.kv_empty[seq % kStages]);
    ++seq;
    if (w.alt && n[1] > 0) {
      if (!wait_stage(seq)) return false;
      tc_fence_after();
      qk(1, q1, seq);
      commit(&S.kv_empty[seq % kStages]);
      ++seq;
    }
    if (n[0] == 1) free_q();
    for (int j = 0; j < n[0]; ++j) {
      int sv = 0, sk = 0;
      for (int slot = 0; slot < 2; ++slot) {
        if (j >= n[slot]) continue;
        const bool more = j + 1 < n[slot];
        const bool fresh = w.alt || slot == 0;   // this slot is the first user of its tiles
        const bool last_use = w.alt || slot == 1;
        if (fresh) {
          sv = seq++;
          if (more) sk = seq++;
          if (!wait_stage(sv)) return false;
        }
        if (!wait_warp(c, &S.p_full[slot], p_par[slot])) return false;
        p_par[slot] ^= 1;
        tc_fence_after();
        pv(slot, sv, j == 0);
        if (last_use) commit(&S.kv_empty[sv % kStages]);
        if (more) {
          if (fresh && !wait_stage(sk)) return false;
          tc_fence_after();
          qk(slot, slot ? q1 : q0, sk);
          if (last_use) commit(&S.kv_empty[sk % kStages]);
        } else {
          commit(&S.o_done[slot]);
        }
      }
      // the last scores are on their way: Q may be replaced once they are done
      if (n[0] > 1 && j == n[0] - 2) free_q();
    }
    ++piece;
  }
}

template <class T, int D>
MK_DEV void run_mma(const AttnParams& P, TileSmem<D>& S, const Ctx& c) {
  if (issue_mmas<T, D>(P, S, c)) return;
  // give up: no MMA may run on after the CTA has left
  uint32_t none = 0;
  if (elect_one()) mma_commit(&S.drained);
  __syncwarp();
  wait_warp(Ctx{&none, c.status}, &S.drained, 0);
}

// ---- softmax (one warpgroup per slot, one thread per row)
template <class T, int D>
MK_DEV void run_softmax(const AttnParams& P, TileSmem<D>& S, const Ctx& c, int slot) {
  const mk_prefix_attn_io& io = P.io;
  const int warp = (threadIdx.x >> 5) & 3, lane = lane_id(), row = warp * 32 + lane;
  const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
  const uint32_t ts = S.tmem + lanes + slot * 128, to = S.tmem + lanes + 256 + slot * 128;
  const int G = P.group, tok_in_tile = row / G, g = row - tok_in_tile * G;
  const float sl2 = P.scale_log2;
  int seq = 0, piece = 0;
  uint32_t s_par = 0, o_par = 0;
  while (true) {
    const int k = piece % kFifo;
    if (!wait_warp(c, &S.fifo_full[k], (piece / kFifo) & 1)) return;
    const Piece w = S.fifo[k];
    __syncwarp();
    if (lane == 0) mbar_arrive(&S.fifo_empty[k]);
    if (w.kind < 0) return;
    ++piece;
    const int n = slot_tiles(w, slot);
    const int seq0 = seq;
    seq += 2 * (w.kt_b - w.kt_a);
    // this thread's row: its token, and the keys [klo, khi) it sees; of a token
    // tree, the bits of `tree` instead from key `tree_at` on
    const int tok = w.tok0 + (w.alt ? 0 : slot * P.tile_tok) + tok_in_tile;
    const bool valid = tok_in_tile < P.tile_tok && tok < w.tok_end;
    int klo = w.klo, khi = w.khi, tree_at = INT_MAX;
    uint64_t tree = 0;
    if (valid) {
      int base = w.base, i = tok - w.cu;
      if (w.kind == 0 && io.window) {  // which request is it?
        int lo = 0, hi = io.n_requests;
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (io.cu_rows[mid] <= tok) lo = mid; else hi = mid;
        }
        const Req r = read_req(P, lo);
        base = r.base;
        i = tok - r.cu;
      }
      if (io.tree_mask) tree = io.tree_mask[tok];
      if (io.window) {
        const int depth = io.tree_mask ? max(1, __popcll(tree)) - 1 : i;
        const int64_t low = static_cast<int64_t>(base) + depth - io.window + 1 +
                            (w.kind == 0 ? io.prefix_len : 0);
        klo = max(klo, clampi(low, 0, w.khi));
      }
      if (w.kind == 1) {
        if (io.tree_mask) tree_at = base;
        else khi = min(khi, clampi(static_cast<int64_t>(base) + i + 1, 0, INT_MAX));
      }
    }
    const bool warp_valid = __any_sync(0xffffffffu, valid);

    float m = -INFINITY, l = 0.f;
    for (int j = 0; j < n; ++j) {
      const int kt = w.kt_a + (w.alt ? 2 * j + slot : j), k0 = kt * kTileKeys;
      if (!wait_warp(c, &S.s_full[slot], s_par)) return;
      s_par ^= 1;
      tc_fence_after();
      if (warp_valid) {
        float s[kTileKeys];
#pragma unroll
        for (int q = 0; q < 4; ++q) tmem_ld32(ts + 32 * q, s + 32 * q);
        tmem_ld_wait();
        const bool edge = klo > k0 || khi < k0 + kTileKeys || tree_at < k0 + kTileKeys;
        if (__any_sync(0xffffffffu, edge)) {
          const int lo = klo - k0, hi = khi - k0, tb = tree_at - k0;
#pragma unroll
          for (int q = 0; q < kTileKeys / 32; ++q) {
            // bit i: key k0 + 32 q + i is seen
            uint32_t see = below(hi - 32 * q) & ~below(lo - 32 * q);
            const int off = tb - 32 * q;
            if (off < 32)
              see &= below(off) | (off >= 0 ? static_cast<uint32_t>(tree) << off
                                   : off > -64 ? static_cast<uint32_t>(tree >> -off) : 0u);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!(see & (1u << i))) s[32 * q + i] = -INFINITY;
          }
        }
        float t8[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) t8[x] = s[x];
#pragma unroll
        for (int x = 8; x < kTileKeys; ++x) t8[x & 7] = fmaxf(t8[x & 7], s[x]);
        const float top = sl2 * fmaxf(fmaxf(fmaxf(t8[0], t8[1]), fmaxf(t8[2], t8[3])),
                                      fmaxf(fmaxf(t8[4], t8[5]), fmaxf(t8[6], t8[7])));
        // rescale only when the maximum has grown by 2^8: until then P is at most
        // 2^8, which its types and the 32-bit sums hold without loss
        const bool grow = valid && top > m + kGrow;
        if (j == 0) {
          m = top;
        } else if (__any_sync(0xffffffffu, grow)) {
          const float f = grow ? exp2_approx(m - top) : 1.f;
          if (grow) m = top;
          l *= f;
#pragma unroll 1
          for (int q = 0; q < D / 32; ++q) {
            float o[32];
            tmem_ld32(to + 32 * q, o);
            tmem_ld_wait();
#pragma unroll
            for (int x = 0; x < 32; ++x) o[x] *= f;
            tmem_st32(to + 32 * q, reinterpret_cast<uint32_t*>(o));
          }
        }
        const float ms = m == -INFINITY ? 0.f : m;
        uint32_t p[kTileKeys / 2];
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int x = 0; x < kTileKeys; x += 2) {
          const float a = exp2_approx(fmaf(s[x], sl2, -ms));
          const float b = exp2_approx(fmaf(s[x + 1], sl2, -ms));
          sum[(x >> 1) & 3] += a + b;
          p[x >> 1] = Types<T>::pack(a, b);
        }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        tmem_st32(ts, p);
        tmem_st32(ts + 32, p + 32);
        tmem_st_wait();
      }
      if (k0 < w.klo || k0 + kTileKeys > w.khi) {
        // keys that no row sees may hold anything: their V rows become zeros, so
        // that a weight of zero leaves no NaN behind
        const int t = w.kt_b - w.kt_a, x = kt - w.kt_a;  // its place among the loads
        const int v_seq = seq0 + (w.alt ? min(2, t) + x + min(x, max(0, t - 2)) : 1 + 2 * x);
        if (!wait_warp(c, &S.kv_full[v_seq % kStages], (v_seq / kStages) & 1)) return;
        if (k0 + row < w.klo || k0 + row >= w.khi) {
#pragma unroll
          for (int f = 0; f < D / 64; ++f)
#pragma unroll
            for (int x = 0; x < 8; ++x)
              reinterpret_cast<uint4*>(S.kv[v_seq % kStages] + f * 128 * 128 + row * 128)[x] =
                  make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.p_full[slot]);
    }

    // the piece's result
    if (n > 0) {
      if (!wait_warp(c, &S.o_done[slot], o_par)) return;
      o_par ^= 1;
      tc_fence_after();
    }
    int64_t at;
    const int64_t by_row = static_cast<int64_t>(tok) * io.n_q_heads + w.h * G + g;
    if (!w.first) at = P.ws.carry + (static_cast<int64_t>(blockIdx.x) * 2 + slot) * 128 + row;
    else if (w.kind == 0) at = w.alt && slot ? P.ws.pre1 + w.h * 128 + row : P.ws.pre0 + by_row;
    else at = (w.alt && slot ? P.ws.own1 : P.ws.own0) + by_row;
    if (valid) P.ws.ml[at] = make_float2(m, l);
    if (n > 0 && warp_valid) {
#pragma unroll 1
      for (int q = 0; q < D / 32; ++q) {
        float o[32];
        tmem_ld32(to + 32 * q, o);
        tmem_ld_wait();
        if (valid) {
          // whole sectors: a thread's row is its own
          float* dst = P.ws.o + at * D + 32 * q;
#pragma unroll
          for (int x = 0; x < 32; x += 8) st_global_8(dst + x, o + x);
        }
      }
      tc_fence_before();
    }
  }
}

template <class T, int D>
__global__ void __launch_bounds__(kTileThreads, 1)
    k_attn_tiles(const __grid_constant__ AttnParams P, const __grid_constant__ CUtensorMap tm_q,
                 const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v) {
  extern __shared__ uint8_t smem_raw[];
  TileSmem<D>& S = *reinterpret_cast<TileSmem<D>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                   ~static_cast<uintptr_t>(1023));
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&S.kv_full[i], 1);
      mbar_init(&S.kv_empty[i], 1);
    }
    mbar_init(&S.drained, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&S.q_full[i], 1);
      mbar_init(&S.q_empty[i], 1);
      mbar_init(&S.s_full[i], 1);
      mbar_init(&S.p_full[i], 4);
      mbar_init(&S.o_done[i], 1);
    }
    for (int i = 0; i < kFifo; ++i) {
      mbar_init(&S.fifo_full[i], 1);
      mbar_init(&S.fifo_empty[i], 10);
    }
    S.abort = 0;
    fence_mbar_init();
    prefetch_tensormap(&tm_q);
    prefetch_tensormap(&tm_k);
    prefetch_tensormap(&tm_v);
  }
  if (warp == 9) {
    tmem_alloc(&S.tmem, 512);
    tmem_relinquish();
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) *P.ws.status = 0;
  lay_out_work<D>(P, S);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_launch_dependents();
  const Ctx c{&S.abort, P.ws.status};
  // 2 x 128 x 208 + 128 x 72 = 62,464 of the 64,512 registers of the launch; all
  // are back at 168 before the common tail
  if (warp < 8) {
    reg_alloc<208>();
    run_softmax<T, D>(P, S, c, warp >> 2);
    __syncwarp();
    reg_dealloc<168>();
  } else {
    reg_dealloc<72>();
    if (warp == 8) run_tile_producer<D>(P, S, c, &tm_q, &tm_k, &tm_v);
    else if (warp == 9) run_mma<T, D>(P, S, c);
    else if (warp == 10) run_scheduler<D>(P, S, c);
    __syncwarp();
    reg_alloc<168>();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc(S.tmem, 512);
}

// ------------------------------------------------------------------ merge

// The stretches of one item that hold a row: by row (its first piece) and by
// the CTAs c0 + 1 .. c1, in one slot or both.
struct Held {
  int64_t main0, main1, carry;  // partial rows; carry of CTA c0 + 1's slot
  int32_t ctas, slots;
  MK_DEV int count() const { return ctas * slots; }
  MK_DEV int64_t at(int e) const {
    const int c = slots == 2 ? e >> 1 : e, s = slots == 2 ? e & 1 : 0;
    return c == 0 ? (s ? main1 : main0) : carry + static_cast<int64_t>(c - 1) * 256 + s * 128;
  }
};
MK_DEV Held held(const AttnParams& P, int64_t share, int64_t start, int tile, int tiles, int kt,
                 int64_t main0, int64_t main1, int row) {
  Held x;
  const bool alt = tile == tiles - 1 && (tiles & 1);
  const int steps = alt ? (kt + 1) >> 1 : kt;
  const int64_t c0 = start / share;
  const int64_t c1 = (start + static_cast<int64_t>(steps - 1) * (alt ? kAltCost : kPairCost)) / share;
  x.ctas = steps > 0 ? static_cast<int>(c1 - c0) + 1 : 0;
  x.slots = alt ? 2 : 1;
  x.main0 = main0;
  x.main1 = main1;
  x.carry = P.ws.carry + (c0 + 1) * 256 + (alt ? 0 : (tile & 1) * 128) + row;
  return x;
}

template <class T, int D>
__global__ void __launch_bounds__(256) k_attn_merge(const __grid_constant__ AttnParams P) {
  const mk_prefix_attn_io& io = P.io;
  constexpr int V = D / 32;
  pdl_wait();
  const Plan plan = *P.ws.plan;
  const int lane = lane_id(), Hq = io.n_q_heads, G = P.group;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int64_t tok64 = item / Hq;
  if (tok64 >= plan.n_used) return;
  const int tok = static_cast<int>(tok64), hq = static_cast<int>(item - tok64 * Hq);
  const int h = hq / G, g = hq - h * G;
  // its request
  int lo = 0, hi = io.n_requests;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (io.cu_rows[mid] <= tok) lo = mid; else hi = mid;
  }
  const Req r = read_req(P, lo);
  const int tt = P.tile_tok;
  Held x[2];
  {
    const int tile = tok / tt, kt = plan.kt1 - plan.kt0;
    const int row = (tok - tile * tt) * G + g;
    const int64_t start = h * head_cost(plan.tiles, kt) +
                          static_cast<int64_t>(tile >> 1) * kt * kPairCost;
    x[0] = held(P, plan.share, start, tile, plan.tiles, kt, P.ws.pre0 + item,
                P.ws.pre1 + h * 128 + row, row);
  }
  {
    const int i = tok - r.cu, tiles = ceil_div(r.n, tt), tile = i / tt, kt = r.kt1 - r.kt0;
    const int row = (i - tile * tt) * G + g;
    const int64_t pair_cost = static_cast<int64_t>(kt) * kPairCost;
    const bool alt = tile == tiles - 1 && (tiles & 1);
    const int64_t start =
        P.ws.cost[lo] + (tile >> 1) * pair_cost * io.n_kv_heads +
        h * (alt ? static_cast<int64_t>((kt + 1) >> 1) * kAltCost : pair_cost);
    x[1] = held(P, plan.share, start, tile, tiles, kt, P.ws.own0 + item, P.ws.own1 + item, row);
  }
  const int n0 = x[0].count(), n = n0 + x[1].count();
  float M = -INFINITY, L = 0.f, acc[V] = {};
  for (int a = 0; a < n; a += 32) {
    const int e = a + lane;
    int64_t at = 0;
    float2 ml = make_float2(-INFINITY, 0.f);
    if (e < n) {
      at = e < n0 ? x[0].at(e) : x[1].at(e - n0);
      ml = P.ws.ml[at];
    }
    float top = ml.x;
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    top = fmaxf(top, M);
    if (top == -INFINITY) continue;
    const float old = exp2f(M - top);
    float wgt = ml.x == -INFINITY ? 0.f : exp2f(ml.x - top);
    float sum = wgt * ml.y;
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    L = L * old + sum;
    M = top;
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] *= old;
    const int cnt = min(32, n - a);
#pragma unroll 4
    for (int k = 0; k < cnt; ++k) {
      const float f = __shfl_sync(0xffffffffu, wgt, k);
      const int64_t p = __shfl_sync(0xffffffffu, at, k);
      if (f == 0.f) continue;
      const float* src = P.ws.o + p * D + lane * V;
      if (V == 4) {
        const float4 y = *reinterpret_cast<const float4*>(src);
        acc[0] += f * y.x, acc[1] += f * y.y, acc[V - 2] += f * y.z, acc[V - 1] += f * y.w;
      } else {
        const float2 y = *reinterpret_cast<const float2*>(src);
        acc[0] += f * y.x, acc[1] += f * y.y;
      }
    }
  }
  const float inv = L != 0.f ? 1.f / L : 0.f;  // no key, or NaN as it comes
  uint32_t out[V / 2];
#pragma unroll
  for (int v = 0; v < V; v += 2) out[v >> 1] = Types<T>::pack(acc[v] * inv, acc[v + 1] * inv);
  T* dst = static_cast<T*>(io.out) + tok * io.out_stride + hq * D + lane * V;
  if (V == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(out[0], out[V / 2 - 1]);
  else *reinterpret_cast<uint32_t*>(dst) = out[0];
  if (lane == 0 && io.lse)
    io.lse[item] = L != 0.f ? (M + log2f(L)) * 0.6931471805599453f : -INFINITY;
}

// ------------------------------------------------------------------- host

mk_status check_shapes(const mk_prefix_attn_io* io) {
  if (!io) return MK_ERR_INVALID_ARG;
  if (io->n_requests < 1 || io->n_requests > 65536 || io->n_rows < 0) return MK_ERR_INVALID_ARG;
  if (io->n_kv_heads < 1 || io->n_q_heads < 1 || io->n_q_heads % io->n_kv_heads)
    return MK_ERR_INVALID_ARG;
  if (io->n_q_heads / io->n_kv_heads > 64 || io->n_q_heads > 4096) return MK_ERR_UNSUPPORTED;
  if (io->head_dim != 64 && io->head_dim != 128) return MK_ERR_UNSUPPORTED;
  if (io->dtype != MK_BF16 && io->dtype != MK_FP16) return MK_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(io->n_rows) * io->n_q_heads > INT32_MAX - 4096) return MK_ERR_UNSUPPORTED;
  return MK_OK;
}

int64_t align256(int64_t v) { return (v + 255) & ~static_cast<int64_t>(255); }

// Lays the workspace out over `base`; returns its size.
int64_t lay_out(const mk_prefix_attn_io* io, int ctas, uint8_t* base, Space* s) {
  const int64_t heads = static_cast<int64_t>(io->n_rows) * io->n_q_heads;
  s->pre0 = 0;
  s->own0 = heads;
  s->own1 = 2 * heads;
  s->pre1 = 3 * heads;
  s->carry = s->pre1 + io->n_kv_heads * 128ll;
  const int64_t rows = s->carry + ctas * 256ll;
  int64_t at = 0;
  s->status = reinterpret_cast<uint32_t*>(base);
  s->plan = reinterpret_cast<Plan*>(base + 64);
  at = 256;
  s->cost = reinterpret_cast<int64_t*>(base + at);
  at = align256(at + (io->n_requests + 1) * 8ll);
  s->ml = reinterpret_cast<float2*>(base + at);
  at = align256(at + rows * 8);
  s->o = reinterpret_cast<float*>(base + at);
  return align256(at + rows * io->head_dim * 4);
}

// 3-D map over [n2][n1][n0] 16-bit values (n0 contiguous), box of 64 values x
// b1 x b2, 128-byte swizzle; out-of-range coordinates read as zeros.
mk_status encode_tmap_3d(CUtensorMap* map, int dtype, const void* base, uint64_t n0, uint64_t n1,
                         uint64_t n2, uint64_t stride1, uint64_t stride2, uint32_t b1,
                         uint32_t b2) {
  PFN_encodeTiled fn = get_encode_fn();
  if (!fn) return MK_ERR_CUDA;
  cuuint64_t dims[3] = {n0, n1, n2};
  cuuint64_t strides[2] = {stride1, stride2};
  cuuint32_t box[3] = {64, b1, b2};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = fn(map, dtype == MK_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                  3, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? MK_OK : MK_ERR_INVALID_ARG;
}

template <class T, int D>
mk_status launch_attn(const AttnParams& A, const CUtensorMap& q, const CUtensorMap& k,
                      const CUtensorMap& v, cudaStream_t s) {
  constexpr int smem = sizeof(TileSmem<D>) + 1024;
  MK_CUDA_TRY(cudaFuncSetAttribute(k_attn_tiles<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
  k_attn_tiles<T, D><<<A.ctas, kTileThreads, smem, s>>>(A, q, k, v);
  MK_CUDA_TRY(cudaGetLastError());
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(static_cast<unsigned>((static_cast<int64_t>(A.io.n_rows) * A.io.n_q_heads + 7) / 8));
  lc.blockDim = dim3(256);
  lc.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = attr;
  lc.numAttrs = 1;
  MK_CUDA_TRY(cudaLaunchKernelEx(&lc, k_attn_merge<T, D>, A));
  return MK_OK;
}

}  // namespace

}  // namespace mk

using namespace mk;

extern "C" {

mk_status mk_prefix_attn_workspace(const mk_prefix_attn_io* io, int64_t* bytes) {
  if (!bytes) return MK_ERR_INVALID_ARG;
  *bytes = 0;
  mk_status st = check_shapes(io);
  if (st != MK_OK) return st;
  int dev = -1, sms = 0;
  MK_CUDA_TRY(cudaGetDevice(&dev));
  MK_CUDA_TRY(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
  Space s;
  *bytes = lay_out(io, sms, nullptr, &s);
  return MK_OK;
}

mk_status mk_prefix_attn(const mk_prefix_attn_io* io, void* workspace, int64_t workspace_bytes,
                         void* stream) {
  mk_status st = check_shapes(io);
  if (st != MK_OK) return st;
  const int64_t P = io->page_size, cap = static_cast<int64_t>(io->max_pages) * P;
  if (P < 16 || P > 65536 || (P & (P - 1))) return MK_ERR_UNSUPPORTED;
  if (io->n_pages < 0 || io->n_pages * P > INT32_MAX || io->prefix_len < 0 || io->max_pages < 0 ||
      io->table_stride < io->max_pages || io->window < 0)
    return MK_ERR_INVALID_ARG;
  if (cap + io->prefix_len > INT32_MAX - 256) return MK_ERR_INVALID_ARG;
  if (!(io->scale >= 0.f && io->scale <= FLT_MAX)) return MK_ERR_INVALID_ARG;
  if (io->tree_mask && io->window > 0 && io->window < 64) return MK_ERR_UNSUPPORTED;
  if (!io->lens || !io->cu_rows || !workspace) return MK_ERR_INVALID_ARG;
  if (io->max_pages && !io->block_table) return MK_ERR_INVALID_ARG;
  if (io->prefix_len && !io->prefix_pages) return MK_ERR_INVALID_ARG;
  if (io->n_rows && (!io->q || !io->out || io->q == io->out)) return MK_ERR_INVALID_ARG;
  if (io->n_pages && (!io->k_cache || !io->v_cache)) return MK_ERR_INVALID_ARG;
  const int64_t width = static_cast<int64_t>(io->n_q_heads) * io->head_dim;
  if (io->q_stride % 8 || io->out_stride % 8 || io->q_stride < width || io->out_stride < width)
    return MK_ERR_INVALID_ARG;
  if (misaligned(io->q, 16) || misaligned(io->out, 16) || misaligned(io->k_cache, 16) ||
      misaligned(io->v_cache, 16) || misaligned(workspace, 256) || misaligned(io->lens, 4) ||
      misaligned(io->cu_rows, 4) || misaligned(io->block_table, 4) ||
      misaligned(io->prefix_pages, 4) || misaligned(io->tree_mask, 8) || misaligned(io->lse, 4))
    return MK_ERR_INVALID_ARG;
  if (io->n_rows == 0) return MK_OK;
  AttnParams A;
  A.io = *io;
  st = check_device(workspace, nullptr, &A.ctas);
  if (st != MK_OK) return st;
  if (workspace_bytes < lay_out(io, A.ctas, static_cast<uint8_t*>(workspace), &A.ws))
    return MK_ERR_INVALID_ARG;
  const float scale = io->scale != 0.f ? io->scale : 1.f / std::sqrt(static_cast<float>(io->head_dim));
  A.scale_log2 = scale * 1.4426950408889634f;
  A.group = io->n_q_heads / io->n_kv_heads;
  A.tile_tok = 128 / A.group;
  A.box = static_cast<int>(std::min<int64_t>(P, kTileKeys));
  A.page_shift = __builtin_ctz(static_cast<uint32_t>(P));
  const uint64_t d = io->head_dim, Hq = io->n_q_heads, Hk = io->n_kv_heads;
  CUtensorMap q, k, v;
  st = encode_tmap_3d(&q, io->dtype, io->q, d, Hq, io->n_rows, d * 2, io->q_stride * 2, A.group, A.tile_tok);
  if (st != MK_OK) return st;
  // a pool without pages is never read
  const uint64_t slots = std::max<int64_t>(1, io->n_pages * P);
  const void* kp = io->n_pages ? io->k_cache : io->q;
  const void* vp = io->n_pages ? io->v_cache : io->q;
  st = encode_tmap_3d(&k, io->dtype, kp, d, Hk, slots, d * 2, Hk * d * 2, 1, A.box);
  if (st != MK_OK) return st;
  st = encode_tmap_3d(&v, io->dtype, vp, d, Hk, slots, d * 2, Hk * d * 2, 1, A.box);
  if (st != MK_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (io->dtype == MK_BF16)
    return io->head_dim == 128 ? launch_attn<__nv_bfloat16, 128>(A, q, k, v, s)
                               : launch_attn<__nv_bfloat16, 64>(A, q, k, v, s);
  return io->head_dim == 128 ? launch_attn<__half, 128>(A, q, k, v, s)
                             : launch_attn<__half, 64>(A, q, k, v, s);
}

mk_status mk_prefix_attn_status(const void* workspace) {
  if (!workspace) return MK_ERR_INVALID_ARG;
  uint32_t s = 0;
  MK_CUDA_TRY(cudaMemcpy(&s, workspace, sizeof(s), cudaMemcpyDeviceToHost));
  return s == 0 ? MK_OK : MK_ERR_TIMEOUT;
}

}  // extern "C"
