// prefix_attn.cu -- attention of a batch whose requests share a prefix
// (mk_prefix_attn), on the 5th-generation tensor cores.
//
// For one KV head, the rows (token, q head of the group) of ALL requests form
// one matrix Q against the prefix, and each request's rows one against its own
// keys.  Both are the same computation on a row tile (up to 128 rows) and a
// range of 128-key tiles, with running maximum m and sum l (log2 units):
//   S = Q K^T,  m' >= m near the maximum so far,  P = 2^(S - m'),
//   l' = l 2^(m - m') + rowsum P,  O' = O 2^(m - m') + P V.
// Each stretch of key tiles leaves (O, m, l); the second kernel joins a row's
// stretches: out = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i.
//
// Work comes in two kinds:
//   pairs  two row tiles on the same key tiles: bound by the tensor cores; a
//          CTA's two slots take a row tile each;
//   solos  one tile of up to 64 rows (what is left of a row set behind its
//          pairs, most requests' own rows): bound by the K and V bytes; each slot
//          takes one.
// All pairs lie on one line and all solos on another, measured in time; every CTA
// works them out from the lengths (only the GPU knows them).  With A and B their
// lengths, each of the C CTAs (one per SM) gets the time T = (A + B / 2) / C: the
// first A / T of them take the pairs, the others' slots the solos, whatever
// heads, requests and keys a stretch crosses.  So the tensor cores and HBM are
// both busy from beginning to end.
// Two launches, the second one chained with programmatic dependent launch:
// k_attn_tiles does all that, k_attn_merge joins the partial results of each
// row.
#include <algorithm>
#include <atomic>
#include <cfloat>
#include <climits>
#include <cmath>
#include <cstring>
#include <cuda_fp16.h>

#include "../../include/mk_selftest.h"
#include "batch.h"
#include "ptx.cuh"

namespace mk {

namespace {

constexpr int kPair = 0, kSolo = 1;  // the two kinds of work
// Time of a key tile, and what an item (a row set's tile or pair of tiles and a
// KV head) takes on top of its key tiles: filling the pipeline and writing the
// result.  In units of about 0.2 us (of 0.4, 0.8 or 1.6 us in calls so large that
// the lines would not fit into 32 bits).  Of 20 settings around these none was
// better over twelve mixes of prefix and own keys; dearer solo tiles cost 1 to 4 %,
// cheaper solo items 1 to 3 %.
constexpr int kTileCost[2] = {8, 10}, kItemCost[2] = {24, 12};

constexpr int kTileKeys = 128;
constexpr uint32_t kTimeout = 1, kFalling = 2;  // values of the status word
constexpr int kFifo = 4;            // pieces handed out ahead
constexpr int kTileThreads = 384;
constexpr float kMost = 16384.f;    // a row's sum of P over a tile, in units of 2^m, at most
// Limits of the waits: for a hand-off, and so many times that for what may take as
// long as a CTA's whole work (a wait that runs out ends that work, too).
constexpr uint64_t kWaitNs = 2000ull * 1000 * 1000;
constexpr int kLongWait = 100;

// Hand-offs that a self-test withholds, so that waits run out: a tile's scores, a
// tile's weights, a slot's row tile after use, the buffers after a slot's pairs.
enum Withhold { kNothing = 0, kScores = 1, kWeights = 2, kRowTile = 3, kBuffers = 4 };

// How the lines are laid out (every CTA of k_attn_tiles works it out for itself).
struct Plan {
  int32_t total[2];        // of each line
  int32_t share;           // T
  int32_t prefix_cost[2];  // the prefix items come first
  int32_t n_used;          // rows in use
  int32_t kt0, kt1;        // key tiles of the prefix that some row sees
  int32_t lo;              // first prefix key that some row sees
  // The solos start in CTA solo_cta, whose slots have solo_len of them each; of
  // the CTAs behind it each slot has `share`.
  int32_t solo_cta;
  int32_t solo_len;
  int32_t first;           // kind of work that this CTA starts with
  MK_DEV int32_t begin(int kind, int slot) const {
    const int c = static_cast<int>(blockIdx.x);
    if (kind == kPair) return c * share;
    if (c <= solo_cta) return c < solo_cta ? total[kSolo] : slot * solo_len;
    return 2 * solo_len + (2 * (c - solo_cta - 1) + slot) * share;
  }
  MK_DEV int32_t length(int kind) const {
    return kind == kSolo && static_cast<int>(blockIdx.x) == solo_cta ? solo_len : share;
  }
  // How many stretches behind this one (a CTA's of pairs, a slot's of solos) the
  // one with a place on the line is.
  MK_DEV int behind(int kind, int slot, int32_t at) const {
    uint32_t past = at - begin(kind, slot);
    if (kind == kSolo && static_cast<int>(blockIdx.x) == solo_cta) {
      past = at - 2 * solo_len;  // (from the next CTA on, or negative)
      if (at < 2 * solo_len) return at >= solo_len && slot == 0;
      return 2 - slot + past / share;
    }
    return past / share;
  }
};

// One row's result of one stretch of key tiles; its O is beside it (in an order of
// its own: see softmax).
struct Partial {
  float m, l;
  // of an item's first stretch: 2 * (stretches behind it) + kind, and the row's
  // place in this stretch's part of the carry region, from which those of the
  // stretches behind it follow
  int32_t more, carry;
};

// Workspace layout.
struct Space {
  uint32_t* status;  // [0] the status, [1] whether any row sees a prefix key
  Partial* part;
  float* o;          // D values per partial row
  // first partial row of each region: the prefix's and the requests' own
  // results by row and head; those of stretches that start in the middle of an
  // item, [kind][CTA][slot][128]
  int64_t pre, own, carry;
};

struct AttnParams {
  mk_prefix_attn_io io;
  float scale_log2;  // scale * log2(e)
  int32_t group;     // G: q heads per KV head
  int32_t tile_tok;  // tokens per row tile: floor(128 / G)
  int32_t half_tok;  // tokens per solo: floor(64 / G)
  int32_t box, box_shift;  // keys per TMA box: min(page_size, 128) = 128 >> box_shift
  int32_t page_shift;
  int32_t ctas;
  int32_t tile_cost[2], item_cost[2];  // kTileCost, kItemCost in this call's units
  // quotients without divisions, whose code, run for the first time at a CTA's
  // start, delays its first loads
  Divisor by_pair, by_heads, by_ctas, by_cost[2];
  Space ws;
  // of a self-test: limit of a wait for a hand-off; which hand-off to withhold, and
  // the how manieth
  uint64_t wait_ns;
  int32_t withhold, withhold_at;
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

// Items of a row set of n tokens for one head: pairs of row tiles, the last one
// of what is left if that is more than 64 rows; a solo of what is left otherwise.
MK_DEV int items_of(const AttnParams& P, int kind, int n) {
  const int full = quotient(n, P.by_pair), left = n - full * 2 * P.tile_tok;
  return kind == kPair ? full + (left > P.half_tok) : left > 0 && left <= P.half_tok;
}
MK_DEV int32_t item_cost(const AttnParams& P, int kind, int kt) {
  return P.item_cost[kind] + kt * P.tile_cost[kind];
}
// Cost of all of a row set's items against kt key tiles.
MK_DEV int32_t set_cost(const AttnParams& P, int kind, int n, int kt) {
  return kt > 0 ? items_of(P, kind, n) * item_cost(P, kind, kt) * P.io.n_kv_heads : 0;
}

// ------------------------------------------------------------------ tiles

// A stretch of key tiles of one item, as a producer hands it out.
struct Piece {
  int32_t own;       // 0 prefix, 1 a request's own keys, -1 no more
  int32_t h, b;
  int32_t tok0;      // first token (row of q) of the (first) row tile
  int32_t tok_end;   // behind the last token of the prefix rows / the request
  int32_t kt_a, kt_b;
  int32_t klo, khi;  // keys that some row sees
  int32_t first;     // starts its item: leaves its result by row, else by CTA
  int32_t more;      // stretches of the item behind this one (of a first one)
  int32_t split;     // tokens of slot 0's row tile of a pair
  int32_t cu, base;
};

// Barriers of one ring of K and V tiles, with those of the row tiles and the
// pieces that go with it.
constexpr int kMaxStages = 8;
struct Ring {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t q_full[2], q_empty[2];
  uint64_t fifo_full[kFifo], fifo_empty[kFifo];
  Piece fifo[kFifo];
  // Once the producer is done: the K and V tiles whose copies were issued, how often
  // those of all row tiles were, and how many row tiles' once more.
  int32_t loads, q_rounds, q_more;
};
// A place in a ring: the stage and how often the ring has gone round (mod 2).
struct Place {
  int st = 0;
  uint32_t round = 0;
  MK_DEV Place next(int stages) const {
    Place p{st + 1, round};
    if (p.st == stages) p.st = 0, p.round ^= 1;
    return p;
  }
};

template <int D>
struct alignas(1024) TileSmem {
  // Row tiles and K and V tiles in flight.  Pairs: two row tiles, then kStages
  // tiles.  Solos: for each slot its row tile of 64 rows, then kSoloStages tiles.
  // (A solo's MMA reads 128 rows: those behind the 64 are whatever lies there, and
  // so are the rows of the result that nobody reads.)  Three stages per slot instead of two keep a K or V tile on its way
  // while the two before it are in use.
  static constexpr int kTile = 128 * D * 2;
  static constexpr int kStages = D == 128 ? 5 : 8;
  static constexpr int kSoloStages = D == 128 ? 3 : 6;
  static constexpr int kArena = (kStages + 2 > 2 * kSoloStages + 1 ? kStages + 2 : 2 * kSoloStages + 1) * kTile;
  uint8_t arena[kArena];
  Ring ring[3];      // of pairs, of slot 0's solos, of slot 1's
  uint64_t s_full[2], p_full[2], o_done[2];
  uint64_t turn_of[2];  // pairs: the other slot's issuer has had its turn
  uint64_t turn;     // both slots' MMAs of the first kind of work are done
  uint64_t drained[2];
  Plan plan;
  int32_t sum[2][kTileThreads / 32];
  int32_t low[kTileThreads / 32];
  int32_t low_cu;    // first row of the (last) request with the lowest position of all
  // the first request with work on a line's stretch and where it starts: the
  // CTA's of pairs, the two slots' of solos
  int32_t first_at[3];
  int32_t first[3];
  uint32_t tmem;
  // some wait of the CTA has run out: while it works, while it drains what it gave up
  uint32_t abort, drain_abort;
};

template <bool kTest>
struct Ctx {
  volatile uint32_t* abort;
  uint32_t* status;
  uint64_t wait_ns;  // of a self-test
  MK_DEV uint64_t limit(int work) const {
    return (kTest ? wait_ns : kWaitNs) * (work ? kLongWait : 1);
  }
};

// One kind of work as one slot's warps see it.
template <int D>
struct View {
  Ring* ring;
  uint8_t* kv;       // its part of the buffers
  uint8_t* q;        // the slot's row tile
  int kind, slot, stages;
  MK_DEV View(TileSmem<D>& S, int kind_, int slot_) : kind(kind_), slot(slot_) {
    const bool pair = kind == kPair;
    ring = &S.ring[pair ? 0 : 1 + slot];
    stages = pair ? TileSmem<D>::kStages : TileSmem<D>::kSoloStages;
    constexpr int kTile = TileSmem<D>::kTile;
    uint8_t* part = S.arena + slot * (kTile / 2 + TileSmem<D>::kSoloStages * kTile);  // of a solo's slot
    kv = pair ? S.arena + 2 * kTile : part + kTile / 2;
    q = pair ? S.arena + slot * kTile : part;
  }
};

// Bounded waits: false once any wait of the CTA has run out.  The clock is read
// now and then only: reading it takes longer than a hand-off.  (With limits that come
// from memory ragged verify steps take 1.2 us longer: 16 requests of up to 16 tokens
// over 16384 keys 47.6 instead of 46.4.)
template <bool kTest>
MK_DEV bool wait_bar(const Ctx<kTest>& c, uint64_t* bar, uint32_t parity, int work) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (*c.abort) return false;
    if (globaltimer() - t0 > c.limit(work)) {
      *c.abort = 1;
      atomicExch(c.status, kTimeout);
      return false;
    }
  }
}
template <bool kTest>
MK_DEV bool wait_warp(const Ctx<kTest>& c, uint64_t* bar, uint32_t parity, int work = 0) {
  return __all_sync(0xffffffffu, wait_bar(c, bar, parity, work));
}

// Of work that was given up: waits for the copies into a ring that may still be on
// their way, the last one into each stage and each row tile.
MK_DEV void drain_ring(const Ctx<false>& c, Ring& R, int stages, int q_tiles) {
  for (int q = max(0, R.loads - stages); q < R.loads; ++q)
    wait_warp(c, &R.full[q % stages], (q / stages) & 1);
  for (int t = 0; t < q_tiles; ++t) {
    const int n = R.q_rounds + (t < R.q_more);
    if (n > 0) wait_warp(c, &R.q_full[t], (n - 1) & 1);
  }
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
// 16 lanes x 32 columns: of every 8 columns, thread t has columns 2 (t % 4) and the
// next of lane t / 4, then the same of lane t / 4 + 8.
MK_DEV void tmem_ld_16rows(uint32_t taddr, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32"
      " {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
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
  static constexpr uint32_t kExponent = 0x7f80;  // all ones: infinity or NaN
};
template <> struct Types<__half> {
  static constexpr uint32_t kFormat = 0;
  static constexpr uint32_t kExponent = 0x7c00;
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

// Pairs of float32 operations in one instruction, and the largest of three.
MK_DEV float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n .reg .b64 a, b, c, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mov.b64 c, {%6, %7};\n"
      " fma.rn.f32x2 d, a, b, c;\n mov.b64 {%0, %1}, d;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
MK_DEV float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n"
      " add.rn.f32x2 d, a, b;\n mov.b64 {%0, %1}, d;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
MK_DEV float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// The larger one, or NaN if either is.
MK_DEV float max_or_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
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

// ---- the lines of work, worked out by the whole CTA: each thread takes
// consecutive requests (one, up to 384 of them)
template <int D>
MK_DEV void lay_out_work(const AttnParams& P, TileSmem<D>& S) {
  const mk_prefix_attn_io& io = P.io;
  const int B = io.n_requests, lane = lane_id(), warp = threadIdx.x >> 5;
  const int each = ceil_div(B, kTileThreads), b0 = threadIdx.x * each, b1 = min(B, b0 + each);
  const int n_used = clampi(io.cu_rows[B], 0, io.n_rows);
  int32_t mine[2] = {0, 0};
  int low = INT_MAX, low_cu = 0;
  bool falls = false;  // the lines are measured for rows that belong to one request each
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    const Req r = read_req(P, b);
    falls |= io.cu_rows[b + 1] < io.cu_rows[b];
    for (int k = 0; k < 2; ++k) mine[k] += set_cost(P, k, r.n, r.kt1 - r.kt0);
    if (r.n && r.base < low) low = r.base, low_cu = r.cu;
  }
  const int my_low = low;
  int32_t v[2] = {mine[0], mine[1]};
#pragma unroll
  for (int o = 1; o < 32; o <<= 1)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int32_t u = __shfl_up_sync(0xffffffffu, v[k], o);
      if (lane >= o) v[k] += u;
    }
  if (lane == 31) S.sum[0][warp] = v[0], S.sum[1][warp] = v[1];
  low = __reduce_min_sync(0xffffffffu, low);
  if (lane == 0) S.low[warp] = low;
  falls = __syncthreads_or(falls);
  Plan p;
  const bool some = lane < kTileThreads / 32;  // a lane per warp
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int32_t x = some ? S.sum[k][lane] : 0;
    v[k] += __reduce_add_sync(0xffffffffu, lane < warp ? x : 0);
    p.total[k] = __reduce_add_sync(0xffffffffu, x);
  }
  low = __reduce_min_sync(0xffffffffu, some ? S.low[lane] : INT_MAX);
  if (my_low == low) atomicMax(&S.low_cu, low_cu);
  // the lowest position of any row decides where the prefix starts to be seen
  const int64_t lo64 =
      io.window && low != INT_MAX ? static_cast<int64_t>(io.prefix_len) + low - io.window + 1 : 0;
  p.n_used = n_used;
  p.lo = clampi(lo64, 0, io.prefix_len);
  p.kt1 = ceil_div(io.prefix_len, kTileKeys);
  p.kt0 = p.lo >= io.prefix_len ? p.kt1 : p.lo / kTileKeys;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    p.prefix_cost[k] = set_cost(P, k, p.n_used, p.kt1 - p.kt0);
    p.total[k] += p.prefix_cost[k];
    if (falls) p.total[k] = 0;
  }
  // At least one key tile each, so that every stretch inside an item has one: what
  // is left of the last pairs' CTA is used only if it holds one (the sum has room
  // for what then is not).
  const int32_t most = max(P.tile_cost[0], P.tile_cost[1]);
  p.share = max(static_cast<int32_t>(quotient(p.total[kPair] + ((p.total[kSolo] + 1) >> 1) + most + P.ctas - 1, P.by_ctas)), most);
  p.solo_cta = static_cast<uint32_t>(p.total[kPair]) / static_cast<uint32_t>(p.share);
  p.solo_len = (p.solo_cta + 1) * p.share - p.total[kPair];
  if (p.solo_len < most) ++p.solo_cta, p.solo_len = p.share;
  p.first = p.begin(kPair, 0) < p.total[kPair] ? kPair : kSolo;
  if (threadIdx.x == 0) {
    S.plan = p;
    if (blockIdx.x == 0) {
      P.ws.status[0] = falls ? kFalling : 0;
      P.ws.status[1] = p.kt1 > p.kt0;
    }
  }
  // the requests that this CTA's stretches start in
#pragma unroll 1
  for (int j = 0; j < 3; ++j) {
    const int k = j > 0;
    const int32_t begin = p.begin(k, j - 1), cost = k ? mine[1] : mine[0];
    int32_t here = (k ? p.prefix_cost[1] + v[1] : p.prefix_cost[0] + v[0]) - cost;
    if (threadIdx.x == 0 && begin < here) S.first[j] = 0, S.first_at[j] = here;
    if (begin >= here && begin < here + cost) {
      int b = b0;
#pragma unroll 1
      for (; b < b1 - 1; ++b) {
        const Req r = read_req(P, b);
        const int32_t next = here + set_cost(P, k, r.n, r.kt1 - r.kt0);
        if (begin < next) break;
        here = next;
      }
      S.first[j] = b;
      S.first_at[j] = here;
    }
  }
}

// ---- a stretch of a line, piece by piece: emit(Piece) for each
template <class Emit>
MK_DEV bool walk(const AttnParams& P, const Plan& plan, int kind, int slot, int first,
                 int32_t first_at, const Emit& emit) {
  const mk_prefix_attn_io& io = P.io;
  const int Hk = io.n_kv_heads, lane = lane_id(), step = P.tile_cost[kind];
  const int32_t begin = plan.begin(kind, slot);
  const int32_t end = min(plan.total[kind], begin + plan.length(kind));
  if (begin >= end) return true;
  // the items of a row set of n tokens (row tile by row tile, head by head) from
  // cost `at`
  auto items = [&](Piece& w, int32_t at, int tok, int n, int kt0, int kt1) -> bool {
    const int kt = kt1 - kt0, rows = items_of(P, kind, n), count = rows * Hk;
    if (kt <= 0 || count == 0) return true;
    const int left = n - (rows - 1) * 2 * P.tile_tok;  // of the last pair
    const int32_t cost = item_cost(P, kind, kt);
    int i = begin > at ? static_cast<uint32_t>(begin - at) / static_cast<uint32_t>(cost) : 0;
    int p = quotient(i, P.by_heads), h = i - p * Hk;
    int32_t s = at + i * cost + P.item_cost[kind];  // of the item's first key tile
    for (; i < count && s < end; ++i, s += cost) {
      const int s0 = s >= begin ? 0 : quotient(begin - s + step - 1, P.by_cost[kind]);
      const int s1 = min(kt, static_cast<int>(quotient(end - s + step - 1, P.by_cost[kind])));
      if (s0 < s1) {
        w.h = h;
        // (behind its pairs the row set's solo)
        w.tok0 = tok + 2 * P.tile_tok * (kind == kPair ? p : quotient(n, P.by_pair));
        w.split = kind == kPair && p == rows - 1 && left <= 2 * P.half_tok ? P.half_tok : P.tile_tok;
        w.kt_a = kt0 + s0;
        w.kt_b = kt0 + s1;
        w.first = s0 == 0;
        const int32_t last = s + (kt - 1) * step;
        w.more = last < end ? 0 : plan.behind(kind, slot, last);
        if (!emit(w)) return false;
      }
      if (++h == Hk) h = 0, ++p;
    }
    return true;
  };
  Piece w;
  std::memset(&w, 0, sizeof(w));
  if (begin < plan.prefix_cost[kind]) {
    w.tok_end = plan.n_used;
    w.klo = plan.lo;
    w.khi = io.prefix_len;
    if (!items(w, 0, 0, plan.n_used, plan.kt0, plan.kt1)) return false;
  }
  w.own = 1;
  int32_t at = first_at;
  for (int b0 = first; at < end && b0 < io.n_requests; b0 += 32) {
    // 32 requests' lengths at a time
    Req req{0, 0, 0, 0, 0, 0};
    if (b0 + lane < io.n_requests) req = read_req(P, b0 + lane);
    for (int i = 0; at < end && i < 32 && b0 + i < io.n_requests; ++i) {
      const int n = __shfl_sync(0xffffffffu, req.n, i), len = __shfl_sync(0xffffffffu, req.len, i);
      const int kt0 = __shfl_sync(0xffffffffu, req.kt0, i), kt1 = __shfl_sync(0xffffffffu, req.kt1, i);
      w.b = b0 + i;
      w.cu = __shfl_sync(0xffffffffu, req.cu, i);
      w.base = max(0, len - n);
      w.tok_end = w.cu + n;
      w.klo = io.window ? clampi(static_cast<int64_t>(w.base) - io.window + 1, 0, len) : 0;
      w.khi = len;
      if (!items(w, at, w.cu, n, kt0, kt1)) return false;
      at += set_cost(P, kind, n, kt1 - kt0);
    }
  }
  return true;
}

// ---- producer of one kind of work: hands the pieces out and loads row tiles
// and K and V tiles (K0 V0 K1 V1 ...)
template <int D, bool kTest>
MK_DEV bool produce(const AttnParams& P, TileSmem<D>& S, const Ctx<kTest>& c, const View<D>& V,
                    const CUtensorMap* tm_q, const CUtensorMap* tm_k, const CUtensorMap* tm_v,
                    uint64_t* after) {
  const mk_prefix_attn_io& io = P.io;
  constexpr int kHalves = D / 64;
  const int lane = lane_id(), kind = V.kind, slot = V.slot, q_tiles = kind == kPair ? 2 : 1;
  Ring& R = *V.ring;
  const int boxes = 1 << P.box_shift;           // per tile and half
  const int group_shift = 5 - P.box_shift;
  const int group_tiles = 1 << group_shift;     // key tiles whose pages one lane each holds
  Place at;          // of the next load
  int loads = 0, n_loaded = 0, n_out = 0;
  // First slot of box number 32 g + lane of a piece; -1: no row sees its keys.
  // A page outside the pool: behind the end, where the copy fills in zeros.
  auto fetch = [&](const volatile Piece& w, int g) -> int {
    const int box = 32 * g + lane, key = w.kt_a * kTileKeys + box * P.box;
    if (box >= (w.kt_b - w.kt_a) * boxes || key >= w.khi || key + P.box <= w.klo) return -1;
    const int page = key >> P.page_shift;
    const int id = w.own ? io.block_table[w.b * io.table_stride + page] : io.prefix_pages[page];
    return id >= 0 && id < io.n_pages ? (id << P.page_shift) + (key & (io.page_size - 1))
                                      : max(1, io.n_pages << P.page_shift);
  };
  auto push = [&](const Piece& w) -> bool {
    const int k = n_out % kFifo;
    if (n_out >= kFifo && !wait_warp(c, &R.fifo_empty[k], ((n_out / kFifo) - 1) & 1, 1))
      return false;
    if (lane == 0) {
      R.fifo[k] = w;
      mbar_arrive(&R.fifo_full[k]);
    }
    __syncwarp();
    ++n_out;
    return true;
  };
  // (a piece is read in the fifo's place, which nobody but this warp reuses:
  // registers are short here)
  auto load_piece = [&](const volatile Piece& w, int pages) -> bool {
    // the buffers belong to the other kind of work until its MMAs are done
    if (after && !wait_warp(c, after, 0, 1)) return false;
    after = nullptr;
    const int n = w.kt_b - w.kt_a;
    int ahead = n > group_tiles ? fetch(w, 1) : -1, group = 0;
    auto load = [&](const CUtensorMap* map, int x) -> bool {
      const int g = x >> group_shift;
      if (g > group) {  // (K is loaded before V of the same tile: x never falls)
        pages = ahead;
        group = g;
        if (n > (g + 1) * group_tiles) ahead = fetch(w, g + 1);
      }
      // lane = half * boxes + box
      const int box = lane & (boxes - 1), half = lane >> P.box_shift;
      const int key = __shfl_sync(0xffffffffu, pages, ((x & (group_tiles - 1)) << P.box_shift) + box);
      const bool mine = lane < boxes * kHalves && key >= 0;
      const uint32_t cnt = __popc(__ballot_sync(0xffffffffu, mine));
      if (loads >= V.stages && !wait_warp(c, &R.empty[at.st], at.round ^ 1)) return false;
      if (lane == 0) mbar_arrive_expect_tx(&R.full[at.st], cnt * P.box * 128);
      __syncwarp();
      if (mine)
        tma_load_3d(V.kv + at.st * (128 * D * 2) + half * 128 * 128 + box * P.box * 128, map,
                    &R.full[at.st], half * 64, w.h, key);
      at = at.next(V.stages);
      ++loads;
      return true;
    };
    if (!load(tm_k, 0)) return false;
    for (int t = 0; t < q_tiles; ++t) {
      if (n_loaded > 0 && !wait_warp(c, &R.q_empty[t], (n_loaded - 1) & 1)) {
        if (lane == 0) R.q_more = t;
        return false;
      }
      if (lane == 0) {
        const int toks = kind == kPair ? P.tile_tok : P.half_tok;
        mbar_arrive_expect_tx(&R.q_full[t], kHalves * P.group * toks * 128);
        for (int f = 0; f < kHalves; ++f)
          tma_load_3d(V.q + t * TileSmem<D>::kTile + f * (kind == kPair ? 128 : 64) * 128, tm_q,
                      &R.q_full[t], f * 64, w.h * P.group, w.tok0 + t * w.split);
      }
      __syncwarp();
    }
    ++n_loaded;
    for (int x = 0; x < n; ++x) {
      if (!load(tm_v, x)) return false;
      if (x + 1 < n && !load(tm_k, x + 1)) return false;
    }
    return true;
  };
  // the next piece's pages are read before the piece at hand is loaded: each
  // read is a round trip to L2 or HBM
  int held_pages = -1;
  const int line = kind == kPair ? 0 : 1 + slot;
  bool ok = walk(P, S.plan, kind, slot, S.first[line], S.first_at[line], [&](const Piece& w) -> bool {
    if (!push(w)) return false;
    const int pages = fetch(w, 0);
    if (n_out > 1 && !load_piece(R.fifo[(n_out - 2) % kFifo], held_pages)) return false;
    held_pages = pages;
    return true;
  });
  if (ok) {
    Piece none;
    std::memset(&none, 0, sizeof(none));
    none.own = -1;
    ok = push(none) && (n_out < 2 || load_piece(R.fifo[(n_out - 2) % kFifo], held_pages));
  }
  if (lane == 0) R.loads = loads, R.q_rounds = n_loaded;
  return ok;
}

// ---- MMA issuer of a slot: the whole warp walks the pieces, one elected lane
// issues, so that descriptors and addresses are warp-uniform; false once a wait
// has run out.  The issuers of a pair's slots take turns, a tile's P V and the next
// tile's scores at a time: with the products of both slots mixed, slots that make
// their P at the same time go on doing so, and a tile takes 2.5 us; with one warp
// issuing for both, its waits and commits (0.1 us each) make it 1.8.  For the
// commits' sake only scores and results are announced by one; what they tell about
// the buffers, the softmax warps that wait for them pass on.
struct SlotParity {
  uint32_t s = 0, p = 0, o = 0;
  int cold = 1;  // nothing has run yet
  int tile = 0;  // (counted in a self-test only)
};

// Whether a self-test withholds this hand-off.
template <bool kTest>
MK_DEV bool withheld(const AttnParams& P, Withhold what, int tile) {
  return kTest && P.withhold == what && P.withhold_at == tile;
}

template <class T, int D, bool kTest>
MK_DEV bool issue_mmas(const AttnParams& P, TileSmem<D>& S, const Ctx<kTest>& c, const View<D>& V, SlotParity& par) {
  constexpr uint32_t kIdS = idesc_of<T>(kTileKeys, false), kIdO = idesc_of<T>(D, true);
  const bool pair = V.kind == kPair;
  const int slot = V.slot;
  const uint32_t ts = S.tmem + slot * 128, to = S.tmem + 256 + slot * 128;
  Ring& R = *V.ring;
  uint64_t* const q_full = &R.q_full[pair ? slot : 0];
  const uint64_t qd = sdesc_kmajor_sw128(smem_u32(V.q));
  const uint32_t q_half = (pair ? 128 : 64) * 128 >> 4;  // to a row's second 64 values
  const uint32_t kv = smem_u32(V.kv);
  Place at;  // of the next K tile
  int piece = 0;
  uint32_t turns = 0;
  auto wait_stage = [&](Place p) { return wait_warp(c, &R.full[p.st], p.round); };
  auto my_turn = [&]() -> bool {
    const uint32_t k = turns++ + slot;  // turns of the other slot that come first
    return !pair || k == 0 || wait_warp(c, &S.turn_of[slot], (k - 1) & 1);
  };
  // the scores of a tile
  auto qk = [&](Place p) {
    const uint64_t kd = sdesc_kmajor_sw128(kv + p.st * TileSmem<D>::kTile);
#pragma unroll
    for (int k = 0; k < D / 16; ++k)
      mma_bf16(ts, qd + (k >> 2) * q_half + (k & 3) * 2, kd + (k >> 2) * (128 * 128 >> 4) + (k & 3) * 2,
               kIdS, k);
  };
  while (true) {
    const int f = piece % kFifo;
    if (!wait_warp(c, &R.fifo_full[f], (piece / kFifo) & 1)) return false;
    const int own = R.fifo[f].own, n = R.fifo[f].kt_b - R.fifo[f].kt_a;
    __syncwarp();
    if (elect_one()) mbar_arrive(&R.fifo_empty[f]);
    if (own < 0) return true;
    if (!wait_warp(c, q_full, piece & 1) || !wait_stage(at) || !my_turn()) return false;
    tc_fence_after();
    if (elect_one()) {
      qk(at);
      if (pair) mbar_arrive(&S.turn_of[slot ^ 1]);
      if (!withheld<kTest>(P, kScores, par.tile)) mma_commit(&S.s_full[slot]);
    }
    if (kTest) ++par.tile;
    __syncwarp();
    for (int j = 0; j < n; ++j) {
      const Place sv = at.next(V.stages), sk = sv.next(V.stages);
      const bool more = j + 1 < n;
      if (!wait_stage(sv) || (more && !wait_stage(sk))) return false;
      if (!my_turn() || !wait_warp(c, &S.p_full[slot], par.p)) return false;
      par.p ^= 1;
      tc_fence_after();
      const uint64_t vd = sdesc_mnmajor_sw128(kv + sv.st * TileSmem<D>::kTile, 128 * 128);
      if (elect_one()) {
        // P V, then the next scores right behind, which take P's place
#pragma unroll
        for (int k = 0; k < kTileKeys / 16; ++k)
          mma_ts(to, ts + 8 * k, vd + k * (16 * 128 >> 4), kIdO, j > 0 || k > 0);
        if (more) qk(sk);
        if (pair) mbar_arrive(&S.turn_of[slot ^ 1]);
        if (!more || !withheld<kTest>(P, kScores, par.tile)) mma_commit(more ? &S.s_full[slot] : &S.o_done[slot]);
      }
      __syncwarp();
      if (kTest && more) ++par.tile;
      at = sk;
    }
    ++piece;
  }
}

// ---- softmax of one slot (a warpgroup, one thread per row)
// Whether a row of V in shared memory holds an infinity or a NaN.  (A call: inlined, it
// costs every softmax 2 %.)
template <class T, int D>
__device__ __noinline__ bool row_not_finite(const uint8_t* v, int row) {
  constexpr uint32_t kLow = Types<T>::kExponent, kHigh = kLow << 16;
  bool found = false;
#pragma unroll 1
  for (int x = 0; x < D / 8; ++x) {  // (neighbouring rows start at different banks)
    const uint4 u = reinterpret_cast<const uint4*>(v + (x >> 3) * 128 * 128)[(x ^ row) & 7];
    const uint32_t words[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) found |= (words[i] & kLow) == kLow || (words[i] & kHigh) == kHigh;
  }
  return found;
}

template <class T, int D, bool kTest>
MK_DEV bool softmax(const AttnParams& P, TileSmem<D>& S, const Ctx<kTest>& c, const View<D>& W,
                    SlotParity& par) {
  const mk_prefix_attn_io& io = P.io;
  const int slot = W.slot, kind = W.kind;
  Ring& R = *W.ring;
  const int warp = (threadIdx.x >> 5) & 3, lane = lane_id(), row = warp * 32 + lane;
  const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
  const uint32_t ts = S.tmem + lanes + slot * 128, to = S.tmem + lanes + 256 + slot * 128;
  const int G = P.group, tok_in_tile = row / G, g = row - tok_in_tile * G;
  const float sl2 = P.scale_log2;
  Place at;  // of the tile's K
  int piece = 0;
  while (true) {
    const int f = piece % kFifo;
    if (!wait_warp(c, &R.fifo_full[f], (piece / kFifo) & 1)) return false;
    const Piece w = R.fifo[f];
    __syncwarp();
    if (lane == 0) mbar_arrive(&R.fifo_empty[f]);
    if (w.own < 0) return true;
    ++piece;
    const int n = w.kt_b - w.kt_a;
    // this thread's row: its token, and the keys [klo, khi) it sees; of a token
    // tree, the bits of `tree` instead from key `tree_at` on
    const int tok = w.tok0 + (kind == kPair ? slot * w.split : 0) + tok_in_tile;
    const int toks = kind == kSolo ? P.half_tok : slot ? P.tile_tok : w.split;
    const bool valid = tok_in_tile < toks && tok < w.tok_end;
    int klo = w.klo, khi = w.khi, tree_at = INT_MAX;
    uint64_t tree = 0;
    if (valid) {
      int base = w.base, i = tok - w.cu;
      if (!w.own && io.window) {  // which request is it?
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
                            (w.own ? 0 : io.prefix_len);
        klo = max(klo, clampi(low, 0, w.khi));
      }
      if (w.own) {
        if (io.tree_mask) tree_at = base;
        else khi = min(khi, clampi(static_cast<int64_t>(base) + i + 1, 0, INT_MAX));
      }
    }
    const bool warp_valid = __any_sync(0xffffffffu, valid);
    // So many keys from klo on may be seen by no row: klo is the window of a row with
    // no bit but its own, and if the first row of the request that it belongs to is not
    // one, all windows may start later.
    const int late =
        io.tree_mask && io.window && __popcll(io.tree_mask[w.own ? w.cu : S.low_cu]) > 1 ? 63 : 0;

    // (The CTA's first tile goes through the motions on what lies in tensor memory,
    // without waiting or leaving anything, while its scores are being made: this
    // code then is in the instruction cache.)
    float m = -INFINITY, l = 0.f;
    for (int j = par.cold ? -1 : 0; j < n; ++j) {
      const int k0 = (w.kt_a + j) * kTileKeys;
      if (j >= 0 && (k0 < w.klo + late || k0 + kTileKeys > w.khi)) {
        // keys that no row sees may hold anything: their V rows become zeros, so
        // that a weight of zero leaves no NaN behind
        const Place sv = at.next(W.stages);
        if (!wait_warp(c, &R.full[sv.st], sv.round)) return false;
        uint8_t* v = W.kv + sv.st * (128 * D * 2) + row * 128;
        bool unseen = k0 + row < w.klo || k0 + row >= w.khi;
        // (one that may be seen has to be finite)
        if (!unseen && k0 + row < w.klo + late) unseen = row_not_finite<T, D>(v, row);
        if (unseen) {
#pragma unroll
          for (int x = 0; x < D / 8; ++x)
            reinterpret_cast<uint4*>(v + (x >> 3) * 128 * 128)[x & 7] = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
      }
      if (j >= 0) {
        if (!wait_warp(c, &S.s_full[slot], par.s)) return false;
        par.s ^= 1;
        tc_fence_after();
        // These scores are done, and so is all that this slot's issuer sent before
        // them: the slot no longer needs the tile's K, the V of the tile before and,
        // with the last tile, its row tile.
        if (warp == 0 && lane == 0) {
          mbar_arrive(&R.empty[at.st]);
          if (j > 0) mbar_arrive(&R.empty[at.st == 0 ? W.stages - 1 : at.st - 1]);
          if (j == n - 1 && !withheld<kTest>(P, kRowTile, 2 * (piece - 1) + slot)) mbar_arrive(&R.q_empty[kind == kPair ? slot : 0]);
        }
        __syncwarp();  // (loads from tensor memory are for whole warps)
      }
      if (warp_valid) {
        // P = 2^(S - m), with the m of the tiles before as long as the row's sum
        // stays below 2^14 (which the weights' types and the 32-bit sums hold
        // without loss): the maximum itself is looked for only in a piece's first
        // tile and where that fails, in a second pass over the scores (they lie in
        // tensor memory until P is stored).  Taking it in every tile is 0.19 us of
        // the 1.6 that a tile takes.
        bool look = j <= 0 || __any_sync(0xffffffffu, valid && m == -INFINITY);
        uint32_t p[kTileKeys / 2];
        float total;
#pragma unroll 1
        while (true) {
          float s[kTileKeys];
#pragma unroll
          for (int q = 0; q < 4; ++q) tmem_ld32(ts + 32 * q, s + 32 * q);
          tmem_ld_wait();
          const bool edge = klo > k0 || khi < k0 + kTileKeys || tree_at < k0 + kTileKeys || j < 0;
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
          if (look) {
            float t4[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) t4[y] = max3(s[y], s[y + 4], s[y + 8]);
#pragma unroll
            for (int x = 12; x < kTileKeys - 4; x += 8)
#pragma unroll
              for (int y = 0; y < 4; ++y) t4[y] = max3(t4[y], s[x + y], s[x + y + 4]);
#pragma unroll
            for (int y = 0; y < 4; ++y) t4[y] = fmaxf(t4[y], s[kTileKeys - 4 + y]);
            const float top = sl2 * fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3]));
            if (j <= 0) {
              m = top;
              l = 0.f;
            } else {
              const bool grow = valid && top > m;
              const float x = grow ? exp2_approx(m - top) : 1.f;
              if (grow) m = top;
              l *= x;
              if (__any_sync(0xffffffffu, grow)) {
#pragma unroll 1
                for (int q = 0; q < D / 32; ++q) {
                  float o[32];
                  tmem_ld32(to + 32 * q, o);
                  tmem_ld_wait();
#pragma unroll
                  for (int y = 0; y < 32; ++y) o[y] *= x;
                  tmem_st32(to + 32 * q, reinterpret_cast<uint32_t*>(o));
                }
              }
            }
          }
          const float ms = m == -INFINITY ? 0.f : m;
          float2 sum[2] = {{0.f, 0.f}, {0.f, 0.f}};
          // P goes into the product rounded to the tensors' type, which is all that operand
          // A takes; its sum is of the 32-bit values. A low part beside it, as the layer
          // kernel keeps one, would double P V (a pair's products 1.05 -> 1.57 us). Without
          // it out is off by 0.0023 of its norm in bf16 (0.00029 in fp16), where rounding
          // out itself leaves 0.0017 (0.00021).
#pragma unroll
          for (int x = 0; x < kTileKeys; x += 2) {
            float2 y = fma2(make_float2(s[x], s[x + 1]), make_float2(sl2, sl2), make_float2(-ms, -ms));
            y.x = exp2_approx(y.x);
            y.y = exp2_approx(y.y);
            sum[(x >> 1) & 1] = add2(sum[(x >> 1) & 1], y);
            p[x >> 1] = Types<T>::pack(y.x, y.y);
          }
          const float2 both = add2(sum[0], sum[1]);
          total = both.x + both.y;
          // (the comparison is false for NaN)
          if (look || !__any_sync(0xffffffffu, valid && !(total <= kMost))) break;
          look = true;
        }
        l += total;
        if (j >= 0) {
          tmem_st32(ts, p);
          tmem_st32(ts + 32, p + 32);
          tmem_st_wait();
        } else {
          par.cold += p[0] == 1u && p[63] == 1u;  // (keeps the work)
        }
      }
      if (j >= 0) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0 && !withheld<kTest>(P, kWeights, par.tile)) mbar_arrive(&S.p_full[slot]);
        if (kTest) ++par.tile;
        at = at.next(W.stages).next(W.stages);
      }
    }
    par.cold = 0;

    // the piece's result
    if (!wait_warp(c, &S.o_done[slot], par.o)) return false;
    par.o ^= 1;
    tc_fence_after();
    if (warp == 0 && lane == 0)  // the last V
      mbar_arrive(&R.empty[at.st == 0 ? W.stages - 1 : at.st - 1]);
    const int32_t carry = ((kind * P.ctas + blockIdx.x) * 2 + slot) * 128 + row;
    const int64_t to_row = w.first ? (w.own ? P.ws.own : P.ws.pre) +
                                         static_cast<int64_t>(tok) * io.n_q_heads + w.h * G + g
                                   : P.ws.carry + carry;
    // (a NaN among the scores is in l, while the maximum passes it by)
    if (valid) P.ws.part[to_row] = Partial{l == l ? m : l, l, 2 * w.more + kind, carry};
    if (warp_valid) {
      // Four threads write 128 bytes of a row, 8 values each as they come from tensor
      // memory: of 16 pairs of columns, pair 4 i + c lies in place 4 c + i.  (With a
      // row per thread each store touched 32 lines, 2 to 3 us for a pair's tiles: 41.8
      // and 36.1 us instead of 40.7 and 35.2 for 64 requests' decode step and 24
      // token trees under a window.)
      const uint32_t rows = __ballot_sync(0xffffffffu, valid);
#pragma unroll 1
      for (int half = 0; half < 32 && rows >> half; half += 16) {
        const int at0 = half + (lane >> 2), at1 = at0 + 8;
        float* dst0 = P.ws.o + __shfl_sync(0xffffffffu, to_row, at0) * D + (lane & 3) * 8;
        float* dst1 = P.ws.o + __shfl_sync(0xffffffffu, to_row, at1) * D + (lane & 3) * 8;
#pragma unroll 1
        for (int q = 0; q < D / 32; ++q) {
          float o[16], x[16];
          __syncwarp();  // (loads from tensor memory are for whole warps)
          tmem_ld_16rows(to + (static_cast<uint32_t>(half) << 16) + 32 * q, o);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) x[2 * i + e] = o[4 * i + e], x[8 + 2 * i + e] = o[4 * i + 2 + e];
          if (rows >> at0 & 1) st_global_8(dst0 + 32 * q, x);
          if (rows >> at1 & 1) st_global_8(dst1 + 32 * q, x + 8);
        }
      }
      tc_fence_before();
    }
  }
}

// Warps 0-3 and 4-7: softmax of slot 0 and 1.  Warps 8 and 9: producers (8 for
// pairs and slot 0's solos, 9 for slot 1's solos).  Warps 10 and 11: MMA issuers.
// A CTA's way to its first scores is a chain of round trips (lengths, page numbers,
// K: 3 us with cold caches) and of code that it runs for the first time, which is
// slower to fetch than to run: the plan without divisions and
// unrolled copies, and CTAs without pairs that go to their solos at once, took 1 to
// 2 us off every call (64 requests over 4096 + up to 1000 keys: 44.5 to 42.6 us).
// Measured, 32 q heads on 8 KV heads of 128, bf16: 64 x 8 rows over a prefix of
// 32768 keys run at 1,160 TFLOP/s (237 us; a pair of tiles takes 1.55 us, its products
// alone 1.05); one row of each of 256 requests over 1000 to 2000 keys of its own, 16
// to a page (1.6 GB), at 6.2 TB/s (255 us), 91 % of a plain copy.
template <class T, int D, bool kTest>
__global__ void __launch_bounds__(kTileThreads, 1)
    k_attn_tiles(const __grid_constant__ AttnParams P, const __grid_constant__ CUtensorMap tm_q,
                 const __grid_constant__ CUtensorMap tm_q64, const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_v) {
  extern __shared__ uint8_t smem_raw[];
  TileSmem<D>& S = *reinterpret_cast<TileSmem<D>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                   ~static_cast<uintptr_t>(1023));
  const int warp = threadIdx.x >> 5;
  if (warp == 11) {
    // one barrier per lane and turn
    for (int i = lane_id(); i < 3 * kMaxStages; i += 32) {
      mbar_init(&S.ring[i / kMaxStages].full[i % kMaxStages], 1);
      mbar_init(&S.ring[i / kMaxStages].empty[i % kMaxStages], i < kMaxStages ? 2 : 1);
    }
    for (int i = lane_id(); i < 3 * kFifo; i += 32) {
      mbar_init(&S.ring[i / kFifo].fifo_full[i % kFifo], 1);
      mbar_init(&S.ring[i / kFifo].fifo_empty[i % kFifo], i < kFifo ? 10 : 5);
    }
    if (lane_id() < 3) {
      Ring& R = S.ring[lane_id()];
      R.loads = R.q_rounds = R.q_more = 0;
    }
    if (lane_id() < 6) {
      mbar_init(&S.ring[lane_id() >> 1].q_full[lane_id() & 1], 1);
      mbar_init(&S.ring[lane_id() >> 1].q_empty[lane_id() & 1], 1);
    }
    if (lane_id() < 2) {
      mbar_init(&S.s_full[lane_id()], 1);
      mbar_init(&S.p_full[lane_id()], 4);
      mbar_init(&S.o_done[lane_id()], 1);
      mbar_init(&S.drained[lane_id()], 1);
      mbar_init(&S.turn_of[lane_id()], 1);
    }
    if (lane_id() == 0) {
      mbar_init(&S.turn, 2);
      S.abort = S.drain_abort = 0;
      S.low_cu = 0;
    }
    fence_mbar_init();
  }
  if (warp == 10) {
    tmem_alloc(&S.tmem, 512);
    tmem_relinquish();
  }
  if (warp == 9 && lane_id() == 0) {
    prefetch_tensormap(&tm_q);
    prefetch_tensormap(&tm_q64);
    prefetch_tensormap(&tm_k);
    prefetch_tensormap(&tm_v);
  }
  pdl_wait();  // (what lies before it overlaps the end of the kernel before)
  lay_out_work<D>(P, S);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_launch_dependents();
  const Ctx<kTest> c{&S.abort, P.ws.status, P.wait_ns};
  // 2 x 128 x 208 + 128 x 88 = 64,512, all registers of the launch; all are back
  // at 168 before the common tail
  if (warp < 8) {
    reg_alloc<208>();
    const int slot = warp >> 2;
    SlotParity par;
    bool ok = true;
#pragma unroll 1
    for (int turn = S.plan.first; ok && turn < 2; ++turn)
      ok = softmax<T, D, kTest>(P, S, c, View<D>(S, turn, slot), par);
    __syncwarp();
    reg_dealloc<168>();
  } else {
    reg_dealloc<88>();
    const int slot = warp & 1;
    bool ok = true;
    if (warp < 10) {
#pragma unroll 1
      for (int turn = S.plan.first; ok && turn < 2; ++turn)
        if (turn == kSolo || slot == 0)
          ok = produce<D, kTest>(P, S, c, View<D>(S, turn, slot), turn == kSolo ? &tm_q64 : &tm_q,
                          &tm_k, &tm_v, turn > S.plan.first ? &S.turn : nullptr);
    } else {
      SlotParity par;
#pragma unroll 1
      for (int turn = S.plan.first; ok && turn < 2; ++turn) {
        ok = issue_mmas<T, D, kTest>(P, S, c, View<D>(S, turn, slot), par);
        if (ok && turn == 0) {
          if (elect_one() && !withheld<kTest>(P, kBuffers, slot)) mma_commit(&S.turn);
          __syncwarp();
        }
      }
    }
    __syncwarp();
    reg_alloc<168>();
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (S.abort) {
    // A wait has run out (none behind the barrier writes the word).  Whichever it was,
    // and whoever was done by then: no copy may land and no product run on after the
    // CTA has left.
    const Ctx<false> last{&S.drain_abort, c.status, 0};
    if (warp == 8) drain_ring(last, S.ring[0], TileSmem<D>::kStages, 2);
    if (warp == 8 || warp == 9) drain_ring(last, S.ring[warp - 7], TileSmem<D>::kSoloStages, 1);
    if (warp >= 10) {
      if (elect_one()) mma_commit(&S.drained[warp & 1]);
      __syncwarp();
      wait_warp(last, &S.drained[warp & 1], 0);
    }
    __syncthreads();
  }
  if (warp == 10) tmem_dealloc(S.tmem, 512);
}

// ------------------------------------------------------------------ merge


constexpr int kMergeThreads = 256, kMergePerSm = 5;
constexpr int kMergeSmem = 220 * 1024;  // less than an SM has

template <int V>
struct Vals {
  float v[V];
};
template <int V>
MK_DEV Vals<V> load_vals(const float* p) {
  Vals<V> x;
  if (V == 2) {
    const float2 y = *reinterpret_cast<const float2*>(p);
    x.v[0] = y.x, x.v[1] = y.y;
  } else {
#pragma unroll
    for (int i = 0; i + 3 < V; i += 4) {
      const float4 y = *reinterpret_cast<const float4*>(p + i);
      x.v[i] = y.x, x.v[i + 1] = y.y, x.v[i + 2] = y.z, x.v[i + 3] = y.w;
    }
  }
  return x;
}

// What does not depend on the tiles (the row's request) comes before the wait for
// them; behind it the first stretches' results of the prefix and of the request's
// own keys, by row, and then those of the stretches that carried on.  Each is a
// round trip to L2; they and the launch bound it (3 to 4 us behind the last tile).
// Its CTAs become resident on the SMs that are done first, as many as fit, so that
// registers are kept low (a CTA that has to wait for others' end costs 3 us) and no
// SM takes more than its even share: 16 requests of up to 16 tokens over 16384 keys
// 45.4 us instead of 47.3, of 2 tokens over 32768 keys 44.4 instead of 46.2 (and
// 47.6 with low registers alone).  A row and head has N lanes: 32, or 16 where
// there are so many rows that they come in waves (64 requests of 8 tokens, 32 heads
// of 128: 10 us less; with 32 tokens and 20 results each 16 lanes would take 6 us
// longer).
template <class T, int D, int N>
__global__ void __launch_bounds__(kMergeThreads, kMergePerSm)
    k_attn_merge(const __grid_constant__ AttnParams P) {
  const mk_prefix_attn_io& io = P.io;
  constexpr int V = D / N, kAtOnce = N == 32 ? 4 : 2;
  const int lane = threadIdx.x % N, Hq = io.n_q_heads;
  // the item's lanes
  const uint32_t lanes = N == 32 ? 0xffffffffu : (threadIdx.x & 16) ? 0xffff0000u : 0xffffu;
  const uint32_t item = blockIdx.x * static_cast<uint32_t>(kMergeThreads / N) + threadIdx.x / N;
  const int tok = static_cast<int>(item / static_cast<uint32_t>(Hq));
  const bool in = tok >= io.cu_rows[0] && tok < clampi(io.cu_rows[io.n_requests], 0, io.n_rows);
  bool own = false;
  if (in) {
    // its request: the lanes look at N places at once
    int lo = 0;
    for (int n = io.n_requests; n > 1;) {
      const int step = (n + N - 1) / N, at = lane * step;
      const uint32_t below = __ballot_sync(lanes, at < n && io.cu_rows[lo + at] <= tok) & lanes;
      const int skip = max(0, __popc(below) - 1) * step;
      lo += skip;
      n = min(step, n - skip);
    }
    const Req r = read_req(P, lo);
    own = r.kt1 > r.kt0;
  }
  pdl_wait();
  if (!in) return;
  const Partial* part = P.ws.part;
  Partial first[2];
  Vals<V> x[2];
  const bool pre = P.ws.status[1] != 0;
  first[0] = part[P.ws.pre + item];
  first[1] = part[P.ws.own + item];
  x[0] = load_vals<V>(P.ws.o + (P.ws.pre + item) * D + lane * V);
  x[1] = load_vals<V>(P.ws.o + (P.ws.own + item) * D + lane * V);
  if (!pre) first[0] = Partial{-INFINITY, 0.f, 0, 0};
  if (!own) first[1] = Partial{-INFINITY, 0.f, 0, 0};
  float M = max_or_nan(first[0].m, first[1].m), L = 0.f, acc[V] = {};
  if (M != -INFINITY) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float w = first[i].m == -INFINITY ? 0.f : exp2f(first[i].m - M);
      if (w != 0.f) {  // (what was not written may hold anything)
        L += w * first[i].l;
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] += w * x[i].v[v];
      }
    }
  }
  const int most = 2 * P.ctas;  // (a wrong cu_rows must not lead out of the workspace)
  const int n0 = clampi(first[0].more >> 1, 0, most), n = n0 + clampi(first[1].more >> 1, 0, most);
  for (int a = 0; a < n; a += N) {
    const int e = a + lane, k0 = e < n0 ? e : e - n0;
    const int kind = (e < n0 ? first[0].more : first[1].more) & 1;
    const int64_t c = (e < n0 ? first[0].carry : first[1].carry) +
                      static_cast<int64_t>(k0 + 1) * (kind == kPair ? 256 : 128);
    const bool ok = e < n && c >= 0 && c < 512ll * P.ctas;
    const int64_t at = P.ws.carry + (ok ? c : 0);
    Partial mine{-INFINITY, 0.f, 0, 0};
    if (ok) mine = part[at];
    float top = mine.m;
#pragma unroll
    for (int o = N / 2; o; o >>= 1) top = max_or_nan(top, __shfl_xor_sync(lanes, top, o));
    top = max_or_nan(top, M);
    if (top == -INFINITY) continue;
    const float old = exp2f(M - top), w = mine.m == -INFINITY ? 0.f : exp2f(mine.m - top);
    float sum = w * mine.l;
#pragma unroll
    for (int o = N / 2; o; o >>= 1) sum += __shfl_xor_sync(lanes, sum, o);
    L = L * old + sum;
    M = top;
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] *= old;
    const int cnt = min(N, n - a);
    for (int k = 0; k < cnt; k += kAtOnce) {  // that many rows on their way at once
      Vals<V> y[kAtOnce];
      float f[kAtOnce];
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        f[u] = __shfl_sync(lanes, w, (k + u) & (N - 1), N);
        const int64_t p = __shfl_sync(lanes, at, (k + u) & (N - 1), N);
        if (k + u >= cnt) f[u] = 0.f;
        y[u] = load_vals<V>(P.ws.o + p * D + lane * V);
      }
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u)
        if (f[u] != 0.f)
#pragma unroll
          for (int v = 0; v < V; ++v) acc[v] += f[u] * y[u].v[v];
    }
  }
  const float inv = L != 0.f ? 1.f / L : 0.f;  // no key, or NaN as it comes
  uint32_t out[V / 2];
#pragma unroll
  for (int v = 0; v < V; v += 2) out[v >> 1] = Types<T>::pack(acc[v] * inv, acc[v + 1] * inv);
  const int hq = static_cast<int>(item) - tok * Hq;
  // From the order of the partial results (see softmax: of 16 pairs of columns, pair
  // 4 i + c lies in place 4 c + i) to that of the columns.
  uint32_t cols[V / 2];
#pragma unroll
  for (int v = 0; v < V / 2; ++v) {
    const int pair = lane * (V / 2) + v, place = (pair & ~15) + (pair & 3) * 4 + ((pair >> 2) & 3);
#pragma unroll
    for (int k = 0; k < V / 2; ++k) {
      const uint32_t x = __shfl_sync(lanes, out[k], place / (V / 2), N);
      if (place % (V / 2) == k) cols[v] = x;
    }
  }
  T* dst = static_cast<T*>(io.out) + tok * io.out_stride + hq * D + lane * V;
  if (V == 8) *reinterpret_cast<uint4*>(dst) = make_uint4(cols[0], cols[V / 8], cols[V / 4], cols[V / 2 - 1]);
  else if (V == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(cols[0], cols[V / 2 - 1]);
  else *reinterpret_cast<uint32_t*>(dst) = cols[0];
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
  s->pre = 0;
  s->own = heads;
  s->carry = 2 * heads;
  const int64_t rows = s->carry + 2 * ctas * 256ll;
  int64_t at = 0;
  s->status = reinterpret_cast<uint32_t*>(base);
  at = 256;
  s->part = reinterpret_cast<Partial*>(base + at);
  at = align256(at + rows * static_cast<int64_t>(sizeof(Partial)));
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

template <class T, int D, bool kTest = false>
mk_status launch_attn(const AttnParams& A, const CUtensorMap& q, const CUtensorMap& q64,
                      const CUtensorMap& k, const CUtensorMap& v, int device, cudaStream_t s) {
  constexpr int smem = sizeof(TileSmem<D>) + 1024;
  // (once per device: it takes as long as a launch)
  static std::atomic<uint64_t> ready{0};
  const uint64_t bit = device < 64 ? uint64_t{1} << device : 0;
  if (!(ready.load(std::memory_order_relaxed) & bit)) {
    MK_CUDA_TRY(cudaFuncSetAttribute(k_attn_tiles<T, D, kTest>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
    MK_CUDA_TRY(cudaFuncSetAttribute(k_attn_merge<T, D, 32>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMergeSmem));
    MK_CUDA_TRY(cudaFuncSetAttribute(k_attn_merge<T, D, 16>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMergeSmem));
    ready.fetch_or(bit, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t lc = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = attr;
  lc.numAttrs = 1;
  lc.stream = s;
  lc.gridDim = dim3(A.ctas);
  lc.blockDim = dim3(kTileThreads);
  lc.dynamicSmemBytes = smem;
  MK_CUDA_TRY(cudaLaunchKernelEx(&lc, k_attn_tiles<T, D, kTest>, A, q, q64, k, v));
  const int64_t items = static_cast<int64_t>(A.io.n_rows) * A.io.n_q_heads;
  const int n = items > 32ll * A.ctas ? 16 : 32;
  lc.gridDim = dim3(static_cast<unsigned>((items * n + kMergeThreads - 1) / kMergeThreads));
  lc.blockDim = dim3(kMergeThreads);
  // (shared memory that nobody uses: no SM takes more than its share of the CTAs)
  const int share = static_cast<int>((lc.gridDim.x + A.ctas - 1) / A.ctas);
  lc.dynamicSmemBytes = share < kMergePerSm ? kMergeSmem / share - 1024 : 0;
  if (n == 32) MK_CUDA_TRY(cudaLaunchKernelEx(&lc, k_attn_merge<T, D, 32>, A));
  else MK_CUDA_TRY(cudaLaunchKernelEx(&lc, k_attn_merge<T, D, 16>, A));
  return MK_OK;
}

// What a self-test sets about the waits.
struct Waits {
  uint64_t ns;
  int32_t withhold, which;
};

mk_status attn(const mk_prefix_attn_io* io, void* workspace, int64_t workspace_bytes, void* stream,
               const Waits* test) {
  mk_status st = check_shapes(io);
  if (st != MK_OK) return st;
  const int64_t P = io->page_size, cap = static_cast<int64_t>(io->max_pages) * P;
  if (P < 16 || P > 65536 || (P & (P - 1))) return MK_ERR_UNSUPPORTED;
  if (io->n_pages < 0 || io->n_pages * P > INT32_MAX || io->prefix_len < 0 || io->max_pages < 0 ||
      io->table_stride < io->max_pages || io->window < 0)
    return MK_ERR_INVALID_ARG;
  if (cap + io->prefix_len > INT32_MAX - 256) return MK_ERR_INVALID_ARG;
  if (!(io->scale >= 0.f && io->scale <= FLT_MAX / 2)) return MK_ERR_INVALID_ARG;
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
  AttnParams A;
  A.io = *io;
  A.wait_ns = test ? test->ns : kWaitNs;
  A.withhold = test ? test->withhold : kNothing;
  A.withhold_at = test ? test->which : 0;
  A.group = io->n_q_heads / io->n_kv_heads;
  A.tile_tok = 128 / A.group;
  A.half_tok = 64 / A.group;
  A.by_pair = make_divisor(2 * A.tile_tok);
  A.by_heads = make_divisor(io->n_kv_heads);
  // the longest that the lines of work can be, by the capacity of the tables
  const int64_t pairs = io->n_rows / (2 * A.tile_tok) + 1;
  const int64_t own = pairs + std::min(io->n_requests, io->n_rows);
  const int64_t kt = (io->prefix_len + kTileKeys - 1) / kTileKeys, own_kt = (cap + kTileKeys - 1) / kTileKeys;
  int unit = 0;
  for (;; ++unit) {
    int64_t t = 1, i = 1;
    for (int k = 0; k < 2; ++k) {
      A.tile_cost[k] = std::max(1, kTileCost[k] >> unit);
      A.item_cost[k] = std::max(1, kItemCost[k] >> unit);
      t = std::max<int64_t>(t, A.tile_cost[k]);
      i = std::max<int64_t>(i, A.item_cost[k]);
    }
    const double most = static_cast<double>(io->n_kv_heads) *
                        (static_cast<double>(pairs) * (kt * t + i) + static_cast<double>(own) * (own_kt * t + i));
    if (most < 1 << 29) break;
    if (unit == 3) return MK_ERR_UNSUPPORTED;
  }
  int device = 0;
  st = check_device(workspace, &device, &A.ctas);
  if (st != MK_OK) return st;
  A.by_ctas = make_divisor(A.ctas);
  for (int k = 0; k < 2; ++k) A.by_cost[k] = make_divisor(A.tile_cost[k]);
  if (workspace_bytes < lay_out(io, A.ctas, static_cast<uint8_t*>(workspace), &A.ws))
    return MK_ERR_INVALID_ARG;
  if (io->n_rows == 0) {
    MK_CUDA_TRY(cudaMemsetAsync(A.ws.status, 0, sizeof(uint32_t), static_cast<cudaStream_t>(stream)));
    return MK_OK;
  }
  const float scale = io->scale != 0.f ? io->scale : 1.f / std::sqrt(static_cast<float>(io->head_dim));
  A.scale_log2 = scale * 1.4426950408889634f;
  A.box = static_cast<int>(std::min<int64_t>(P, kTileKeys));
  A.box_shift = __builtin_ctz(kTileKeys / A.box);
  A.page_shift = __builtin_ctz(static_cast<uint32_t>(P));
  const uint64_t d = io->head_dim, Hq = io->n_q_heads, Hk = io->n_kv_heads;
  CUtensorMap q, q64, k, v;
  st = encode_tmap_3d(&q, io->dtype, io->q, d, Hq, io->n_rows, d * 2, io->q_stride * 2, A.group, A.tile_tok);
  if (st != MK_OK) return st;
  st = encode_tmap_3d(&q64, io->dtype, io->q, d, Hq, io->n_rows, d * 2, io->q_stride * 2, A.group, A.half_tok);
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
  if (test) return launch_attn<__nv_bfloat16, 64, true>(A, q, q64, k, v, device, s);
  if (io->dtype == MK_BF16)
    return io->head_dim == 128 ? launch_attn<__nv_bfloat16, 128>(A, q, q64, k, v, device, s)
                               : launch_attn<__nv_bfloat16, 64>(A, q, q64, k, v, device, s);
  return io->head_dim == 128 ? launch_attn<__half, 128>(A, q, q64, k, v, device, s)
                             : launch_attn<__half, 64>(A, q, q64, k, v, device, s);
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
  return attn(io, workspace, workspace_bytes, stream, nullptr);
}

mk_status mk_selftest_attn_waits(const mk_prefix_attn_io* io, void* workspace, int64_t workspace_bytes,
                                 uint64_t wait_ns, int32_t withhold, int32_t which, void* stream) {
  if (!io || !wait_ns || wait_ns > kWaitNs || withhold < kNothing || withhold > kBuffers || which < 0)
    return MK_ERR_INVALID_ARG;
  if (io->dtype != MK_BF16 || io->head_dim != 64) return MK_ERR_UNSUPPORTED;
  const Waits w{wait_ns, withhold, which};
  const mk_status st = attn(io, workspace, workspace_bytes, stream, &w);
  if (st != MK_OK) return st;
  MK_CUDA_TRY(cudaStreamSynchronize(static_cast<cudaStream_t>(stream)));
  return mk_prefix_attn_status(workspace);
}

mk_status mk_prefix_attn_status(const void* workspace) {
  if (!workspace) return MK_ERR_INVALID_ARG;
  uint32_t s = 0;
  MK_CUDA_TRY(cudaMemcpy(&s, workspace, sizeof(s), cudaMemcpyDeviceToHost));
  return s == 0 ? MK_OK : s == kFalling ? MK_ERR_INVALID_ARG : MK_ERR_TIMEOUT;
}

}  // extern "C"
