// linear.cu -- projection with bias, activation and residual (mk_linear), on the
// 5th-generation tensor cores.
//
//   out^T = act(w x^T + bias) + residual^T
// in tiles of 128 outputs (the rows of tensor memory) by up to 256 rows of x (its
// columns), over blocks of 64 inputs that TMA brings into a ring of stages.  With
// the weights as the first operand a call with few rows wastes no tensor core rows
// on them, and reads every weight once; a result's bias is a thread's own.
//
// Few tiles: a cluster of CTAs shares a tile's inputs, each with a range of them;
// their sums meet in distributed shared memory, where each CTA adds up a part of
// the rows in the order of the ranks.  Many tiles: one CTA per SM works through
// them, the tensor cores on the next tile while the last one's results leave.
//
// What bounds it: 4096 rows, 4096 -> 12288, SiLU: 217 to 229 us, 1.8 to 1.9 PFLOP/s, the tensor
// cores.  64 rows, 4096 -> 6144: 14.5 us, of which 50 MB of weights take 9; 250 rows,
// 4096 -> 4096: 17.5 us, of which 6 go for what each SM takes in and 6 for the sums' way.
#include <algorithm>
#include <atomic>
#include <climits>

#include "../../include/mk_selftest.h"
#include "attn_ptx.cuh"
#include "batch.h"
#include "rope.h"

namespace mk {

namespace {

constexpr int kFeat = 128;        // outputs of a tile
constexpr int kBlock = 64;        // inputs of a block: 128 bytes, the width of the swizzle
constexpr int kMaxStages = 12;
constexpr int kOutWarps = 8;      // of results: two to 32 outputs, for every other 16 rows
constexpr int kThreads = 32 * (2 + kOutWarps);  // producer, MMA issuer, these
constexpr uint64_t kWaitNs = 2000ull * 1000 * 1000;
constexpr uint32_t kTimeout = 1;
constexpr int kSmem = 222 * 1024;  // of a CTA, at most
// At least: more than half of an SM's, so that no two CTAs are on one. Clusters and pairs
// take tensor memory on several SMs, and each of two might wait for what the other holds.
constexpr int kSmemLeast = 120 * 1024;

// Hand-offs that a self-test withholds, so that waits run out: copies from a block on, a
// stage after use, a tile's sums, a tile's columns after use.
enum Withhold { kNothing = 0, kCopies = 1, kStage = 2, kSums = 3, kColumns = 4 };

struct LinearParams {
  mk_linear_io io;
  uint32_t* status;
  int32_t cols;        // N: rows of x per tile, a multiple of 16
  int32_t row_tiles;   // tiles along the rows of x
  int32_t tiles;       // all tiles
  int32_t blocks;      // of inputs
  int32_t split;       // CTAs (pairs of CTAs) per tile
  int32_t pair;        // a tile is 256 outputs, of two CTAs
  int32_t stages;
  int32_t tmem_cols;   // allocated; two tiles' where a CTA has several
  uint32_t idesc;
  int32_t vec;         // out and residual take four values at a time
  // of a self-test: limit of a wait; which hand-off to withhold, the how manieth, and of
  // a pair in which CTA
  uint64_t wait_ns;
  int32_t withhold, withhold_at, withhold_half;
};

struct LinearBars {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t drained;
  uint32_t tmem, abort;
  int32_t loads;  // blocks that the producer has brought
};

// y = act(y) of N values (the choice outside of the loop, so that their chains overlap).
template <int N>
MK_DEV void activate(float (&y)[N], int act) {
  if (act == MK_ACT_SILU) {
#pragma unroll
    for (int i = 0; i < N; ++i) y[i] = __fdividef(y[i], 1.f + __expf(-y[i]));
  } else if (act == MK_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      // y (1 + erf(y / sqrt 2)) / 2 = max(y, 0) - |y| erfc(x) / 2 with x = |y| / sqrt 2, and
      // erfc(x) e^(x^2) / 2 as t times a polynomial in t = 1 / (1 + 0.45 x), of the least
      // relative error up to x = 9.6: it alternates nine times between +-2^-21.5, with the
      // rounding 2^-18.9 for y > -6.
      // (2935 rows, 360 -> 10456: 59 us, with erff, whose ranges
      // diverge, 72.)
      const float a = fminf(fabsf(y[i]), 15.f), t = __fdividef(1.f, fmaf(a, 0.31819805f, 1.f));
      float q = 0.033216566f;
      q = fmaf(q, t, -0.119189195f);
      q = fmaf(q, t, 0.10271385f);
      q = fmaf(q, t, 0.021787712f);
      q = fmaf(q, t, 0.09341932f);
      q = fmaf(q, t, 0.11432297f);
      q = fmaf(q, t, 0.12677133f);
      q = fmaf(q, t, 0.1269576f);
      const float tail = (y[i] < 0.f ? -y[i] : a) * (q * t * exp2_approx(a * a * -0.72134752f));
      y[i] = (y[i] < 0.f ? 0.f : y[i]) - tail;
    }
  } else if (act == MK_ACT_GELU_TANH) {
#pragma unroll
    for (int i = 0; i < N; ++i) {  // (1 + tanh u) / 2 = 1 / (1 + e^-2u)
      const float u = 0.7978845608028654f * fmaf(0.044715f * y[i] * y[i], y[i], y[i]);
      y[i] = __fdividef(y[i], 1.f + __expf(-2.f * u));
    }
  }
}

// Pairs of CTAs: each holds half of a tile's outputs and brings half of the rows of x;
// the first one's issuer multiplies for both.
MK_DEV uint32_t address_in(const void* p, uint32_t rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
// Bounded wait: false once any wait of the CTA, or of another one of its cluster, has run
// out: they wait for one another, and none reads the sums of one that gave up.
template <bool kTest>
MK_DEV bool wait_bar(const LinearParams& P, LinearBars& B, uint64_t* bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (*const_cast<volatile uint32_t*>(&B.abort)) return false;
    if (globaltimer() - t0 > (kTest ? P.wait_ns : kWaitNs)) {
      uint32_t ctas;
      asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ctas));
      for (uint32_t r = 0; r < ctas; ++r)
        asm volatile("st.relaxed.cluster.shared::cluster.u32 [%0], %1;" ::"r"(address_in(&B.abort, r)), "r"(1u) : "memory");
      atomicExch(P.status, kTimeout);
      return false;
    }
  }
}
template <bool kTest>
MK_DEV bool withheld(const LinearParams& P, int what, int at, int half) {
  return kTest && P.withhold == what && P.withhold_at == at && P.withhold_half == half;
}

template <bool PAIR>
MK_DEV void load_box(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, uint64_t policy, uint32_t leader) {
  if (!PAIR) {
    tma_load_2d(dst, map, bar, x, y, policy);
    return;
  }
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
      ".L2::cache_hint [%0], [%1, {%3, %4}], [%2], %5;" ::"r"(smem_u32(dst)),
      "l"(map), "r"(address_in(bar, leader)), "r"(x), "r"(y), "l"(policy)
      : "memory");
}
template <bool PAIR>
MK_DEV void multiply(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  if (!PAIR) {
    mma_bf16(d_tmem, adesc, bdesc, idesc, accumulate);
    return;
  }
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrives on `bar` (of both CTAs of a pair, whose ranks `mask` names) when the products
// issued so far are done.
template <bool PAIR>
MK_DEV void commit(uint64_t* bar, uint32_t mask) {
  if (!PAIR) {
    mma_commit(bar);
    return;
  }
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"(static_cast<uint16_t>(mask))
      : "memory");
}
template <bool PAIR>
MK_DEV void alloc_columns(uint32_t* to, uint32_t cols) {
  if (!PAIR) {
    tmem_alloc(to, cols);
    tmem_relinquish();
    return;
  }
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(to)), "r"(cols) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
template <bool PAIR>
MK_DEV void free_columns(uint32_t at, uint32_t cols) {
  if (!PAIR) tmem_dealloc(at, cols);
  else asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(cols) : "memory");
}
MK_DEV void arrive_at(uint32_t bar) {
  // (relaxed: tensor memory has been read, and the arrival need not wait for what the
  // thread has stored elsewhere: 2935 rows, 360 -> 10456, 46.5 us without, 42.6 with)
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Bytes of copies that do not come, as if they had.
MK_DEV void complete_bytes(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}

MK_DEV void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");
}
MK_DEV int32_t load_cluster_word(const int32_t* p, uint32_t rank) {
  int32_t v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(address_in(p, rank)) : "memory");
  return v;
}
MK_DEV float4 load_cluster(uint32_t addr, uint32_t rank) {
  uint32_t a;
  float4 v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(a)
               : "memory");
  return v;
}

MK_DEV void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// Of a split tile: adds up the ranks' sums of rows c0 .. c1-1 (four outputs per
// lane, a row per warp at a time, kRows rows on their way) and writes the results.
template <class T, bool VEC>
MK_DEV void join_sums(const LinearParams& P, uint32_t sums, int feat0, int row0, int c0, int c1, int half) {
  constexpr int kRows = 4, kWarps = kThreads / 32;
  const mk_linear_io& io = P.io;
  const int warp = threadIdx.x / 32, feat = feat0 + static_cast<int>(lane_id()) * 4;
  const int mine = min(4, io.n_out - feat);  // outputs of this lane
  float bias[4] = {};
  if (io.bias)
    for (int j = 0; j < mine; ++j) bias[j] = static_cast<float>(static_cast<const T*>(io.bias)[feat + j]);
  for (int col = c0 + warp; col < c1; col += kRows * kWarps) {
    float4 y[kRows];
    float r[kRows][4];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int at = col + i * kWarps;
      const T* res = static_cast<const T*>(io.residual) + static_cast<int64_t>(row0 + at) * io.residual_stride + feat;
      const bool there = io.residual && at < c1;
      if (VEC) {
        uint2 w = make_uint2(0, 0);
        if (there && mine == 4) w = *reinterpret_cast<const uint2*>(res);
        const float2 a = Pack<T>::get(w.x), b = Pack<T>::get(w.y);
        r[i][0] = a.x, r[i][1] = a.y, r[i][2] = b.x, r[i][3] = b.y;
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) r[i][j] = there && j < mine ? static_cast<float>(res[j]) : 0.f;
      }
      y[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int k = 0; k < P.split; ++k)
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const float4 v = load_cluster(sums + min(col + i * kWarps, c1 - 1) * (kFeat * 4) + lane_id() * 16, P.pair ? 2 * k + half : k);
        y[i].x += v.x, y[i].y += v.y, y[i].z += v.z, y[i].w += v.w;
      }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int at = col + i * kWarps;
      if (at >= c1) continue;
      T* out = static_cast<T*>(io.out) + static_cast<int64_t>(row0 + at) * io.out_stride + feat;
      float z[4] = {y[i].x + bias[0], y[i].y + bias[1], y[i].z + bias[2], y[i].w + bias[3]};
      activate(z, io.act);
#pragma unroll
      for (int j = 0; j < 4; ++j) z[j] += r[i][j];
      if (VEC) {
        if (mine == 4) *reinterpret_cast<uint2*>(out) = make_uint2(Pack<T>::put(z[0], z[1]), Pack<T>::put(z[2], z[3]));
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (j < mine) out[j] = static_cast<T>(z[j]);
      }
    }
  }
}

template <class T, bool PAIR, bool kTest>
__global__ void __launch_bounds__(kThreads, 1)
    k_linear(const __grid_constant__ LinearParams P, const __grid_constant__ CUtensorMap wmap,
             const __grid_constant__ CUtensorMap xmap) {
  extern __shared__ uint8_t raw_smem[];
  __shared__ LinearBars B;
  const mk_linear_io& io = P.io;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw_smem) + 1023) & ~uintptr_t{1023});
  const int warp = threadIdx.x / 32, lane = lane_id();
  constexpr int kCtas = PAIR ? 2 : 1, kTileFeat = kFeat * kCtas;
  const int x_rows = P.cols / kCtas;  // that this CTA brings
  const uint32_t stage_bytes = kFeat * 128 + x_rows * 128;
  const int in_cluster = blockIdx.x % (P.split * kCtas), rank = in_cluster / kCtas, half = in_cluster % kCtas;
  const uint32_t leader = in_cluster - half, both = 3u << leader;
  const int first = blockIdx.x / (P.split * kCtas), step = gridDim.x / (P.split * kCtas);
  // this CTA's blocks of every tile
  const int k0 = static_cast<int>(static_cast<int64_t>(P.blocks) * rank / P.split);
  const int k1 = static_cast<int>(static_cast<int64_t>(P.blocks) * (rank + 1) / P.split);
  const int acc_cols = P.cols <= 32 ? 32 : P.cols <= 64 ? 64 : P.cols <= 128 ? 128 : 256;

  if (warp == 0 && elect_one()) {
    prefetch_tensormap(&wmap);
    prefetch_tensormap(&xmap);
    for (int i = 0; i < P.stages; ++i) mbar_init(&B.full[i], 1), mbar_init(&B.empty[i], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&B.acc_full[i], 1), mbar_init(&B.acc_empty[i], kOutWarps * kCtas);
    mbar_init(&B.drained, 1);
    B.abort = 0;
    fence_mbar_init();
  }
  __syncwarp();
  if (PAIR) cluster_sync();  // (barriers that the other CTA arrives at)
  if (warp == 1) {
    alloc_columns<PAIR>(&B.tmem, P.tmem_cols);
    // (not before: a dependent grid that took the columns first would wait for this one,
    // which would wait for the columns)
    pdl_launch_dependents();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = B.tmem;
  pdl_wait();
  if (blockIdx.x == 0 && threadIdx.x == 0) *P.status = 0;

  if (warp == 0) {
    if (elect_one()) {
      const uint64_t keep = policy_evict_normal(), once = P.row_tiles == 1 ? policy_evict_first() : keep;
      bool ok = true;
      int loads = 0;
      for (int tile = first; tile < P.tiles && ok; tile += step) {
        const int f = tile / P.row_tiles * kTileFeat + half * kFeat, r = tile % P.row_tiles * P.cols + half * x_rows;
        for (int k = k0; k < k1; ++k, ++loads) {
          const int st = loads % P.stages, round = loads / P.stages;
          ok = !withheld<kTest>(P, kCopies, loads, half) &&
               (!round || wait_bar<kTest>(P, B, &B.empty[st], (round - 1) & 1));
          if (!ok) break;
          uint8_t* a = smem + st * stage_bytes;
          if (half == 0) mbar_arrive_expect_tx(&B.full[st], stage_bytes * kCtas);
          load_box<PAIR>(a, &wmap, &B.full[st], k * kBlock, f, once, leader);
          load_box<PAIR>(a + kFeat * 128, &xmap, &B.full[st], k * kBlock, r, keep, leader);
        }
      }
      // (what the first CTA's products say about the second one's stages comes before that
      // one leaves)
      for (int i = max(0, loads - P.stages); PAIR && i < loads && ok; ++i)
        ok = wait_bar<kTest>(P, B, &B.empty[i % P.stages], (i / P.stages) & 1);
      B.loads = loads;
    }
    __syncwarp();
  } else if (warp == 1) {
    if (half == 0 && elect_one()) {
      bool ok = true;
      int used = 0, n = 0;
      for (int tile = first; tile < P.tiles && ok; tile += step, ++n) {
        const int buf = n & 1;
        if (n >= 2 && !wait_bar<kTest>(P, B, &B.acc_empty[buf], ((n >> 1) - 1) & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        for (int k = k0; k < k1; ++k, ++used) {
          const int st = used % P.stages;
          if (!wait_bar<kTest>(P, B, &B.full[st], (used / P.stages) & 1)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a = smem_u32(smem + st * stage_bytes);
          const uint64_t ad = sdesc_kmajor_sw128(a), bd = sdesc_kmajor_sw128(a + kFeat * 128);
#pragma unroll
          for (int i = 0; i < kBlock / 16; ++i)  // 16 inputs: 32 bytes on in the swizzled rows
            multiply<PAIR>(tmem + buf * acc_cols, ad + 2 * i, bd + 2 * i, P.idesc, k > k0 || i > 0);
          if (!withheld<kTest>(P, kStage, used, 0)) commit<PAIR>(&B.empty[st], both);
        }
        if (ok && !withheld<kTest>(P, kSums, n, 0)) commit<PAIR>(&B.acc_full[buf], both);
      }
    }
    __syncwarp();
  } else {
    const int quad = warp & 3, col0 = (warp - 2) / 4 * 16;
    const uint32_t lane_at = static_cast<uint32_t>(quad * 32) << 16;
    int n = 0;
    bool ok = true;
    float* sums = reinterpret_cast<float*>(smem);  // of a split tile: [cols][128]
    for (int tile = first; tile < P.tiles; tile += step, ++n) {
      const int buf = n & 1;
      const int feat = tile / P.row_tiles * kTileFeat + half * kFeat + quad * 32 + lane;
      const int row0 = tile % P.row_tiles * P.cols, rows = min(P.cols, io.n_rows - row0);
      const bool mine = feat < io.n_out;
      const float bias = io.bias && mine ? static_cast<float>(static_cast<const T*>(io.bias)[feat]) : 0.f;
      const T* res = static_cast<const T*>(io.residual) + static_cast<int64_t>(row0) * io.residual_stride + feat;
      T* out = static_cast<T*>(io.out) + static_cast<int64_t>(row0) * io.out_stride + feat;
      // (the residual of the columns behind the next ones is on its way)
      T ahead[2][16];
      auto fetch = [&](int col, T (&to)[16]) {
        if (!io.residual || P.split > 1) return;
#pragma unroll
        for (int i = 0; i < 16; ++i)
          to[i] = mine && col + i < rows ? res[static_cast<int64_t>(col + i) * io.residual_stride] : static_cast<T>(0.f);
      };
      // (the next tile's on its way into L2, as the loads here keep few bytes in flight)
      if (io.residual && P.split == 1) {
        for (int to = n ? tile + step : tile; to <= tile + step && to < P.tiles; to += step) {
          const int f = to / P.row_tiles * kTileFeat + half * kFeat, r = to % P.row_tiles * P.cols;
          const char* from = static_cast<const char*>(io.residual) + (static_cast<int64_t>(r) * io.residual_stride + f) * 2;
          const int bytes = min(kFeat, io.n_out - f) * 2, count = min(P.cols, io.n_rows - r);
          for (int i = threadIdx.x - 64; i < 2 * count; i += kOutWarps * 32)
            if ((i & 1) * 128 < bytes) prefetch_l2(from + (i >> 1) * io.residual_stride * 2 + (i & 1) * 128);
        }
      }
      fetch(col0, ahead[0]);
      fetch(col0 + 32, ahead[1]);
      ok = __all_sync(0xffffffffu, wait_bar<kTest>(P, B, &B.acc_full[buf], (n >> 1) & 1));
      if (!ok) break;
      tc_fence_after();
      for (int col = col0; col < rows; col += 32) {
        float v[16], r[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          r[i] = static_cast<float>(ahead[0][i]);
          ahead[0][i] = ahead[1][i];
        }
        fetch(col + 64, ahead[1]);
        tmem_ld16(tmem + lane_at + buf * acc_cols + col, v);
        if (P.split > 1) {
#pragma unroll
          for (int i = 0; i < 16; ++i) sums[(col + i) * kFeat + quad * 32 + lane] = v[i];
          continue;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] += bias;
        activate(v, io.act);
        if (io.residual)
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] += r[i];
        T* to = out + static_cast<int64_t>(col) * io.out_stride;
        if (mine && col + 16 <= rows) {
#pragma unroll
          for (int i = 0; i < 16; ++i, to += io.out_stride) *to = static_cast<T>(v[i]);
        } else if (mine) {
          for (int i = 0; i < 16; ++i, to += io.out_stride)
            if (col + i < rows) *to = static_cast<T>(v[i]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0 && !withheld<kTest>(P, kColumns, n, half)) {
        if (half == 0) mbar_arrive(&B.acc_empty[buf]);
        else arrive_at(address_in(&B.acc_empty[buf], leader));
      }
      __syncwarp();
    }
  }
  // Every warp of the CTA, of the whole cluster, is through: whether any of them gave up
  // is settled, and the same in all of them.
  const bool cluster = PAIR || P.split > 1;
  auto meet = [&] {
    __syncwarp();
    tc_fence_before();
    if (cluster) cluster_sync();
    else __syncthreads();
    tc_fence_after();
  };
  meet();
  const bool gave_up = *const_cast<volatile uint32_t*>(&B.abort) != 0;
  if (gave_up) {
    // Whichever wait it was, and whoever was done by then: no copy may land and no product
    // run on after the CTA has left.
    if (warp == 0 && half == 0 && elect_one()) {
      // (of a pair: this CTA's barriers count both CTAs' copies, and one may have brought
      // blocks, fewer than there are stages, that the other has not)
      const int mine = B.loads, other = PAIR ? load_cluster_word(&B.loads, leader + 1) : mine, most = max(mine, other);
      for (int i = max(0, most - P.stages); i < most; ++i) {
        uint64_t* bar = &B.full[i % P.stages];
        if (i >= mine) mbar_arrive_expect_tx(bar, stage_bytes);
        else if (i >= other) complete_bytes(bar, stage_bytes);
        mbar_wait_bounded(bar, (i / P.stages) & 1, kWaitNs);
      }
    }
    if (warp == 1) {
      if (half == 0 && elect_one()) commit<PAIR>(&B.drained, both);
      __syncwarp();
      mbar_wait_bounded(&B.drained, 0, kWaitNs);
    }
  } else if (P.split > 1) {
    // (a CTA of a cluster has one tile)
    const int feat0 = first / P.row_tiles * kTileFeat + half * kFeat;
    const int row0 = first % P.row_tiles * P.cols, rows = min(P.cols, io.n_rows - row0);
    const int c0 = rows * rank / P.split, c1 = rows * (rank + 1) / P.split;
    if (P.vec) join_sums<T, true>(P, smem_u32(smem), feat0, row0, c0, c1, half);
    else join_sums<T, false>(P, smem_u32(smem), feat0, row0, c0, c1, half);
  }
  // (no CTA leaves while another one reads its sums or its word, or copies into it)
  if (gave_up || P.split > 1) meet();
  __syncwarp();
  if (warp == 1) free_columns<PAIR>(tmem, P.tmem_cols);
}

// 2-D map over [rows][inner] 16-bit values, box of 64 x box_rows, 128-byte swizzle;
// what is out of range reads as zeros.
mk_status encode_tmap(CUtensorMap* map, int dtype, const void* base, uint64_t inner, uint64_t rows, int64_t stride,
                      uint32_t box_rows) {
  PFN_encodeTiled fn = get_encode_fn();
  if (!fn) return MK_ERR_CUDA;
  cuuint64_t dims[2] = {inner, rows};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(stride) * 2};
  cuuint32_t box[2] = {kBlock, box_rows};
  cuuint32_t estr[2] = {1, 1};
  const CUresult r = fn(map, dtype == MK_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
                        const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? MK_OK : MK_ERR_INVALID_ARG;
}

// How many clusters of 2 .. 8 CTAs, one CTA per SM, run at the same time: less than
// the SMs divided by their size, as a cluster's SMs lie side by side.
template <class T, bool kTest>
mk_status max_clusters(int device, int sms, int (&most)[9]) {
  static std::atomic<int> known[64][9];
  for (int c = 1; c <= 8; ++c) {
    int n = c == 1 ? sms : device < 64 ? known[device][c].load(std::memory_order_relaxed) : 0;
    if (n == 0) {
      cudaLaunchConfig_t lc = {};
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = c;
      attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
      lc.attrs = attr;
      lc.numAttrs = 1;
      lc.gridDim = dim3(c * sms);
      lc.blockDim = dim3(kThreads);
      lc.dynamicSmemBytes = kSmem;
      MK_CUDA_TRY(cudaOccupancyMaxActiveClusters(&n, k_linear<T, false, kTest>, &lc));
      if (device < 64) known[device][c].store(n, std::memory_order_relaxed);
    }
    most[c] = n;
  }
  return MK_OK;
}

int columns_of(int cols) { return cols <= 32 ? 32 : cols <= 64 ? 64 : cols <= 128 ? 128 : 256; }

// Sizes of the tiles and how many CTAs share one; returns how many CTAs work.
int choose(LinearParams* P, const int (&most)[9], int ctas) {
  const int64_t m = P->io.n_rows, n = P->io.n_out;
  const int64_t row_tiles = (m + 255) / 256, each = (m + row_tiles - 1) / row_tiles;
  const int unit = 16 * ctas, feat = kFeat * ctas;
  P->pair = ctas == 2;
  P->blocks = (P->io.n_in + kBlock - 1) / kBlock;
  P->cols = static_cast<int32_t>((each + unit - 1) / unit * unit);
  P->row_tiles = static_cast<int32_t>((m + P->cols - 1) / P->cols);
  P->tiles = P->row_tiles * static_cast<int32_t>((n + feat - 1) / feat);
  // as many CTAs per tile as run at the same time, of four blocks at least
  P->split = 1;
  for (int s = 2; s * ctas <= 8; ++s)
    if (P->tiles <= most[s * ctas] && P->blocks >= 4 * s) P->split = s;
  const int stage = (kFeat + P->cols / ctas) * 128;
  P->stages = std::min({kMaxStages, (kSmem - 1024) / stage, std::max(2, P->blocks / P->split + 1)});
  P->tmem_cols = 2 * columns_of(P->cols);
  return ctas * std::min(P->tiles * P->split, most[ctas]);
}

// With more than 128 rows what a CTA copies per block, its weights and all rows, takes
// longer than its products: a pair halves the rows (4096 rows, 4096 -> 12288: 264 us,
// with pairs 223).  Few tiles do better one by one if that keeps more CTAs busy, a
// quarter more (250 rows, 4096 -> 4096: 128 CTAs 17.1 us, 48 pairs 18.8).
void choose(LinearParams* P, const int (&most)[9]) {
  const int single = choose(P, most, 1);
  if (P->cols <= 128 || P->io.n_out <= kFeat) return;
  if (choose(P, most, 2) * 5 < single * 4) choose(P, most, 1);
}

template <class T, bool PAIR, bool kTest>
mk_status launch(const LinearParams& P, const CUtensorMap& w, const CUtensorMap& x, const int (&most)[9],
                 cudaStream_t s) {
  constexpr int kCtas = PAIR ? 2 : 1;
  cudaLaunchConfig_t lc = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = P.split * kCtas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  lc.attrs = attr;
  lc.numAttrs = P.split * kCtas > 1 ? 2 : 1;
  lc.stream = s;
  lc.gridDim = dim3(P.split > 1 ? P.tiles * P.split * kCtas : std::min(P.tiles, most[kCtas]) * kCtas);
  lc.blockDim = dim3(kThreads);
  // (a split tile's sums lie where the stages were)
  lc.dynamicSmemBytes = std::max(P.stages * (kFeat + P.cols / kCtas) * 128, P.split > 1 ? P.cols * kFeat * 4 : 0) + 1024;
  lc.dynamicSmemBytes = std::max<size_t>(lc.dynamicSmemBytes, kSmemLeast);
  MK_CUDA_TRY(cudaLaunchKernelEx(&lc, k_linear<T, PAIR, kTest>, P, w, x));
  return MK_OK;
}

template <class T, bool kTest = false>
mk_status linear(LinearParams* P, int device, int sms, cudaStream_t s) {
  static std::atomic<uint64_t> ready{0};  // (once per device: it takes as long as a launch)
  const uint64_t bit = device < 64 ? uint64_t{1} << device : 0;
  if (!(ready.load(std::memory_order_relaxed) & bit)) {
    MK_CUDA_TRY(cudaFuncSetAttribute(k_linear<T, false, kTest>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem));
    MK_CUDA_TRY(cudaFuncSetAttribute(k_linear<T, true, kTest>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem));
    ready.fetch_or(bit, std::memory_order_relaxed);
  }
  int most[9] = {};
  mk_status st = max_clusters<T, kTest>(device, sms, most);
  if (st != MK_OK) return st;
  choose(P, most);
  const mk_linear_io& io = P->io;
  // M, N of a product; fp16 is type 0, bf16 type 1
  P->idesc = idesc_bf16(P->pair ? 2 * kFeat : kFeat, P->cols);
  if (io.dtype == MK_FP16) P->idesc &= ~((1u << 7) | (1u << 10));
  CUtensorMap w, x;
  st = encode_tmap(&w, io.dtype, io.w, io.n_in, io.n_out, io.w_stride, kFeat);
  if (st != MK_OK) return st;
  st = encode_tmap(&x, io.dtype, io.x, io.n_in, io.n_rows, io.x_stride, P->pair ? P->cols / 2 : P->cols);
  if (st != MK_OK) return st;
  return P->pair ? launch<T, true, kTest>(*P, w, x, most, s) : launch<T, false, kTest>(*P, w, x, most, s);
}

mk_status check_shapes(const mk_linear_io* io) {
  if (!io) return MK_ERR_INVALID_ARG;
  if (io->dtype != MK_BF16 && io->dtype != MK_FP16) return MK_ERR_UNSUPPORTED;
  if (io->n_rows < 0 || io->n_in < 1 || io->n_out < 1) return MK_ERR_INVALID_ARG;
  if (io->n_in % 8) return MK_ERR_UNSUPPORTED;
  // (tiles and outputs are counted in 32 bits)
  if (((io->n_rows + 255ll) / 256 + 1) * ((io->n_out + 127ll) / 128) > INT32_MAX || io->n_out > INT32_MAX - 256 ||
      io->n_rows > INT32_MAX - 256)
    return MK_ERR_UNSUPPORTED;
  if (io->act < MK_ACT_NONE || io->act > MK_ACT_GELU_TANH) return MK_ERR_INVALID_ARG;
  return MK_OK;
}

// What a self-test sets about the waits.
struct Waits {
  uint64_t ns;
  int32_t withhold, which, half;
};

mk_status call_linear(const mk_linear_io* io, void* workspace, int64_t workspace_bytes, void* stream,
                      const Waits* test) {
  mk_status st = check_shapes(io);
  if (st != MK_OK) return st;
  const int64_t m = io->n_rows, n = io->n_out, k = io->n_in;
  if (!io->w || !workspace) return MK_ERR_INVALID_ARG;
  if (io->x_stride % 8 || io->w_stride % 8 || io->w_stride < k) return MK_ERR_INVALID_ARG;
  if (misaligned(io->x, 16) || misaligned(io->w, 16) || misaligned(workspace, 256) || misaligned(io->bias, 2) ||
      misaligned(io->residual, 2) || misaligned(io->out, 2))
    return MK_ERR_INVALID_ARG;
  if (m) {
    if (!io->x || !io->out || io->x_stride < k || io->out_stride < n) return MK_ERR_INVALID_ARG;
    if (io->residual && io->residual_stride < n) return MK_ERR_INVALID_ARG;
    const int64_t to = span_bytes(m, n, io->out_stride, 2);
    const bool in_place = io->residual == io->out && (m == 1 || io->residual_stride == io->out_stride);
    struct Range { const void* p; int64_t n; };
    const Range in[] = {{io->x, span_bytes(m, k, io->x_stride, 2)}, {io->w, span_bytes(n, k, io->w_stride, 2)},
                        {io->bias, n * 2}, {io->residual, span_bytes(m, n, io->residual_stride, 2)}};
    for (int i = 0; i < 4; ++i) {
      if (!(i == 3 && in_place) && overlap(in[i].p, in[i].n, io->out, to)) return MK_ERR_INVALID_ARG;
      if (overlap(in[i].p, in[i].n, workspace, workspace_bytes)) return MK_ERR_INVALID_ARG;
    }
    if (overlap(io->out, to, workspace, workspace_bytes)) return MK_ERR_INVALID_ARG;
  }
  if (workspace_bytes < 256) return MK_ERR_INVALID_ARG;
  int device = 0, sms = 0;
  st = check_device(workspace, &device, &sms);
  if (st != MK_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (m == 0) {
    MK_CUDA_TRY(cudaMemsetAsync(workspace, 0, sizeof(uint32_t), s));
    return MK_OK;
  }
  LinearParams P;
  P.io = *io;
  P.status = static_cast<uint32_t*>(workspace);
  P.vec = n % 4 == 0 && io->out_stride % 4 == 0 && !misaligned(io->out, 8) &&
          (!io->residual || (io->residual_stride % 4 == 0 && !misaligned(io->residual, 8)));
  P.wait_ns = test ? test->ns : kWaitNs;
  P.withhold = test ? test->withhold : kNothing;
  P.withhold_at = test ? test->which : 0;
  P.withhold_half = test ? test->half : 0;
  if (test) return linear<__nv_bfloat16, true>(&P, device, sms, s);
  return io->dtype == MK_BF16 ? linear<__nv_bfloat16>(&P, device, sms, s) : linear<__half>(&P, device, sms, s);
}

}  // namespace

}  // namespace mk

using namespace mk;

extern "C" {

mk_status mk_linear_workspace(const mk_linear_io* io, int64_t* bytes) {
  if (!bytes) return MK_ERR_INVALID_ARG;
  *bytes = 0;
  const mk_status st = check_shapes(io);
  if (st != MK_OK) return st;
  *bytes = 256;
  return MK_OK;
}

mk_status mk_linear(const mk_linear_io* io, void* workspace, int64_t workspace_bytes, void* stream) {
  return call_linear(io, workspace, workspace_bytes, stream, nullptr);
}

mk_status mk_selftest_linear_waits(const mk_linear_io* io, void* workspace, int64_t workspace_bytes,
                                   uint64_t wait_ns, int32_t withhold, int32_t which, int32_t half, void* stream) {
  if (!io || !wait_ns || wait_ns > kWaitNs || withhold < kNothing || withhold > kColumns || which < 0 ||
      (half & ~1) || (half && (withhold == kStage || withhold == kSums)))
    return MK_ERR_INVALID_ARG;
  if (io->dtype != MK_BF16) return MK_ERR_UNSUPPORTED;
  const Waits w{wait_ns, withhold, which, half};
  const mk_status st = call_linear(io, workspace, workspace_bytes, stream, &w);
  if (st != MK_OK) return st;
  MK_CUDA_TRY(cudaStreamSynchronize(static_cast<cudaStream_t>(stream)));
  return mk_linear_status(workspace);
}

mk_status mk_linear_status(const void* workspace) {
  if (!workspace) return MK_ERR_INVALID_ARG;
  uint32_t s = 0;
  MK_CUDA_TRY(cudaMemcpy(&s, workspace, sizeof(s), cudaMemcpyDeviceToHost));
  return s == 0 ? MK_OK : MK_ERR_TIMEOUT;
}

}  // extern "C"
