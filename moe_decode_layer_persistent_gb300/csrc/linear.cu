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
#include <algorithm>
#include <atomic>
#include <climits>

#include "batch.h"
#include "rope.h"

namespace mk {

namespace {

constexpr int kFeat = 128;        // outputs of a tile
constexpr int kBlock = 64;        // inputs of a block: 128 bytes, the width of the swizzle
constexpr int kMaxStages = 12;
constexpr int kThreads = 192;     // producer, MMA issuer, four warps of results
constexpr uint64_t kWaitNs = 2000ull * 1000 * 1000;
constexpr uint32_t kTimeout = 1;

struct LinearParams {
  mk_linear_io io;
  uint32_t* status;
  int32_t cols;        // N: rows of x per tile, a multiple of 16
  int32_t row_tiles;   // tiles along the rows of x
  int32_t tiles;       // all tiles
  int32_t blocks;      // of inputs
  int32_t split;       // CTAs per tile
  int32_t stages;
  int32_t tmem_cols;   // allocated; two tiles' where a CTA has several
  uint32_t idesc;
  int32_t vec;         // out and residual take four values at a time
};

struct LinearBars {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t drained;
  uint32_t tmem, abort;
};

MK_DEV float activated(float y, int act) {
  if (act == MK_ACT_SILU) return y / (1.f + expf(-y));
  if (act == MK_ACT_GELU) return 0.5f * y * (1.f + erff(y * 0.7071067811865476f));
  if (act == MK_ACT_GELU_TANH)
    return 0.5f * y * (1.f + tanhf(0.7978845608028654f * (y + 0.044715f * y * y * y)));
  return y;
}

// Bounded wait: false once any wait of the CTA has run out.
MK_DEV bool wait_bar(const LinearParams& P, LinearBars& B, uint64_t* bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (*const_cast<volatile uint32_t*>(&B.abort)) return false;
    if (globaltimer() - t0 > kWaitNs) {
      *const_cast<volatile uint32_t*>(&B.abort) = 1;
      atomicExch(P.status, kTimeout);
      return false;
    }
  }
}

MK_DEV void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");
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

// Of a split tile: adds up the ranks' sums of rows c0 .. c1-1 (four outputs per
// lane, a row per warp at a time, kRows rows on their way) and writes the results.
template <class T, bool VEC>
MK_DEV void join_sums(const LinearParams& P, uint32_t sums, int feat0, int row0, int c0, int c1) {
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
        const float4 v = load_cluster(sums + min(col + i * kWarps, c1 - 1) * (kFeat * 4) + lane_id() * 16, k);
        y[i].x += v.x, y[i].y += v.y, y[i].z += v.z, y[i].w += v.w;
      }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int at = col + i * kWarps;
      if (at >= c1) continue;
      T* out = static_cast<T*>(io.out) + static_cast<int64_t>(row0 + at) * io.out_stride + feat;
      const float z[4] = {activated(y[i].x + bias[0], io.act) + r[i][0], activated(y[i].y + bias[1], io.act) + r[i][1],
                          activated(y[i].z + bias[2], io.act) + r[i][2], activated(y[i].w + bias[3], io.act) + r[i][3]};
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

template <class T>
__global__ void __launch_bounds__(kThreads, 1)
    k_linear(const __grid_constant__ LinearParams P, const __grid_constant__ CUtensorMap wmap,
             const __grid_constant__ CUtensorMap xmap) {
  extern __shared__ uint8_t raw_smem[];
  __shared__ LinearBars B;
  const mk_linear_io& io = P.io;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw_smem) + 1023) & ~uintptr_t{1023});
  const int warp = threadIdx.x / 32, lane = lane_id();
  const uint32_t stage_bytes = kFeat * 128 + P.cols * 128;
  const int rank = blockIdx.x % P.split;
  const int first = blockIdx.x / P.split, step = gridDim.x / P.split;
  // this CTA's blocks of every tile
  const int k0 = static_cast<int>(static_cast<int64_t>(P.blocks) * rank / P.split);
  const int k1 = static_cast<int>(static_cast<int64_t>(P.blocks) * (rank + 1) / P.split);
  const int acc_cols = P.cols <= 32 ? 32 : P.cols <= 64 ? 64 : P.cols <= 128 ? 128 : 256;

  pdl_launch_dependents();
  if (warp == 0 && elect_one()) {
    prefetch_tensormap(&wmap);
    prefetch_tensormap(&xmap);
    for (int i = 0; i < P.stages; ++i) mbar_init(&B.full[i], 1), mbar_init(&B.empty[i], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&B.acc_full[i], 1), mbar_init(&B.acc_empty[i], 4);
    mbar_init(&B.drained, 1);
    B.abort = 0;
    fence_mbar_init();
  }
  __syncwarp();
  if (warp == 1) {
    tmem_alloc(&B.tmem, P.tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = B.tmem;
  pdl_wait();
  if (blockIdx.x == 0 && threadIdx.x == 0) *P.status = 0;

  int loads = 0;  // of the producer
  if (warp == 0) {
    if (elect_one()) {
      const uint64_t keep = policy_evict_normal(), once = P.row_tiles == 1 ? policy_evict_first() : keep;
      bool ok = true;
      for (int tile = first; tile < P.tiles && ok; tile += step) {
        const int f = tile / P.row_tiles * kFeat, r = tile % P.row_tiles * P.cols;
        for (int k = k0; k < k1; ++k, ++loads) {
          const int st = loads % P.stages, round = loads / P.stages;
          if (round && !wait_bar(P, B, &B.empty[st], (round - 1) & 1)) {
            ok = false;
            break;
          }
          uint8_t* a = smem + st * stage_bytes;
          mbar_arrive_expect_tx(&B.full[st], stage_bytes);
          tma_load_2d(a, &wmap, &B.full[st], k * kBlock, f, once);
          tma_load_2d(a + kFeat * 128, &xmap, &B.full[st], k * kBlock, r, keep);
        }
      }
      // of work that was given up: the copies on their way, the last one into each stage
      if (!ok)
        for (int i = max(0, loads - P.stages); i < loads; ++i) mbar_wait_bounded(&B.full[i % P.stages], (i / P.stages) & 1, kWaitNs);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (elect_one()) {
      bool ok = true;
      int used = 0, n = 0;
      for (int tile = first; tile < P.tiles && ok; tile += step, ++n) {
        const int buf = n & 1;
        if (n >= 2 && !wait_bar(P, B, &B.acc_empty[buf], ((n >> 1) - 1) & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        for (int k = k0; k < k1; ++k, ++used) {
          const int st = used % P.stages;
          if (!wait_bar(P, B, &B.full[st], (used / P.stages) & 1)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a = smem_u32(smem + st * stage_bytes);
          const uint64_t ad = sdesc_kmajor_sw128(a), bd = sdesc_kmajor_sw128(a + kFeat * 128);
#pragma unroll
          for (int i = 0; i < kBlock / 16; ++i)  // 16 inputs: 32 bytes on in the swizzled rows
            mma_bf16(tmem + buf * acc_cols, ad + 2 * i, bd + 2 * i, P.idesc, k > k0 || i > 0);
          mma_commit(&B.empty[st]);
        }
        if (ok) mma_commit(&B.acc_full[buf]);
      }
      if (!ok) {
        mma_commit(&B.drained);
        mbar_wait_bounded(&B.drained, 0, kWaitNs);
      }
    }
    __syncwarp();
  } else {
    const int quad = warp & 3;
    const uint32_t lane_at = static_cast<uint32_t>(quad * 32) << 16;
    int n = 0;
    bool ok = true;
    float* sums = reinterpret_cast<float*>(smem);  // of a split tile: [cols][128]
    for (int tile = first; tile < P.tiles; tile += step, ++n) {
      const int buf = n & 1;
      ok = __all_sync(0xffffffffu, wait_bar(P, B, &B.acc_full[buf], (n >> 1) & 1));
      if (!ok) break;
      tc_fence_after();
      const int feat = tile / P.row_tiles * kFeat + quad * 32 + lane;
      const int row0 = tile % P.row_tiles * P.cols, rows = min(P.cols, io.n_rows - row0);
      const bool mine = feat < io.n_out;
      const float bias = io.bias && mine ? static_cast<float>(static_cast<const T*>(io.bias)[feat]) : 0.f;
      const T* res = static_cast<const T*>(io.residual) + static_cast<int64_t>(row0) * io.residual_stride + feat;
      T* out = static_cast<T*>(io.out) + static_cast<int64_t>(row0) * io.out_stride + feat;
      for (int col = 0; col < rows; col += 16) {
        float v[16], r[16];
        if (io.residual && P.split == 1)
#pragma unroll
          for (int i = 0; i < 16; ++i)
            r[i] = mine && col + i < rows ? static_cast<float>(res[static_cast<int64_t>(col + i) * io.residual_stride]) : 0.f;
        tmem_ld16(tmem + lane_at + buf * acc_cols + col, v);
        if (P.split > 1) {
#pragma unroll
          for (int i = 0; i < 16; ++i) sums[(col + i) * kFeat + quad * 32 + lane] = v[i];
          continue;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          if (!mine || col + i >= rows) continue;
          float y = activated(v[i] + bias, io.act);
          if (io.residual) y += r[i];
          out[static_cast<int64_t>(col + i) * io.out_stride] = static_cast<T>(y);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&B.acc_empty[buf]);
    }
  }
  if (P.split > 1) {
    __syncwarp();
    cluster_sync();
    // (a CTA of a cluster has one tile)
    if (!*const_cast<volatile uint32_t*>(&B.abort)) {
      const int feat0 = first / P.row_tiles * kFeat;
      const int row0 = first % P.row_tiles * P.cols, rows = min(P.cols, io.n_rows - row0);
      const int c0 = rows * rank / P.split, c1 = rows * (rank + 1) / P.split;
      if (P.vec) join_sums<T, true>(P, smem_u32(smem), feat0, row0, c0, c1);
      else join_sums<T, false>(P, smem_u32(smem), feat0, row0, c0, c1);
    }
    __syncwarp();
    cluster_sync();  // no CTA leaves while another one reads its sums
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) tmem_dealloc(tmem, P.tmem_cols);
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

// Sizes of the tiles and how many CTAs share one.
void choose(LinearParams* P, int sms) {
  const int64_t m = P->io.n_rows;
  const int64_t row_tiles = (m + 255) / 256, each = (m + row_tiles - 1) / row_tiles;
  P->cols = static_cast<int32_t>((each + 15) / 16 * 16);
  P->row_tiles = static_cast<int32_t>((m + P->cols - 1) / P->cols);
  P->tiles = P->row_tiles * static_cast<int32_t>((P->io.n_out + kFeat - 1) / kFeat);
  P->blocks = (P->io.n_in + kBlock - 1) / kBlock;
  P->split = 1;
  if (P->tiles < sms) P->split = std::max(1, std::min({8, sms / P->tiles, P->blocks / 4}));
  const int stage = (kFeat + P->cols) * 128;
  P->stages = std::min({kMaxStages, 220 * 1024 / stage, std::max(2, P->blocks / P->split + 1)});
  const int acc = P->cols <= 32 ? 32 : P->cols <= 64 ? 64 : P->cols <= 128 ? 128 : 256;
  P->tmem_cols = 2 * acc;
}

template <class T>
mk_status launch(const LinearParams& P, const CUtensorMap& w, const CUtensorMap& x, int device, int sms, cudaStream_t s) {
  static std::atomic<uint64_t> ready{0};  // (once per device: it takes as long as a launch)
  const uint64_t bit = device < 64 ? uint64_t{1} << device : 0;
  if (!(ready.load(std::memory_order_relaxed) & bit)) {
    MK_CUDA_TRY(cudaFuncSetAttribute(k_linear<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, 221 * 1024 + 1024));
    ready.fetch_or(bit, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t lc = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = P.split;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  lc.attrs = attr;
  lc.numAttrs = P.split > 1 ? 2 : 1;
  lc.stream = s;
  lc.gridDim = dim3(P.split > 1 ? P.tiles * P.split : std::min(P.tiles, sms));
  lc.blockDim = dim3(kThreads);
  const int stage = (kFeat + P.cols) * 128;
  // (a split tile's sums lie where the stages were)
  lc.dynamicSmemBytes = std::max(P.stages * stage, P.split > 1 ? P.cols * kFeat * 4 : 0) + 1024;
  MK_CUDA_TRY(cudaLaunchKernelEx(&lc, k_linear<T>, P, w, x));
  return MK_OK;
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
    const bool in_place = io->residual == io->out && io->residual_stride == io->out_stride;
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
  choose(&P, sms);
  // M 128, N the tile's columns; fp16 is type 0, bf16 type 1
  P.idesc = io->dtype == MK_BF16 ? idesc_bf16(kFeat, P.cols) : idesc_bf16(kFeat, P.cols) & ~((1u << 7) | (1u << 10));
  P.vec = n % 4 == 0 && io->out_stride % 4 == 0 && !misaligned(io->out, 8) &&
          (!io->residual || (io->residual_stride % 4 == 0 && !misaligned(io->residual, 8)));
  CUtensorMap w, x;
  st = encode_tmap(&w, io->dtype, io->w, k, n, io->w_stride, kFeat);
  if (st != MK_OK) return st;
  st = encode_tmap(&x, io->dtype, io->x, k, m, io->x_stride, P.cols);
  if (st != MK_OK) return st;
  return io->dtype == MK_BF16 ? launch<__nv_bfloat16>(P, w, x, device, sms, s) : launch<__half>(P, w, x, device, sms, s);
}

mk_status mk_linear_status(const void* workspace) {
  if (!workspace) return MK_ERR_INVALID_ARG;
  uint32_t s = 0;
  MK_CUDA_TRY(cudaMemcpy(&s, workspace, sizeof(s), cudaMemcpyDeviceToHost));
  return s == 0 ? MK_OK : MK_ERR_TIMEOUT;
}

}  // extern "C"
