// prefix_attn.cu -- attention of a batch whose requests share a prefix
// (mk_prefix_attn): softmax(scale q K^T) V per row over the prefix's pages and
// its request's own, with online maximum and sum.
#include <algorithm>
#include <cfloat>
#include <climits>
#include <cmath>
#include <cuda_fp16.h>

#include "batch.h"
#include "ptx.cuh"

namespace mk {

namespace {

struct AttnParams {
  mk_prefix_attn_io io;
  float scale_log2;  // scale * log2(e)
  uint32_t* status;
};

MK_DEV float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
MK_DEV float to_f(__half v) { return __half2float(v); }
template <class T> MK_DEV T from_f(float v);
template <> MK_DEV __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> MK_DEV __half from_f<__half>(float v) { return __float2half_rn(v); }

MK_DEV int clampi(int64_t v, int lo, int hi) {
  return v < lo ? lo : v > hi ? hi : static_cast<int>(v);
}

// One CTA per (row, q head); each warp takes every fourth key, its lanes the
// head's values; the warps' maxima, sums and outputs are joined at the end.
template <class T, int D>
__global__ void __launch_bounds__(128) k_prefix_attn(const __grid_constant__ AttnParams P) {
  const mk_prefix_attn_io& io = P.io;
  constexpr int V = D / 32;
  __shared__ float s_o[4][D];
  __shared__ float s_m[4], s_l[4];
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *P.status = 0;
  const int row = blockIdx.x, hq = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int hk = hq / (io.n_q_heads / io.n_kv_heads);
  if (row >= clampi(io.cu_rows[io.n_requests], 0, io.n_rows)) return;
  int lo = 0, hi = io.n_requests;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (io.cu_rows[mid] <= row) lo = mid; else hi = mid;
  }
  const int b = lo, cu = clampi(io.cu_rows[b], 0, io.n_rows);
  const int n = clampi(io.cu_rows[b + 1], cu, io.n_rows) - cu, i = row - cu;
  const int64_t cap = static_cast<int64_t>(io.max_pages) * io.page_size;
  const int len = clampi(io.lens[b], 0, static_cast<int>(cap));
  const int base = max(0, len - n);
  const uint64_t tree = io.tree_mask ? io.tree_mask[row] : 0;
  const int depth = io.tree_mask ? max(1, __popcll(tree)) - 1 : i;
  const int64_t low = io.window ? static_cast<int64_t>(io.prefix_len) + base + depth - io.window + 1 : 0;
  const int own_end = io.tree_mask ? len : clampi(static_cast<int64_t>(base) + i + 1, 0, len);
  const int64_t first = low < 0 ? 0 : low;
  const int64_t end = static_cast<int64_t>(io.prefix_len) + own_end;

  float q[V], o[V] = {};
  const T* qp = static_cast<const T*>(io.q) + row * io.q_stride + hq * D + lane * V;
#pragma unroll
  for (int e = 0; e < V; ++e) q[e] = to_f(qp[e]) * P.scale_log2;
  float m = -INFINITY, l = 0.f;
  for (int64_t pos = first + warp; pos < end; pos += 4) {
    const bool pre = pos < io.prefix_len;
    const int j = static_cast<int>(pre ? pos : pos - io.prefix_len);
    if (!pre && io.tree_mask && j >= base && !(j - base < 64 && (tree >> (j - base) & 1))) continue;
    const int id = pre ? io.prefix_pages[j / io.page_size]
                       : io.block_table[b * io.table_stride + j / io.page_size];
    const bool ok = id >= 0 && id < io.n_pages;
    const int64_t at = ((static_cast<int64_t>(id) * io.page_size + j % io.page_size) * io.n_kv_heads + hk) * D + lane * V;
    float s = 0.f, v[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      s += ok ? q[e] * to_f(static_cast<const T*>(io.k_cache)[at + e]) : 0.f;
      v[e] = ok ? to_f(static_cast<const T*>(io.v_cache)[at + e]) : 0.f;
    }
#pragma unroll
    for (int w = 16; w; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
    const float top = fmaxf(m, s), c = exp2f(m - top), p = exp2f(s - top);
    l = l * c + p;
    m = top;
#pragma unroll
    for (int e = 0; e < V; ++e) o[e] = o[e] * c + p * v[e];
  }
#pragma unroll
  for (int e = 0; e < V; ++e) s_o[warp][lane * V + e] = o[e];
  if (lane == 0) s_m[warp] = m, s_l[warp] = l;
  __syncthreads();
  const float top = fmaxf(fmaxf(s_m[0], s_m[1]), fmaxf(s_m[2], s_m[3]));
  float total = 0.f, w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    w[k] = top == -INFINITY ? 0.f : exp2f(s_m[k] - top);
    total += w[k] * s_l[k];
  }
  if (threadIdx.x < D) {
    float acc = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) acc += w[k] * s_o[k][threadIdx.x];
    static_cast<T*>(io.out)[row * io.out_stride + hq * D + threadIdx.x] =
        from_f<T>(total > 0.f ? acc / total : 0.f);
  }
  if (threadIdx.x == 0 && io.lse)
    io.lse[static_cast<int64_t>(row) * io.n_q_heads + hq] =
        total > 0.f ? (top + log2f(total)) * 0.6931471805599453f : -INFINITY;
}

mk_status check_shapes(const mk_prefix_attn_io* io) {
  if (!io) return MK_ERR_INVALID_ARG;
  if (io->n_requests < 1 || io->n_requests > 65536 || io->n_rows < 0) return MK_ERR_INVALID_ARG;
  if (io->n_kv_heads < 1 || io->n_q_heads < 1 || io->n_q_heads % io->n_kv_heads)
    return MK_ERR_INVALID_ARG;
  if (io->n_q_heads / io->n_kv_heads > 64 || io->n_q_heads > 4096) return MK_ERR_UNSUPPORTED;
  if (io->head_dim != 64 && io->head_dim != 128) return MK_ERR_UNSUPPORTED;
  if (io->dtype != MK_BF16 && io->dtype != MK_FP16) return MK_ERR_UNSUPPORTED;
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
  *bytes = 256;
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
  if (cap > INT32_MAX - io->prefix_len) return MK_ERR_INVALID_ARG;
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
  int64_t need = 0;
  st = mk_prefix_attn_workspace(io, &need);
  if (st != MK_OK) return st;
  if (workspace_bytes < need) return MK_ERR_INVALID_ARG;
  if (io->n_rows == 0) return MK_OK;
  st = check_device(workspace, nullptr, nullptr);
  if (st != MK_OK) return st;
  AttnParams A;
  A.io = *io;
  const float scale = io->scale != 0.f ? io->scale : 1.f / std::sqrt(static_cast<float>(io->head_dim));
  A.scale_log2 = scale * 1.4426950408889634f;
  A.status = static_cast<uint32_t*>(workspace);
  const dim3 grid(io->n_rows, io->n_q_heads);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (io->dtype == MK_BF16) {
    if (io->head_dim == 128) k_prefix_attn<__nv_bfloat16, 128><<<grid, 128, 0, s>>>(A);
    else k_prefix_attn<__nv_bfloat16, 64><<<grid, 128, 0, s>>>(A);
  } else {
    if (io->head_dim == 128) k_prefix_attn<__half, 128><<<grid, 128, 0, s>>>(A);
    else k_prefix_attn<__half, 64><<<grid, 128, 0, s>>>(A);
  }
  MK_CUDA_TRY(cudaGetLastError());
  return MK_OK;
}

mk_status mk_prefix_attn_status(const void* workspace) {
  if (!workspace) return MK_ERR_INVALID_ARG;
  uint32_t s = 0;
  MK_CUDA_TRY(cudaMemcpy(&s, workspace, sizeof(s), cudaMemcpyDeviceToHost));
  return s == 0 ? MK_OK : MK_ERR_TIMEOUT;
}

}  // extern "C"
