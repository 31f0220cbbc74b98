// kvq_attn.cu -- attention over a paged cache in 4 bits (mk_kvq_attn).
#include <algorithm>
#include <cfloat>
#include <climits>
#include <cmath>

#include "kvq.cuh"
#include "rope.h"

namespace mk {

namespace {

struct KvqParams {
  mk_kvq_attn_io io;
  float scale_log2;  // scale * log2(e)
  int32_t group;
  int32_t page_shift;
  uint32_t* status;
};

MK_DEV int clampi(int64_t v, int lo, int hi) { return v < lo ? lo : v > hi ? hi : static_cast<int>(v); }

// One row and q head per CTA, a key per warp at a time.
template <class T, int D>
__global__ void __launch_bounds__(128) k_kvq_simple(const __grid_constant__ KvqParams P) {
  const mk_kvq_attn_io& io = P.io;
  const mk_kvq_cache& c = io.kvq;
  constexpr int V = D / 32;
  __shared__ float part[4][D + 2];
  const int row = blockIdx.x / io.n_q_heads, hq = blockIdx.x % io.n_q_heads, h = hq / P.group;
  const int lane = lane_id(), warp = threadIdx.x / 32;
  if (blockIdx.x == 0 && threadIdx.x == 0) *P.status = 0;
  int lo = 0, hi = io.n_requests;  // last b with cu_rows[b] <= row
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (io.cu_rows[mid] <= row) lo = mid;
    else hi = mid;
  }
  if (io.cu_rows[lo] > row || io.cu_rows[lo + 1] <= row) return;
  const int cu = clampi(io.cu_rows[lo], 0, io.n_rows), n = clampi(io.cu_rows[lo + 1], cu, io.n_rows) - cu;
  const int len = clampi(io.lens[lo], 0, io.max_pages << P.page_shift);
  const int base = max(0, len - n), i = row - cu;
  const uint64_t mask = io.tree_mask ? io.tree_mask[row] : 0;
  const int p = base + (io.tree_mask ? __popcll(mask) - 1 : i);
  const int first = io.window ? max(0, p - io.window + 1) : 0;
  const int last = io.tree_mask ? len : min(len, base + i + 1);
  const T* q = static_cast<const T*>(io.q) + row * io.q_stride + hq * D + lane * V;
  float x[V], acc[V] = {}, m = -INFINITY, sum = 0.f;
  const float unit_k = pow2(c.k_exp ? clamp_exp(c.k_exp[h]) : 0), unit_v = pow2(c.v_exp ? clamp_exp(c.v_exp[h]) : 0);
  for (int v = 0; v < V; ++v) x[v] = static_cast<float>(q[v]);
  for (int j = first + warp; j < last; j += 4) {
    if (io.tree_mask && j >= base && !(j - base < 64 && mask >> (j - base) & 1)) continue;
    const int page = io.block_table[lo * io.table_stride + (j >> P.page_shift)];
    float kv[2][V] = {};
    if (page >= 0 && page < c.n_pages) {
      const int64_t at = ((static_cast<int64_t>(page) * c.n_kv_heads + h) << P.page_shift) + (j & (c.page_size - 1));
      for (int k = 0; k < 2; ++k) {
        const uint8_t* codes = static_cast<const uint8_t*>(k ? c.v_codes : c.k_codes) + at * (D / 2) + lane * V / 2;
        const float s = e4m3_to_float((static_cast<const uint8_t*>(k ? c.v_scales : c.k_scales) + at * (D / 16))[lane * V / 16]);
        for (int v = 0; v < V; ++v) kv[k][v] = (static_cast<int>(codes[v / 2] >> (4 * (v & 1)) & 15) - 8) * s;
      }
    }
    float dot = 0.f;
    for (int v = 0; v < V; ++v) dot += x[v] * kv[0][v];
    for (int o = 16; o; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    const float s = dot * unit_k * P.scale_log2, top = s > m ? s : m != m ? m : s != s ? s : m;
    const float old = exp2f(m - top), w = exp2f(s - top);
    sum = sum * old + w;
    for (int v = 0; v < V; ++v) acc[v] = acc[v] * old + w * kv[1][v];
    m = top;
  }
  for (int v = 0; v < V; ++v) part[warp][lane * V + v] = acc[v];
  if (lane == 0) part[warp][D] = m, part[warp][D + 1] = sum;
  __syncthreads();
  if (warp) return;
  float top = -INFINITY;
  for (int w = 0; w < 4; ++w) top = part[w][D] > top || part[w][D] != part[w][D] ? part[w][D] : top;
  float all = 0.f, out[V] = {};
  for (int w = 0; w < 4; ++w) {
    const float f = part[w][D] == -INFINITY ? 0.f : exp2f(part[w][D] - top);
    all += f * part[w][D + 1];
    for (int v = 0; v < V; ++v) out[v] += f * part[w][lane * V + v];
  }
  T* to = static_cast<T*>(io.out) + row * io.out_stride + hq * D + lane * V;
  const float inv = all != 0.f ? unit_v / all : 0.f;
  for (int v = 0; v < V; ++v) to[v] = static_cast<T>(out[v] * inv);
  if (lane == 0 && io.lse) io.lse[static_cast<int64_t>(row) * io.n_q_heads + hq] = all != 0.f ? (top + log2f(all)) * 0.6931471805599453f : -INFINITY;
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

}  // namespace

}  // namespace mk

using namespace mk;

extern "C" {

mk_status mk_kvq_attn_workspace(const mk_kvq_attn_io* io, int64_t* bytes) {
  if (!bytes) return MK_ERR_INVALID_ARG;
  *bytes = 0;
  const mk_status st = check_shapes(io);
  if (st != MK_OK) return st;
  *bytes = 256;
  return MK_OK;
}

mk_status mk_kvq_attn(const mk_kvq_attn_io* io, void* workspace, int64_t workspace_bytes, void* stream) {
  mk_status st = check_shapes(io);
  if (st != MK_OK) return st;
  st = check_kvq(io->kvq, true);
  if (st != MK_OK) return st;
  const mk_kvq_cache& c = io->kvq;
  const int64_t d = c.head_dim, n = io->n_rows, slots = static_cast<int64_t>(c.n_pages) * c.page_size;
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
  if (workspace_bytes < 256) return MK_ERR_INVALID_ARG;
  st = check_device(workspace, nullptr, nullptr);
  if (st != MK_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (n == 0) {
    MK_CUDA_TRY(cudaMemsetAsync(workspace, 0, sizeof(uint32_t), s));
    return MK_OK;
  }
  KvqParams P;
  P.io = *io;
  P.scale_log2 = (io->scale != 0.f ? io->scale : 1.f / std::sqrt(static_cast<float>(d))) * 1.4426950408889634f;
  P.group = io->n_q_heads / c.n_kv_heads;
  P.page_shift = __builtin_ctz(static_cast<uint32_t>(c.page_size));
  P.status = static_cast<uint32_t*>(workspace);
  const unsigned grid = static_cast<unsigned>(n * io->n_q_heads);
  if (io->dtype == MK_BF16) {
    if (d == 128) k_kvq_simple<__nv_bfloat16, 128><<<grid, 128, 0, s>>>(P);
    else k_kvq_simple<__nv_bfloat16, 64><<<grid, 128, 0, s>>>(P);
  } else {
    if (d == 128) k_kvq_simple<__half, 128><<<grid, 128, 0, s>>>(P);
    else k_kvq_simple<__half, 64><<<grid, 128, 0, s>>>(P);
  }
  MK_CUDA_TRY(cudaGetLastError());
  return MK_OK;
}

mk_status mk_kvq_attn_status(const void* workspace) {
  if (!workspace) return MK_ERR_INVALID_ARG;
  uint32_t s = 0;
  MK_CUDA_TRY(cudaMemcpy(&s, workspace, sizeof(s), cudaMemcpyDeviceToHost));
  return s == 0 ? MK_OK : MK_ERR_TIMEOUT;
}

}  // extern "C"
