// linear.cu -- projection with bias, activation and residual (mk_linear).
#include <algorithm>
#include <climits>

#include "batch.h"
#include "rope.h"

namespace mk {

namespace {

struct LinearParams {
  mk_linear_io io;
  uint32_t* status;
};

MK_DEV float activated(float y, int act) {
  if (act == MK_ACT_SILU) return y / (1.f + expf(-y));
  if (act == MK_ACT_GELU) return 0.5f * y * (1.f + erff(y * 0.7071067811865476f));
  if (act == MK_ACT_GELU_TANH)
    return 0.5f * y * (1.f + tanhf(0.7978845608028654f * (y + 0.044715f * y * y * y)));
  return y;
}

// 16 x 16 results per CTA, one per thread.
template <class T>
__global__ void __launch_bounds__(256) k_linear_simple(const __grid_constant__ LinearParams P) {
  const mk_linear_io& io = P.io;
  __shared__ float xs[16][17], ws[16][17];
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  const int64_t m = blockIdx.y * 16ll + ty, n = blockIdx.x * 16ll + tx, n_ld = blockIdx.x * 16ll + ty;
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *P.status = 0;
  float acc = 0.f;
  for (int k0 = 0; k0 < io.n_in; k0 += 16) {
    const int k = k0 + tx;
    xs[ty][tx] = m < io.n_rows && k < io.n_in ? static_cast<float>(static_cast<const T*>(io.x)[m * io.x_stride + k]) : 0.f;
    ws[ty][tx] = n_ld < io.n_out && k < io.n_in ? static_cast<float>(static_cast<const T*>(io.w)[n_ld * io.w_stride + k]) : 0.f;
    __syncthreads();
    for (int i = 0; i < 16; ++i) acc += xs[ty][i] * ws[tx][i];
    __syncthreads();
  }
  if (m >= io.n_rows || n >= io.n_out) return;
  if (io.bias) acc += static_cast<float>(static_cast<const T*>(io.bias)[n]);
  acc = activated(acc, io.act);
  if (io.residual) acc += static_cast<float>(static_cast<const T*>(io.residual)[m * io.residual_stride + n]);
  static_cast<T*>(io.out)[m * io.out_stride + n] = static_cast<T>(acc);
}

mk_status check_shapes(const mk_linear_io* io) {
  if (!io) return MK_ERR_INVALID_ARG;
  if (io->dtype != MK_BF16 && io->dtype != MK_FP16) return MK_ERR_UNSUPPORTED;
  if (io->n_rows < 0 || io->n_in < 1 || io->n_out < 1) return MK_ERR_INVALID_ARG;
  if (io->n_in % 8) return MK_ERR_UNSUPPORTED;
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
  st = check_device(workspace, nullptr, nullptr);
  if (st != MK_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (m == 0) {
    MK_CUDA_TRY(cudaMemsetAsync(workspace, 0, sizeof(uint32_t), s));
    return MK_OK;
  }
  LinearParams P;
  P.io = *io;
  P.status = static_cast<uint32_t*>(workspace);
  if ((m + 15) / 16 > 65535) return MK_ERR_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>((n + 15) / 16), static_cast<unsigned>((m + 15) / 16));
  if (io->dtype == MK_BF16) k_linear_simple<__nv_bfloat16><<<grid, 256, 0, s>>>(P);
  else k_linear_simple<__half><<<grid, 256, 0, s>>>(P);
  MK_CUDA_TRY(cudaGetLastError());
  return MK_OK;
}

mk_status mk_linear_status(const void* workspace) {
  if (!workspace) return MK_ERR_INVALID_ARG;
  uint32_t s = 0;
  MK_CUDA_TRY(cudaMemcpy(&s, workspace, sizeof(s), cudaMemcpyDeviceToHost));
  return s == 0 ? MK_OK : MK_ERR_TIMEOUT;
}

}  // extern "C"
