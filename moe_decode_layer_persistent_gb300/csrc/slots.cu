// slots.cu -- block tables and slot maps of a batch from its request lengths
// (mk_build_slots), and the device check the batched operators share.
//
// With c_b cached and n_b new tokens of request b and pages of P tokens:
//   cu_b    = sum_{a<b} n_a                      rows of request b
//   need_b  = ceil((c_b+n_b)/P) - ceil(c_b/P)    pages it gets
//   first_b = head + sum_{a<b} need_a            their place in the free list
// so the whole of it is two exclusive sums over the batch and a write per row and
// per page.  Each CTA sums the lengths before its own requests itself, in one
// launch: reading the batch again from L2 costs less than a second launch or a
// wait for other CTAs.  With few rows per request a handful of dependent reads bounds
// it, not the bytes: 16 requests take 6 us, 4096 with 196,000 rows (3.3 MB) 9 us.  A
// CTA has 32 requests (more, beyond 9,700), and their rows and pages are its alone,
// 512 at a time with a search and a page read each: 131,072 rows take 7.5 us as those
// of 4096 requests, 163 us as those of 32, 77 us as those of one.
#include <algorithm>
#include <atomic>
#include <climits>

#include "batch.h"
#include "ptx.cuh"

namespace mk {

namespace {

constexpr int kSlotThreads = 512;

struct SlotsParams {
  mk_slots_io io;
  Divisor page;
  int32_t per_cta;  // requests of one CTA
};

// Sums over a batch, or a part of it.
struct Sums {
  int64_t rows, need;
};

// One request's lengths.
struct Request {
  int32_t cached, rows, need;  // need: pages, if its rows fit
  bool lengths_ok;
};

MK_DEV Request read_request(const SlotsParams& P, int b) {
  const mk_slots_io& io = P.io;
  const int32_t c = io.cached_lens[b], n = io.new_lens[b];
  Request r;
  r.cached = c;
  r.rows = max(n, 0);
  // (max_pages * page_size is below 2^31)
  r.lengths_ok = c >= 0 && n >= 0 && static_cast<int64_t>(c) + n <= io.max_pages * io.page_size;
  r.need = 0;
  if (r.lengths_ok)
    r.need = quotient(c + n + io.page_size - 1u, P.page) - quotient(c + io.page_size - 1u, P.page);
  return r;
}

// Inclusive sums of a value pair per thread over the CTA; *total = those of all.
MK_DEV Sums cta_scan(Sums v, Sums* warp_sums, Sums* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t a = __shfl_up_sync(0xffffffffu, v.rows, o), b = __shfl_up_sync(0xffffffffu, v.need, o);
    if (lane >= o) v.rows += a, v.need += b;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  Sums before{0, 0}, all{0, 0};
#pragma unroll
  for (int w = 0; w < kSlotThreads / 32; ++w) {
    const Sums x = warp_sums[w];
    if (w < warp) before.rows += x.rows, before.need += x.need;
    all.rows += x.rows, all.need += x.need;
  }
  *total = all;
  return Sums{v.rows + before.rows, v.need + before.need};
}

MK_DEV int64_t warp_sum(int64_t v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__global__ void __launch_bounds__(kSlotThreads)
    k_build_slots(const __grid_constant__ SlotsParams P) {
  const mk_slots_io& io = P.io;
  __shared__ Sums warp_sums[kSlotThreads / 32];
  __shared__ int64_t part[kSlotThreads / 32][5];
  __shared__ int64_t s_cu[kSlotThreads];    // first row of each request of the chunk
  __shared__ int64_t s_need[kSlotThreads];  // pages before each request of the chunk
  __shared__ int32_t s_cached[kSlotThreads];
  __shared__ uint8_t s_granted[kSlotThreads];

  const int B = io.n_requests, page = io.page_size, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b0 = min(B, static_cast<int>(blockIdx.x) * P.per_cta), b1 = min(B, b0 + P.per_cta);
  int64_t head = io.free_head ? *io.free_head : 0;
  head = head < 0 ? 0 : head > io.n_free ? io.n_free : head;
  const int64_t avail = io.n_free - head;

  // sums over the requests before b0 and over all, and how many lengths are wrong
  Sums before{0, 0}, all{0, 0};
  int64_t wrong = 0;
#pragma unroll 4
  for (int b = threadIdx.x; b < B; b += kSlotThreads) {
    const Request r = read_request(P, b);
    all.rows += r.rows, all.need += r.need;
    if (b < b0) before.rows += r.rows, before.need += r.need;
    wrong += !r.lengths_ok;
  }
  {
    const int64_t v[5] = {warp_sum(before.rows), warp_sum(before.need), warp_sum(all.rows),
                          warp_sum(all.need), warp_sum(wrong)};
    if (lane == 0)
#pragma unroll
      for (int i = 0; i < 5; ++i) part[warp][i] = v[i];
    __syncthreads();
    int64_t sum[5] = {0, 0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < kSlotThreads / 32; ++w)
#pragma unroll
      for (int i = 0; i < 5; ++i) sum[i] += part[w][i];
    before = Sums{sum[0], sum[1]};
    all = Sums{sum[2], sum[3]};
    wrong = sum[4];
  }
  const int64_t rows_all = all.rows;
  const int64_t rows_used = rows_all < io.n_rows ? rows_all : io.n_rows;
  int64_t taken = all.need, refused = wrong;
  if (rows_all > io.n_rows || all.need > avail) {
    // Some request's rows or pages do not fit.  One whose rows do not needs no
    // pages, nor do those behind it, so that the page sums go by each one's last
    // row: a pass over the batch in order.
    Sums at{0, 0};
    before.need = taken = refused = 0;
    for (int a = 0; a < B; a += kSlotThreads) {
      const int b = a + threadIdx.x;
      Request r{0, 0, 0, false};
      if (b < B) r = read_request(P, b);
      Sums total;
      const int64_t end = at.rows + cta_scan(Sums{r.rows, 0}, warp_sums, &total).rows;
      at.rows += total.rows;
      const bool fits = b < B && r.lengths_ok && end <= io.n_rows;
      const int64_t want = fits ? r.need : 0;
      const int64_t need_end = at.need + cta_scan(Sums{0, want}, warp_sums, &total).need;
      at.need += total.need;
      const bool granted = fits && (want == 0 || need_end <= avail);
      cta_scan(Sums{granted ? want : 0, b < B && !granted}, warp_sums, &total);
      taken += total.rows;
      refused += total.need;
      cta_scan(Sums{0, b < b0 ? want : 0}, warp_sums, &total);
      before.need += total.need;
    }
    all.need = at.need;
  }

  for (int a = b0; a < b1; a += kSlotThreads) {
    const int m = min(kSlotThreads, b1 - a), i = threadIdx.x, b = a + i;
    Request r{0, 0, 0, false};
    if (i < m) r = read_request(P, b);
    // (the rows first: whether they fit decides about the pages)
    Sums total, need_total;
    const int64_t row_end = before.rows + cta_scan(Sums{r.rows, 0}, warp_sums, &total).rows;
    const bool fits = i < m && r.lengths_ok && row_end <= io.n_rows;
    const int64_t want = fits ? r.need : 0;
    const int64_t need_end = before.need + cta_scan(Sums{0, want}, warp_sums, &need_total).need;
    const bool granted = fits && (want == 0 || need_end <= avail);
    if (i < m) {
      io.cu_rows[b] = static_cast<int32_t>(min(row_end - r.rows, static_cast<int64_t>(io.n_rows)));
      io.lens[b] = granted ? r.cached + r.rows : max(0, min(r.cached, io.max_pages * page));
      s_cached[i] = r.cached;
      s_granted[i] = granted;
    }
    s_cu[i] = row_end - r.rows;
    s_need[i] = need_end - want;
    __syncthreads();

    // the new pages of the chunk's requests, one thread per page
    const int64_t e1 = min(before.need + need_total.need, avail);
    for (int64_t e = before.need + threadIdx.x; e < e1; e += kSlotThreads) {
      int lo = 0, hi = m;  // the last request with s_need <= e, which has a page at e
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_need[mid] <= e) lo = mid; else hi = mid;
      }
      if (s_granted[lo])
        io.block_table[static_cast<int64_t>(a + lo) * io.table_stride +
                       quotient(s_cached[lo] + page - 1u, P.page) + (e - s_need[lo])] =
            io.free_pages[head + e];
    }
    // the chunk's rows, one thread per row; a row takes its page from where it
    // is handed out, not from the table, which this CTA is writing
    const int64_t r1 = min(before.rows + total.rows, static_cast<int64_t>(io.n_rows));
    for (int64_t row = before.rows + threadIdx.x; row < r1; row += kSlotThreads) {
      int lo = 0, hi = m;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_cu[mid] <= row) lo = mid; else hi = mid;
      }
      const int64_t at = static_cast<int64_t>(s_cached[lo]) + (row - s_cu[lo]);
      int64_t slot = -1;
      if (s_granted[lo]) {
        const uint32_t t = static_cast<uint32_t>(at), col = quotient(t, P.page);
        const uint32_t held = quotient(s_cached[lo] + page - 1u, P.page);
        const int32_t id =
            col < held ? io.block_table[static_cast<int64_t>(a + lo) * io.table_stride + col]
                       : io.free_pages[head + s_need[lo] + (col - held)];
        if (id >= 0 && id < io.n_pages) slot = static_cast<int64_t>(id) * page + (t - col * page);
      }
      io.positions[row] = static_cast<int32_t>(min(io.prefix_len + at, static_cast<int64_t>(INT_MAX)));
      io.slots[row] = slot;
      if (io.row_request) io.row_request[row] = a + lo;
    }
    before.rows += total.rows;
    before.need += need_total.need;
    __syncthreads();
  }

  // rows behind the last request, shared out over the grid
  for (int64_t row = rows_used + static_cast<int64_t>(blockIdx.x) * kSlotThreads + threadIdx.x;
       row < io.n_rows; row += static_cast<int64_t>(gridDim.x) * kSlotThreads) {
    io.positions[row] = 0;
    io.slots[row] = -1;
    if (io.row_request) io.row_request[row] = -1;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    io.cu_rows[B] = static_cast<int32_t>(rows_used);
    io.summary[0] = static_cast<int32_t>(head + taken);
    io.summary[1] = static_cast<int32_t>(rows_used);
    io.summary[2] = static_cast<int32_t>(refused);
    io.summary[3] = static_cast<int32_t>(all.need < INT_MAX ? all.need : INT_MAX);
  }
}

}  // namespace

mk_status check_device(const void* p, int* device, int* sm_count) {
  // SM count of each device once asked, -1 for another architecture (a fact of the
  // machine; asking takes longer than the rest of a call)
  static std::atomic<int> known[64];
  int dev = -1;
  MK_CUDA_TRY(cudaGetDevice(&dev));
  int sms = dev < 64 ? known[dev].load(std::memory_order_relaxed) : 0;
  if (sms == 0) {
    int major = 0, minor = 0;
    MK_CUDA_TRY(cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev));
    MK_CUDA_TRY(cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev));
    MK_CUDA_TRY(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
    if (major != 10 || minor != 3) sms = -1;
    if (dev < 64) known[dev].store(sms, std::memory_order_relaxed);
  }
  if (sms < 0) return MK_ERR_UNSUPPORTED;
  cudaPointerAttributes at;
  MK_CUDA_TRY(cudaPointerGetAttributes(&at, p));
  if (at.type != cudaMemoryTypeDevice && at.type != cudaMemoryTypeManaged) return MK_ERR_INVALID_ARG;
  if (at.type == cudaMemoryTypeDevice && at.device != dev) return MK_ERR_INVALID_ARG;
  if (device) *device = dev;
  if (sm_count) *sm_count = sms;
  return MK_OK;
}

}  // namespace mk

using namespace mk;

extern "C" mk_status mk_build_slots(const mk_slots_io* io, void* stream) {
  if (!io) return MK_ERR_INVALID_ARG;
  if (io->n_requests < 0 || io->n_requests > 65536) return MK_ERR_INVALID_ARG;
  if (io->n_rows < 0 || io->page_size < 1 || io->max_pages < 0 || io->n_pages < 0 ||
      io->n_free < 0 || io->prefix_len < 0 || io->table_stride < io->max_pages)
    return MK_ERR_INVALID_ARG;
  const int64_t B = io->n_requests;
  if ((io->max_pages + 1ll) * io->page_size > INT32_MAX - io->prefix_len) return MK_ERR_INVALID_ARG;
  if (!io->cu_rows || !io->summary) return MK_ERR_INVALID_ARG;
  if (B && (!io->cached_lens || !io->new_lens || !io->lens)) return MK_ERR_INVALID_ARG;
  if (B && io->max_pages && !io->block_table) return MK_ERR_INVALID_ARG;
  if (io->n_rows && (!io->positions || !io->slots)) return MK_ERR_INVALID_ARG;
  if (io->n_free && !io->free_pages) return MK_ERR_INVALID_ARG;
  struct Range {
    const void* p;
    int64_t bytes;
    int align;
  };
  const Range in[] = {{io->cached_lens, B * 4, 4},
                      {io->new_lens, B * 4, 4},
                      {io->free_pages, io->n_free * 4ll, 4},
                      {io->free_head, 4, 4}};
  const Range out[] = {{io->block_table, span_bytes(B, io->max_pages, io->table_stride, 4), 4},
                       {io->cu_rows, (B + 1) * 4, 4},
                       {io->lens, B * 4, 4},
                       {io->positions, io->n_rows * 4ll, 4},
                       {io->slots, io->n_rows * 8ll, 8},
                       {io->row_request, io->n_rows * 4ll, 4},
                       {io->summary, 16, 4}};
  for (const Range& r : in)
    if (misaligned(r.p, r.align)) return MK_ERR_INVALID_ARG;
  for (const Range& r : out) {
    if (misaligned(r.p, r.align)) return MK_ERR_INVALID_ARG;
    for (const Range& i : in)
      if (overlap(r.p, r.bytes, i.p, i.bytes)) return MK_ERR_INVALID_ARG;
    for (const Range& o : out)
      if (&o != &r && overlap(r.p, r.bytes, o.p, o.bytes)) return MK_ERR_INVALID_ARG;
  }
  int sms = 0;
  mk_status st = check_device(io->summary, nullptr, &sms);
  if (st != MK_OK) return st;
  SlotsParams P;
  P.io = *io;
  P.page = make_divisor(static_cast<uint32_t>(io->page_size));
  const int64_t grid = std::max<int64_t>(1, std::min<int64_t>((B + 31) / 32, 2 * sms));
  P.per_cta = static_cast<int32_t>((B + grid - 1) / grid);
  k_build_slots<<<static_cast<unsigned>(grid), kSlotThreads, 0, static_cast<cudaStream_t>(stream)>>>(P);
  MK_CUDA_TRY(cudaGetLastError());
  return MK_OK;
}
