// slots.cu -- block tables and slot maps of a batch from its request lengths
// (mk_build_slots), and the device check the batched operators share.
//
// With c_b cached and n_b new tokens of request b and pages of P tokens:
//   cu_b    = sum_{a<b} n_a                      rows of request b
//   need_b  = ceil((c_b+n_b)/P) - ceil(c_b/P)    pages it gets
//   first_b = head + sum_{a<b} need_a            their place in the free list
// so the whole of it is two exclusive scans over the batch and a write per row
// and per page.  Bound by launch latency at every batch size in use.
#include <algorithm>
#include <atomic>
#include <climits>

#include "batch.h"
#include "ptx.cuh"

namespace mk {

namespace {

constexpr int kSlotThreads = 256;

struct SlotsParams {
  mk_slots_io io;
  int32_t per_cta;  // requests of one CTA
};

// Lengths of one request as every CTA reads them.
struct Request {
  int64_t rows;  // rows in the row layout
  int64_t need;  // pages, if its rows fit
  bool lengths_ok;
};

MK_DEV int64_t pages_of(int64_t tokens, int32_t page) { return (tokens + page - 1) / page; }

MK_DEV Request read_request(const mk_slots_io& io, int b) {
  const int64_t c = io.cached_lens[b], n = io.new_lens[b];
  Request r;
  r.rows = n > 0 ? n : 0;
  r.lengths_ok = c >= 0 && n >= 0 && c + n <= static_cast<int64_t>(io.max_pages) * io.page_size;
  r.need = r.lengths_ok ? pages_of(c + n, io.page_size) - pages_of(c, io.page_size) : 0;
  return r;
}

// Inclusive sums of one value per thread over the CTA; *total = the sum of all.
MK_DEV int64_t cta_scan(int64_t v, int64_t* warp_sums, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  int64_t before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kSlotThreads / 32; ++w) {
    if (w < warp) before += warp_sums[w];
    all += warp_sums[w];
  }
  __syncthreads();
  *total = all;
  return v + before;
}

MK_DEV int64_t cta_sum(int64_t v, int64_t* warp_sums) {
  int64_t total;
  cta_scan(v, warp_sums, &total);
  return total;
}

// Each CTA owns per_cta consecutive requests.  It sums the lengths of the
// requests before its own (and of all, for the end of the rows) itself:
// reading the batch's lengths again costs less than a second launch or a wait
// for the CTAs before it.
__global__ void __launch_bounds__(kSlotThreads)
    k_build_slots(const __grid_constant__ SlotsParams P) {
  const mk_slots_io& io = P.io;
  __shared__ int64_t warp_sums[kSlotThreads / 32];
  __shared__ int64_t s_cu[kSlotThreads + 1];     // first row of each request of the chunk
  __shared__ int64_t s_need[kSlotThreads + 1];   // pages before each request of the chunk
  __shared__ int32_t s_cached[kSlotThreads];
  __shared__ uint8_t s_granted[kSlotThreads];

  const int B = io.n_requests, page = io.page_size;
  const int b0 = min(B, static_cast<int>(blockIdx.x) * P.per_cta), b1 = min(B, b0 + P.per_cta);
  int64_t head = io.free_head ? *io.free_head : 0;
  head = head < 0 ? 0 : head > io.n_free ? io.n_free : head;
  const int64_t avail = io.n_free - head;

  // sums over the requests before b0 and over all
  int64_t rows_before = 0, rows_all = 0, need_before = 0, need_all = 0;
  for (int b = threadIdx.x; b < B; b += kSlotThreads) {
    const Request r = read_request(io, b);
    rows_all += r.rows;
    need_all += r.need;
    if (b < b0) rows_before += r.rows, need_before += r.need;
  }
  rows_before = cta_sum(rows_before, warp_sums);
  rows_all = cta_sum(rows_all, warp_sums);
  need_before = cta_sum(need_before, warp_sums);
  need_all = cta_sum(need_all, warp_sums);
  if (rows_all > io.n_rows) {
    // some request's rows do not fit: it and those behind it need no pages, so
    // the page sums have to go by each request's last row
    int64_t row = 0;
    need_before = need_all = 0;
    for (int a = 0; a < B; a += kSlotThreads) {
      const int b = a + threadIdx.x;
      Request r{0, 0, false};
      if (b < B) r = read_request(io, b);
      int64_t rows, need;
      const int64_t end = row + cta_scan(r.rows, warp_sums, &rows);
      cta_scan(end <= io.n_rows ? r.need : 0, warp_sums, &need);
      need_all += need;
      if (b1 > b0) need_before += cta_sum(b < b0 && end <= io.n_rows ? r.need : 0, warp_sums);
      row += rows;
    }
  }
  const int64_t rows_used = rows_all < io.n_rows ? rows_all : io.n_rows;

  for (int a = b0; a < b1; a += kSlotThreads) {
    const int m = min(kSlotThreads, b1 - a), i = threadIdx.x, b = a + i;
    Request r{0, 0, false};
    int64_t c = 0, n = 0;
    if (i < m) {
      r = read_request(io, b);
      c = io.cached_lens[b];
      n = r.rows;
    }
    int64_t rows, need;
    const int64_t row_end = rows_before + cta_scan(r.rows, warp_sums, &rows);
    const bool fits = i < m && r.lengths_ok && row_end <= io.n_rows;
    const int64_t want = fits ? r.need : 0;
    const int64_t need_end = need_before + cta_scan(want, warp_sums, &need);
    const bool granted = fits && (want == 0 || need_end <= avail);
    if (i < m) {
      const int64_t cap = static_cast<int64_t>(io.max_pages) * page;
      io.cu_rows[b] = static_cast<int32_t>(min(row_end - r.rows, static_cast<int64_t>(io.n_rows)));
      io.lens[b] = static_cast<int32_t>(granted ? c + n : c < 0 ? 0 : min(c, cap));
      s_cached[i] = static_cast<int32_t>(c);
      s_granted[i] = granted;
    }
    s_cu[i] = row_end - r.rows;
    s_need[i] = need_end - want;
    if (i == kSlotThreads - 1) {
      s_cu[kSlotThreads] = row_end;
      s_need[kSlotThreads] = need_end;
    }
    __syncthreads();

    // the new pages of the chunk's requests, one thread per page
    for (int64_t e = need_before + threadIdx.x; e < need_before + need && e < avail;
         e += kSlotThreads) {
      int lo = 0, hi = m;  // the last request with s_need <= e, which has a page at e
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_need[mid] <= e) lo = mid; else hi = mid;
      }
      if (s_granted[lo])
        io.block_table[static_cast<int64_t>(a + lo) * io.table_stride +
                       pages_of(s_cached[lo], page) + (e - s_need[lo])] = io.free_pages[head + e];
    }
    // the chunk's rows, one thread per row; a row takes its page from where it
    // is handed out, not from the table, which this CTA is writing
    const int64_t r1 = min(rows_before + rows, static_cast<int64_t>(io.n_rows));
    for (int64_t row = rows_before + threadIdx.x; row < r1; row += kSlotThreads) {
      int lo = 0, hi = m;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_cu[mid] <= row) lo = mid; else hi = mid;
      }
      const int64_t at = static_cast<int64_t>(s_cached[lo]) + (row - s_cu[lo]);
      int64_t slot = -1;
      if (s_granted[lo]) {
        const int64_t col = at / page, held = pages_of(s_cached[lo], page);
        const int32_t id =
            col < held ? io.block_table[static_cast<int64_t>(a + lo) * io.table_stride + col]
                       : io.free_pages[head + s_need[lo] + (col - held)];
        if (id >= 0 && id < io.n_pages) slot = static_cast<int64_t>(id) * page + at % page;
      }
      io.positions[row] = static_cast<int32_t>(min(io.prefix_len + at, static_cast<int64_t>(INT_MAX)));
      io.slots[row] = slot;
      if (io.row_request) io.row_request[row] = a + lo;
    }
    rows_before += rows;
    need_before += need;
    __syncthreads();
  }

  // rows behind the last request, shared out over the grid
  for (int64_t row = rows_used + static_cast<int64_t>(blockIdx.x) * kSlotThreads + threadIdx.x;
       row < io.n_rows; row += static_cast<int64_t>(gridDim.x) * kSlotThreads) {
    io.positions[row] = 0;
    io.slots[row] = -1;
    if (io.row_request) io.row_request[row] = -1;
  }
  if (blockIdx.x == gridDim.x - 1) {
    // what was taken and refused: a pass over the batch in order
    int64_t row = 0, upto = 0, taken = 0, refused = 0;
    for (int a = 0; a < B; a += kSlotThreads) {
      const int b = a + threadIdx.x;
      Request r{0, 0, false};
      if (b < B) r = read_request(io, b);
      int64_t rows, need;
      const int64_t end = row + cta_scan(r.rows, warp_sums, &rows);
      const bool fits = b < B && r.lengths_ok && end <= io.n_rows;
      const int64_t want = fits ? r.need : 0;
      const int64_t need_end = upto + cta_scan(want, warp_sums, &need);
      const bool granted = fits && (want == 0 || need_end <= avail);
      taken += granted ? want : 0;
      refused += b < B && !granted;
      row += rows;
      upto += need;
    }
    taken = cta_sum(taken, warp_sums);
    refused = cta_sum(refused, warp_sums);
    if (threadIdx.x == 0) {
      io.cu_rows[B] = static_cast<int32_t>(rows_used);
      io.summary[0] = static_cast<int32_t>(head + taken);
      io.summary[1] = static_cast<int32_t>(rows_used);
      io.summary[2] = static_cast<int32_t>(refused);
      io.summary[3] = static_cast<int32_t>(need_all < INT_MAX ? need_all : INT_MAX);
    }
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
  if (static_cast<int64_t>(io->max_pages) * io->page_size > INT32_MAX - io->prefix_len)
    return MK_ERR_INVALID_ARG;
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
  const int64_t grid = std::max<int64_t>(1, std::min<int64_t>((B + 31) / 32, 2 * sms));
  P.per_cta = static_cast<int32_t>((B + grid - 1) / grid);
  k_build_slots<<<static_cast<unsigned>(grid), kSlotThreads, 0, static_cast<cudaStream_t>(stream)>>>(P);
  MK_CUDA_TRY(cudaGetLastError());
  return MK_OK;
}
