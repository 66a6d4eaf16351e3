// pages.cu -- the new rows of every request get pages and slots (the way back from evict.cu's
// free list into the page tables), and K/V rows are stored at their slots.
//
// assign_kernel.  Request b appends rows L_b - n_b .. L_b - 1.  A page whose first row is new
// has nothing in it yet, so which pages a request needs follows from its two lengths alone:
//   need_b = ceil(L_b / 16) - ceil((L_b - n_b) / 16),
// and the k-th page needed, requests in order, is free_pages[count - 1 - k].  Everything is a
// prefix sum over the requests, so the result does not depend on the order of CTAs.  Each CTA
// takes 512 of the packed rows; it sums over all requests itself, which costs less than a
// second launch, and notes the requests that start in its rows; a running maximum over the rows
// then gives each row its request.  Bound, for a step's few rows, by the chain of dependent loads
// (lengths, sums, page id, slot; 2.9 us); for many rows by issue as well, as each CTA goes over all
// requests twice with 64-bit sums.  Measured: 1024 requests of 32 .. 512 new rows (530 CTAs, 5.6 M
// instructions, issue slots 57 % busy) 8.6 us, 12.5 with 512 requests summed at a time.
//
// write_kernel.  A copy bound by HBM; the rows do not wait for their slots, both are loaded
// together.
#include "common.cuh"
#include "internal.h"

namespace dsa {
namespace {

constexpr int kAssignThreads = 512;

// A request whose rows start (or go on) in a CTA's tile.
struct TileRequest {
  int32_t b, row, first;  // request; the row at its place in the tile; first fresh page
  int32_t served;         // the free list holds all that it needs
  int32_t take;           // served: index in the free list of the first fresh page
};

__device__ __forceinline__ int64_t warp_scan(int64_t x, int lane) {
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, x, s);
    if (lane >= s) x += v;
  }
  return x;
}

__global__ void __launch_bounds__(kAssignThreads) assign_kernel(const AssignLaunch a) {
  constexpr int kWarps = kAssignThreads / 32;
  __shared__ TileRequest req[kAssignThreads];
  __shared__ int32_t owner[kAssignThreads];
  __shared__ int64_t rows_of[kWarps], pages_of[kWarps];
  __shared__ int32_t owner_of[kWarps], taken_of[kWarps];
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kAssignThreads;
  const bool first_cta = blockIdx.x == 0;
  // Eviction counts past a list that was too small; the list is full then.
  int count = *a.free_count;
  if (count < 0 || count > a.capacity) {
    if (first_cta && tid == 0) set_error(a.err, DSA_DEV_BAD_COUNT);
    count = count < 0 ? 0 : a.capacity;
  }
  owner[tid] = -1;
  // Every thread has some requests side by side: their sums, the sums before them, then each
  // of them again (its lengths are in the SM's cache by then).
  const int per = (a.batch + kAssignThreads - 1) / kAssignThreads;
  const int first_b = tid * per, end_b = min(a.batch, first_b + per);
  struct Request {
    int L, n, first, need;  // rows, new ones; first fresh page, fresh pages
  };
  auto request = [&](int b, bool report) -> Request {
    Request r{__ldg(a.seq_len + b), a.new_len != nullptr ? __ldg(a.new_len + b) : 1, 0, 0};
    int code = 0;
    if (r.L < 1 || r.L > a.max_pages * kPage) code = DSA_DEV_BAD_SEQ_LEN;
    else if (r.n < 0 || r.n > r.L) code = DSA_DEV_BAD_QLEN;
    if (code != 0) {
      if (report) set_error(a.err, code);
      r.L = r.n = 0;
    }
    r.first = (r.L - r.n + kPage - 1) / kPage;
    r.need = (r.L + kPage - 1) / kPage - r.first;
    return r;
  };
  int64_t rows = 0, pages = 0;
#pragma unroll 4
  for (int b = first_b; b < end_b; ++b) {
    const Request r = request(b, first_cta);
    rows += r.n;
    pages += r.need;
  }
  const int64_t own_rows = rows, own_pages = pages;
  rows = warp_scan(rows, lane);
  pages = warp_scan(pages, lane);
  if (lane == 31) {
    rows_of[warp] = rows;
    pages_of[warp] = pages;
  }
  __syncthreads();
  // The last CTA to come by here stores the count at its end: all have read theirs.
  bool last = gridDim.x == 1;
  if (tid == 0 && !last) {
    __threadfence();
    last = atomicAdd(a.done, 1) == static_cast<int32_t>(gridDim.x) - 1;
  }
  int64_t total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) {
      rows += rows_of[w];
      pages += pages_of[w];
    }
    total += rows_of[w];
  }
  rows -= own_rows;  // before this thread's requests
  pages -= own_pages;
  int32_t taken = 0;  // pages up to the last request that is served
  for (int b = first_b; b < end_b; ++b) {
    const Request r = request(b, false);
    if (first_cta && a.token_start != nullptr)
      a.token_start[b] = static_cast<int32_t>(rows < INT32_MAX ? rows : INT32_MAX);
    const bool served = r.need == 0 || pages + r.need <= count;
    if (r.need > 0 && served) taken = static_cast<int32_t>(pages + r.need);
    if (!served && first_cta) set_error(a.err, DSA_DEV_FREE_LIST_EMPTY);
    // the request's first row in this tile, if it has one
    const int64_t at = rows > t0 ? rows : t0;
    if (r.n > 0 && at < t0 + kAssignThreads && at < rows + r.n) {
      const int x = static_cast<int>(at - t0);
      req[x] = TileRequest{b, static_cast<int32_t>(r.L - r.n + (at - rows)), r.first, served,
                           served && r.need > 0 ? count - 1 - static_cast<int32_t>(pages) : 0};
      owner[x] = x;
    }
    rows += r.n;
    pages += r.need;
  }
  taken = __reduce_max_sync(0xffffffffu, taken);
  if (lane == 0) taken_of[warp] = taken;
  __syncthreads();
  const bool fits = total <= a.max_tokens;
  if (first_cta && tid == 0) {
    if (a.token_start != nullptr)
      a.token_start[a.batch] = static_cast<int32_t>(total < INT32_MAX ? total : INT32_MAX);
    if (!fits) set_error(a.err, DSA_DEV_BAD_COUNT);
  }
  // the request of a row: the last one that starts at or before it
  int own = owner[tid];
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, own, s);
    if (lane >= s) own = max(own, v);
  }
  if (lane == 31) owner_of[warp] = own;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w)
    if (w < warp) own = max(own, owner_of[w]);
  const int64_t t = t0 + tid;
  if (t < a.max_tokens) {
    int32_t slot = -1, row = 0;
    if (fits && t < total && own >= 0) {
      const TileRequest r = req[own];
      row = r.row + (tid - own);
      const int p = row / kPage;
      if (r.served != 0) {
        int32_t pg;
        int32_t* entry = a.page_table + static_cast<size_t>(r.b) * a.max_pages + p;
        if (p >= r.first) {
          pg = a.free_pages[r.take - (p - r.first)];
          if (static_cast<uint32_t>(pg) >= static_cast<uint32_t>(a.num_pages)) {
            set_error(a.err, DSA_DEV_BAD_PAGE);
            pg = -1;
          }
          if (row % kPage == 0) *entry = pg;
        } else {
          pg = *entry;
          if (static_cast<uint32_t>(pg) >= static_cast<uint32_t>(a.num_pages)) {
            set_error(a.err, DSA_DEV_BAD_PAGE);
            pg = -1;
          }
        }
        if (pg >= 0) slot = pg * kPage + row % kPage;
      }
    }
    a.row_slot[t] = slot;
    if (a.row_pos != nullptr) a.row_pos[t] = row;
  }
  if (tid == 0 && last) {
    if (gridDim.x > 1) *a.done = 0;
    for (int w = 1; w < kWarps; ++w) taken = max(taken, taken_of[w]);
    *a.free_out = count - (fits ? taken : 0);
  }
}

constexpr int kWriteThreads = 256;
constexpr int kWriteVecs = 4;  // 16-byte pieces of a thread

// A warp takes 2 KB of a row of K or V.
__global__ void __launch_bounds__(kWriteThreads) write_kernel(const RowsLaunch a, int parts, int both,
                                                             int64_t units) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * (kWriteThreads / 32) + (threadIdx.x >> 5);
  if (unit >= units) return;
  const int part = static_cast<int>(unit % parts);
  const int64_t rest = unit / parts;
  const int x = both != 0 ? static_cast<int>(rest & 1) : (a.rows[0] != nullptr ? 0 : 1);
  const int64_t t = both != 0 ? rest >> 1 : rest;
  const int32_t slot = __ldg(a.row_slot + t);
  const unsigned char* from = static_cast<const unsigned char*>(a.rows[x]) + t * a.stride[x];
  uint4 v[kWriteVecs];
  const int at = part * (512 * kWriteVecs) + 16 * lane;
#pragma unroll
  for (int i = 0; i < kWriteVecs; ++i)
    if (at + 512 * i < a.row_bytes) v[i] = __ldg(reinterpret_cast<const uint4*>(from + at + 512 * i));
  if (slot < 0) return;  // a row without a slot
  if (slot >= a.slots) {
    if (lane == 0) set_error(a.err, DSA_DEV_BAD_PAGE);
    return;
  }
  unsigned char* to = static_cast<unsigned char*>(a.pages[x]) + static_cast<int64_t>(slot) * a.row_bytes;
#pragma unroll
  for (int i = 0; i < kWriteVecs; ++i)
    if (at + 512 * i < a.row_bytes) *reinterpret_cast<uint4*>(to + at + 512 * i) = v[i];
}

}  // namespace

cudaError_t launch_assign_pages(const AssignLaunch& a, cudaStream_t s) {
  const int64_t tiles = (static_cast<int64_t>(a.max_tokens) + kAssignThreads - 1) / kAssignThreads;
  return launch_pdl(assign_kernel, dim3(static_cast<unsigned>(tiles > 1 ? tiles : 1)),
                    dim3(kAssignThreads), 0, s, a);
}

cudaError_t launch_write_rows(const RowsLaunch& a, cudaStream_t s) {
  const int parts = (a.row_bytes + 512 * kWriteVecs - 1) / (512 * kWriteVecs);
  const int both = a.rows[0] != nullptr && a.rows[1] != nullptr;
  const int64_t units = static_cast<int64_t>(a.tokens) * (1 + both) * parts;
  const int64_t ctas = (units + kWriteThreads / 32 - 1) / (kWriteThreads / 32);
  if (ctas > INT32_MAX) return cudaErrorInvalidValue;
  return launch_pdl(write_kernel, dim3(static_cast<unsigned>(ctas)), dim3(kWriteThreads), 0, s, a, parts,
                    both, units);
}

}  // namespace dsa
