// host.h -- host-side helpers shared by the C entry points: checks of the dims
// and pointers, the device's SM count, and the regions of the workspace.
#pragma once

#include <atomic>
#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

#include "common.cuh"
#include "dsa.h"
#include "internal.h"

namespace dsa {

constexpr int kMaxDevices = 64;

// Resident CTAs per SM of one kernel at one shared-memory size, and the permission to
// launch with it, asked of the runtime once per device (each call of it costs a
// microsecond of a decode step's launch).  One object per kernel; any thread.
class KernelSlots {
 public:
  // `all_shared`: an SM that runs the kernel is set up with all the shared memory there is, so
  // that CTAs of another kernel fit beside it.
  cudaError_t get(const void* kern, int threads, int smem, int* per_sm, bool all_shared = false) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool known = dev >= 0 && dev < kMaxDevices;
    const uint64_t want = (static_cast<uint64_t>(static_cast<uint32_t>(smem)) << 32) | 0x80000000u;
    if (known) {
      const uint64_t v = cache_[dev].load(std::memory_order_acquire);
      if ((v & ~0x7fffffffull) == want) {
        *per_sm = static_cast<int>(v & 0x7fffffffu);
        return cudaSuccess;
      }
    }
    // the permission never shrinks: a launch of another size on another thread keeps it
    int most = 0;
    e = cudaDeviceGetAttribute(&most, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
    if (e != cudaSuccess) return e;
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, kern);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             most - static_cast<int>(fa.sharedSizeBytes));
    if (e != cudaSuccess) return e;
    if (all_shared) {
      e = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout,
                               cudaSharedmemCarveoutMaxShared);
      if (e != cudaSuccess) return e;
    }
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(per_sm, kern, threads, smem);
    if (e != cudaSuccess) return e;
    if (known) cache_[dev].store(want | static_cast<uint32_t>(*per_sm), std::memory_order_release);
    return *per_sm < 1 ? cudaErrorLaunchOutOfResources : cudaSuccess;
  }

 private:
  std::atomic<uint64_t> cache_[kMaxDevices] = {};
};

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline bool dims_valid(const dsa_dims* d) {
  if (d == nullptr) return false;
  if (d->batch < 0 || d->hq < 1 || d->hkv < 1 || d->head_dim < 1) return false;
  if (d->hq % d->hkv != 0) return false;
  if (d->num_pages < 1 || d->max_pages_per_req < 1 || d->max_window < 0) return false;
  if (d->mask_words < 1 || static_cast<int64_t>(d->mask_words) * 32 < d->max_window) return false;
  if (d->max_kept < 1) return false;
  if (d->q_dtype != DSA_F32 && d->q_dtype != DSA_BF16) return false;
  if (d->kv_dtype != DSA_F32 && d->kv_dtype != DSA_BF16) return false;
  // page_table entries index rows as page * 16 * hkv * head_dim elements in 64-bit math;
  // logical positions are int32.
  if (static_cast<int64_t>(d->max_pages_per_req) * kPage > INT32_MAX / 2) return false;
  return true;
}

inline bool dims_supported(const dsa_dims* d) {
  const int g = d->hq / d->hkv;
  return d->page_size == kPage && (d->head_dim == 64 || d->head_dim == 128) &&
         (g == 1 || g == 2 || g == 4 || g == 8);
}

inline dsa_status check_dims(const dsa_dims* d) {
  if (!dims_valid(d)) return DSA_ERR_INVALID_ARG;
  if (!dims_supported(d)) return DSA_ERR_UNSUPPORTED;
  return DSA_OK;
}

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Upper bound of chunks per (request, kv head) for a row count n_max.
inline int chunk_bound(int64_t n_max) {
  const int64_t c = ceil_div(n_max, kChunkQuantum);
  return static_cast<int>(c < kMaxChunks ? (c < 1 ? 1 : c) : kMaxChunks);
}

inline int64_t dense_rows(const dsa_dims* d) { return static_cast<int64_t>(d->max_pages_per_req) * kPage; }

inline size_t partial_bytes(const dsa_dims* d, int per_head_floats) {
  const int64_t n_max = dense_rows(d) > d->max_kept ? dense_rows(d) : d->max_kept;
  return static_cast<size_t>(d->batch) * d->hq * chunk_bound(n_max) * per_head_floats *
         sizeof(float);
}

inline int sm_count() {
  static int cache[kMaxDevices] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 1;
  if (dev >= 0 && dev < kMaxDevices && cache[dev] > 0) return cache[dev];
  int n = 1;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1)
    n = 1;
  if (dev >= 0 && dev < kMaxDevices) cache[dev] = n;
  return n;
}

inline dsa_status from_cuda(cudaError_t e) { return e == cudaSuccess ? DSA_OK : DSA_ERR_CUDA; }

inline int32_t* err_word(void* ws) { return reinterpret_cast<int32_t*>(ws); }

inline float* partials(void* ws) {
  return reinterpret_cast<float*>(reinterpret_cast<unsigned char*>(ws) + kWsHeader);
}

inline size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// Partials region of the workspace, the same for every entry point.
inline size_t partials_region(const dsa_dims* d) {
  const size_t dec = partial_bytes(d, d->head_dim + 2);
  const size_t mass = partial_bytes(d, 6);
  // dsa_prefill_sparse's split parts: at most one wave of resident CTAs, at
  // most kMultiPartWarpsPerSm warps of 16 (query, head) rows each per SM
  const size_t multi = static_cast<size_t>(sm_count()) * kMultiPartWarpsPerSm * 16 *
                       (d->head_dim + 2) * sizeof(float);
  size_t r = dec > mass ? dec : mass;
  if (multi > r) r = multi;
  return round_up(r, 256);
}

// [batch][hkv] kept counts of dsa_decode_sparse_masked, after the partials.
inline int32_t* unit_rows(const dsa_dims* d, void* ws) {
  return reinterpret_cast<int32_t*>(reinterpret_cast<unsigned char*>(ws) + kWsHeader +
                                    partials_region(d));
}

inline size_t unit_ints_region(const dsa_dims* d) {
  return round_up(static_cast<size_t>(d->batch) * d->hkv * sizeof(int32_t), 256);
}

// [batch] request schedule dsa_build_index leaves for dsa_decode_sparse, after
// the kept counts of the fused call.
inline int32_t* sched_region(const dsa_dims* d, void* ws) {
  return reinterpret_cast<int32_t*>(reinterpret_cast<unsigned char*>(ws) + kWsHeader +
                                    partials_region(d) + unit_ints_region(d));
}

inline size_t sched_bytes(const dsa_dims* d) {
  return round_up(static_cast<size_t>(d->batch) * sizeof(int32_t), 256);
}

// Arrival counters of dsa_prefill_sparse's split units, after the schedule.
inline int32_t* multi_count_region(const dsa_dims* d, void* ws) {
  return reinterpret_cast<int32_t*>(reinterpret_cast<unsigned char*>(ws) + kWsHeader +
                                    partials_region(d) + unit_ints_region(d) + sched_bytes(d));
}

constexpr size_t kMultiCountBytes = kMultiCounters * sizeof(int32_t);

// The calls over a shared prefix.  Their states lie in the partials region; behind the counters
// are [batch][hq] numbers of prefix states, zero between calls, and, for dims whose partials region
// does not hold four states of each (request, query head), kSharedExtra of them.
inline int shared_in_part(const dsa_dims* d) {
  const int64_t n_max = dense_rows(d) > d->max_kept ? dense_rows(d) : d->max_kept;
  return chunk_bound(n_max) * (d->head_dim + 2) / (d->head_dim + 4);
}
inline size_t shared_piece_bytes(const dsa_dims* d) {
  return round_up(static_cast<size_t>(d->batch) * d->hq * sizeof(int32_t), 256);
}
inline int32_t* shared_pieces(const dsa_dims* d, void* ws) {
  return multi_count_region(d, ws) + kMultiCounters;
}
inline float* shared_extra(const dsa_dims* d, void* ws) {
  return reinterpret_cast<float*>(shared_pieces(d, ws) + shared_piece_bytes(d) / sizeof(int32_t));
}
inline bool shared_few(const dsa_dims* d) { return shared_in_part(d) < 4; }
inline size_t shared_bytes(const dsa_dims* d) {
  const size_t extra = shared_few(d) ? static_cast<size_t>(d->batch) * d->hq * kSharedExtra *
                                           (d->head_dim + 4) * sizeof(float)
                                     : 0;
  return shared_piece_bytes(d) + round_up(extra, 256);
}

// Whether a row stride is at least `least` elements and whole 16-byte pieces.
inline bool row_stride_ok(int64_t stride, int64_t least, int elt) {
  return stride >= least && (stride * elt) % 16 == 0;
}

dsa_status make_rope_launch(const dsa_dims* dims, const dsa_rope* rope, int32_t tokens,
                       const int32_t* positions, const void* q, int64_t q_stride, const void* k,
                       int64_t k_stride, void* q_out, int64_t q_out_stride, void* k_out,
                       int64_t k_out_stride, RopeLaunch* launch);

}  // namespace dsa
