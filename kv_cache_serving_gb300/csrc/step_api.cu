// step_api.cu -- the extern "C" entry points around the cache that a serving step calls beside
// the attention (declared in dsa.h): pages and slots for new rows, head norms with the rotary
// positions, rows stored at their slots, and decode attention for requests that share a prefix.
// Host-side checks and dispatch.
#include <cmath>
#include <cstdint>

#include <cuda_runtime.h>

#include "common.cuh"
#include "dsa.h"
#include "host.h"
#include "internal.h"

namespace dsa {
namespace {

// Half waves of resident warps that the rows behind the prefixes are cut for (the host knows a
// bound of a request's rows only), and the rows that a chunk is a multiple of.  128 requests of
// nine prompts, 1 .. 1024 own rows: 60 us cut for six half waves, 63 for eight, ten or twelve.  64
// images, 40 kept rows on the average: 24 us for two half waves, 21.5 for three or four, 22.5 for
// five or six.  Eight requests of 1 .. 300 own rows: 12.8 us in chunks of 64, 13.3 of 32 (more to
// join), 17.8 of 128.
constexpr int kSharedDenseWaves = 6, kSharedMaskWaves = 4, kSharedChunk = 64;

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

dsa_status decode_shared(const dsa_dims* d, bool mask, const dsa_shared_prefix* sh, const void* q,
                         const void* k, const void* v, const int32_t* page_table,
                         const int32_t* seq_len, const int32_t* prompt_len, const int32_t* window,
                         const uint32_t* keep_mask, float scale, void* out, float* lse, void* ws,
                         void* stream) {
  const dsa_status st = check_dims(d);
  if (st != DSA_OK) return st;
  if (sh == nullptr || sh->groups < 0 || sh->max_prefix < 0 || sh->max_suffix < 0)
    return DSA_ERR_INVALID_ARG;
  if (d->batch == 0) return DSA_OK;
  if (!q || !k || !v || !page_table || !seq_len || !out || !ws || !sh->prefix_len ||
      (sh->max_prefix > 0 && (sh->groups < 1 || !sh->group_start)))
    return DSA_ERR_INVALID_ARG;
  if (mask && (!prompt_len || !window || !keep_mask)) return DSA_ERR_INVALID_ARG;
  const size_t bytes = static_cast<size_t>(d->batch) * d->hq * d->head_dim * 2;
  if (!std::isfinite(scale) || !aligned(ws, 256) || !aligned(q, 16) || !aligned(k, 16) ||
      !aligned(v, 16) || !aligned(out, 8) || !aligned(lse, 4) || sh->max_prefix > dense_rows(d) ||
      overlap(q, bytes, out, bytes))
    return DSA_ERR_INVALID_ARG;
  if (d->q_dtype != DSA_BF16 || d->kv_dtype != DSA_BF16 || d->batch > 65535 || d->hkv > 65535 ||
      (mask && d->max_window > kMaskModeMaxWindow))
    return DSA_ERR_UNSUPPORTED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int group = d->hq / d->hkv;
  // blocks of all tiles of the prefixes, and chunks of the rows behind them, are counted in 32 bits
  const int64_t units = static_cast<int64_t>(d->batch) * d->hkv;
  const int64_t tiles = sh->groups + (static_cast<int64_t>(d->batch) * group) / kSharedRows;
  if (sh->groups == INT32_MAX || units * kMaxChunks > INT32_MAX || units * group > INT32_MAX ||
      (sh->max_prefix > 0 &&
       ceil_div(sh->max_prefix, kSharedBlock) > INT32_MAX / 2 / (tiles * d->hkv)))
    return DSA_ERR_UNSUPPORTED;
  RestLaunch a{};
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.page_table = page_table;
  a.seq_len = seq_len;
  a.prefix_len = sh->prefix_len;
  a.prompt_len = prompt_len;
  a.window = window;
  a.keep_mask = keep_mask;
  a.batch = d->batch;
  a.hq = d->hq;
  a.hkv = d->hkv;
  a.head_dim = d->head_dim;
  a.max_pages = d->max_pages_per_req;
  a.num_pages = d->num_pages;
  a.max_window = d->max_window;
  a.mask_words = d->mask_words;
  a.max_prefix = sh->max_prefix;
  a.max_suffix = sh->max_suffix;
  a.early = sh->max_prefix > 0;
  a.scale_log2 = scale * kLog2e;
  a.unit_rows = unit_rows(d, ws);
  a.pieces = shared_pieces(d, ws);
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  a.err = err_word(ws);
  // chunks of the rows behind the prefix, a warp each: some waves of warps, at most half of the
  // states in the workspace
  int warps = 0;
  if (shared_rest_warps(d->head_dim, group, mask, &warps) != cudaSuccess) return DSA_ERR_CUDA;
  // states of a (request, query head): in the partials region where that holds four or more
  const bool few = shared_few(d);
  const int slots = few ? kSharedExtra : shared_in_part(d);
  int64_t parts = static_cast<int64_t>(sm_count()) * warps *
                  (mask ? kSharedMaskWaves : kSharedDenseWaves) / (units * 2);
  if (parts > slots / 2) parts = slots / 2;
  if (parts < 1) parts = 1;
  int64_t rows = sh->max_suffix < dense_rows(d) ? sh->max_suffix : dense_rows(d);
  if (rows < 1) rows = 1;
  a.chunk = static_cast<int32_t>(ceil_div(ceil_div(rows, parts), kSharedChunk) * kSharedChunk);
  a.num_chunks = static_cast<int32_t>(ceil_div(rows, a.chunk));
  a.prefix_slots = slots - a.num_chunks;
  a.states.floats = d->head_dim + 4;
  a.states.apart = static_cast<int64_t>(d->batch) * d->hq * a.states.floats;
  a.states.chunks = few ? shared_extra(d, ws) : partials(ws);
  a.states.pieces = a.states.chunks + a.num_chunks * a.states.apart;
  a.deep = units * a.num_chunks <= static_cast<int64_t>(sm_count()) * 8;
  if (a.early != 0) {
    SharedLaunch p{};
    p.q = a.q;
    p.k = k;
    p.v = v;
    p.page_table = page_table;
    p.group_start = sh->group_start;
    p.prefix_len = sh->prefix_len;
    p.groups = sh->groups;
    p.batch = d->batch;
    p.hq = d->hq;
    p.hkv = d->hkv;
    p.group_log2 = group == 1 ? 0 : group == 2 ? 1 : group == 4 ? 2 : 3;
    p.head_dim = d->head_dim;
    p.max_pages = d->max_pages_per_req;
    p.num_pages = d->num_pages;
    p.max_prefix = sh->max_prefix;
    p.prefix_slots = a.prefix_slots;
    p.scale_log2 = a.scale_log2;
    p.states = a.states;
    p.pieces = a.pieces;
    p.err = a.err;
    p.sms = sm_count();
    if (launch_shared_prefix(p, s) != cudaSuccess) return DSA_ERR_CUDA;
  }
  return from_cuda(launch_shared_rest(a, mask, s));
}

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" {

dsa_status dsa_decode_dense_shared(const dsa_dims* dims, const dsa_shared_prefix* shared,
                                   const void* q, const void* k_pages, const void* v_pages,
                                   const int32_t* page_table, const int32_t* seq_len, float scale,
                                   void* out, float* lse, void* ws, void* stream) {
  return decode_shared(dims, false, shared, q, k_pages, v_pages, page_table, seq_len, nullptr,
                       nullptr, nullptr, scale, out, lse, ws, stream);
}

dsa_status dsa_decode_sparse_masked_shared(const dsa_dims* dims, const dsa_shared_prefix* shared,
                                           const void* q, const void* k_pages, const void* v_pages,
                                           const int32_t* page_table, const int32_t* seq_len,
                                           const int32_t* prompt_len, const int32_t* window,
                                           const uint32_t* keep_mask, float scale, void* out,
                                           float* lse, void* ws, void* stream) {
  return decode_shared(dims, true, shared, q, k_pages, v_pages, page_table, seq_len, prompt_len,
                       window, keep_mask, scale, out, lse, ws, stream);
}

dsa_status dsa_assign_pages(const dsa_dims* dims, const int32_t* seq_len, const int32_t* new_len,
                            const int32_t* free_pages, int32_t capacity,
                            const int32_t* free_count, int32_t* free_count_out,
                            int32_t* page_table, int32_t max_tokens, int32_t* token_start,
                            int32_t* row_slot, int32_t* row_pos, void* ws, void* stream) {
  const dsa_status st = check_dims(dims);
  if (st != DSA_OK) return st;
  if (capacity < 0 || max_tokens < 0 || (capacity > 0 && !free_pages) || !free_count ||
      !free_count_out || !ws || !aligned(ws, 256) || (max_tokens > 0 && !row_slot))
    return DSA_ERR_INVALID_ARG;
  if (dims->batch > 0 && (!seq_len || !page_table)) return DSA_ERR_INVALID_ARG;
  // slots are int32
  if (dims->num_pages > INT32_MAX / kPage) return DSA_ERR_UNSUPPORTED;
  AssignLaunch a{};
  a.seq_len = seq_len;
  a.new_len = new_len;
  a.free_pages = free_pages;
  a.free_count = free_count;
  a.free_out = free_count_out;
  a.page_table = page_table;
  a.token_start = token_start;
  a.row_slot = row_slot;
  a.row_pos = row_pos;
  a.batch = dims->batch;
  a.max_pages = dims->max_pages_per_req;
  a.num_pages = dims->num_pages;
  a.capacity = capacity;
  a.max_tokens = max_tokens;
  a.err = err_word(ws);
  a.done = err_word(ws) + kWsAssignCount;
  return from_cuda(launch_assign_pages(a, static_cast<cudaStream_t>(stream)));
}

dsa_status dsa_write_rows(const dsa_dims* dims, int32_t tokens, const int32_t* row_slot,
                          const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                          void* k_pages, void* v_pages, void* ws, void* stream) {
  const dsa_status st = check_dims(dims);
  if (st != DSA_OK) return st;
  if (tokens < 0 || (k == nullptr) != (k_pages == nullptr) || (v == nullptr) != (v_pages == nullptr))
    return DSA_ERR_INVALID_ARG;
  if (tokens == 0 || (k == nullptr && v == nullptr)) return DSA_OK;
  const int elt = dims->kv_dtype == DSA_BF16 ? 2 : 4;
  const int64_t row = static_cast<int64_t>(dims->hkv) * dims->head_dim;
  if (!row_slot || !aligned(row_slot, 4) || !ws || !aligned(ws, 256) || !aligned(k, 16) ||
      !aligned(v, 16) || !aligned(k_pages, 16) || !aligned(v_pages, 16) ||
      (k != nullptr && !row_stride_ok(k_stride, row, elt)) ||
      (v != nullptr && !row_stride_ok(v_stride, row, elt)))
    return DSA_ERR_INVALID_ARG;
  // a row's bytes, and the warps of 2 KB of a launch, are int32
  if (row * elt > INT32_MAX / 2 ||
      2 * static_cast<int64_t>(tokens) * (ceil_div(row * elt, 2048)) / 8 >= INT32_MAX)
    return DSA_ERR_UNSUPPORTED;
  RowsLaunch a{};
  a.row_slot = row_slot;
  a.rows[0] = k;
  a.rows[1] = v;
  a.pages[0] = k_pages;
  a.pages[1] = v_pages;
  a.stride[0] = k_stride * elt;
  a.stride[1] = v_stride * elt;
  a.slots = static_cast<int64_t>(dims->num_pages) * kPage;
  a.tokens = tokens;
  a.row_bytes = static_cast<int32_t>(row * elt);
  a.err = err_word(ws);
  return from_cuda(launch_write_rows(a, static_cast<cudaStream_t>(stream)));
}

dsa_status dsa_qk_norm_rope(const dsa_dims* dims, const dsa_qk_norm* norm, const dsa_rope* rope,
                            int32_t tokens, const int32_t* positions, const void* q,
                            int64_t q_stride, const void* k, int64_t k_stride, void* q_out,
                            int64_t q_out_stride, void* k_out, int64_t k_out_stride,
                            void* stream) {
  NormLaunch a{};
  const dsa_status st = make_rope_launch(dims, rope, tokens, positions, q, q_stride, k, k_stride,
                                         q_out, q_out_stride, k_out, k_out_stride, &a.rope);
  if (st != DSA_OK) return st;
  if (norm == nullptr || (norm->kind != DSA_NORM_RMS && norm->kind != DSA_NORM_LAYER) ||
      (norm->weight_dtype != DSA_F32 && norm->weight_dtype != DSA_BF16) ||
      !std::isfinite(norm->eps) || norm->eps < 0.f || !aligned(norm->q_weight, 16) ||
      !aligned(norm->k_weight, 16) || !aligned(norm->q_bias, 16) || !aligned(norm->k_bias, 16))
    return DSA_ERR_INVALID_ARG;
  if (a.rope.tokens == 0) return DSA_OK;
  a.weight[0] = norm->q_weight;
  a.weight[1] = norm->k_weight;
  a.bias[0] = norm->q_bias;
  a.bias[1] = norm->k_bias;
  a.layer = norm->kind == DSA_NORM_LAYER;
  a.per_head = norm->per_head != 0;
  a.weight_bf16 = norm->weight_dtype == DSA_BF16;
  a.eps = norm->eps;
  return from_cuda(launch_qk_norm_rope(a, sm_count(), static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
