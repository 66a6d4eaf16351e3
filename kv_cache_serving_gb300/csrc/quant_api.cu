// quant_api.cu -- the extern "C" entry points of the 8-bit K/V cache and of the rotary
// positions (declared in dsa.h): host-side checks and dispatch.
#include <cmath>
#include <cstdint>
#include <cstring>

#include <cuda_runtime.h>

#include "common.cuh"
#include "dsa.h"
#include "host.h"
#include "internal.h"

namespace dsa {
namespace {

dsa_status check_cache(const dsa_dims* d, const dsa_quant_cache* c) {
  if (c == nullptr || !c->k_codes || !c->v_codes || !c->k_scale || !c->v_scale)
    return DSA_ERR_INVALID_ARG;
  if (!aligned(c->k_codes, 16) || !aligned(c->v_codes, 16) || !aligned(c->k_scale, 4) ||
      !aligned(c->v_scale, 4))
    return DSA_ERR_INVALID_ARG;
  // rows of a pool are numbered in 32 bits
  if (static_cast<int64_t>(d->num_pages) * d->hkv * kPage > UINT32_MAX) return DSA_ERR_UNSUPPORTED;
  return DSA_OK;
}

int64_t part_floats(const dsa_dims* d) {
  return static_cast<int64_t>(partials_region(d) / sizeof(float));
}

bool finite(float x) { return std::isfinite(x); }

dsa_status decode_quant(const dsa_dims* d, int mode, const void* q, const dsa_quant_cache* c,
                        const int32_t* page_table, const int32_t* seq_len, QuantDecodeLaunch a,
                        float scale, void* out, float* lse, void* ws, void* stream) {
  dsa_status st = check_dims(d);
  if (st != DSA_OK) return st;
  if (d->batch == 0) return DSA_OK;
  if (!q || !page_table || !seq_len || !out || !ws) return DSA_ERR_INVALID_ARG;
  if (mode == kModeList && (!a.kept_idx || !a.kept_cnt)) return DSA_ERR_INVALID_ARG;
  if (mode == kModeMask && (!a.prompt_len || !a.window || !a.keep_mask)) return DSA_ERR_INVALID_ARG;
  if (!finite(scale) || !aligned(ws, 256) || !aligned(q, 16) || !aligned(out, 16) ||
      !aligned(lse, 4))
    return DSA_ERR_INVALID_ARG;
  st = check_cache(d, c);
  if (st != DSA_OK) return st;
  if (mode == kModeMask && d->max_window > kMaskModeMaxWindow) return DSA_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(d->batch) * d->hkv * kQuantMaxParts > INT32_MAX)
    return DSA_ERR_UNSUPPORTED;
  a.q = q;
  a.q_bf16 = d->q_dtype == DSA_BF16;
  a.k = static_cast<const uint8_t*>(c->k_codes);
  a.v = static_cast<const uint8_t*>(c->v_codes);
  a.k_scale = c->k_scale;
  a.v_scale = c->v_scale;
  a.page_table = page_table;
  a.seq_len = seq_len;
  if (mode == kModeList) {
    a.sched = sched_region(d, ws);
    a.sched_tag = err_word(ws) + kWsSchedTag;
    a.sched_expect = kSchedMagic ^ d->batch;
  }
  a.batch = d->batch;
  a.hq = d->hq;
  a.hkv = d->hkv;
  a.group = d->hq / d->hkv;
  a.head_dim = d->head_dim;
  a.max_pages = d->max_pages_per_req;
  a.num_pages = d->num_pages;
  a.max_kept = d->max_kept;
  a.max_window = d->max_window;
  a.mask_words = d->mask_words;
  a.scale_log2 = scale * kLog2e;
  a.out = out;
  a.lse = lse;
  a.part = partials(ws);
  a.part_cap = part_floats(d);
  a.count = multi_count_region(d, ws);
  a.err = err_word(ws);
  a.sms = sm_count();
  return from_cuda(launch_quant_decode(a, mode, static_cast<cudaStream_t>(stream)));
}

// Pages that `rows` consecutive rows can touch, whatever row they start at.
int64_t page_slots(int64_t rows) { return (rows + kPage - 2) / kPage + 1; }

dsa_status rows_common(const dsa_dims* d, const dsa_quant_cache* c, int32_t max_rows,
                       const int32_t* page_table, const int32_t* seq_len, void* ws,
                       QuantRowsLaunch* a) {
  a->k = static_cast<uint8_t*>(c->k_codes);
  a->v = static_cast<uint8_t*>(c->v_codes);
  a->k_scale = c->k_scale;
  a->v_scale = c->v_scale;
  a->rows_bf16 = d->kv_dtype == DSA_BF16;
  a->page_table = page_table;
  a->seq_len = seq_len;
  a->batch = d->batch;
  a->hkv = d->hkv;
  a->head_dim = d->head_dim;
  a->max_pages = d->max_pages_per_req;
  a->num_pages = d->num_pages;
  a->max_rows = max_rows;
  const int64_t slots = page_slots(max_rows);
  const int64_t most = d->max_pages_per_req;
  a->slots = static_cast<int32_t>(slots < most ? slots : most);
  a->err = err_word(ws);
  if (static_cast<int64_t>(d->batch) * a->slots > INT32_MAX / (2 * static_cast<int64_t>(d->hkv)))
    return DSA_ERR_UNSUPPORTED;
  return DSA_OK;
}

// f radians (0 <= f <= 2 pi) in turns, as a 64-bit fraction (a whole turn is none), to half a unit:
// the double's whole mantissa times 1 / (2 pi) to 128 bits, so that a position of 31 bits times
// the result is still good to 2^-34 turns.
uint64_t turns_of(double f) {
  using u128 = unsigned __int128;
  uint64_t bits;
  std::memcpy(&bits, &f, sizeof bits);
  if ((bits >> 52) == 0) return 0;  // 0, or a subnormal: no turn at any position
  const int e = static_cast<int>(bits >> 52) - 1022;
  const uint64_t m = (bits & ((1ull << 52) - 1)) | (1ull << 52);  // f = m 2^(e - 53)
  // 2^130 / (2 pi), rounded down
  constexpr uint64_t hi = 0xa2f9836e4e441529ull, lo = 0xfc2757d1f534ddc0ull;
  const u128 p = static_cast<u128>(m) * hi + ((static_cast<u128>(m) * lo) >> 64);  // m / (2 pi) 2^66
  const int shift = 55 - e;  // to f / (2 pi) 2^64; at least 52, as f < 2^3
  return shift >= 127 ? 0 : static_cast<uint64_t>((p + (static_cast<u128>(1) << (shift - 1))) >> shift);
}

}  // namespace

// The checks and the launch of dsa_rope_axes and dsa_qk_norm_rope; tokens 0: nothing to do.
dsa_status make_rope_launch(const dsa_dims* dims, const dsa_rope* rope, int32_t tokens,
                       const int32_t* positions, const void* q, int64_t q_stride, const void* k,
                       int64_t k_stride, void* q_out, int64_t q_out_stride, void* k_out,
                       int64_t k_out_stride, RopeLaunch* launch) {
  const dsa_status st = check_dims(dims);
  if (st != DSA_OK) return st;
  if (rope == nullptr || tokens < 0 || (q == nullptr) != (q_out == nullptr) ||
      (k == nullptr) != (k_out == nullptr))
    return DSA_ERR_INVALID_ARG;
  if (rope->axes < 1 || rope->axes > 4 ||
      (rope->pairing != DSA_ROPE_HALVES && rope->pairing != DSA_ROPE_NEIGHBOURS))
    return DSA_ERR_INVALID_ARG;
  const int pairs = dims->head_dim / 2;
  RopeLaunch& a = *launch;
  a = RopeLaunch{};
  for (int i = 0; i < pairs; ++i) {
    const double f = rope->inv_freq[i];
    if (!std::isfinite(f) || std::fabs(f) > 6.283185307179587 || rope->pair_axis[i] >= rope->axes)
      return DSA_ERR_INVALID_ARG;
    const uint64_t t = turns_of(std::fabs(f));
    a.turn[i] = f < 0 ? 0 - t : t;
    a.pair_axis[i] = rope->pair_axis[i];
  }
  if (tokens == 0 || (q == nullptr && k == nullptr)) return DSA_OK;
  if (positions == nullptr || !aligned(positions, 4)) return DSA_ERR_INVALID_ARG;
  const int qe = dims->q_dtype == DSA_BF16 ? 2 : 4, ke = dims->kv_dtype == DSA_BF16 ? 2 : 4;
  const int64_t qw = static_cast<int64_t>(dims->hq) * dims->head_dim;
  const int64_t kw = static_cast<int64_t>(dims->hkv) * dims->head_dim;
  if (q != nullptr && (!aligned(q, 16) || !aligned(q_out, 16) || !row_stride_ok(q_stride, qw, qe) ||
                       !row_stride_ok(q_out_stride, qw, qe) ||
                       (q == q_out && q_stride != q_out_stride)))
    return DSA_ERR_INVALID_ARG;
  if (k != nullptr && (!aligned(k, 16) || !aligned(k_out, 16) || !row_stride_ok(k_stride, kw, ke) ||
                       !row_stride_ok(k_out_stride, kw, ke) ||
                       (k == k_out && k_stride != k_out_stride)))
    return DSA_ERR_INVALID_ARG;
  if (4 * (qw + kw) / 16 > INT32_MAX) return DSA_ERR_UNSUPPORTED;
  a.q = q;
  a.k = k;
  a.q_out = q_out;
  a.k_out = k_out;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.q_out_stride = q_out_stride;
  a.k_out_stride = k_out_stride;
  a.positions = positions;
  a.tokens = tokens;
  a.hq = dims->hq;
  a.hkv = dims->hkv;
  a.head_dim = dims->head_dim;
  a.axes = rope->axes;
  a.neighbours = rope->pairing == DSA_ROPE_NEIGHBOURS;
  a.q_bf16 = dims->q_dtype == DSA_BF16;
  a.k_bf16 = dims->kv_dtype == DSA_BF16;
  return DSA_OK;
}

}  // namespace dsa

using namespace dsa;

extern "C" {

dsa_status dsa_rope_axes(const dsa_dims* dims, const dsa_rope* rope, int32_t tokens,
                         const int32_t* positions, const void* q, int64_t q_stride, const void* k,
                         int64_t k_stride, void* q_out, int64_t q_out_stride, void* k_out,
                         int64_t k_out_stride, void* stream) {
  RopeLaunch a{};
  const dsa_status st = make_rope_launch(dims, rope, tokens, positions, q, q_stride, k, k_stride,
                                         q_out, q_out_stride, k_out, k_out_stride, &a);
  if (st != DSA_OK || a.tokens == 0) return st;
  return from_cuda(launch_rope(a, sm_count(), static_cast<cudaStream_t>(stream)));
}

dsa_status dsa_quant_write(const dsa_dims* dims, const dsa_quant_cache* cache, int32_t max_new,
                           const void* k_new, const void* v_new, int64_t new_stride,
                           const int32_t* page_table, const int32_t* seq_len,
                           const int32_t* new_len, void* ws, void* stream) {
  dsa_status st = check_dims(dims);
  if (st != DSA_OK) return st;
  if (max_new < 0) return DSA_ERR_INVALID_ARG;
  if (dims->batch == 0 || max_new == 0) return DSA_OK;
  if (!k_new || !v_new || !page_table || !seq_len || !ws) return DSA_ERR_INVALID_ARG;
  if (!aligned(ws, 256) || !aligned(k_new, 16) || !aligned(v_new, 16) ||
      !row_stride_ok(new_stride, static_cast<int64_t>(dims->hkv) * dims->head_dim,
                     dims->kv_dtype == DSA_BF16 ? 2 : 4))
    return DSA_ERR_INVALID_ARG;
  st = check_cache(dims, cache);
  if (st != DSA_OK) return st;
  QuantRowsLaunch a{};
  st = rows_common(dims, cache, max_new, page_table, seq_len, ws, &a);
  if (st != DSA_OK) return st;
  a.k_rows = k_new;
  a.v_rows = v_new;
  a.stride = new_stride;
  a.count = new_len;
  return from_cuda(launch_quant_write(a, static_cast<cudaStream_t>(stream)));
}

dsa_status dsa_quant_read(const dsa_dims* dims, const dsa_quant_cache* cache, int32_t max_rows,
                          const int32_t* page_table, const int32_t* seq_len,
                          const int32_t* row_start, const int32_t* row_count, void* k_out,
                          void* v_out, void* ws, void* stream) {
  dsa_status st = check_dims(dims);
  if (st != DSA_OK) return st;
  if (max_rows < 0) return DSA_ERR_INVALID_ARG;
  if (dims->batch == 0 || max_rows == 0 || (!k_out && !v_out)) return DSA_OK;
  if (!page_table || !seq_len || !row_start || !row_count || !ws) return DSA_ERR_INVALID_ARG;
  if (!aligned(ws, 256) || !aligned(k_out, 16) || !aligned(v_out, 16)) return DSA_ERR_INVALID_ARG;
  st = check_cache(dims, cache);
  if (st != DSA_OK) return st;
  QuantRowsLaunch a{};
  st = rows_common(dims, cache, max_rows, page_table, seq_len, ws, &a);
  if (st != DSA_OK) return st;
  a.k_out = k_out;
  a.v_out = v_out;
  a.start = row_start;
  a.count = row_count;
  return from_cuda(launch_quant_read(a, static_cast<cudaStream_t>(stream)));
}

dsa_status dsa_decode_dense_quant(const dsa_dims* dims, const void* q,
                                  const dsa_quant_cache* cache, const int32_t* page_table,
                                  const int32_t* seq_len, float scale, void* out, float* lse,
                                  void* ws, void* stream) {
  return decode_quant(dims, kModeDense, q, cache, page_table, seq_len, QuantDecodeLaunch{}, scale,
                      out, lse, ws, stream);
}

dsa_status dsa_decode_sparse_quant(const dsa_dims* dims, const void* q,
                                   const dsa_quant_cache* cache, const int32_t* page_table,
                                   const int32_t* seq_len, const int32_t* kept_idx,
                                   const int32_t* kept_cnt, float scale, void* out, float* lse,
                                   void* ws, void* stream) {
  QuantDecodeLaunch a{};
  a.kept_idx = kept_idx;
  a.kept_cnt = kept_cnt;
  return decode_quant(dims, kModeList, q, cache, page_table, seq_len, a, scale, out, lse, ws,
                      stream);
}

dsa_status dsa_decode_sparse_masked_quant(const dsa_dims* dims, const void* q,
                                          const dsa_quant_cache* cache, const int32_t* page_table,
                                          const int32_t* seq_len, const int32_t* prompt_len,
                                          const int32_t* window, const uint32_t* keep_mask,
                                          const int32_t* request_order, float scale, void* out,
                                          float* lse, void* ws, void* stream) {
  QuantDecodeLaunch a{};
  a.prompt_len = prompt_len;
  a.window = window;
  a.keep_mask = keep_mask;
  a.order = request_order;
  return decode_quant(dims, kModeMask, q, cache, page_table, seq_len, a, scale, out, lse, ws,
                      stream);
}

dsa_status dsa_prefill_sparse_quant(const dsa_dims* dims, int32_t max_q, const void* q,
                                    const dsa_quant_cache* cache, const int32_t* page_table,
                                    const int32_t* seq_len, const int32_t* q_len,
                                    const int32_t* prompt_len, const int32_t* window,
                                    const uint32_t* keep_mask, const int32_t* request_order,
                                    float scale, void* out, float* lse, void* ws, void* stream) {
  dsa_status st = check_dims(dims);
  if (st != DSA_OK) return st;
  if (max_q < 0) return DSA_ERR_INVALID_ARG;
  if (dims->q_dtype != DSA_BF16 || dims->max_window > kMultiMaxWindow) return DSA_ERR_UNSUPPORTED;
  if (dims->batch == 0 || max_q == 0) return DSA_OK;
  if (!q || !page_table || !seq_len || !q_len || !prompt_len || !window ||
      !keep_mask || !out || !ws)
    return DSA_ERR_INVALID_ARG;
  if (!finite(scale) || !aligned(ws, 256) || !aligned(q, 16) || !aligned(out, 16) ||
      !aligned(lse, 4))
    return DSA_ERR_INVALID_ARG;
  st = check_cache(dims, cache);
  if (st != DSA_OK) return st;
  if (static_cast<int64_t>(dims->batch) * dims->hkv > INT32_MAX / kQuantMaxParts ||
      static_cast<int64_t>(dims->batch) * dims->hkv * ceil_div(max_q, 4) > INT32_MAX)
    return DSA_ERR_UNSUPPORTED;
  // queries of a tile may be read again after its first output (NaN in V)
  const uintptr_t bytes = static_cast<uintptr_t>(dims->batch) * max_q * dims->hq * dims->head_dim * 2;
  const uintptr_t qa = reinterpret_cast<uintptr_t>(q), oa = reinterpret_cast<uintptr_t>(out);
  if (qa < oa + bytes && oa < qa + bytes) return DSA_ERR_INVALID_ARG;
  QuantChunkLaunch a{};
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint8_t*>(cache->k_codes);
  a.v = static_cast<const uint8_t*>(cache->v_codes);
  a.k_scale = cache->k_scale;
  a.v_scale = cache->v_scale;
  a.page_table = page_table;
  a.seq_len = seq_len;
  a.q_len = q_len;
  a.prompt_len = prompt_len;
  a.window = window;
  a.keep_mask = keep_mask;
  a.order = request_order;
  a.batch = dims->batch;
  a.hq = dims->hq;
  a.hkv = dims->hkv;
  const int g = dims->hq / dims->hkv;
  a.group_log2 = g == 1 ? 0 : g == 2 ? 1 : g == 4 ? 2 : 3;
  a.head_dim = dims->head_dim;
  a.max_pages = dims->max_pages_per_req;
  a.num_pages = dims->num_pages;
  a.max_window = dims->max_window;
  a.mask_words = dims->mask_words;
  a.max_q = max_q;
  a.scale_log2 = scale * kLog2e;
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  a.part = partials(ws);
  a.part_cap = part_floats(dims);
  a.count = multi_count_region(dims, ws);
  a.err = err_word(ws);
  a.sms = sm_count();
  a.split_setting = dsa_get_prefill_split();
  return from_cuda(launch_quant_chunk(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
