// internal.h -- host-side launch interface between the C ABI and the kernels.
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

namespace dsa {

// Rows of one decode / mass work unit are split into chunks of `chunk` rows;
// each chunk is one CTA.  At most kMaxChunks chunks per (request, kv head).
constexpr int kMaxChunks = 32;
// Largest cluster of decode CTAs sharing one (request, kv head).
constexpr int kMaxCluster = 8;
constexpr int kChunkQuantum = 64;  // chunk sizes are multiples of this

// States (acc[head_dim], reference, sum, padding) that the calls over a shared prefix leave in the
// workspace: those of the prefix's pieces and those of chunks, of one (request, query head)
// `apart` floats from each other (few of them are used, so those read lie together).  They lie in
// the partials region, or, where that holds fewer than four of them, in kSharedExtra of their own.
constexpr int kSharedExtra = 3;
constexpr int kSharedRows = 128, kSharedBlock = 128;  // query rows of a tile, cache rows of a block
struct SharedStates {
  float* pieces;
  float* chunks;
  int64_t apart;
  int32_t floats;  // of a state: head_dim + 4
};

struct DecodeLaunch {
  const void* q;
  int q_bf16;
  const void* k;
  const void* v;
  const int32_t* page_table;
  const int32_t* seq_len;
  const int32_t* kept_idx;  // kRowsList only
  const int32_t* kept_cnt;  // kRowsList only
  const int32_t* prompt_len;  // kRowsMask only
  const int32_t* window;      // kRowsMask only
  const uint32_t* keep_mask;  // kRowsMask only: [batch][hkv][mask_words]
  int32_t* unit_rows;         // kRowsMask only: [batch][hkv] kept count or -error
  const int32_t* order;       // [batch] request scheduled at each grid z, or null (z itself)
  const int32_t* sched;       // kRowsList: [batch] schedule left by dsa_build_index, used
  const int32_t* sched_tag;   //   when *sched_tag == sched_expect (else z itself), or null
  int32_t sched_expect;
  const void* k_new;          // [batch][hkv][head_dim] K/V of row seq_len-1, or null (the
  const void* v_new;          //   cache already holds it); written into its page slot
  int32_t batch, hq, hkv, head_dim, max_pages, num_pages, max_kept;
  int32_t max_window, mask_words;  // kRowsMask only
  int32_t chunk, num_chunks;
  int32_t cluster;   // > 1: the num_chunks (== cluster) CTAs of a unit merge in a cluster
  int32_t warps;     // warps per CTA of the build to launch (see DecodeShape)
  int32_t build;     // kBuildDefault / kBuildBig / kBuildSmall (see DecodeShape)
  float scale_log2;  // softmax scale * log2(e)
  float* out;
  float* lse;
  float* part;  // [batch][hq][num_chunks][head_dim + 2]
  int32_t* err;
};

// The rows behind shared prefixes, and the joining (shared_rest.cu): bf16 q, pages and out.
struct RestLaunch {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  const int32_t* page_table;
  const int32_t* seq_len;
  const int32_t* prefix_len;  // [batch]
  const int32_t* prompt_len;  // masks only
  const int32_t* window;      // masks only
  const uint32_t* keep_mask;  // masks only
  int32_t batch, hq, hkv, head_dim, max_pages, num_pages, max_window, mask_words;
  int32_t max_prefix, max_suffix;
  int32_t chunk, num_chunks;  // rows of a chunk, chunks of a unit at most
  int32_t early;              // behind a prefix kernel
  int32_t deep;               // few warps: more of a warp's rows on their way at a time
  int32_t prefix_slots;       // states that the pieces of a prefix have room for
  float scale_log2;
  SharedStates states;
  int32_t* unit_rows;         // [batch][hkv] rows behind the prefix, or -error
  int32_t* pieces;            // [batch][hq] states of the prefix
  uint16_t* out;
  float* lse;
  int32_t* err;
};

// The prefixes of groups of requests (shared_prefix.cu): bf16 q and pages.
struct SharedLaunch {
  const uint16_t* q;
  const void* k;
  const void* v;
  const int32_t* page_table;
  const int32_t* group_start;  // [groups + 1]
  const int32_t* prefix_len;   // [batch]
  int32_t groups, batch, hq, hkv, group_log2, head_dim, max_pages, num_pages, max_prefix;
  int32_t prefix_slots;        // >= 2
  float scale_log2;
  SharedStates states;
  int32_t* pieces;
  int32_t leave;       // rows of the prefixes leave the L2 first
  int32_t* err;
  int32_t sms;
};

struct MassLaunch {
  const void* q;
  int q_bf16;
  const void* k;
  const int32_t* page_table;
  const int32_t* seq_len;
  const int32_t* prompt_len;
  const int32_t* window;
  const int32_t* grid_w;
  int32_t batch, hq, hkv, head_dim, max_pages, num_pages, max_window;
  int32_t r_local, r_diag;
  int32_t chunk, num_chunks;
  float scale_log2;
  float* mass;         // [batch][hq][4]
  float* offset_mass;  // [batch][hq][max_window+1] or null
  float* part;         // [batch][hq][num_chunks][6]
  int32_t* err;
};

struct CompactLaunch {
  const int32_t* seq_len;
  const int32_t* prompt_len;
  const int32_t* window;
  const uint32_t* keep_mask;
  int32_t* kept_idx;
  int32_t* kept_cnt;
  int32_t batch, hkv, max_pages, max_window, mask_words, max_kept;
  int32_t* err;
  int32_t* sched;       // [batch] requests by decreasing kept rows (written by the last CTA)
  int32_t* sched_tag;   // set to kSchedMagic ^ batch once sched is written
  int32_t* done_count;  // CTAs done; zero between calls
};

struct EvictLaunch {
  const int32_t* seq_len;
  const int32_t* prompt_len;
  const int32_t* window;
  int32_t* page_table;   // [batch][max_pages], evicted entries set to -1
  int32_t* freed;        // [capacity] freed page ids
  int32_t* freed_count;  // appended to atomically
  int32_t batch, max_pages, max_window, capacity;
  int32_t* err;
};

// Several query tokens per request (prefill.cu): q [batch][max_q][hq][head_dim].
struct MultiLaunch {
  const void* q;
  const void* k;
  const void* v;
  const int32_t* page_table;
  const int32_t* seq_len;
  const int32_t* q_len;       // [batch] query tokens of each request (its last rows)
  const int32_t* prompt_len;
  const int32_t* window;
  const uint32_t* keep_mask;  // [batch][hkv][mask_words]
  const int32_t* order;       // [batch] request handed to the GPU at each position, or null
  int32_t batch, hq, hkv, head_dim, max_pages, num_pages, max_window, mask_words, max_q;
  int32_t q_tiles;            // CTAs along the query axis of one (request, kv head)
  int32_t warps;              // warps per CTA (multi_warps)
  float scale_log2;
  float* out;                 // [batch][max_q][hq][head_dim]
  float* lse;                 // [batch][max_q][hq] or null
  int32_t* err;
  // Units are (query tile, kv head, request) in that order, x fastest.  The first
  // n_whole run whole, one CTA each; every later one is split along its scanned
  // rows into `split` parts whose partial states the unit's last-arriving part
  // merges.  Filled by launch_multi from the fields below it.
  int32_t n_whole, split;
  float* part;                // [split unit][part][16 warps][head_dim + 2]
  int32_t* part_count;        // [split unit] arrivals, 0 between launches
  // host only: split setting (0 automatic, 1 never, n: every unit in n parts),
  // partial rows the workspace holds, arrival counters it holds, SMs
  int32_t split_setting;
  int64_t part_rows_cap;
  int32_t count_cap, sms;
};

// Row sources of a decode launch (`mode` below).
constexpr int kModeDense = 0;  // rows 0..L-1
constexpr int kModeList = 1;   // kept_idx / kept_cnt from dsa_build_index
constexpr int kModeMask = 2;   // kept set built in the kernel from keep_mask

// Largest max_window of kModeMask: the kernel holds the window's mask bits one
// 32-bit word per lane of a warp.
constexpr int kMaskModeMaxWindow = 1024;

// Each returns cudaSuccess or the launch error.
cudaError_t launch_decode_bf16(const DecodeLaunch& a, int mode, cudaStream_t s);
cudaError_t launch_decode_f32(const DecodeLaunch& a, int mode, cudaStream_t s);
cudaError_t launch_merge(const DecodeLaunch& a, int mode, cudaStream_t s);
// Rows behind shared prefixes, dense or the kept set of the mask; warps of an SM at a time.
cudaError_t launch_shared_rest(const RestLaunch& a, bool mask, cudaStream_t s);
cudaError_t shared_rest_warps(int head_dim, int group, bool mask, int* warps);
cudaError_t launch_shared_prefix(const SharedLaunch& a, cudaStream_t s);
cudaError_t launch_mass(const MassLaunch& a, bool kv_bf16, cudaStream_t s);
// Rows one pass of all warps of an attention-mass CTA covers, and its resident
// CTAs per SM (>= 1), for the host's chunk choice.
int mass_rows_per_pass(int head_dim, int group, bool kv_bf16, bool q_bf16);
// The attention-mass build for these dtypes scores on the tensor cores.
bool mass_uses_tensor_cores(bool kv_bf16, bool q_bf16, int group);
int mass_ctas_per_sm(int head_dim, int group, bool kv_bf16, bool q_bf16);
cudaError_t launch_compact(const CompactLaunch& a, cudaStream_t s);
// Several query tokens per request: bf16 q and KV only.  Warps per CTA for a
// call (2 when max_q x group fits 32 (query, head) rows, else 4) and the query
// tokens a CTA of that many warps holds.
// The launch of a multi-query call: warps per CTA, units, units run whole,
// parts of each later unit, resident CTAs per SM, CTAs launched.
struct MultiPlan {
  int32_t warps, units, n_whole, parts, ctas_per_sm, ctas;
};
// Plans the launch (into *plan when not null) and launches it unless `launch`
// is false (then nothing is enqueued).
cudaError_t launch_multi(const MultiLaunch& a, cudaStream_t s, MultiPlan* plan = nullptr,
                         bool launch = true);
int multi_warps(int max_q, int group);
int multi_queries_per_cta(int warps, int group);
// Largest max_window of the multi-query call (its mask words sit in shared memory).
constexpr int kMultiMaxWindow = 32768;
// Arrival counters of split multi-query units in the workspace, and the most
// parts a unit is split into.
constexpr int kMultiCounters = 4096;
constexpr int kMultiMaxParts = 8;
// Resident warps per SM of the multi-query kernel the workspace's partials
// region is sized for (6 CTAs of 2 warps, or 3 of 4).
constexpr int kMultiPartWarpsPerSm = 12;
cudaError_t launch_evict(const EvictLaunch& a, cudaStream_t s);

// Host copies of a step (hostio.cu): a copy kernel when the host side is
// page-locked memory the device can address, else cudaMemcpyAsync.
cudaError_t copy_host_to_device(void* dev, const void* host, size_t bytes, cudaStream_t s);
cudaError_t copy_device_to_host(void* host, const void* dev, size_t bytes, cudaStream_t s);

// Builds of the decode kernel.  The sparse calls with bf16 KV have three more
// besides the default: one for batches of more than two waves of units (more
// warps per SM), one for batches that fit one wave only with it (5 warps of a
// single stage, each warp about one tile of a unit), and one for batches of at
// most one unit per SM (8 warps of a single stage: a unit's rows spread over
// the warps of one CTA, merged in its shared memory, no cluster).
enum : int { kBuildDefault = 0, kBuildBig = 1, kBuildSmall = 2, kBuildWide = 3 };

// Host-side facts about one build of the decode kernel, for the chunk choice.
struct DecodeShape {
  int rows_per_pass;  // warps x tile rows
  int ctas_per_sm;    // resident CTAs per SM (>= 1)
  int cluster_limit;  // largest cluster whose merge buffer fits the rings
  int warps;          // warps per CTA of this build
  int tile_rows;      // rows per tile of this build
  int build;          // which build this is
};
// The requested build of (head_dim, group, mode) when there is one, else the
// default build.
DecodeShape decode_shape_bf16(int head_dim, int group, int mode, int build);
DecodeShape decode_shape_f32(int head_dim, int group, int mode, int build);

// ---- 8-bit K/V cache (quant_*.cu) and rotary positions (rope.cu) ----

struct QuantDecodeLaunch {
  const void* q;
  int q_bf16;                // else fp32; out has the same type
  const uint8_t* k;          // [num_pages][hkv][16][head_dim] e4m3
  const uint8_t* v;
  const float* k_scale;      // [num_pages][hkv]
  const float* v_scale;
  const int32_t* page_table;
  const int32_t* seq_len;
  const int32_t* kept_idx;    // kModeList only
  const int32_t* kept_cnt;    // kModeList only
  const int32_t* prompt_len;  // kModeMask only
  const int32_t* window;      // kModeMask only
  const uint32_t* keep_mask;  // kModeMask only
  const int32_t* order;       // kModeMask only: request at each position, or null
  const int32_t* sched;       // kModeList only: as in DecodeLaunch
  const int32_t* sched_tag;
  int32_t sched_expect;
  int32_t batch, hq, hkv, group, head_dim, max_pages, num_pages, max_kept;
  int32_t max_window, mask_words;
  float scale_log2;
  void* out;
  float* lse;
  float* part;       // partial states, quant_part_floats() each
  int32_t* count;    // arrival counters, 0 between launches
  int32_t* err;
  int32_t parts;     // sparse rows: CTAs per unit at most (set by the launch)
  int32_t min_tiles; // dense rows: least tiles per CTA (set by the launch)
  int64_t part_cap;  // floats the workspace holds at `part`
  int32_t sms;
};

// Floats of one partial state of `group` heads, whole 16-byte pieces.
constexpr __host__ __device__ int quant_part_floats(int group, int head_dim) {
  return (group * (head_dim + 2) + 3) / 4 * 4;
}
// Most CTAs that share one unit of sparse rows, and the least tiles (16 rows) a CTA of the
// dense call takes, unless that would leave fewer CTAs than units: four for each of its warps
// (48 units of 2 .. 4 rows: 25 us with 3 CTAs, 3.6 with 48).
constexpr int kQuantMaxParts = 8;
constexpr int kQuantMinTiles = 16;

// Pages of a request up to which the tcgen05 chunk kernels take few tiles too (2048 rows).
constexpr int kQuantWholePages = 128;

// Several query tokens per request over the 8-bit cache: q and out bf16.
struct QuantChunkLaunch {
  const uint16_t* q;  // [batch][max_q][hq][head_dim] bf16
  const uint8_t* k;
  const uint8_t* v;
  const float* k_scale;
  const float* v_scale;
  const int32_t* page_table;
  const int32_t* seq_len;
  const int32_t* q_len;
  const int32_t* prompt_len;
  const int32_t* window;
  const uint32_t* keep_mask;
  const int32_t* order;
  int32_t batch, hq, hkv, group_log2, head_dim, max_pages, num_pages;
  int32_t max_window, mask_words, max_q;
  float scale_log2;
  uint16_t* out;
  float* lse;
  float* part;
  int32_t* count;
  int32_t* err;
  int64_t part_cap;
  int32_t q_tiles, parts;  // set by the launch
  int32_t sms;
  int32_t split_setting;   // dsa_set_prefill_split
};

struct QuantRowsLaunch {
  uint8_t* k;
  uint8_t* v;
  float* k_scale;
  float* v_scale;
  int rows_bf16;             // type of the rows outside the cache, else fp32
  const void* k_rows;        // write: new rows
  const void* v_rows;
  void* k_out;               // read: where the rows go, or null
  void* v_out;
  int64_t stride;            // write: elements between two row slots
  const int32_t* page_table;
  const int32_t* seq_len;
  const int32_t* start;      // read: first row of each request
  const int32_t* count;      // rows of each request, or null (max_rows each)
  int32_t batch, hkv, head_dim, max_pages, num_pages;
  int32_t max_rows, slots;   // row slots per request; pages they can touch
  int32_t* err;
};

struct RopeLaunch {
  const void* q;
  const void* k;
  void* q_out;
  void* k_out;
  int64_t q_stride, k_stride, q_out_stride, k_out_stride;  // elements between tokens
  const int32_t* positions;  // [tokens][axes]
  int32_t tokens, hq, hkv, head_dim, axes, neighbours;
  int q_bf16, k_bf16;
  uint64_t turn[64];         // pair i: 2^64 turns per position, modulo 2^64
  uint8_t pair_axis[64];
};

// ---- head norms (qk_norm.cu), pages and rows (pages.cu) ----

struct NormLaunch {
  RopeLaunch rope;
  // per head kind (0: q, 1: k): weight and bias, or null; of every head's own when per_head
  const void* weight[2];
  const void* bias[2];
  int32_t layer, per_head, weight_bf16;
  float eps;
  // set by the launch: heads of q and of k, tokens per CTA, threads per token, tokens side by
  // side, whether a pair does not turn
  int32_t q_heads, k_heads, tile, lanes, subs, still;
};

struct AssignLaunch {
  const int32_t* seq_len;
  const int32_t* new_len;    // or null: one row each
  const int32_t* free_pages;
  const int32_t* free_count;
  int32_t* free_out;         // may be free_count
  int32_t* page_table;
  int32_t* token_start;      // [batch + 1], or null
  int32_t* row_slot;         // [max_tokens]
  int32_t* row_pos;          // [max_tokens], or null
  int32_t batch, max_pages, num_pages, capacity, max_tokens;
  int32_t* err;
  int32_t* done;             // CTAs done, zero between calls
};

struct RowsLaunch {
  const int32_t* row_slot;
  const void* rows[2];       // K, V; null: not written
  void* pages[2];
  int64_t stride[2];         // bytes between two rows
  int64_t slots;             // num_pages * 16
  int32_t tokens, row_bytes;
  int32_t* err;
};

cudaError_t launch_qk_norm_rope(NormLaunch a, int sms, cudaStream_t s);
cudaError_t launch_assign_pages(const AssignLaunch& a, cudaStream_t s);
cudaError_t launch_write_rows(const RowsLaunch& a, cudaStream_t s);

cudaError_t launch_quant_decode(const QuantDecodeLaunch& a, int mode, cudaStream_t s);
cudaError_t launch_quant_chunk(const QuantChunkLaunch& a, cudaStream_t s);
// The tcgen05 kernels of the call (_tc: head_dim 128), and whether one takes a call: _tc with the
// queries as columns (few of them per request), _rows with the queries as rows.
bool quant_chunk_rows_fits(const QuantChunkLaunch& a);
cudaError_t launch_quant_chunk_rows(const QuantChunkLaunch& a, cudaStream_t s);
bool quant_chunk_tc_fits(const QuantChunkLaunch& a);
cudaError_t launch_quant_chunk_tc(const QuantChunkLaunch& a, cudaStream_t s);
cudaError_t launch_quant_write(const QuantRowsLaunch& a, cudaStream_t s);
cudaError_t launch_quant_read(const QuantRowsLaunch& a, cudaStream_t s);
cudaError_t launch_rope(const RopeLaunch& a, int sms, cudaStream_t s);

}  // namespace dsa
