// shared_prefix.cu -- decode attention over the prefix that the requests of a group share, once
// for the whole group, on the 5th-generation tensor cores.
//
// For a group of n requests with the same first S rows, the queries of one kv head are a matrix
// Q of n * (hq / hkv) rows, and the prefix part of their attention is
//   S = Q K^T,   P = 2^(scale log2(e) S - ref),   acc = P V,   l = sum P,
// one pass over the prefix with a running reference per query row.  The state (acc, ref, l) of
// each row goes to the workspace; shared_rest.cu takes the request's other rows and joins the
// states.
//
// A tile is 128 query rows of one (group, kv head); a block is 128 cache rows.  All blocks of all
// tiles, tiles of one (group, kv head) side by side, form one line that is cut into equal
// pieces, one per CTA, whatever the groups' sizes: a CTA takes parts of a tile or several tiles,
// and a tile has as many states as pieces touch it.  (Beginning a tile counts as blocks too.)
//
// Seven warps: two load (K, and V; a page's 16 rows of 64 dims per tensor copy, into the swizzled
// tiles that the products read), one issues the products, four weigh, one query row per thread.
// The queries lie in tensor memory.  Scores exist twice, so that the scores of a block are made
// while the one before it is weighed; weights go back to tensor memory as the left operand of P V,
// as two bf16 numbers (V's type asks for bf16; the second is what the first leaves out, so that a
// weight is good to 2^-16, as in the library's other decode calls): the first to a place of their
// own, the second over the scores that they were.  The reference follows the row's maximum when
// that passes it by 2^8, so that acc is rarely rescaled.  The sum is taken of the fp32 weights.
//
// All members keep every row of the prefix, so there is no mask; rows of the last page behind the
// prefix (another request's, or nothing yet) get weight 0 and V rows of zeros.
//
// What bounds it: weighing, one warp per scheduler: 1.04 us of a block's 1.11, and 1.41 of 1.52
// beside the rest kernel, whose warps share the schedulers.  (With weights of one bf16 number a block
// took 1.06 us by itself, and 64 requests behind 16391 rows 36.5 as a whole.)
// Before the first scores there are the groups' two dependent loads, page ids and rows (5 us, 7
// beside), behind the last block the states of 128 rows (1.7 us).  Measured, whole calls: 64
// requests of 32/8 heads behind 16391 rows 40.7 us (31.4 where the requests have one own row each).
// A CTA leaves room for two CTAs of the rest kernel (160 registers a thread, 145 KB): without, that
// one started behind it (128 requests of nine prompts 77 us, 71 with it).  In its place, warps of 8
// query rows with mma.sync for groups of few rows: 28 us for 64 images of four prompts where this
// took 24.
#include <cuda.h>
#include <math.h>

#include <atomic>

#include "common.cuh"
#include "host.h"
#include "internal.h"
#include "mma.cuh"
#include "tcgen05.cuh"

namespace dsa {
namespace {

constexpr int kPRows = kSharedRows;    // query rows per tile
constexpr int kPBlock = kSharedBlock;  // cache rows per block ...
constexpr int kPPages = kPBlock / 16;  // ... and pages
constexpr int kPThreads = 224;         // 4 weighing warps, two loading ones, an issuing one
constexpr int kHalfBytes = 128 * 128;  // 128 rows of 64 bf16
constexpr float kSlackLog2 = 8.f, kNoRef = -3e38f;

template <int D>
struct PrefixShape {
  static constexpr int kHalves = D / 64;
  static constexpr int kTile = kHalves * kHalfBytes;  // 128 rows
  static constexpr int kSlots = D == 128 ? 4 : 6;     // tiles of K and V in shared memory
  static constexpr int kRing = 0, kStage = kSlots * kTile;  // the ring; 4 KB of each weighing warp
  static constexpr int kBar = kStage + 4 * 4096;
  static constexpr int kSmem = 1024 + kBar + 256;     // the base is rounded up to 1024
  // tensor memory: S twice, P, O, Q
  static constexpr int kS = 0, kP = 256, kO = 320, kQ = 320 + D, kTmem = 512;
};

constexpr uint32_t kBf16Operands = (1u << 7) | (1u << 10);

// How long rows stay in the L2: prefixes that fit there as usual, for the next step; those that do
// not (kStayBytes of K and V, by the host's bounds) leave first, which keeps the states there until
// the join.  64 requests behind 16391 rows (67 MB) 40.4 us, as usual 42.2; 128 of nine prompts (73
// MB) 60.3 and 61.7; but eight requests (6 MB) 13.2 and 12.6.
constexpr int64_t kStayBytes = 48 << 20;
__device__ __forceinline__ uint64_t l2_policy(bool leave) {
  uint64_t first, usual;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(first));
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(usual));
  return leave ? first : usual;
}

__device__ __forceinline__ void tensor_copy(uint32_t dst, const CUtensorMap* map, int x, int slot,
                                            int head, int page, uint64_t* bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%2, %3, %4, %5}], [%6], %7;" ::"r"(dst),
      "l"(map), "r"(x), "r"(slot), "r"(head), "r"(page), "r"(smem_addr(bar)), "l"(policy)
      : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ void sts128(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y),
               "r"(v.z), "r"(v.w)
               : "memory");
}

struct Group {
  int b0, n, rows, tiles, blocks;  // first request, requests, prefix rows; of one kv head
  bool sound;                      // its ends lie in order within the batch
};

// Group g as the arrays say; one that is wrong has no work.  `err`: where to flag it, or null.
__device__ __forceinline__ Group load_group(const SharedLaunch& a, int g, int32_t* err) {
  Group r{0, 0, 0, 0, 0, true};
  const int lo = __ldg(a.group_start + g), hi = __ldg(a.group_start + g + 1);
  if (lo < 0 || hi < lo || hi > a.batch || (g == 0 && lo != 0) || (g == a.groups - 1 && hi != a.batch)) {
    if (err != nullptr) set_error(err, DSA_DEV_BAD_GROUP);
    r.sound = false;
    return r;
  }
  if (hi == lo) return r;
  const int rows = __ldg(a.prefix_len + lo);
  if (rows < 0 || rows > a.max_prefix || rows > a.max_pages * kPage) {
    if (err != nullptr) set_error(err, DSA_DEV_BAD_PREFIX);
    return r;
  }
  r.b0 = lo;
  r.n = hi - lo;
  r.rows = rows;
  r.blocks = (rows + kPBlock - 1) / kPBlock;
  r.tiles = ((r.n << a.group_log2) + kPRows - 1) / kPRows;
  return r;
}

// Blocks that beginning another tile is worth (queries, the first rows, the state: 5 us), none for a
// tile of few blocks, which is better not cut; the line has so many places before the tile's own.
// 64 requests behind 16391 rows 40.6 us, 47.5 with tiles begun for nothing, 45.8 with 4 blocks,
// 43.5 with 8.
__device__ __forceinline__ int tile_cost(const Group& g) { return min(6, g.blocks >> 3); }

// A CTA's place on the line of blocks.
struct Cursor {
  int at, end;  // places done and to do, counted over all tiles
  int g, hk, t, blk;
  Group grp;
};

template <int D>
// 160 registers: two warps of it leave a quarter of an SM room for two warps of the rest kernel
__global__ void __maxnreg__(160)
    prefix_kernel(const SharedLaunch a, const __grid_constant__ CUtensorMap kmap,
                  const __grid_constant__ CUtensorMap vmap) {
  using Sh = PrefixShape<D>;
  constexpr int kHalves = Sh::kHalves;
  extern __shared__ unsigned char smem_raw[];
  __shared__ int32_t scan[kPThreads / 32];
  __shared__ int32_t most_of[kPThreads / 32];
  __shared__ int32_t found_before, found;
  __shared__ uint32_t tmem_slot;
  __shared__ int32_t failed_word;
  unsigned char* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  const uint32_t sm = smem_addr(smem);
  volatile int32_t* failed = &failed_word;
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);

  uint64_t* full = reinterpret_cast<uint64_t*>(smem + Sh::kBar);  // a tile of K or V is there
  uint64_t* empty = full + Sh::kSlots;                           // the products are done with it
  uint64_t* s_done = empty + Sh::kSlots;                         // scores of an even, odd block
  uint64_t* p_full = s_done + 2;                                 // its weights
  uint64_t* o_done = s_done + 4;                                 // its second product
  uint64_t* q_full = s_done + 6;                                 // a tile's queries are there
  if (warp == 5) tmem_alloc<Sh::kTmem>(&tmem_slot);
  if (tid == 128 || tid == 192)
    asm volatile("prefetch.tensormap [%0];" ::"l"(tid == 128 ? &kmap : &vmap) : "memory");
  if (tid == 128) {
    for (int s = 0; s < Sh::kSlots; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, 1);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      mbar_init(s_done + e, 1);
      mbar_init(p_full + e, 4);
      mbar_init(o_done + e, 1);
    }
    mbar_init(q_full, 4);
    fence_mbar_init();
    failed_word = 0;
    found = -1;
  }

  // ---- this CTA's piece of the line ----
  // blocks of all tiles of a group, summed over the groups
  auto units_of = [&](const Group& g) { return g.tiles * (g.blocks + tile_cost(g)) * a.hkv; };
  int sum = 0, mine0 = 0;  // mine0: of the first group this thread looks at
  int most = 0, wrong = 0;
  for (int g = tid; g < a.groups; g += kPThreads) {
    const Group r = load_group(a, g, blockIdx.x == 0 ? a.err : nullptr);
    wrong |= !r.sound;
    sum += units_of(r);
    if (g == tid) mine0 = sum;
    most = max(most, r.blocks + tile_cost(r));
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, o);
    most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
  }
  if (lane == 0) {
    scan[warp] = sum;
    most_of[warp] = most;
  }
  // Groups that do not rise from 0 to the batch may overlap and be more than the host has counted
  // with: then no prefix is computed at all.  (The barrier is that of the mbarriers and of the
  // tensor-memory address too.)
  wrong = __syncthreads_or(wrong);
  const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_slot, 0);
  sum = 0;
#pragma unroll
  for (int w = 0; w < kPThreads / 32; ++w) {
    sum += scan[w];
    most = max(most, most_of[w]);
  }
  if (wrong != 0) sum = 0;
  // a tile of `most` blocks is touched by at most ceil(most / per) + 1 pieces
  const int grid = static_cast<int>(gridDim.x);
  const int per = max(max((sum + grid - 1) / grid, 1), (most + a.prefix_slots - 2) / (a.prefix_slots - 1));
  Cursor c0;
  c0.at = static_cast<int>(min(static_cast<int64_t>(sum), static_cast<int64_t>(per) * blockIdx.x));
  c0.end = min(sum, c0.at + per);
  // the group that holds the first block
  int before = 0;
  __syncthreads();  // scan is used again
  for (int g0 = 0; g0 < a.groups && c0.at < c0.end; g0 += kPThreads) {
    const int g = g0 + tid;
    const int u = g0 == 0 ? mine0 : g < a.groups ? units_of(load_group(a, g, nullptr)) : 0;
    int x = u;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, x, s);
      if (lane >= s) x += v;
    }
    if (lane == 31) scan[warp] = x;
    __syncthreads();
    int all = 0;
    x += before;
#pragma unroll
    for (int w = 0; w < kPThreads / 32; ++w) {
      if (w < warp) x += scan[w];
      all += scan[w];
    }
    if (x - u <= c0.at && c0.at < x) {
      found = g;
      found_before = x - u;
    }
    before += all;
    __syncthreads();
  }
  bool work = c0.at < c0.end && found >= 0;
  if (work) {
    c0.g = found;
    c0.grp = load_group(a, c0.g, nullptr);
    int in = c0.at - found_before;
    const int cost = tile_cost(c0.grp), per_tile = c0.grp.blocks + cost;
    c0.t = in / per_tile;
    in -= c0.t * per_tile;
    c0.hk = c0.t / c0.grp.tiles;
    c0.t -= c0.hk * c0.grp.tiles;
    c0.blk = max(in - cost, 0);
    c0.at += max(cost - in, 0);
    work = c0.at < c0.end;
  }
  // Blocks of the cursor's tile that are this CTA's; then on to the next tile.
  auto blocks_here = [&](const Cursor& c) { return min(c.grp.blocks - c.blk, c.end - c.at); };
  auto next_tile = [&](Cursor& c) {
    c.at += blocks_here(c);
    c.blk = 0;
    if (++c.t == c.grp.tiles) {
      c.t = 0;
      if (++c.hk == a.hkv) {
        c.hk = 0;
        if (c.at >= c.end) return;
        do c.grp = load_group(a, ++c.g, nullptr);
        while (c.grp.blocks == 0 && c.g + 1 < a.groups);
      }
    }
    c.at += tile_cost(c.grp);
  };

  bool ok = true;
  int count = 0;  // blocks done, over all tiles of the CTA
  if (!work) {
  } else if (warp == 4 || warp == 6) {
    // ================= loading: K, or V, of every block into the ring =================
    // One elected lane issues, from values that the whole warp holds: sixteen lanes with a page
    // half each took 95 cycles a copy, three times a block's products.
    const bool k = warp == 4;
    const CUtensorMap* map = k ? &kmap : &vmap;
    const uint64_t policy = l2_policy(a.leave != 0);
    for (Cursor c = c0; ok && c.at < c.end; next_tile(c)) {
      const int nb = blocks_here(c);
      const int32_t* pt = a.page_table + static_cast<size_t>(c.grp.b0) * a.max_pages;
      const int all_pages = (c.grp.rows + 15) >> 4;
      auto load_id = [&](int blk) {
        const int p = blk * kPPages + (lane & 7);
        return p < all_pages ? __ldg(pt + p) : 0;
      };
      int id = load_id(c.blk);
      for (int i = 0; i < nb; ++i, ++count) {
        const int pages = min(kPPages, all_pages - (c.blk + i) * kPPages);
        if ((lane & 7) < pages && static_cast<unsigned>(id) >= static_cast<unsigned>(a.num_pages)) {
          set_error(a.err, DSA_DEV_BAD_PAGE);
          id = 0;
        }
        int ids[kPPages];
#pragma unroll
        for (int x = 0; x < kPPages; ++x) ids[x] = __shfl_sync(0xffffffffu, id, x);
        if (i + 1 < nb) id = load_id(c.blk + i + 1);
        const int item = 2 * count + (k ? 0 : 1), s = item % Sh::kSlots;
        if (item >= Sh::kSlots)
          ok = mbar_wait(empty + s, static_cast<uint32_t>(item / Sh::kSlots - 1) & 1u);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (elect_one()) {
          mbar_arrive_expect_tx(full + s, static_cast<uint32_t>(pages * 16 * D * 2));
          const uint32_t to = sm + Sh::kRing + s * Sh::kTile;
#pragma unroll
          for (int x = 0; x < kPPages; ++x)
            if (x < pages) {
#pragma unroll
              for (int h = 0; h < kHalves; ++h)
                tensor_copy(to + h * kHalfBytes + x * 2048, map, 64 * h, 0, c.hk, ids[x], full + s,
                            policy);
            }
        }
        __syncwarp();
      }
    }
    if (!ok) {
      *failed = 1;
      // copies in flight get a bounded time to land
      for (int n = max(0, count - Sh::kSlots / 2); n < count; ++n) {
        const int item = 2 * n + (k ? 0 : 1);
        mbar_wait(full + item % Sh::kSlots, static_cast<uint32_t>(item / Sh::kSlots) & 1u);
      }
    }
  } else if (warp == 5) {
    // ================= issuing =================
    const uint64_t k_desc = tc_desc(sm + Sh::kRing, 16, 1024, kSwizzle128);
    const uint64_t v_desc = tc_desc(sm + Sh::kRing, kHalfBytes, 1024, kSwizzle128);
    int tiles = 0;
    for (Cursor c = c0; ok && c.at < c.end; next_tile(c), ++tiles) {
      const int nb = blocks_here(c);
      auto pages_of = [&](int i) {
        return min(kPPages, ((c.grp.rows + 15) >> 4) - (c.blk + i) * kPPages);
      };
      auto issue_s = [&](int i) {  // S = Q K^T into the place of block count + i
        const int item = 2 * (count + i), s = item % Sh::kSlots, e = (count + i) & 1;
        ok = mbar_wait(full + s, static_cast<uint32_t>(item / Sh::kSlots) & 1u) && ok;
        tc_fence_after();
        if (!__all_sync(0xffffffffu, ok)) return;
        if (elect_one()) {
          const uint32_t id_s = tc_idesc(128, 16 * pages_of(i), false) | kBf16Operands;
          const uint64_t kd = k_desc + (s * Sh::kTile >> 4);
#pragma unroll
          for (int x = 0; x < D / 16; ++x) {
            tc_mma_f16_ta(tmem + Sh::kS + e * 128, tmem + Sh::kQ + 8 * x,
                          kd + (((x >> 2) * kHalfBytes + (x & 3) * 32) >> 4), id_s, x > 0);
          }
          tc_commit(s_done + e);
          tc_commit(empty + s);
        }
        __syncwarp();
      };
      ok = mbar_wait(q_full, static_cast<uint32_t>(tiles) & 1u) && ok;
      issue_s(0);
      for (int i = 0; ok && i < nb; ++i) {
        const int now = count + i, e = now & 1;
        if (i + 1 < nb) {  // into the place of the block before, when its weights' second parts are used
          if (i > 0) ok = mbar_wait(o_done + (e ^ 1), static_cast<uint32_t>((now - 1) >> 1) & 1u) && ok;
          issue_s(i + 1);
        }
        const int item = 2 * now + 1, s = item % Sh::kSlots;
        ok = mbar_wait(full + s, static_cast<uint32_t>(item / Sh::kSlots) & 1u) &&
             mbar_wait(p_full + e, static_cast<uint32_t>(now >> 1) & 1u) && ok;
        tc_fence_after();
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (elect_one()) {  // O += P V, two steps for each page
          constexpr uint32_t id_o = tc_idesc_b_rows(128, D) | kBf16Operands;
          const uint64_t vd = v_desc + (s * Sh::kTile >> 4);
          const uint32_t high = tmem + Sh::kP, low = tmem + Sh::kS + e * 128;
          const int pages = pages_of(i);
          for (int x = 0; x < pages; ++x) {
            tc_mma_f16_ta(tmem + Sh::kO, high + 8 * x, vd + (x * 2048 >> 4), id_o, i > 0 || x > 0);
            tc_mma_f16_ta(tmem + Sh::kO, low + 8 * x, vd + (x * 2048 >> 4), id_o, true);
          }
          tc_commit(o_done + e);
          tc_commit(empty + s);
        }
        __syncwarp();
      }
      count += nb;
    }
    if (!ok) *failed = 1;
  } else {
    // ================= weighing: one query row per thread =================
    const int r = tid, lg = a.group_log2, per_tile = kPRows >> lg;
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(32 * warp) << 16);
    // at least the smallest fp32 number, so that a masked score (-inf) times it stays one; a finite
    // score (below 2^128) times that is nothing, as with scale 0
    const float c1 = fmaxf(fabsf(a.scale_log2), 0x1p-149f);
    const uint32_t flip = a.scale_log2 < 0.f ? 0x80008000u : 0u;  // q changes its sign
    for (Cursor c = c0; ok && c.at < c.end; next_tile(c)) {
      const int nb = blocks_here(c);
      const int req0 = c.t * per_tile;  // first request of the tile, within the group
      const bool idle = req0 + ((32 * warp) >> lg) >= c.grp.n;
      const bool mine = req0 + (r >> lg) < c.grp.n;
      const int b = c.grp.b0 + req0 + (r >> lg);
      // The row's query into tensor memory (zeros where there is no request); the products that
      // read the last tile's are done: its scores were.
      if (!idle) {
        const size_t qh = static_cast<size_t>(b) * a.hq + (c.hk << lg) + (r & ((1 << lg) - 1));
        const uint4* from = reinterpret_cast<const uint4*>(a.q + (mine ? qh : 0) * D);
#pragma unroll
        for (int h = 0; h < D / 64; ++h) {
          uint32_t w[32];
#pragma unroll
          for (int y = 0; y < 8; ++y) {
            const uint4 v = mine ? __ldg(from + 8 * h + y) : make_uint4(0u, 0u, 0u, 0u);
            w[4 * y] = v.x ^ flip;
            w[4 * y + 1] = v.y ^ flip;
            w[4 * y + 2] = v.z ^ flip;
            w[4 * y + 3] = v.w ^ flip;
          }
          tmem_store16(t_lane + Sh::kQ + 32 * h, w);
          tmem_store16(t_lane + Sh::kQ + 32 * h + 16, w + 16);
        }
        tc_wait_st();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
      bool same = true;  // a member states the group's prefix
      if (mine && __ldg(a.prefix_len + b) != c.grp.rows) {
        set_error(a.err, DSA_DEV_BAD_PREFIX);
        same = false;
      }
      float ref = kNoRef, l = 0.f;
      for (int i = 0; i < nb; ++i) {
        const int now = count + i, e = now & 1;
        const uint32_t phase = static_cast<uint32_t>(now >> 1) & 1u;
        const int left = c.grp.rows - (c.blk + i) * kPBlock, valid = min(left, kPBlock);
        ok = mbar_wait(s_done + e, phase) && ok;
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        if ((valid & 15) != 0) {
          // V rows of the last page behind the prefix: zeros (weight 0 times NaN is NaN)
          const int item = 2 * now + 1, s = item % Sh::kSlots;
          ok = mbar_wait(full + s, static_cast<uint32_t>(item / Sh::kSlots) & 1u) && ok;
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          const int rows = 16 - (valid & 15);
          for (int y = tid; y < rows * (D / 8); y += 128) {
            const int row = valid + y / (D / 8), piece = y % (D / 8);
            sts128(sm + Sh::kRing + s * Sh::kTile + (piece >> 3) * kHalfBytes + row * 128 + 16 * (piece & 7),
                   make_uint4(0u, 0u, 0u, 0u));
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        if (!idle) {
          const uint32_t t_s = t_lane + Sh::kS + e * 128;
          // 64 columns at a time: the second half for its maximum, the first for its maximum and
          // its weights, the second again
          uint32_t s[2][32];
          auto load_half = [&](int h) {
            tmem_load<32>(t_s + 64 * h, s[0]);
            tmem_load<32>(t_s + 64 * h + 32, s[1]);
            tc_wait_ld();
            if (valid < kPBlock) {
#pragma unroll
              for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int q = 0; q < 32; ++q)
                  if (64 * h + 32 * x + q >= valid) s[x][q] = 0xff800000u;
            }
          };
          float m[4];
#pragma unroll
          for (int h = 1; h >= 0; --h) {
            load_half(h);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              float& t = m[2 * h + x];
              t = __uint_as_float(s[x][0]);
#pragma unroll
              for (int q = 1; q < 32; ++q) t = fmaxf(t, __uint_as_float(s[x][q]));
            }
          }
          const float top = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])) * c1;
          const bool over = top - ref > kSlackLog2;
          const float to = over ? top : ref, down = ex2_approx(ref - to);
          ref = to;
          l *= down;
          const f32x2 a1 = pack2(c1, c1), a2 = pack2(-ref, -ref), minus1 = pack2(-1.f, -1.f);
          f32x2 sums[2] = {pack2(0.f, 0.f), pack2(0.f, 0.f)};
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (h == 1) load_half(1);
            uint32_t w[2][16], rest[2][16];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
#pragma unroll
              for (int q = 0; q < 32; q += 2) {
                float z0, z1;
                unpack2(fma2(pack2(__uint_as_float(s[x][q]), __uint_as_float(s[x][q + 1])), a1, a2), z0, z1);
                z0 = ex2_approx(z0);
                z1 = ex2_approx(z1);
                const f32x2 z = pack2(z0, z1);
                sums[(q >> 1) & 1] = add2(sums[(q >> 1) & 1], z);
                const uint32_t high = bf16x2_rn(z0, z1);
                unpack2(fma2(pack2(bf16_lo(high), bf16_hi(high)), minus1, z), z0, z1);
                w[x][q / 2] = high;
                rest[x][q / 2] = bf16x2_rn(z0, z1);
              }
            }
            // (the first half's scores are in registers or done with, and these lie over them)
            tmem_store16(t_s + 32 * h, rest[0]);
            tmem_store16(t_s + 32 * h + 16, rest[1]);
            if (h == 0 && now > 0) {
              // the last weights and O are free when the second product of the block before is done
              ok = mbar_wait(o_done + (e ^ 1), static_cast<uint32_t>((now - 1) >> 1) & 1u) && ok;
              __syncwarp();
              tc_fence_after();
              if (i > 0 && __any_sync(0xffffffffu, over)) {
#pragma unroll 1
                for (int y = 0; y < D / 16; ++y) {
                  uint32_t o[16];
                  tmem_load<16>(t_lane + Sh::kO + 16 * y, o);
                  tc_wait_ld();
#pragma unroll
                  for (int q = 0; q < 16; ++q) o[q] = __float_as_uint(__uint_as_float(o[q]) * down);
                  tmem_store16(t_lane + Sh::kO + 16 * y, o);
                }
              }
            }
            tmem_store16(t_lane + Sh::kP + 32 * h, w[0]);
            tmem_store16(t_lane + Sh::kP + 32 * h + 16, w[1]);
          }
          float u, v;
          unpack2(add2(sums[0], sums[1]), u, v);
          l += u + v;
          tc_wait_st();
        }
        tc_fence_before();
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane == 0) mbar_arrive(p_full + e);
      }
      if (!ok) break;
      count += nb;
      const int last = count - 1;
      ok = mbar_wait(o_done + (last & 1), static_cast<uint32_t>(last >> 1) & 1u);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      // the state of the row, at the number of this piece among those of its tile
      const int tile_at = c.at - c.blk;
      const int slot = static_cast<int>(blockIdx.x) - tile_at / per;
      if (!idle) {
        tc_fence_after();
        const size_t qh = static_cast<size_t>(b) * a.hq + (c.hk << lg) + (r & ((1 << lg) - 1));
        float* to = a.states.pieces + slot * a.states.apart + (mine ? qh : 0) * a.states.floats;
        // 32 dims of the warp's 32 rows at a time, by way of shared memory (swizzled), so that 8
        // lanes store a row's line: a thread that stores its row alone touches 32 lines with every
        // store
        const uint32_t stage = sm + Sh::kStage + warp * 4096;
#pragma unroll 1
        for (int h = 0; h < D / 32; ++h) {
          uint32_t o[32];
          tmem_load<32>(t_lane + Sh::kO + 32 * h, o);
          tc_wait_ld();
          __syncwarp();
#pragma unroll
          for (int q = 0; q < 8; ++q)
            sts128(stage + lane * 128 + ((q ^ (lane & 7)) << 4),
                   make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]));
          __syncwarp();
#pragma unroll
          for (int y = 0; y < 8; ++y) {
            const int row = 4 * y + (lane >> 3);  // of the warp
            const uint64_t base = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(to), row);
            const uint4 v = lds128(stage + row * 128 + (((lane & 7) ^ (row & 7)) << 4));
            if (req0 + ((32 * warp + row) >> lg) < c.grp.n)
              reinterpret_cast<uint4*>(reinterpret_cast<float*>(base) + 32 * h)[lane & 7] = v;
          }
        }
        if (mine)
          *reinterpret_cast<float2*>(to + D) = make_float2(same ? ref : __int_as_float(0x7fc00000), l);
        if (mine && slot == 0)
          a.pieces[qh] = (tile_at + c.grp.blocks - 1) / per - tile_at / per + 1;
        tc_fence_before();
      }
    }
    if (!ok) *failed = 1;
  }
  __syncthreads();
  if (*failed != 0) {
    // products in flight get a bounded time to finish before the memory goes back
    if (tid == 0) set_error(a.err, DSA_DEV_TIMEOUT);
    const uint64_t t0 = global_ns();
    while (global_ns() - t0 < 2000000ull) {}
    __syncthreads();
  }
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc<Sh::kTmem>(tmem);
  }
}

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                 const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                 const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// CUDA's encoder, asked for once (the library links the runtime alone).
EncodeTiled encoder() {
  static std::atomic<void*> known{nullptr};
  void* p = known.load(std::memory_order_acquire);
  if (p == nullptr) {
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      return nullptr;
    known.store(p, std::memory_order_release);
  }
  return reinterpret_cast<EncodeTiled>(p);
}

// Pages [num_pages][16][hkv][d] as (dim, slot, head, page); a copy takes 64 dims of the 16
// rows of one head and page.
bool encode_pages(CUtensorMap* map, const void* pages, const SharedLaunch& a) {
  const EncodeTiled encode = encoder();
  if (encode == nullptr) return false;
  const cuuint64_t row = static_cast<cuuint64_t>(a.hkv) * a.head_dim * 2;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(a.head_dim), 16, static_cast<cuuint64_t>(a.hkv),
                              static_cast<cuuint64_t>(a.num_pages)};
  const cuuint64_t strides[3] = {row, static_cast<cuuint64_t>(a.head_dim) * 2, 16 * row};
  const cuuint32_t box[4] = {64, 16, 1, 1}, step[4] = {1, 1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(pages), dims, strides,
                box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t launch_one(SharedLaunch a, const CUtensorMap& kmap, const CUtensorMap& vmap,
                       cudaStream_t s) {
  auto kern = prefix_kernel<D>;
  static KernelSlots cache;
  int per_sm = 0;
  const cudaError_t e =
      cache.get(reinterpret_cast<const void*>(kern), kPThreads, PrefixShape<D>::kSmem, &per_sm, true);
  if (e != cudaSuccess) return e;
  // no more CTAs than blocks there can be
  const int64_t tiles = a.groups + ((static_cast<int64_t>(a.batch) << a.group_log2) / kPRows);
  const int64_t blocks = tiles * a.hkv * ceil_div(a.max_prefix, kPBlock);
  // A quarter of the blocks, but half of the SMs at least: a CTA keeps the rest kernel's CTAs from
  // most of its SM, so few blocks are better on some SMs alone.
  int64_t ctas = blocks / 4 > a.sms / 2 ? blocks / 4 : a.sms / 2;
  ctas = ctas < a.sms ? ctas : a.sms;
  ctas = ctas < blocks ? ctas : blocks;
  a.leave = static_cast<int64_t>(a.groups) * a.max_prefix * a.hkv * D * 4 > kStayBytes;
  return launch_pdl(kern, dim3(static_cast<unsigned>(ctas)), dim3(kPThreads),
                    static_cast<size_t>(PrefixShape<D>::kSmem), s, a, kmap, vmap);
}

}  // namespace

cudaError_t launch_shared_prefix(const SharedLaunch& a, cudaStream_t s) {
  CUtensorMap kmap, vmap;
  if (!encode_pages(&kmap, a.k, a) || !encode_pages(&vmap, a.v, a)) return cudaErrorInvalidValue;
  return a.head_dim == 128 ? launch_one<128>(a, kmap, vmap, s) : launch_one<64>(a, kmap, vmap, s);
}

}  // namespace dsa
