// shared_rest.cu -- decode attention over the rows that requests do not share, and the joining of
// all states of a batch with shared prefixes (shared_prefix.cu leaves those of the prefixes).
//
// rest_kernel.  A work item is a chunk of the rows of one (request, kv head) behind the prefix:
// dense rows, or the kept set of the mask without the prefix.  A warp takes an item by itself, with
// its own ring of shared memory, and leaves a state (acc, m, l) per query head in the workspace:
// no two warps wait for each other, and short units (a few tens of kept rows) occupy a warp each.
// The warps of a CTA have neighbouring kv heads of the same rows, which lie side by side in
// memory and end together.  The kernel runs beside the prefix kernel: it starts as soon as that
// one's CTAs do, waits for nothing of it, and takes the places that its CTAs leave.
// What bounds it: HBM while most warps are there (in the middle of 128 requests of nine prompts
// 6.9 TB/s, 4.4 beside the prefix kernel's 2.3), at both ends the latency of a tile, 1.3 us alone
// and 2.1 in company, times the tiles of a chunk; an item takes 0.9 us to its lengths and page
// ids and 2.2 us to its first rows.  Measured: those 128 requests 60 us as a whole (floor 43), this
// kernel's last rows at 56.  Twice the buffers and half of the warps: 65; items fetched by warps
// from a counter: 70 where this took 65; CTAs that took a unit, waited for the prefix kernel and
// joined the states themselves: 77 for 73; rows in 16-byte copies instead of one each: 73 for 73.
//
// join_kernel.  A warp per (request, query head): the log-sum-exp sum of the prefix's states and
// the chunks', in their order, so results do not depend on who was first.  Three dependent loads
// (counts; weights and dims), 3 us for few states, 4 for 18 MB of them, 5 for 15 MB of up to 14 a
// head.
#include <math.h>

#include <type_traits>

#include "common.cuh"
#include "host.h"
#include "internal.h"
#include "mma.cuh"
#include "rows.cuh"
#include "warp_attn.cuh"

namespace dsa {
namespace {

constexpr int kRestWarps = 4;

// A row that nobody reads again: first to leave the L2, so that the states and the prefixes stay
// there until the join and the next step.  128 requests of nine prompts 63 us, without 65; 64
// images of four prompts 21, without 23.
__device__ __forceinline__ uint64_t leaves_first() {
  uint64_t policy;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
  return policy;
}
__device__ __forceinline__ void row_copy(void* dst, const void* src, uint32_t bytes, uint64_t* bar,
                                         uint64_t policy) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint "
      "[%0], [%1], %2, [%3], %4;" ::"r"(smem_addr(dst)),
      "l"(src), "r"(bytes), "r"(smem_addr(bar)), "l"(policy)
      : "memory");
}

template <int D, int G, bool DEEP>
struct RestShape {
  static constexpr bool kMma = G >= 2;
  static constexpr int kRowBytes = 2 * D;
  static constexpr int kRows = (kMma || D == 64) ? 16 : 8;  // of a tile
  static constexpr int kRowStride = kRowBytes + (kMma ? 16 : 0);
  static constexpr int kTile = kRows * kRowStride;          // K or V of a tile
  // K and V buffers of a warp: about 8 KB in all, so that some 20 warps fit an SM; twice as many
  // where there are few warps and the latency of a tile counts
  static constexpr int kBufs = (kTile > 4096 ? 1 : 2) * (DEEP ? 2 : 1);
  static constexpr int kWarp = 2 * kBufs * kTile;
  static constexpr int kBars = kRestWarps * kWarp;
  static constexpr int kSmem = kBars + kRestWarps * 2 * kBufs * 8;
  static constexpr bool kBulk = D == 128;  // a copy per row; rows of 128 bytes go in 16-byte pieces
};

template <int D, int G, bool MASK, bool DEEP>
__global__ void __launch_bounds__(kRestWarps * 32, 20 / kRestWarps) rest_kernel(const RestLaunch a) {
  using Sh = RestShape<D, G, DEEP>;
  constexpr int T = Sh::kRows, NB = Sh::kBufs;
  extern __shared__ __align__(128) unsigned char smem[];
  // Behind a prefix kernel nothing is waited for here: that one has waited for its own
  // predecessor before this grid could start.  What was written before is read past the SM's
  // own cache, which may hold lines from earlier.
  if (a.early == 0) griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
  const uint32_t item = blockIdx.x * kRestWarps + warp;
  const int hk = static_cast<int>(item % a.hkv);
  const int b = static_cast<int>(item / a.hkv % a.batch);
  const int c = static_cast<int>(item / a.hkv / a.batch);
  if (c < a.num_chunks) {
    const int L = __ldcg(a.seq_len + b), S0 = __ldcg(a.prefix_len + b);
    int n = 0, np = 0;
    MaskRows rows;
    if constexpr (MASK) {
      const uint32_t raw = lane < a.mask_words
                               ? __ldcg(a.keep_mask + (static_cast<size_t>(b) * a.hkv + hk) * a.mask_words + lane)
                               : 0u;
      n = rows.init(raw, L, __ldcg(a.prompt_len + b), __ldcg(a.window + b), a.max_pages, a.max_window,
                    INT32_MAX, lane);
      np = rows.np;
    } else {
      n = L < 1 || L > a.max_pages * kPage ? -DSA_DEV_BAD_SEQ_LEN : L;
      np = L;
    }
    // all of the prefix is kept, and left to the prefix kernel
    if (n >= 0)
      n = S0 < 0 || S0 > a.max_prefix || S0 > np || n - S0 > a.max_suffix ? -DSA_DEV_BAD_PREFIX : n - S0;
    np -= S0;
    if (c == 0 && lane == 0) {
      a.unit_rows[static_cast<size_t>(b) * a.hkv + hk] = n;
      if (n < 0) set_error(a.err, -n);
    }
    const int row0 = c * a.chunk, row1 = min(n, row0 + a.chunk);
    const int tiles = row1 > row0 ? (row1 - row0 + T - 1) / T : 0;
    unsigned char* kst = smem + warp * Sh::kWarp;
    unsigned char* vst = kst + NB * Sh::kTile;
    uint64_t* kbar = reinterpret_cast<uint64_t*>(smem + Sh::kBars) + warp * 2 * NB;
    uint64_t* vbar = kbar + NB;
    const int32_t* pt = a.page_table + static_cast<size_t>(b) * a.max_pages;
    const int my_r = lane & (T - 1);
    auto rows_of = [&](int t) { return min(T, row1 - (row0 + t * T)); };
    // Logical row of this lane in tile t (all lanes take part).
    auto row_of = [&](int t) -> int {
      const int r = row0 + t * T + my_r;
      int j = S0 + r;
      if constexpr (MASK)
        if (t < tiles && row0 + t * T + rows_of(t) > np) {  // the tile reaches window rows
          const int w = rows.window_row(r - np);
          if (r >= np) j = w;
        }
      return j;
    };
    // Where the row lies: its page, asked for a tile ahead, and its slot.
    struct Place {
      int page, slot;
    };
    auto place_of = [&](int t, int j) -> Place {
      if (t >= tiles || my_r >= rows_of(t)) return Place{0, 0};
      return Place{__ldcg(pt + (j >> 4)), j & (kPage - 1)};
    };
    // K (half 0) or V of tile t on its way into its buffer.
    const uint64_t policy = leaves_first();
    auto issue = [&](int t, int half, const Place& p) {
      const int nrows = rows_of(t), s = t % NB;
      uint64_t* bar = (half == 0 ? kbar : vbar) + s;
      unsigned char* to = (half == 0 ? kst : vst) + s * Sh::kTile;
      const uint16_t* base = half == 0 ? a.k : a.v;
      int64_t at = static_cast<int64_t>(p.page) * kPage + p.slot;
      if (my_r < nrows && static_cast<uint32_t>(p.page) >= static_cast<uint32_t>(a.num_pages)) {
        set_error(a.err, DSA_DEV_BAD_PAGE);
        at = 0;
      }
      if constexpr (Sh::kBulk) {
        if (lane == 0) mbar_arrive_expect_tx(bar, static_cast<uint32_t>(nrows * Sh::kRowBytes));
        __syncwarp();
        if (lane < nrows)
          row_copy(to + lane * Sh::kRowStride, base + (static_cast<size_t>(at) * a.hkv + hk) * D,
                   Sh::kRowBytes, bar, policy);
      } else {
        constexpr int kLanes = Sh::kRowBytes / 16, kStep = 32 / kLanes;
        const int piece = lane % kLanes;
#pragma unroll
        for (int y = 0; y < T / kStep; ++y) {
          const int r = kStep * y + lane / kLanes;
          const int64_t src = __shfl_sync(0xffffffffu, at, r);
          if (r < nrows)
            cp_async16(to + r * Sh::kRowStride + 16 * piece,
                       reinterpret_cast<const unsigned char*>(
                           base + (static_cast<size_t>(src) * a.hkv + hk) * D) + 16 * piece);
        }
        cp_async_arrive(bar);
      }
    };

    if (tiles > 0) {
      bool ok = true;
      if (lane == 0) {
#pragma unroll
        for (int s = 0; s < 2 * NB; ++s) mbar_init(kbar + s, Sh::kBulk ? 1 : 32);
        fence_mbar_init();
      }
      __syncwarp();
      WarpAttn<D, bf16_t, G, true, T> wa;
      static_assert(WarpAttn<D, bf16_t, G, true, T>::kRowStride == Sh::kRowStride, "row stride");
      WarpQ<D, bf16_t, G, true> q;
      const size_t qh0 = static_cast<size_t>(b) * a.hq + hk * G;
      Place at[NB + 1];
#pragma unroll
      for (int t = 0; t <= NB; ++t) at[t] = place_of(t, row_of(t));
      q.template load<true>(a.q, true, qh0, lane);
      wa.reset();
#pragma unroll
      for (int t = 0; t < NB; ++t)
        if (t < tiles) {
          issue(t, 0, at[t]);
          issue(t, 1, at[t]);
        }
      Place next = at[NB];  // of tile t + NB
      int t = 0;
      for (; t < tiles; ++t) {
        const int s = t % NB, nrows = rows_of(t);
        const uint32_t phase = static_cast<uint32_t>(t / NB) & 1u;
        const Place now = next;
        ok = mbar_wait(kbar + s, phase);
        if constexpr (Sh::kMma) {
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          wa.qk_softmax(q, kst + s * Sh::kTile, nrows, a.scale_log2, lane);
          __syncwarp();
          fence_proxy_async_smem();
          if (t + NB < tiles) issue(t + NB, 0, now);
          next = place_of(t + NB + 1, row_of(t + NB + 1));
          ok = __all_sync(0xffffffffu, mbar_wait(vbar + s, phase));
          if (!ok) break;
          wa.pv(vst + s * Sh::kTile, nrows, lane);
          __syncwarp();
          fence_proxy_async_smem();
          if (t + NB < tiles) issue(t + NB, 1, now);
        } else {
          ok = __all_sync(0xffffffffu, mbar_wait(vbar + s, phase) && ok);
          if (!ok) break;
          wa.tile(q, kst + s * Sh::kTile, vst + s * Sh::kTile, nrows, a.scale_log2, lane);
          __syncwarp();
          fence_proxy_async_smem();
          if (t + NB < tiles) {
            issue(t + NB, 0, now);
            issue(t + NB, 1, now);
          }
          next = place_of(t + NB + 1, row_of(t + NB + 1));
        }
      }
      if (!ok) {
        // copies still in flight get a bounded time to land
        if (lane == 0) set_error(a.err, DSA_DEV_TIMEOUT);
        for (int s = 0; s < 2 * NB; ++s) {
          mbar_wait(kbar + s, 0);
          mbar_wait(kbar + s, 1);
        }
      }
      wa.flush(a.states.chunks + c * a.states.apart + qh0 * a.states.floats, lane, a.states.floats);
    }
  }
  // The grid ends behind the prefix kernel, so that whoever waits for it has waited for both.
  if (a.early != 0 && blockIdx.x == 0) griddep_wait();
}

constexpr int kJoinWarps = 4;

// A warp joins the states of one (request, query head): lane p weighs piece p and chunk p, all
// lanes add.  The first states are asked for together with their weights; fewer of them (MANY)
// where the warps are more than an SM holds at once otherwise, 16: 128 requests of 32 heads 61.7 us
// for 63.4, but 64 of them with up to 14 pieces 43.3 for 42.2.
template <int D, bool MANY>
__global__ void __launch_bounds__(kJoinWarps * 32, MANY ? 7 : 4) join_kernel(const RestLaunch a) {
  constexpr int kDims = D / 32;  // of a lane
  constexpr int kPieces = MANY ? 6 : 8, kChunks = MANY ? 4 : 6;
  using Vec = typename std::conditional<kDims == 4, float4, float2>::type;
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const uint32_t qh = blockIdx.x * kJoinWarps + (threadIdx.x >> 5);
  if (qh >= static_cast<uint32_t>(a.batch) * a.hq) return;
  const uint32_t b = qh / a.hq, hk = (qh - b * a.hq) / (static_cast<uint32_t>(a.hq) / a.hkv);
  const int n = __ldcg(a.unit_rows + static_cast<size_t>(b) * a.hkv + hk), S0 = __ldcg(a.prefix_len + b);
  int pieces = __ldcg(a.pieces + qh);
  if (pieces != 0 && lane == 0) a.pieces[qh] = 0;  // the next call's prefix kernel states it anew
  int chunks = n > 0 ? (n + a.chunk - 1) / a.chunk : 0;
  bool bad = n < 0;
  if (S0 <= 0) {
    bad = bad || pieces != 0;  // its group has a prefix (flagged where that was computed)
  } else if (!bad && (pieces < 1 || pieces > a.prefix_slots)) {
    // no group holds this request, or its group's first has another prefix
    if (lane == 0) set_error(a.err, DSA_DEV_BAD_GROUP);
    bad = true;
  }
  if (bad) pieces = chunks = 0;
  static_assert(kMaxChunks <= 32, "a piece and a chunk per lane");
  const int64_t apart = a.states.apart;
  const float* piece = a.states.pieces + static_cast<int64_t>(qh) * a.states.floats;
  const float* chunk = a.states.chunks + static_cast<int64_t>(qh) * a.states.floats;
  auto weight_of = [&](const float* s, int count) {
    return lane < count ? __ldcg(reinterpret_cast<const float2*>(s + lane * apart + D))
                        : make_float2(-INFINITY, 0.f);
  };
  auto dims_of = [&](const float* s, int p) { return __ldcg(reinterpret_cast<const Vec*>(s + p * apart) + lane); };
  const float2 mp = weight_of(piece, pieces), mc = weight_of(chunk, chunks);
  Vec vp[kPieces], vc[kChunks];
#pragma unroll
  for (int y = 0; y < kPieces; ++y)
    if (y < pieces) vp[y] = dims_of(piece, y);
#pragma unroll
  for (int y = 0; y < kChunks; ++y)
    if (y < chunks) vc[y] = dims_of(chunk, y);
  float m = warp_max(fmaxf(mp.x, mc.x));
  // (a NaN reference, which the maximum passes over, makes its weight NaN)
  const float sp = mp.x == -INFINITY ? 0.f : exp2f(mp.x - m), sc = mc.x == -INFINITY ? 0.f : exp2f(mc.x - m);
  float l = warp_sum(fmaf(sp, mp.y, sc * mc.y));
  Vec o{};
  auto add = [&](const Vec& v, float w) {
    o.x = fmaf(w, v.x, o.x);
    o.y = fmaf(w, v.y, o.y);
    if constexpr (kDims == 4) {
      o.z = fmaf(w, v.z, o.z);
      o.w = fmaf(w, v.w, o.w);
    }
  };
#pragma unroll
  for (int y = 0; y < kPieces; ++y)
    if (y < pieces) add(vp[y], __shfl_sync(0xffffffffu, sp, y));
  for (int p = kPieces; p < pieces; p += kPieces) {
#pragma unroll
    for (int y = 0; y < kPieces; ++y)
      if (p + y < pieces) vp[y] = dims_of(piece, p + y);
#pragma unroll
    for (int y = 0; y < kPieces; ++y)
      if (p + y < pieces) add(vp[y], __shfl_sync(0xffffffffu, sp, p + y));
  }
#pragma unroll
  for (int y = 0; y < kChunks; ++y)
    if (y < chunks) add(vc[y], __shfl_sync(0xffffffffu, sc, y));
  for (int p = kChunks; p < chunks; p += kChunks) {
#pragma unroll
    for (int y = 0; y < kChunks; ++y)
      if (p + y < chunks) vc[y] = dims_of(chunk, p + y);
#pragma unroll
    for (int y = 0; y < kChunks; ++y)
      if (p + y < chunks) add(vc[y], __shfl_sync(0xffffffffu, sc, p + y));
  }
  if (bad) l = m = __int_as_float(0x7fc00000);
  const float inv = 1.f / l;
  uint32_t* to = reinterpret_cast<uint32_t*>(a.out) + (static_cast<size_t>(qh) * D + kDims * lane) / 2;
  if constexpr (kDims == 4)
    *reinterpret_cast<uint2*>(to) =
        make_uint2(bf16x2_rn(o.x * inv, o.y * inv), bf16x2_rn(o.z * inv, o.w * inv));
  else
    to[0] = bf16x2_rn(o.x * inv, o.y * inv);
  if (a.lse != nullptr && lane == 0) a.lse[qh] = (m + log2f(l)) * kLn2;
}

// One build: the launch when `a` is given, the warps of a wave when `warps` is.
template <int D, int G, bool MASK, bool DEEP>
cudaError_t one(const RestLaunch* a, cudaStream_t s, int* warps) {
  using Sh = RestShape<D, G, DEEP>;
  auto kern = rest_kernel<D, G, MASK, DEEP>;
  static KernelSlots cache;
  int per_sm = 0;
  const cudaError_t e =
      cache.get(reinterpret_cast<const void*>(kern), kRestWarps * 32, Sh::kSmem, &per_sm, true);
  if (e != cudaSuccess) return e;
  if (warps != nullptr) *warps = per_sm * kRestWarps;
  if (a == nullptr) return cudaSuccess;
  const int64_t items = static_cast<int64_t>(a->batch) * a->hkv * a->num_chunks;
  return launch_pdl(kern, dim3(static_cast<unsigned>(ceil_div(items, kRestWarps))), dim3(kRestWarps * 32),
                    static_cast<size_t>(Sh::kSmem), s, *a);
}
template <int D, int G>
cudaError_t build(bool mask, const RestLaunch* a, cudaStream_t s, int* warps) {
  if (a != nullptr && a->deep != 0)
    return mask ? one<D, G, true, true>(a, s, warps) : one<D, G, false, true>(a, s, warps);
  return mask ? one<D, G, true, false>(a, s, warps) : one<D, G, false, false>(a, s, warps);
}

cudaError_t any(int head_dim, int group, bool mask, const RestLaunch* a, cudaStream_t s, int* warps) {
#define DSA_BODY(DD, GG) return build<DD, GG>(mask, a, s, warps);
  if (head_dim == 64 && group == 1) { DSA_BODY(64, 1) }
  if (head_dim == 64 && group == 2) { DSA_BODY(64, 2) }
  if (head_dim == 64 && group == 4) { DSA_BODY(64, 4) }
  if (head_dim == 64 && group == 8) { DSA_BODY(64, 8) }
  if (head_dim == 128 && group == 1) { DSA_BODY(128, 1) }
  if (head_dim == 128 && group == 2) { DSA_BODY(128, 2) }
  if (head_dim == 128 && group == 4) { DSA_BODY(128, 4) }
  if (head_dim == 128 && group == 8) { DSA_BODY(128, 8) }
#undef DSA_BODY
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_shared_rest(const RestLaunch& a, bool mask, cudaStream_t s) {
  const cudaError_t e = any(a.head_dim, a.hq / a.hkv, mask, &a, s, nullptr);
  if (e != cudaSuccess) return e;
  const bool many = static_cast<int64_t>(a.batch) * a.hq > static_cast<int64_t>(sm_count()) * 16;
  auto kern = a.head_dim == 128 ? (many ? join_kernel<128, true> : join_kernel<128, false>)
                                : (many ? join_kernel<64, true> : join_kernel<64, false>);
  return launch_pdl(
      kern, dim3(static_cast<unsigned>(ceil_div(static_cast<int64_t>(a.batch) * a.hq, kJoinWarps))),
      dim3(kJoinWarps * 32), 0, s, a);
}

cudaError_t shared_rest_warps(int head_dim, int group, bool mask, int* warps) {
  return any(head_dim, group, mask, nullptr, nullptr, warps);
}

}  // namespace dsa
