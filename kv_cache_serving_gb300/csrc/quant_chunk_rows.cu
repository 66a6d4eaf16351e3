// quant_chunk_rows.cu -- several query tokens per request over the 8-bit paged K/V cache
// on the 5th-generation tensor cores, for chunks of many (query token, head) rows.
//
// Mathematics as in quant_chunk.cu, with the queries on the lanes of tensor memory: a CTA
// holds 128 rows (query token, head of the kv head's group) of one (request, kv head) and
// walks its pages in blocks of 4 (64 cache rows):
//   S (128 x 64) = Q K^T,   P = weights of S,   O (128 x head_dim) += P V
// so a thread owns a query: its running reference and sum are two registers, a page's
// scales are constants of 16 of its scores, its mask is one shifted word per page, and P
// goes back to tensor memory over S as the left operand of the second product.  The
// reference follows the row's maximum (taken over the raw scores of a page, then scaled
// once) when that passes it by 2^10.  A block that every query keeps whole is not masked.
//
// Nine warps: four weigh, four convert (K and V codes of a page each to fp16 in shared
// memory), one issues the products.  S, P and K exist twice, so the scores of a block are
// ready when the weights of the one before it are done; V once (its place is free again
// before the next weights are).  Codes reach the converters by asynchronous copies into
// shared memory: loads to registers are held up by the few KB of L1 that the tiles leave
// (128 tokens over 4096 rows of 8 requests, 32/8 heads: 107 -> 97 us).  The issuing warp
// elects its lane, which keeps the products' descriptors in uniform registers: issuing a
// product took 150 cycles from a weighing thread and takes 60.  The unrolled prologue was
// a run of instruction-cache misses for every tile; as loops of four rows it brought prompts
// from 485 to 447 us.
//
// What bounds it: latency and instruction issue of the weighing and the prologue, not the
// products (12% of the tensor pipe) and not HBM.  Of a tile of prompts (3.5 blocks on
// average) 2.3 K cycles go by until its sizes and tensor memory are there, 7 K until q is
// converted and the first scores exist, 3 K per block, 4 K for the output; two CTAs per SM
// fill each other's gaps to 1.4 instructions per cycle.
// Measured (head_dim 128): prompts of 32 .. 512 rows of 128 requests, 32/8 heads, 427 us =
// 275 TFLOP/s of kept pairs (694 us with quant_chunk.cu); all 2048 rows of 8 requests 387 us
// (1017).
#include <math.h>

#include <type_traits>

#include "common.cuh"
#include "host.h"
#include "internal.h"
#include "mma.cuh"
#include "quant.cuh"
#include "quant_redo.cuh"
#include "tcgen05.cuh"

namespace dsa {
namespace {

constexpr int kRRows = 128;         // query rows per CTA
constexpr int kRPages = 4;          // pages per block ...
constexpr int kRBlock = 64;         // ... and cache rows
constexpr int kRThreads = 288;      // 4 weighing warps, 4 converting ones, an issuing one
constexpr int kRQHalf = kRRows * 128, kRHalf = kRBlock * 128;  // bytes of 64 dims, fp16
constexpr int kRInfos = 4;          // blocks whose scales are held
constexpr float kRHead = 4.f, kRSlack = 10.f, kRNoRef = -3e38f;  // as in quant_chunk.cu

template <int D>
struct RowsShape {
  static constexpr int kHalves = D / 64;               // of a row of a tile
  static constexpr int kQ = 0, kK = kHalves * kRQHalf;
  static constexpr int kV = kK + 2 * kHalves * kRHalf;  // K twice, V once
  static constexpr int kCodes = kV + kHalves * kRHalf;  // a block's codes: K, V of each page
  // 4 x 4 float4 of a page: see below
  static constexpr int kInfo = kCodes + kRPages * 2 * 16 * D;
  static constexpr int kUp = kInfo + kRInfos * kRPages * 16;  // score factor of a row: 128 floats
  static constexpr int kBar = kUp + 4 * kRRows;        // thirteen barriers, address, flag
  static constexpr int kMask = kBar + 112;
  static constexpr int kSlack = 1024;                  // the base is rounded up to 1024
  static constexpr int kS = 0, kO = 128, kTmem = 256;  // tensor memory: S and P twice, O
  static int smem(int words) { return kSlack + kMask + 4 * words; }
};

__device__ __forceinline__ void sts128(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y),
               "r"(v.z), "r"(v.w)
               : "memory");
}
// 32 bytes in one store: a whole sector.
__device__ __forceinline__ void stg256(void* p, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]),
               "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) { return fmaxf(fmaxf(a, b), c); }

template <int LG>
struct RowsTile {  // the last query tokens, which see the most rows, first
  static constexpr int kColumns = kRRows;
  __device__ __forceinline__ static void at(const QuantChunkLaunch&, int& bpos, int& hk, int& t0) {
    bpos = blockIdx.z;
    hk = blockIdx.y;
    t0 = (gridDim.x - 1 - blockIdx.x) * (kRRows >> LG);
  }
};

template <int D, int LG>
__global__ void __launch_bounds__(kRThreads, 2) quant_chunk_rows_kernel(const QuantChunkLaunch a) {
  using Sh = RowsShape<D>;
  constexpr int kHalves = Sh::kHalves;
  constexpr int per_cta = kRRows >> LG;  // query tokens per CTA
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  const uint32_t sm = smem_addr(smem);
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // known to be the warp's
  // the last query tokens, which see the most rows, first
  const int qt = gridDim.x - 1 - blockIdx.x, hk = blockIdx.y, bpos = blockIdx.z;
  const int b = a.order != nullptr ? __ldg(a.order + bpos) : bpos;
  if (static_cast<unsigned>(b) >= static_cast<unsigned>(a.batch)) {
    if (qt == 0 && hk == 0 && tid == 0) set_error(a.err, DSA_DEV_BAD_ORDER);
    return;
  }
  const int t0 = qt * per_cta;
  const int L = a.seq_len[b], n = a.q_len[b], P = a.prompt_len[b], Wn = a.window[b];
  int code = 0;
  if (L < 1 || L > a.max_pages * kPage) code = DSA_DEV_BAD_SEQ_LEN;
  else if (n < 0 || n > L || n > a.max_q) code = DSA_DEV_BAD_QLEN;
  else if (P < 0) code = DSA_DEV_BAD_PROMPT;
  else if (Wn < 0 || Wn > a.max_window) code = DSA_DEV_BAD_WINDOW;
  if (code != 0) {
    // q_len is not trusted: NaN into every slot of the unit
    if (qt == 0 && hk == 0 && tid == 0) set_error(a.err, code);
    for (int x = tid; x < kRRows * D; x += kRThreads) {
      const int t = t0 + x / (D << LG);
      if (t >= a.max_q) break;
      const size_t qh = (static_cast<size_t>(b) * a.max_q + t) * a.hq + (hk << LG) +
                        (x / D & ((1 << LG) - 1));
      a.out[qh * D + x % D] = 0x7fc0;
      if (a.lse != nullptr && x % D == 0) a.lse[qh] = __int_as_float(0x7fc00000);
    }
    return;
  }
  if (t0 >= n) return;
  const int t1 = min(t0 + per_cta, n);
  const int i_first = L - n + t0, i_last = L - n + t1 - 1;
  // pages scanned: those of the prompt rows [0, pa), then those from the window's start
  const int pa = (min(P, i_last + 1) + 15) >> 4;
  const int pb = max(pa, max(i_first - Wn, 0) >> 4), pe = i_last >> 4;
  const int pages = pa + max(0, pe - pb + 1);
  const int nblocks = (pages + kRPages - 1) / kRPages;
  auto page_of = [&](int x) { return x < pa ? x : pb + (x - pa); };
  // row of q and out of query row r
  const size_t qh0 = (static_cast<size_t>(b) * a.max_q + t0) * a.hq + (hk << LG);
  auto qh_of = [&](int r) {
    return qh0 + static_cast<size_t>(r >> LG) * a.hq + (r & ((1 << LG) - 1));
  };

  float4* info = reinterpret_cast<float4*>(smem + Sh::kInfo);
  float* up = reinterpret_cast<float*>(smem + Sh::kUp);
  // Barriers, one for even blocks and one for odd ones of each kind.
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + Sh::kBar);  // K and scales of a block
  uint64_t* v_full = k_full + 2;                                    // its V
  uint64_t* s_done = k_full + 4;                                    // its scores
  uint64_t* o_done = k_full + 6;                                    // its second product
  uint64_t* p_full = k_full + 8;                                    // its weights
  // k_full as the issuing warp passes it on to the weighing ones: its next phase waits for
  // their weights, so that none can miss one (k_full's next phase waits for s_done alone)
  uint64_t* i_full = k_full + 10;
  uint64_t* q_full = k_full + 12;  // q, its factors and the mask
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(k_full + 13);
  volatile int* failed = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint32_t* msk = reinterpret_cast<uint32_t*>(smem + Sh::kMask);

  const int cw = warp & 3;  // of the converting warps: its page of a block
  struct Page {
    unsigned need;
    size_t ph;
    float ks, vs;
  };
  const int32_t* pt = a.page_table + static_cast<size_t>(b) * a.max_pages;
  auto load_id = [&](int blk) {  // this warp's page of a block
    const int x = blk * kRPages + cw;
    return x < pages ? __ldg(pt + page_of(x)) : 0;
  };
  // The rows of it that some query of the CTA keeps, its place in the pool, its scales.
  auto open_page = [&](int blk, int pg) -> Page {
    Page p{0u, 0, 1.f, 1.f};
    const int x = blk * kRPages + cw;
    if (x >= pages) return p;
    const int j0 = page_of(x) * 16;
    if (j0 + 15 <= i_last && (j0 + 15 < P || j0 >= i_first)) {
      p.need = 0xffffu;
    } else {
      const int j = j0 + (lane & 15);
      bool need = j <= i_last;
      if (need && j >= P && j < i_first) {
        // kept by some query: a set bit among offsets lo + 1 .. hi + 1
        const uint32_t* mrow = a.keep_mask + (static_cast<size_t>(b) * a.hkv + hk) * a.mask_words;
        const int lo = i_first - j - 1, hi = min(Wn, i_last - j) - 1;
        need = false;
        for (int w = lo >> 5; lo <= hi && w <= (hi >> 5); ++w) {
          uint32_t v = __ldg(mrow + w);
          if (w == (lo >> 5)) v &= 0xffffffffu << (lo & 31);
          if (w == (hi >> 5) && (hi & 31) != 31) v &= (2u << (hi & 31)) - 1u;
          need |= v != 0u;
        }
      }
      p.need = __ballot_sync(0xffffffffu, need) & 0xffffu;
    }
    if (p.need != 0u && static_cast<unsigned>(pg) >= static_cast<unsigned>(a.num_pages)) {
      set_error(a.err, DSA_DEV_BAD_PAGE);
      p.need = 0u;
    }
    if (p.need != 0u) {
      p.ph = static_cast<size_t>(pg) * a.hkv + hk;
      p.ks = __ldg(a.k_scale + p.ph);
      p.vs = __ldg(a.v_scale + p.ph);
    }
    return p;
  };
  // The codes of a page on their way to shared memory (not through registers: what an SM can
  // have in flight there is bounded by the few KB of L1 beside the tiles); rows that nobody
  // needs become zeros.
  auto load_codes = [&](const uint8_t* base, const Page& p, uint32_t to) {
    const uint8_t* src = base + p.ph * (16 * D) + 16 * lane;
#pragma unroll
    for (int i = 0; i < D / 32; ++i)  // 512 bytes
      cp_async16_zfill(to + 512 * i + 16 * lane, src + 512 * i,
                       (p.need >> ((512 * i + 16 * lane) / D)) & 1u);
  };
  // Its fp16 values into rows 16 cw .. of a block's tile: 64-dim halves of 64 rows of 128
  // bytes, 16-byte pieces swizzled by the row; a lane has 8 codes of every kStep-th row.
  constexpr int kLanes = D / 8, kStep = 32 / kLanes;
  const uint32_t f16_at = sm + (D == 128 ? (lane >> 3) & 1 : 0) * kRHalf +
                          (16 * cw + lane / kLanes) * 128 + (((lane & 7) ^ (lane / kLanes)) << 4);
  auto take_codes = [&](uint32_t from, uint2 (&v)[D / 16]) {
#pragma unroll
    for (int i = 0; i < D / 16; ++i) v[i] = lds64(from + 256 * i + 8 * lane);
  };
  auto store_f16 = [&](int tile, const uint2 (&v)[D / 16]) {
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
      sts128((f16_at ^ ((kStep * i & 7) << 4)) + tile + i * kStep * 128,
             make_uint4(e4m3x2_f16x2(v[i].x), e4m3x2_f16x2_hi(v[i].x), e4m3x2_f16x2(v[i].y),
                        e4m3x2_f16x2_hi(v[i].y)));
  };
  if (warp == 8) tmem_alloc<Sh::kTmem>(tmem_slot);
  if (tid == 256) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      mbar_init(k_full + e, 4);
      mbar_init(v_full + e, 4);
      mbar_init(s_done + e, 1);
      mbar_init(o_done + e, 1);
      mbar_init(p_full + e, 4);
      mbar_init(i_full + e, 1);
    }
    mbar_init(q_full, 4);
    fence_mbar_init();
    *failed = 0;
  }
  if (tid < 4) quant_redo_clear();
  const bool converts = warp >= 4 && warp < 8;
  const int id0 = converts ? load_id(0) : 0;
  __syncthreads();  // barriers, tensor-memory address
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);

  bool ok = true;
  if (converts) {
    // ================= converters: a page of every block, codes loaded a block ahead =========
    // K goes a block ahead of V, so that the scores after next wait for no V.
    const uint32_t at_k = sm + Sh::kCodes + cw * 2 * 16 * D, at_v = at_k + 16 * D;
    auto put_k = [&](int blk, const Page& p) {  // codes of the block are there
      const int e = blk & 1;
      uint2 x[D / 16];
      take_codes(at_k, x);
      if (lane == 0) {
        // a page's K scale, log2 and reciprocal of its V scale
        const uint32_t ks = __float_as_uint(p.ks), vs = __float_as_uint(p.vs);
        if (!scale_ok(ks) || !scale_ok(vs)) set_error(a.err, DSA_DEV_BAD_SCALE);
        info[(blk & (kRInfos - 1)) * kRPages + cw] =
            make_float4(p.ks, static_cast<float>(scale_exp(vs)),
                        __uint_as_float((254u << 23) - vs), 0.f);
      }
      if (blk > 1)  // its place is free
        ok = mbar_wait(s_done + e, (static_cast<uint32_t>(blk >> 1) - 1u) & 1u) && ok;
      if (blk * kRPages + cw < pages) store_f16(Sh::kK + kHalves * e * kRHalf, x);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(k_full + e);
    };
    Page page = open_page(0, id0);  // of the block whose K comes next
    load_codes(a.k, page, at_k);
    cp_async_commit();
    load_codes(a.v, page, at_v);
    cp_async_commit();
    int id = load_id(1);
    for (int blk = -1; blk < nblocks; ++blk) {
      // K of block blk + 1 (before block 1's there are block 0's V and block 1's K to wait for)
      if (blk == 0) cp_async_wait<0>();
      else cp_async_wait<1>();
      __syncwarp();
      if (blk + 1 < nblocks) put_k(blk + 1, page);
      const Page held = page;
      if (blk + 2 < nblocks) {
        page = open_page(blk + 2, id);
        load_codes(a.k, page, at_k);
        id = load_id(blk + 3);
      }
      cp_async_commit();
      if (blk >= 0) {  // V of block blk
        uint2 x[D / 16];
        cp_async_wait<1>();
        __syncwarp();
        take_codes(at_v, x);
        if (blk > 0)  // the last block's second product is done with its place
          ok = mbar_wait(o_done + (~blk & 1), static_cast<uint32_t>((blk - 1) >> 1) & 1u) && ok;
        if (blk * kRPages + cw < pages) store_f16(Sh::kV, x);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(v_full + (blk & 1));
        if (blk + 1 < nblocks) load_codes(a.v, held, at_v);
        cp_async_commit();
      }
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
    }
    cp_async_wait<0>();
    if (!ok) *failed = 1;
  } else if (warp == 8) {
    // ================= issuing =================
    const uint64_t q_desc = tc_desc(sm + Sh::kQ, 16, 1024, kSwizzle128);
    const uint64_t k_desc = tc_desc(sm + Sh::kK, 16, 1024, kSwizzle128);
    const uint64_t v_desc = tc_desc(sm + Sh::kV, kRHalf, 1024, kSwizzle128);
    auto issue_s = [&](int blk) {  // S = Q K^T over the block's pages, when K is there
      ok = mbar_wait(k_full + (blk & 1), static_cast<uint32_t>(blk >> 1) & 1u) && ok;
      tc_fence_after();
      if (!__all_sync(0xffffffffu, ok)) return;
      const uint32_t id_s = tc_idesc(128, 16 * min(kRPages, pages - blk * kRPages), false);
      const uint32_t to = tmem + Sh::kS + (blk & 1) * kRBlock;
      const uint64_t kd = k_desc + ((blk & 1) * kHalves * kRHalf >> 4);
      if (elect_one()) {
        mbar_arrive(i_full + (blk & 1));
#pragma unroll
        for (int s = 0; s < D / 16; ++s)
          tc_mma_f16(to, q_desc + (((s >> 2) * kRQHalf + (s & 3) * 32) >> 4),
                     kd + (((s >> 2) * kRHalf + (s & 3) * 32) >> 4), id_s, s > 0);
        tc_commit(s_done + (blk & 1));
      }
      __syncwarp();
    };
    ok = mbar_wait(q_full, 0);
    for (int blk = 0; blk < min(2, nblocks); ++blk) issue_s(blk);
    for (int blk = 0; blk < nblocks; ++blk) {
      const int e = blk & 1, present = min(kRPages, pages - blk * kRPages);
      const uint32_t phase = static_cast<uint32_t>(blk >> 1) & 1u;
      ok = mbar_wait(v_full + e, phase) && mbar_wait(p_full + e, phase) && ok;
      tc_fence_after();
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const uint32_t from = tmem + Sh::kS + e * kRBlock;
      if (elect_one()) {  // O += P V, a step for each page
        constexpr uint32_t id_o = tc_idesc_b_rows(128, D);
#pragma unroll
        for (int s = 0; s < kRPages; ++s)
          if (s < present)
            tc_mma_f16_ta(tmem + Sh::kO, from + 8 * s, v_desc + (s * 2048 >> 4), id_o, blk > 0 || s > 0);
        tc_commit(o_done + e);
      }
      __syncwarp();
      if (blk + 2 < nblocks) {  // into the place of these weights
        ok = mbar_wait(o_done + e, phase) && ok;
        issue_s(blk + 2);
      }
    }
    if (!ok) *failed = 1;
  } else {
    // ================= weighing: one query row per thread =================
    const int r = tid;
    const int i = i_first + (r >> LG);
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(32 * warp) << 16);
    // q as fp16, a row (query token, head) scaled by its own power of two: a query's result
    // does not hang on the others of its tile.  The scale's sign goes into q, so that a
    // page's largest score is its largest product.
    // A warp without a query has nothing to weigh (what its rows of S and O hold is theirs
    // alone): it keeps the blocks' count and no more.
    const bool idle = t0 + (32 * warp >> LG) >= t1;
    if (!idle) {
      constexpr int kPass = 4 * kStep;  // rows a pass
      const int piece = lane % kLanes, r0 = 32 * warp + lane / kLanes;
      auto load_q = [&](int g, uint4 (&x)[4]) {
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const int row = r0 + kPass * g + kStep * y;
          x[y] = t0 + (row >> LG) < t1
                     ? __ldg(reinterpret_cast<const uint4*>(a.q + qh_of(row) * D) + piece)
                     : make_uint4(0u, 0u, 0u, 0u);
        }
      };
      uint4 x[4], ahead[4];
      load_q(0, x);
      load_q(1, ahead);
#pragma unroll 1
      for (int g = 0; g < 32 / kPass; ++g) {
        uint32_t m[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          m[y] = x[y].x & 0x7fff7fffu;
          asm("max.bf16x2 %0, %0, %1;" : "+r"(m[y]) : "r"(x[y].y & 0x7fff7fffu));
          asm("max.bf16x2 %0, %0, %1;" : "+r"(m[y]) : "r"(x[y].z & 0x7fff7fffu));
          asm("max.bf16x2 %0, %0, %1;" : "+r"(m[y]) : "r"(x[y].w & 0x7fff7fffu));
        }
#pragma unroll
        for (int o = kLanes / 2; o >= 1; o >>= 1)
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const uint32_t other = __shfl_xor_sync(0xffffffffu, m[y], o);
            asm("max.bf16x2 %0, %0, %1;" : "+r"(m[y]) : "r"(other));
          }
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const int row = r0 + kPass * g + kStep * y;
          const int qe = q_exponent(fmaxf(bf16_lo(m[y]), bf16_hi(m[y])));
          const float down = a.scale_log2 < 0.f ? -pow2i(-qe) : pow2i(-qe);
          // at least 2^-105, so that a masked score (-inf) times it and a page's scale (2^-40
          // and more) stays one; a score so scaled is below 2^-40
          if (piece == 0) up[row] = fmaxf(fabsf(a.scale_log2) * pow2i(qe), 0x1p-105f);
          sts128(sm + Sh::kQ + (piece >> 3) * kRQHalf + row * 128 + (((piece & 7) ^ (row & 7)) << 4),
                 make_uint4(f16x2_rn(bf16_lo(x[y].x) * down, bf16_hi(x[y].x) * down),
                            f16x2_rn(bf16_lo(x[y].y) * down, bf16_hi(x[y].y) * down),
                            f16x2_rn(bf16_lo(x[y].z) * down, bf16_hi(x[y].z) * down),
                            f16x2_rn(bf16_lo(x[y].w) * down, bf16_hi(x[y].w) * down)));
          x[y] = ahead[y];
        }
        if (g + 2 < 32 / kPass) load_q(g + 2, ahead);
      }
    }
    {
      // the mask shifted by one: bit o keeps offset o, 0 (the query itself) and 1 .. window
      const uint32_t* mrow = a.keep_mask + (static_cast<size_t>(b) * a.hkv + hk) * a.mask_words;
      for (int x = tid; x < a.max_window / 32 + 1; x += 128) {
        const uint32_t lo = x == 0 ? 0x80000000u : __ldg(mrow + x - 1);
        const uint32_t hi = x < a.mask_words ? __ldg(mrow + x) : 0u;
        uint32_t m = (hi << 1) | (lo >> 31);
        const int live = Wn + 1 - 32 * x;
        if (live < 32) m = live <= 0 ? 0u : m & ((1u << live) - 1u);
        msk[x] = m;
      }
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(q_full);
    ok = mbar_wait(q_full, 0);  // the other warps' part of the mask
    const float f = up[r];
    float ref = kRNoRef, l = 0.f;
    for (int blk = 0; blk < nblocks; ++blk) {
      const int e = blk & 1, present = min(kRPages, pages - blk * kRPages);
      const uint32_t phase = static_cast<uint32_t>(blk >> 1) & 1u;
      ok = mbar_wait(i_full + e, phase) && (idle || mbar_wait(s_done + e, phase)) && ok;
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      if (idle) {
        if (lane == 0) mbar_arrive(p_full + e);
        continue;
      }
      tc_fence_after();
      const uint32_t t_s = t_lane + Sh::kS + e * kRBlock;
      const float4* in = info + (blk & (kRInfos - 1)) * kRPages;
      uint32_t s[kRPages][16];
#pragma unroll
      for (int x = 0; x < kRPages; ++x)
        if (x < present) tmem_load<16>(t_s + 16 * x, s[x]);
      tc_wait_ld();
      const int j_last = page_of(blk * kRPages + present - 1) * 16 + 15;
      if (j_last >= P || j_last > i_first) {
        // some query does not keep some row: scores that this one does not keep become -inf
#pragma unroll
        for (int x = 0; x < kRPages; ++x) {
          if (x < present) {
            const int j0 = page_of(blk * kRPages + x) * 16;
            // columns up to the query's own row, and of those prompt rows and kept offsets
            const int c = i - j0;  // column of the query itself
            uint32_t on = c < 0 ? 0u : c >= 15 ? 0xffffu : (2u << c) - 1u;
            if (j0 + 15 >= P) {
              const int words = a.max_window / 32 + 1;
              const int base = c - 15;  // offset of column 15
              const int w0 = max(base, 0) >> 5, sh = max(base, 0) & 31;
              const uint32_t lo = w0 < words ? msk[w0] : 0u, hi = w0 + 1 < words ? msk[w0 + 1] : 0u;
              uint32_t win = __funnelshift_r(lo, hi, sh);
              if (base < 0) win = base <= -32 ? 0u : win << -base;
              win = __brev(win) >> 16;  // the bit of column 15 - k to bit 15 - k
              const int np = P - j0;    // prompt rows of the page
              on &= win | (np <= 0 ? 0u : (1u << min(np, 16)) - 1u);
            }
            if (!__all_sync(0xffffffffu, on == 0xffffu)) {
#pragma unroll
              for (int q = 0; q < 16; ++q)
                if (!((on >> q) & 1u)) s[x][q] = 0xff800000u;
            }
          }
        }
      }
      float top = -INFINITY;  // the row's largest score
#pragma unroll
      for (int x = 0; x < kRPages; ++x) {
        if (x < present) {
          float m[4];
#pragma unroll
          for (int q = 0; q < 4; ++q)
            m[q] = fmaxf(max3(__uint_as_float(s[x][q]), __uint_as_float(s[x][4 + q]),
                              __uint_as_float(s[x][8 + q])),
                         __uint_as_float(s[x][12 + q]));
          const float2 pgi = *reinterpret_cast<const float2*>(in + x);
          top = fmaxf(top, fmaf(fmaxf(max3(m[0], m[1], m[2]), m[3]), f * pgi.x, pgi.y));
        }
      }
      // (the difference is exact where it counts; ref + 14 rounds to as much as ref + 16 from
      // 2^25 on, and 2^16 is no fp16)
      const bool over = top - ref > kRHead + kRSlack;
      if (__any_sync(0xffffffffu, over)) {
        const float to = over ? top - kRHead : ref;
        const float down = ex2_approx(ref - to);
        ref = to;
        l *= down;
        if (blk > 0) {
          ok = mbar_wait(o_done + (e ^ 1), static_cast<uint32_t>((blk - 1) >> 1) & 1u) && ok;
          __syncwarp();
          tc_fence_after();
#pragma unroll 1
          for (int h = 0; h < D / 16; ++h) {
            uint32_t o[16];
            tmem_load<16>(t_lane + Sh::kO + 16 * h, o);
            tc_wait_ld();
#pragma unroll
            for (int q = 0; q < 16; ++q) o[q] = __float_as_uint(__uint_as_float(o[q]) * down);
            tmem_store16(t_lane + Sh::kO + 16 * h, o);
          }
        }
      }
      // weights, packed over the scores
#pragma unroll
      for (int x = 0; x < kRPages; ++x) {
        if (x < present) {
          const float4 pgi = in[x];
          const float c1 = f * pgi.x, c2 = pgi.y - ref;
          const f32x2 a1 = pack2(c1, c1), a2 = pack2(c2, c2);
          f32x2 sum = pack2(0.f, 0.f);
          uint32_t w[8];
#pragma unroll
          for (int q = 0; q < 16; q += 2) {
            float z0, z1;
            unpack2(fma2(pack2(__uint_as_float(s[x][q]), __uint_as_float(s[x][q + 1])), a1, a2), z0, z1);
            z0 = ex2_approx(z0);
            z1 = ex2_approx(z1);
            sum = add2(sum, pack2(z0, z1));
            w[q / 2] = f16x2_rn(z0, z1);
          }
          tmem_store8(t_s + 8 * x, w);
          float u, t;
          unpack2(sum, u, t);
          l = fmaf(u + t, pgi.z, l);
        }
      }
      tc_wait_st();
      tc_fence_before();
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      if (lane == 0) mbar_arrive(p_full + e);
    }
    if (ok && !idle)
      ok = mbar_wait(o_done + ((nblocks - 1) & 1), static_cast<uint32_t>((nblocks - 1) >> 1) & 1u);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) *failed = 1;
    if (ok && !idle) {
      tc_fence_after();
      const float inv = 1.f / l;
      const bool mine = t0 + (r >> LG) < t1;
      if (a.lse != nullptr && mine) a.lse[qh_of(r)] = (ref + log2f(l)) * kLn2;
      uint16_t* to = reinterpret_cast<uint16_t*>(a.out) + qh_of(r) * D;
      const bool wide = (reinterpret_cast<uintptr_t>(a.out) & 31u) == 0;  // rows are 256 bytes
      float probe = 0.f;
#pragma unroll 1
      for (int h = 0; h < D / 32; ++h) {
        uint32_t o[32];
        tmem_load<32>(t_lane + Sh::kO + 32 * h, o);
        tc_wait_ld();
        uint32_t w[16];
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          const float u = __uint_as_float(o[2 * q]) * inv, t = __uint_as_float(o[2 * q + 1]) * inv;
          probe += u + t;
          w[q] = bf16x2_rn(u, t);
        }
        if (mine && wide) {
          stg256(to + 32 * h, w);
          stg256(to + 32 * h + 16, w + 8);
        } else if (mine) {
#pragma unroll
          for (int q = 0; q < 4; ++q)
            reinterpret_cast<uint4*>(to + 32 * h)[q] =
                make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
        }
      }
      tc_fence_before();
      // A NaN may come from a row of V that other queries of the CTA keep (weight 0 times
      // NaN), an infinity from a weight past fp16 (scores of 2^20 and more): such a query is done
      // again, from the rows it keeps.
      const unsigned nan =
          __ballot_sync(0xffffffffu, mine && !(fabsf(probe) < INFINITY) && quant_redo_needed(l, ref));
      if (nan != 0u) {
        const unsigned sums = __ballot_sync(0xffffffffu, quant_sum_unsure(l, ref));
        if (lane == 0) {
          quant_redo().out[warp] = nan;
          quant_redo().sum[warp] = sums;
          quant_redo().hit = 1;
        }
      }
    }
  }
  __syncthreads();
  if (*failed != 0) {
    // give products in flight a bounded time to finish before the memory goes back
    if (tid == 0) set_error(a.err, DSA_DEV_TIMEOUT);
    for (int blk = max(0, nblocks - 2); blk < nblocks; ++blk) {
      mbar_wait(s_done + (blk & 1), static_cast<uint32_t>(blk >> 1) & 1u);
      mbar_wait(o_done + (blk & 1), static_cast<uint32_t>(blk >> 1) & 1u);
    }
    __syncthreads();
  }
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc<Sh::kTmem>(tmem);
  }
  if (quant_redo().hit != 0) quant_redo_tile<D, RowsTile<LG>>(a);
}

template <int D, int LG>
cudaError_t launch_one(const QuantChunkLaunch& a, cudaStream_t s) {
  auto kern = quant_chunk_rows_kernel<D, LG>;
  const int smem = RowsShape<D>::smem(a.max_window / 32 + 1);
  static KernelSlots cache;
  int per_sm = 0;
  const cudaError_t e =
      cache.get(reinterpret_cast<const void*>(kern), kRThreads, smem, &per_sm);
  if (e != cudaSuccess) return e;
  constexpr int per_cta = kRRows >> LG;
  return launch_pdl(kern, dim3((a.max_q + per_cta - 1) / per_cta, a.hkv, a.batch), dim3(kRThreads),
                    static_cast<size_t>(smem), s, a);
}

template <int D>
cudaError_t launch_group(const QuantChunkLaunch& a, cudaStream_t s) {
  switch (a.group_log2) {
    case 0: return launch_one<D, 0>(a, s);
    case 1: return launch_one<D, 1>(a, s);
    case 2: return launch_one<D, 2>(a, s);
    default: return launch_one<D, 3>(a, s);
  }
}

}  // namespace

// Which calls this kernel takes: more than 32 rows (fewer are quant_chunk_tc.cu's), when
// their tiles are a quarter of the SMs or more, or no request passes 2048 rows: a tile is
// never cut along its pages, and quant_chunk.cu, which cuts them, was ahead at 32 tiles of
// 4000 rows (62 / 70 us) and behind at 48 (78 / 70); at 8 tiles of 2000 rows 32 / 38, of 1000
// 26 / 22, of 500 19 / 14, and of 2000 rows of which prompt and window leave 110, 18 / 9.
// Measured against the other two (us, this kernel / quant_chunk_tc.cu or quant_chunk.cu,
// batch x kv heads x group, tokens, rows):
//   up to 32 rows of a tile:  128x8x4, 8, 500: 71 / 57;  64x32x1, 32, 1000: 195 / 168
//   33 .. 64:                 128x8x4, 16, 300: 54 / 77 and 80;  64x32x1, 40, 200: 82 / 98
//   more:                     64x8x4, 128, 256: 90 / 150;  8x8x4, 128, 4096: 95 / 271;
//                             8x8x4, 2048, 2048: 396 / 1017
// and with head_dim 64 against quant_chunk.cu: 64x20x1, 8, 300: 46 / 38;  128x8x4, 8, 2000:
// 162 / 141;  64x20x1, 48, 600: 79 / 87;  128x20x1, 400, 400: 341 / 514;  8x8x4, 128, 4096:
// 80 / 224.
bool quant_chunk_rows_fits(const QuantChunkLaunch& a) {
  const int64_t rows = static_cast<int64_t>(a.max_q) << a.group_log2;
  if (rows <= 32 || a.split_setting >= 2 || a.batch > 65535 || a.hkv > 65535) return false;
  return a.split_setting == 1 || a.max_pages <= kQuantWholePages ||
         (rows + kRRows - 1) / kRRows * a.batch * a.hkv * 4 >= a.sms;
}

cudaError_t launch_quant_chunk_rows(const QuantChunkLaunch& a, cudaStream_t s) {
  return a.head_dim == 128 ? launch_group<128>(a, s) : launch_group<64>(a, s);
}

}  // namespace dsa
