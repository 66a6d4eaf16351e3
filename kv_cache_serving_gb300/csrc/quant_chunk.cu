// quant_chunk.cu -- several query tokens per request over the 8-bit paged K/V cache,
// each over its own causal kept set (prompt rows, window offsets of the mask, itself).
//
// Mathematics: as in quant_decode.cu, with a column of the tensor-core products for
// each (query token, head of the kv head's group) and the mask applied to the weights:
//   p_ij = 2^(x_ij + log2 t_j - r_i) if query i keeps row j, else 0.
//
// A tile of rows is one page of one kv head, so its two scales are constants of the
// tile, and a page that no query of the CTA keeps is neither copied nor computed (of a
// page with some kept rows only those are read; the others are zeros).
//
// What bounds it: instruction issue and the legacy tensor path.  Codes become fp16 in
// registers (64 conversions per page and warp) and the scores of every (row, column)
// pass through an exponential, so a warp takes 32 columns: the conversions, the shared
// memory reads and the row bookkeeping of a page are paid once for 32 queries and
// heads, with q and the 32 columns of output in registers (255 of them at D = 128, and 112 to
// 232 bytes spilled: 8 warps per SM; 16 columns and 16 warps measured a third slower).  The
// accumulators hold the output
// transposed (dims x columns), which lets the weights go from the score accumulators to
// the second product by movmatrix alone.
// This kernel serves head_dim 64 up to 32 columns, calls of few tiles over long caches and
// calls whose units are to be cut along their pages; the others go to quant_chunk_tc.cu
// (head_dim 128 up to 32 columns) and quant_chunk_rows.cu.  Measured: 40 tokens over 3000
// rows of one request, 32/8 heads of 128: 36 us in 8 parts (54 whole in quant_chunk_rows.cu).
// Prompts of 32 .. 512 rows of 128 requests, 32/8 heads, take 694 us here, 430 there.
//
// Work split.  A CTA of 4 warps covers 32 KC columns (KC = 4 / KG column groups) of one
// (request, kv head); KG warps share a column group and take its pages in turn, joined
// through shared memory at the end.  Few columns take KG = 4, many KG = 1.  Pages reach
// the CTA through a ring of stages of four pages (one page copied by each warp).  When
// there are too few CTAs the pages of a unit are cut into parts, whose register states
// the last part to arrive sums in order.
#include <math.h>

#include <type_traits>

#include "common.cuh"
#include "host.h"
#include "internal.h"
#include "mma.cuh"
#include "quant.cuh"
#include "quant_redo.cuh"

namespace dsa {
namespace {

constexpr int kCW = 4;          // warps per CTA
constexpr int kCols = 32;       // columns per warp
constexpr int kNT = kCols / 8;  // 8-column tiles per warp
constexpr int kCStages = 3;
// Weights are 2^(y - ref); ref follows the largest y so that it stands for 2^kCHead, once a
// y passes it by kCSlack (as in quant_decode.cu).  Before its first row it is far below
// every score, and finite: -inf - ref stays -inf.
constexpr float kCHead = 4.f, kCSlack = 10.f, kNoRef = -3e38f;

template <int D, int KG>
struct ChunkShape {
  static constexpr int KC = kCW / KG;
  using Tile = QuantTile<D>;
  static constexpr int kPage = 2 * Tile::kBytes;        // K tile, V tile
  static constexpr int kStage = kCW * kPage;
  static constexpr int kStateWords = kNT * (D / 16 * 4 + 4);  // registers of a column group
  // ring, then per stage and page {rows needed, K scale, V scale, -}, then the mask
  static constexpr int kInfoOff = kCStages * kStage;
  static constexpr int kMaskOff = kInfoOff + kCStages * kCW * 16;
  static int smem(int mask_bits_words) { return kMaskOff + 4 * mask_bits_words; }
  // the joining warps' register dumps reuse the ring
  static_assert(KG == 1 || (kCW / 2) * kStateWords * 32 * 4 <= kInfoOff, "dumps fit the ring");
};

// The state of one warp: 32 columns over the rows it has seen.
template <int D>
struct ChunkState {
  static constexpr int NK = D / 16;
  float acc[kNT][NK][4];
  float ref[kNT][2], l[kNT][2];

  __device__ __forceinline__ void reset() {
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        ref[nt][j] = kNoRef;
        l[nt][j] = 0.f;
      }
#pragma unroll
      for (int mt = 0; mt < NK; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[nt][mt][e] = 0.f;
    }
  }
  // Register by register, lanes side by side.
  __device__ __forceinline__ void dump(float* to, int lane) const {
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
      float* p = to + nt * (NK * 4 + 4) * 32 + lane;
#pragma unroll
      for (int mt = 0; mt < NK; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e) p[(mt * 4 + e) * 32] = acc[nt][mt][e];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        p[(NK * 4 + j) * 32] = ref[nt][j];
        p[(NK * 4 + 2 + j) * 32] = l[nt][j];
      }
    }
  }
  // Joins a dumped state (from shared memory, or from global memory past the L1).
  template <bool GLOBAL>
  __device__ __forceinline__ void join(const float* from, int lane) {
    auto get = [&](const float* p) { return GLOBAL ? __ldcg(p) : *p; };
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
      const float* p = from + nt * (NK * 4 + 4) * 32 + lane;
      float wa[2], wb[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float r = get(p + (NK * 4 + j) * 32);
        const float to = fmaxf(ref[nt][j], r);
        wa[j] = ex2_approx(ref[nt][j] - to);
        wb[j] = ex2_approx(r - to);
        ref[nt][j] = to;
        l[nt][j] = l[nt][j] * wa[j] + get(p + (NK * 4 + 2 + j) * 32) * wb[j];
      }
#pragma unroll
      for (int mt = 0; mt < NK; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          acc[nt][mt][e] =
              acc[nt][mt][e] * wa[e & 1] + get(p + (mt * 4 + e) * 32) * wb[e & 1];
    }
  }
};

template <int KG>
struct ChunkTile {  // the last tokens, which see the most rows, first
  static constexpr int kColumns = kCols * (kCW / KG);
  __device__ __forceinline__ static void at(const QuantChunkLaunch& a, int& bpos, int& hk, int& t0) {
    const int unit = blockIdx.x / a.parts;
    bpos = unit / (a.q_tiles * a.hkv);
    hk = unit / a.q_tiles % a.hkv;
    t0 = (a.q_tiles - 1 - unit % a.q_tiles) * (kColumns >> a.group_log2);
  }
};

template <int D, int KG>
__global__ void __launch_bounds__(kCW * 32, D == 128 ? 2 : 3)
    quant_chunk_kernel(const QuantChunkLaunch a) {
  using Sh = ChunkShape<D, KG>;
  using Tile = QuantTile<D>;
  constexpr int NK = D / 16;
  extern __shared__ __align__(128) unsigned char smem[];
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, c = lane & 3;
  const int kg = warp % KG, cg = warp / KG;
  // unit: request, kv head, tile of query tokens (the last tokens, which see the most
  // rows, first); part: its share of the unit's pages
  const int part = blockIdx.x % a.parts, unit = blockIdx.x / a.parts;
  const int qt = a.q_tiles - 1 - unit % a.q_tiles;
  const int hk = unit / a.q_tiles % a.hkv, bpos = unit / (a.q_tiles * a.hkv);
  const int b = a.order != nullptr ? __ldg(a.order + bpos) : bpos;
  if (static_cast<unsigned>(b) >= static_cast<unsigned>(a.batch)) {
    if (qt == 0 && hk == 0 && part == 0 && threadIdx.x == 0) set_error(a.err, DSA_DEV_BAD_ORDER);
    return;
  }
  const int lg = a.group_log2, per_cta = (kCols * Sh::KC) >> lg;
  const int t0 = qt * per_cta;
  const int L = a.seq_len[b], n = a.q_len[b], P = a.prompt_len[b], W = a.window[b];
  int code = 0;
  if (L < 1 || L > a.max_pages * kPage) code = DSA_DEV_BAD_SEQ_LEN;
  else if (n < 0 || n > L || n > a.max_q) code = DSA_DEV_BAD_QLEN;
  else if (P < 0) code = DSA_DEV_BAD_PROMPT;
  else if (W < 0 || W > a.max_window) code = DSA_DEV_BAD_WINDOW;
  if (code != 0) {
    // q_len is not trusted: NaN into every slot of the unit (by part 0)
    if (part != 0) return;
    if (qt == 0 && hk == 0 && threadIdx.x == 0) set_error(a.err, code);
    const int heads = 1 << lg;
    for (int x = threadIdx.x; x < per_cta * heads * D; x += kCW * 32) {
      const int t = t0 + x / (heads * D);
      if (t >= a.max_q) break;
      const size_t qh = (static_cast<size_t>(b) * a.max_q + t) * a.hq + hk * heads + x / D % heads;
      a.out[qh * D + x % D] = 0x7fc0;
      if (a.lse != nullptr && x % D == 0) a.lse[qh] = __int_as_float(0x7fc00000);
    }
    return;
  }
  if (t0 >= n) return;
  const int t1 = min(t0 + per_cta, n);
  const int i_first = L - n + t0, i_last = L - n + t1 - 1;
  // pages scanned: those of the prompt rows [0, pa), then those from the window's start
  const int n_prompt = min(P, i_last + 1);
  const int pa = (n_prompt + 15) >> 4;
  const int pb = max(pa, max(i_first - W, 0) >> 4), pe = i_last >> 4;
  const int pages = pa + max(0, pe - pb + 1);
  const int per_part = (pages + a.parts - 1) / a.parts;
  const int nparts = (pages + per_part - 1) / per_part;
  if (part >= nparts) return;
  const int x0 = part * per_part, x1 = min(pages, x0 + per_part);
  auto page_of = [&](int x) { return x < pa ? x : pb + (x - pa); };

  // the mask shifted by one: bit o of the words keeps offset o, 0 (the query itself)
  // and 1 .. W
  uint32_t* msk = reinterpret_cast<uint32_t*>(smem + Sh::kMaskOff);
  {
    const uint32_t* mrow = a.keep_mask + (static_cast<size_t>(b) * a.hkv + hk) * a.mask_words;
    const int words = a.max_window / 32 + 1;
    for (int x = threadIdx.x; x < words; x += kCW * 32) {
      const uint32_t lo = x == 0 ? 0x80000000u : __ldg(mrow + x - 1);
      const uint32_t hi = x < a.mask_words ? __ldg(mrow + x) : 0u;
      uint32_t v = (hi << 1) | (lo >> 31);
      const int live = W + 1 - 32 * x;  // bits 32x .. that are at most W
      if (live < 32) v = live <= 0 ? 0u : v & ((1u << live) - 1u);
      msk[x] = v;
    }
  }
  const int32_t* pt = a.page_table + static_cast<size_t>(b) * a.max_pages;
  const uint32_t ring = smem_addr(smem);
  int4* info = reinterpret_cast<int4*>(smem + Sh::kInfoOff);
  const int nstages = (x1 - x0 + kCW - 1) / kCW;
  // this warp's page of stage k (its id is loaded a stage before its copies go out)
  auto load_page = [&](int k) {
    const int x = x0 + k * kCW + warp;
    return x < x1 ? __ldg(pt + page_of(x)) : 0;
  };
  auto any_bit = [&](int lo, int hi) {  // bits lo..hi of msk, 0 <= lo <= hi <= W
    for (int w = lo >> 5; w <= (hi >> 5); ++w) {
      uint32_t x = msk[w];
      if (w == (lo >> 5)) x &= 0xffffffffu << (lo & 31);
      if (w == (hi >> 5) && (hi & 31) != 31) x &= (2u << (hi & 31)) - 1u;
      if (x != 0u) return true;
    }
    return false;
  };
  auto issue = [&](int k, int pg) {
    const int x = x0 + k * kCW + warp, s = k % kCStages;
    if (x < x1) {
      const int j = page_of(x) * 16 + (lane & 15);
      bool need = j <= i_last;
      if (need && j >= P && j < i_first) {
        const int lo = i_first - j, hi = min(W, i_last - j);
        need = lo <= hi && any_bit(lo, hi);
      }
      unsigned mask = __ballot_sync(0xffffffffu, need) & 0xffffu;
      if (mask != 0u && static_cast<unsigned>(pg) >= static_cast<unsigned>(a.num_pages)) {
        set_error(a.err, DSA_DEV_BAD_PAGE);
        mask = 0u;
      }
      if (lane == 0) info[s * kCW + warp].x = static_cast<int>(mask);
      if (mask != 0u) {
        const size_t ph = static_cast<size_t>(pg) * a.hkv + hk;
        const uint8_t* kp = a.k + ph * (16 * D);
        const uint8_t* vp = a.v + ph * (16 * D);
        const uint32_t dst = ring + s * Sh::kStage + warp * Sh::kPage;
#pragma unroll
        for (int i = 0; i < Tile::kCopies; ++i) {
          const int r = Tile::copy_row(i, lane), ch = Tile::copy_piece(lane);
          const bool in = (mask >> r) & 1u;
          const uint32_t to = dst + Tile::offset(r, ch);
          cp_async16_zfill(to, kp + r * D + 16 * ch, in);
          cp_async16_zfill(to + Tile::kBytes, vp + r * D + 16 * ch, in);
        }
        if (lane < 2)
          cp_async4_zfill(smem_addr(&info[s * kCW + warp].y) + 4 * lane,
                          (lane == 0 ? a.k_scale : a.v_scale) + ph, true);
      }
    }
    cp_async_commit();
  };
  if (threadIdx.x < 4) quant_redo_clear();
  __syncthreads();  // the mask
  {
    int pg[kCStages - 1];
#pragma unroll
    for (int k = 0; k < kCStages - 1; ++k) pg[k] = load_page(k);
#pragma unroll
    for (int k = 0; k < kCStages - 1; ++k) issue(k, pg[k]);
  }
  int pg_next = load_page(kCStages - 1);

  // q of the column group as B operands: column 8 nt + g of the thread's share
  const int gt0 = t0 + ((cg * kCols) >> lg);         // first token of the group
  const int gt1 = min(gt0 + (kCols >> lg), t1);
  const bool active = gt0 < gt1;
  uint32_t q[kNT][NK][2];
  float f[kNT][2];
#pragma unroll
  for (int nt = 0; nt < kNT; ++nt) {
    const int col = 8 * nt + g, t = gt0 + (col >> lg);
    uint32_t w[D / 8];
#pragma unroll
    for (int i = 0; i < D / 8; ++i) w[i] = 0u;
    if (t < gt1) {
      const size_t qh =
          (static_cast<size_t>(b) * a.max_q + t) * a.hq + (hk << lg) + (col & ((1 << lg) - 1));
      const uint4* p = reinterpret_cast<const uint4*>(a.q + qh * D + c * (D / 4));
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint4 v = __ldg(p + i);
        w[4 * i] = v.x;
        w[4 * i + 1] = v.y;
        w[4 * i + 2] = v.z;
        w[4 * i + 3] = v.w;
      }
    }
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
      amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(w[i])), fabsf(bf16_hi(w[i]))));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    const int e = q_exponent(amax);
    const float down = pow2i(-e);
#pragma unroll
    for (int i = 0; i < NK; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        q[nt][i][h] = f16x2_rn(bf16_lo(w[2 * i + h]) * down, bf16_hi(w[2 * i + h]) * down);
    const float up = a.scale_log2 * pow2i(e);
    f[nt][0] = __shfl_sync(0xffffffffu, up, (2 * c) * 4);
    f[nt][1] = __shfl_sync(0xffffffffu, up, (2 * c + 1) * 4);
  }

  ChunkState<D> st;
  st.reset();
  bool bad = false;
  const int i_lo = L - n + gt0, i_hi = L - n + gt1 - 1;
  for (int k = 0; k < nstages; ++k) {
    cp_async_wait<kCStages - 2>();
    __syncthreads();  // stage k has landed; stage k - 1 is free
    issue(k + kCStages - 1, pg_next);
    pg_next = load_page(k + kCStages);
    if (!active) continue;
    const int s = k % kCStages;
#pragma unroll 1
    for (int e = kg; e < kCW; e += KG) {
      const int x = x0 + k * kCW + e;
      if (x >= x1) break;
      const int4 in = info[s * kCW + e];
      const int j0 = page_of(x) * 16;
      if (in.x == 0 || j0 > i_hi) continue;
      const uint32_t ks = static_cast<uint32_t>(in.y), vs = static_cast<uint32_t>(in.z);
      bad |= !(scale_ok(ks) && scale_ok(vs));
      const float lv = static_cast<float>(scale_exp(vs)), kscale = __uint_as_float(ks);
      const float inv = __uint_as_float((254u << 23) - vs);
      const uint32_t tile = ring + s * Sh::kStage + e * Sh::kPage;
      float z[kNT][4];
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
        for (int v = 0; v < 4; ++v) z[nt][v] = 0.f;
      {
        uint32_t w[2][Tile::kKW];
        Tile::load_k(tile, lane, w);
#pragma unroll
        for (int i = 0; i < NK; ++i) {
          const uint32_t a0 = e4m3x2_f16x2(w[0][i]), a1 = e4m3x2_f16x2(w[1][i]);
          const uint32_t a2 = e4m3x2_f16x2_hi(w[0][i]), a3 = e4m3x2_f16x2_hi(w[1][i]);
#pragma unroll
          for (int nt = 0; nt < kNT; ++nt) mma_f16(z[nt], a0, a1, a2, a3, q[nt][i][0], q[nt][i][1]);
        }
      }
      // Scores to weights.  A page of prompt rows before the group's first query is kept
      // whole and carries no mask arithmetic; else bit 4 nt + v of `keep` tells.
      uint32_t p[kNT][2];
      auto weigh = [&](auto masked, uint32_t keep) {
        bool over = false;
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float c1 = f[nt][h] * kscale;
#pragma unroll
            for (int v = h; v < 4; v += 2) {
              z[nt][v] = fmaf(z[nt][v], c1, lv);
              if (decltype(masked)::value && !((keep >> (4 * nt + v)) & 1u)) z[nt][v] = -INFINITY;
            }
            over |= fmaxf(z[nt][h], z[nt][2 + h]) - st.ref[nt][h] > kCHead + kCSlack;
          }
        if (__any_sync(0xffffffffu, over)) {
#pragma unroll
          for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float mx = fmaxf(z[nt][h], z[nt][2 + h]);
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
              const float to = fmaxf(st.ref[nt][h], mx - kCHead);
              const float down = ex2_approx(st.ref[nt][h] - to);
              st.ref[nt][h] = to;
              st.l[nt][h] *= down;
#pragma unroll
              for (int mt = 0; mt < NK; ++mt) {
                st.acc[nt][mt][h] *= down;
                st.acc[nt][mt][2 + h] *= down;
              }
            }
        }
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) {
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            z[nt][v] = ex2_approx(z[nt][v] - st.ref[nt][v & 1]);
            st.l[nt][v & 1] = fmaf(z[nt][v], inv, st.l[nt][v & 1]);
          }
          p[nt][0] = movmatrix_trans(f16x2_rn(z[nt][0], z[nt][1]));
          p[nt][1] = movmatrix_trans(f16x2_rn(z[nt][2], z[nt][3]));
        }
      };
      if (j0 + 15 < P && j0 + 15 <= i_lo) {
        weigh(std::false_type{}, 0u);
      } else {
        uint32_t keep = 0u;
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            const int j = j0 + g + 8 * (v >> 1);
            const int o = i_lo + ((8 * nt + 2 * c + (v & 1)) >> lg) - j;
            bool on = o >= 0;
            if (on && j >= P) on = o <= W && ((msk[o >> 5] >> (o & 31)) & 1u);
            keep |= on ? 1u << (4 * nt + v) : 0u;
          }
        weigh(std::true_type{}, keep);
      }
      uint32_t w[4][Tile::kVW];
      Tile::load_v(tile + Tile::kBytes, lane, w);
#pragma unroll
      for (int mt = 0; mt < NK; ++mt) {
        uint32_t va[4];
        Tile::frag_v(w, mt, va);
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt)
          mma_f16(st.acc[nt][mt], va[0], va[1], va[2], va[3], p[nt][0], p[nt][1]);
      }
    }
  }
  if (bad) set_error(a.err, DSA_DEV_BAD_SCALE);
  cp_async_wait<0>();

  // the KG warps of a column group join: half of them hand their registers to the
  // other half, until one holds the group's state
  float* dumps = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int half = KG / 2; half >= 1; half /= 2) {
    __syncthreads();
    if (kg >= half && kg < 2 * half)
      st.dump(dumps + (cg * half + kg - half) * Sh::kStateWords * 32, lane);
    __syncthreads();
    if (kg < half) st.template join<false>(dumps + (cg * half + kg) * Sh::kStateWords * 32, lane);
  }
  if (nparts > 1) {
    // this part's state to the workspace; the last part to arrive sums them in order
    float* base = a.part + static_cast<size_t>(unit) * a.parts * (Sh::KC * Sh::kStateWords * 32);
    auto of = [&](int p) { return base + (p * Sh::KC + cg) * Sh::kStateWords * 32; };
    if (kg == 0) st.dump(of(part), lane);
    __shared__ int last;
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) {
      last = atomicAdd(a.count + unit, 1) == nparts - 1;
      if (last) a.count[unit] = 0;  // every part has arrived
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    if (kg == 0) {
      st.reset();
      for (int p = 0; p < nparts; ++p) st.template join<true>(of(p), lane);
    }
  }
  if (kg == 0 && active) {
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float l = st.l[nt][h];
        l += __shfl_xor_sync(0xffffffffu, l, 4);
        l += __shfl_xor_sync(0xffffffffu, l, 8);
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        const int col = 8 * nt + 2 * c + h, t = gt0 + (col >> lg);
        if (t >= gt1) continue;
        const size_t qh =
            (static_cast<size_t>(b) * a.max_q + t) * a.hq + (hk << lg) + (col & ((1 << lg) - 1));
        const float r = 1.f / l;
        float probe = 0.f;
        uint32_t o[NK];
#pragma unroll
        for (int mt = 0; mt < NK; ++mt) {
          o[mt] = bf16x2_rn(st.acc[nt][mt][h] * r, st.acc[nt][mt][2 + h] * r);
          probe += st.acc[nt][mt][h] + st.acc[nt][mt][2 + h];
        }
        // A NaN may come from a row of V that other queries of the tile keep (weight 0 times NaN):
        // such a column is done again, from the rows it keeps.
        if (probe != probe && quant_redo_needed(l, st.ref[nt][h])) {
          quant_redo().hit = 1;
          atomicOr(&quant_redo().out[cg], 1u << col);
          if (quant_sum_unsure(l, st.ref[nt][h])) atomicOr(&quant_redo().sum[cg], 1u << col);
        }
        uint4* to = reinterpret_cast<uint4*>(a.out + qh * D + g * (D / 8));
#pragma unroll
        for (int i = 0; i < NK / 4; ++i)
          to[i] = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
        if (a.lse != nullptr && g == 0)
          a.lse[qh] = (st.ref[nt][h] + log2f(l)) * kLn2;
      }
  }
  __syncthreads();  // after the columns' first output
  if (quant_redo().hit != 0) quant_redo_tile<D, ChunkTile<KG>>(a);
}

template <int D, int KG>
cudaError_t launch_one(QuantChunkLaunch a, cudaStream_t s) {
  using Sh = ChunkShape<D, KG>;
  auto kern = quant_chunk_kernel<D, KG>;
  const int smem = Sh::smem(a.max_window / 32 + 1);
  static KernelSlots cache;
  int per_sm = 0;
  const cudaError_t e = cache.get(reinterpret_cast<const void*>(kern), kCW * 32, smem, &per_sm);
  if (e != cudaSuccess) return e;
  const int per_cta = (kCols * Sh::KC) >> a.group_log2;
  a.q_tiles = (a.max_q + per_cta - 1) / per_cta;
  const int64_t units = static_cast<int64_t>(a.q_tiles) * a.hkv * a.batch;
  const int64_t slots = static_cast<int64_t>(per_sm) * a.sms;
  // parts of a unit: by the setting, else only when the units leave half of the slots
  // empty (a part keeps two stages of pages); as many as the workspace holds
  int64_t parts = 1;
  if (a.split_setting >= 2) {
    parts = a.split_setting;
  } else if (a.split_setting == 0 && units * 2 <= slots) {
    parts = slots / units;
    const int64_t most = (a.max_pages + 2 * kCW - 1) / (2 * kCW);
    if (parts > most) parts = most;
    if (parts > kQuantMaxParts) parts = kQuantMaxParts;
  }
  const int64_t hold = units > kMultiCounters ? 1 : a.part_cap / (units * Sh::KC * Sh::kStateWords * 32);
  if (parts > hold) parts = hold;
  a.parts = parts < 1 ? 1 : static_cast<int32_t>(parts);
  if (units * a.parts > INT32_MAX) return cudaErrorInvalidValue;
  return launch_pdl(kern, dim3(static_cast<unsigned>(units * a.parts)), dim3(kCW * 32),
                    static_cast<size_t>(smem), s, a);
}

template <int D>
cudaError_t launch_cols(const QuantChunkLaunch& a, cudaStream_t s) {
  const int64_t cols = static_cast<int64_t>(a.max_q) << a.group_log2;
  if (cols <= kCols) return launch_one<D, 4>(a, s);
  if (cols <= 2 * kCols) return launch_one<D, 2>(a, s);
  return launch_one<D, 1>(a, s);
}

}  // namespace

cudaError_t launch_quant_chunk(const QuantChunkLaunch& a, cudaStream_t s) {
  if (a.head_dim == 128 && quant_chunk_tc_fits(a)) return launch_quant_chunk_tc(a, s);
  if (quant_chunk_rows_fits(a)) return launch_quant_chunk_rows(a, s);
  return a.head_dim == 128 ? launch_cols<128>(a, s) : launch_cols<64>(a, s);
}

}  // namespace dsa
