// quant_redo.cuh -- queries of a chunk over the 8-bit cache done again, eight at a time.
//
// The chunk kernels multiply a tile of rows with the weights of many queries at once; a
// row that a query does not keep has weight 0 there, which is right for every finite V
// and not for NaN (0 x NaN).  A tile whose output holds NaN therefore looks through V's codes
// of its pages, by all its warps.  Where a query itself keeps the rows that hold NaN, its
// elements are NaN rightly and the others are right; a query with a NaN from a row that it
// does not keep is done again, with zeros in the place of V's NaN codes and NaN in the
// elements that keep them: a warp per eight columns (query token, head), the products of
// quant_decode.cu with fragments read straight from the pages.  Finite data with scores below
// 2^20 never come here, so it is a call, and what it needs is found again, not held by the
// kernels.
//
// Measured with one NaN element in a row that every query keeps (us, without / with it, in
// brackets a warp per query that takes a row at a time): all of 2048 rows of 8 requests, 32/8
// heads of 128, 387 / 495 (218 000); 32 tokens of 64 requests of 320 .. 1280 rows, 32/32 heads,
// 123 / 176 (4 800).  Every query of the former done again: 5 100.
#pragma once

#include "common.cuh"
#include "internal.h"
#include "mma.cuh"
#include "quant.cuh"

namespace dsa {

// Whether a query whose output holds a NaN is to be done again, by its sum and reference.  Not
// one whose sum is NaN too: a score of its own is NaN (or infinite), so all of its output is
// -- unless its scores pass 2^20, where the rounding of the reference alone, up to half a
// unit of its last place, can carry a weight past fp16.
__device__ __forceinline__ bool quant_redo_needed(float l, float ref) {
  return l == l || (fabsf(ref) >= 0x1p20f && fabsf(ref) < 1e38f);
}

// Whether what a sum is made of may be wrong: weights past fp16, or all of them lost.
__device__ __forceinline__ bool quant_sum_unsure(float l, float ref) {
  return !(l > 0.f && l < INFINITY) || fabsf(ref) >= 0x1p20f;
}

// Four codes: 0x80 in the byte of each that is NaN; and from that a bit for each.
__device__ __forceinline__ uint32_t e4m3_nan(uint32_t w) {
  return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
}
__device__ __forceinline__ uint32_t e4m3_nan_bits(uint32_t is) { return (is >> 7) * 0x10204080u >> 28; }

// The columns of a CTA's tile that may have to be done again (`out`), and those whose sum may be
// wrong as well: a bit each, up to 128 columns; `hit`: some output holds a
// NaN or an infinity.  At an address that takes no register.
struct QuantRedo {
  uint32_t out[4], sum[4];
  int hit;
  int lo, hi;  // the tile's pages with NaN in V, first and last
};
__device__ __forceinline__ QuantRedo& quant_redo() {
  __shared__ QuantRedo set;
  return set;
}
__device__ __forceinline__ void quant_redo_clear() {
  quant_redo().out[threadIdx.x & 3] = 0u;
  quant_redo().sum[threadIdx.x & 3] = 0u;
  quant_redo().hit = 0;
}

// Columns col0 .. col0 + 7 of the tile of request b and kv head hk whose first query token is
// t0 (column c: token t0 + c / group, head c % group).  Bit c of `outs`: column col0 + c is
// written (out, and lse where its sum went wrong as well, bit c of `sums`).
template <int D>
__device__ __forceinline__ void quant_redo_columns(const QuantChunkLaunch& a, int b, int hk, int t0,
                                                   int col0, unsigned outs, unsigned sums) {
  using Tile = QuantTile<D>;
  constexpr int NK = D / 16;
  constexpr float kHead = 4.f, kSlack = 10.f;  // as in quant_decode.cu
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int lg = a.group_log2, P = a.prompt_len[b], W = a.window[b];
  const int i0 = a.seq_len[b] - a.q_len[b] + t0;  // row of column 0's query
  auto row_of = [&](int col) { return i0 + ((col0 + col) >> lg); };
  auto qh_of = [&](int col) {
    const int t = t0 + ((col0 + col) >> lg);
    return (static_cast<size_t>(b) * a.max_q + t) * a.hq + (hk << lg) + ((col0 + col) & ((1 << lg) - 1));
  };
  const int32_t* pt = a.page_table + static_cast<size_t>(b) * a.max_pages;
  const uint32_t* mrow = a.keep_mask + (static_cast<size_t>(b) * a.hkv + hk) * a.mask_words;

  uint32_t q[NK][2];
  float f[2];
  {
    const uint32_t* p = reinterpret_cast<const uint32_t*>(a.q + qh_of(g) * D + c * (D / 4));
    const bool on = (outs >> g) & 1u;
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
      q[i / 2][i % 2] = on ? __ldg(p + i) : 0u;
      amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(q[i / 2][i % 2])), fabsf(bf16_hi(q[i / 2][i % 2]))));
    }
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    const int e = q_exponent(amax);
    const float down = pow2i(-e), up = a.scale_log2 * pow2i(e);
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
      q[i / 2][i % 2] = f16x2_rn(bf16_lo(q[i / 2][i % 2]) * down, bf16_hi(q[i / 2][i % 2]) * down);
    f[0] = __shfl_sync(0xffffffffu, up, (2 * c) * 4);
    f[1] = __shfl_sync(0xffffffffu, up, (2 * c + 1) * 4);
  }
  float acc[NK][4], ref[2] = {-3e38f, -3e38f}, l[2] = {0.f, 0.f};
#pragma unroll
  for (int mt = 0; mt < NK; ++mt)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[mt][e] = 0.f;

  // Whether column `col` keeps row j.
  auto keeps = [&](int col, int j) -> bool {
    const int o = row_of(col) - j;
    if (!((outs >> col) & 1u) || o < 0) return false;
    if (o == 0 || j < P) return true;
    return o <= W && ((__ldg(mrow + ((o - 1) >> 5)) >> ((o - 1) & 31)) & 1u);
  };
  // pages scanned: those of the prompt rows [0, pa), then those from the window's start
  const int first = row_of(__ffs(outs) - 1), last = row_of(31 - __clz(outs));
  const int pa = (min(P, last + 1) + 15) >> 4;
  const int pb = max(pa, max(first - W, 0) >> 4), pages = pa + max(0, (last >> 4) - pb + 1);
  auto page_of = [&](int x) { return x < pa ? x : pb + (x - pa); };
  int pg_next = __ldg(pt + page_of(0));
#pragma unroll 1
  for (int x = 0; x < pages; ++x) {
    const int j0 = page_of(x) * 16, pg = pg_next;
    if (x + 1 < pages) pg_next = __ldg(pt + page_of(x + 1));
    if (static_cast<unsigned>(pg) >= static_cast<unsigned>(a.num_pages)) continue;
    const size_t ph = static_cast<size_t>(pg) * a.hkv + hk;
    const float ks = __ldg(a.k_scale + ph), vs = __ldg(a.v_scale + ph);
    uint32_t v[4][Tile::kVW];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const uint8_t* p = a.v + ph * (16 * D) + (2 * c + (r & 1) + 8 * (r >> 1)) * D + g * (D / 8);
#pragma unroll
      for (int k = 0; k < Tile::kVW; k += 2) {
        const uint2 u = __ldg(reinterpret_cast<const uint2*>(p + 4 * k));
        v[r][k] = u.x;
        v[r][k + 1] = u.y;
      }
    }
    uint32_t w[2][Tile::kKW];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const uint8_t* p = a.k + ph * (16 * D) + (g + 8 * r) * D + c * (D / 4);
#pragma unroll
      for (int k = 0; k < Tile::kKW / 4; ++k) {
        const uint4 u = __ldg(reinterpret_cast<const uint4*>(p) + k);
        w[r][4 * k] = u.x;
        w[r][4 * k + 1] = u.y;
        w[r][4 * k + 2] = u.z;
        w[r][4 * k + 3] = u.w;
      }
    }
    // (the page is on its way before it is known whether a query keeps any of it)
    unsigned keep = 15u;  // rows g (bits 0, 1) and g + 8 (2, 3), columns 2c and 2c + 1
    if (j0 + 15 >= P || j0 + 15 > first) {
      keep = 0u;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (keeps(2 * c + (e & 1), j0 + g + 8 * (e >> 1))) keep |= 1u << e;
      if (!__any_sync(0xffffffffu, keep != 0u)) continue;
    }
    float s[4] = {0.f, 0.f, 0.f, 0.f}, s2[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NK; ++i)
      mma_f16((i & 1) ? s2 : s, e4m3x2_f16x2(w[0][i]), e4m3x2_f16x2(w[1][i]), e4m3x2_f16x2_hi(w[0][i]),
              e4m3x2_f16x2_hi(w[1][i]), q[i][0], q[i][1]);
    const uint32_t vbits = __float_as_uint(vs);
    const float lv = static_cast<float>(scale_exp(vbits)), inv = __uint_as_float((254u << 23) - vbits);
    float y[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      y[e] = (keep >> e) & 1u ? fmaf(s[e] + s2[e], f[e & 1] * ks, lv) : -INFINITY;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float mx = fmaxf(y[j], y[2 + j]);
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
      // where an fp32 no longer holds a score to a part of one, the reference is the largest
      const bool coarse = fabsf(mx) >= 0x1p20f;
      if (mx - ref[j] > (coarse ? 0.f : kHead + kSlack)) {
        const float to = mx - (coarse ? 0.f : kHead), down = ex2_approx(ref[j] - to);
        ref[j] = to;
        l[j] *= down;
#pragma unroll
        for (int mt = 0; mt < NK; ++mt) {
          acc[mt][j] *= down;
          acc[mt][2 + j] *= down;
        }
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      y[e] = ex2_approx(y[e] - ref[e & 1]);
      l[e & 1] = fmaf(y[e], inv, l[e & 1]);
    }
    uint32_t any = 0u;
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int k = 0; k < Tile::kVW; ++k) any |= e4m3_nan(v[r][k]);
    any = __any_sync(0xffffffffu, any != 0u);
    // bit of each of this lane's D / 8 dims that is NaN, for rows 2c, 2c + 1, 2c + 8, 2c + 9
    uint32_t nan[4] = {0u, 0u, 0u, 0u};
    if (any != 0u) {
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int k = 0; k < Tile::kVW; ++k) {
          const uint32_t is = e4m3_nan(v[r][k]);
          nan[r] |= e4m3_nan_bits(is) << (4 * k);
          v[r][k] &= ~((is >> 7) * 0xffu);
        }
    }
    const uint32_t p0 = movmatrix_trans(f16x2_rn(y[0], y[1]));
    const uint32_t p1 = movmatrix_trans(f16x2_rn(y[2], y[3]));
#pragma unroll
    for (int mt = 0; mt < NK; ++mt) {
      uint32_t va[4];
      Tile::frag_v(v, mt, va);
      mma_f16(acc[mt], va[0], va[1], va[2], va[3], p0, p1);
    }
    if (any != 0u) {
#pragma unroll 1
      for (int r = 0; r < 16; ++r) {
        const int slot = (r & 1) + 2 * (r >> 3);
        const uint32_t mine = slot == 0 ? nan[0] : slot == 1 ? nan[1] : slot == 2 ? nan[2] : nan[3];
        const uint32_t bits = __shfl_sync(0xffffffffu, mine, (g << 2) | ((r & 7) >> 1));
        const bool k0 = keeps(2 * c, j0 + r), k1 = keeps(2 * c + 1, j0 + r);
#pragma unroll
        for (int mt = 0; mt < NK; ++mt)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (((bits >> (2 * mt + (e >> 1))) & 1u) && (e & 1 ? k1 : k0))
              acc[mt][e] = __int_as_float(0x7fc00000);
      }
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float sum = l[h];
    sum += __shfl_xor_sync(0xffffffffu, sum, 4);
    sum += __shfl_xor_sync(0xffffffffu, sum, 8);
    sum += __shfl_xor_sync(0xffffffffu, sum, 16);
    const int col = 2 * c + h;
    if (!((outs >> col) & 1u)) continue;
    uint32_t* to = reinterpret_cast<uint32_t*>(a.out + qh_of(col) * D + g * (D / 8));
#pragma unroll
    for (int mt = 0; mt < NK; ++mt) to[mt] = bf16x2_rn(acc[mt][h] / sum, acc[mt][2 + h] / sum);
    if (a.lse != nullptr && g == 0 && ((sums >> col) & 1u))
      a.lse[qh_of(col)] = (ref[h] + log2f(sum)) * kLn2;
  }
}

// The NaN codes of this lane's part of V of the page (pieces lane, lane + 32 ..): a bit each.
template <int D>
__device__ __forceinline__ void quant_nan_codes(const QuantChunkLaunch& a, const int32_t* pt, int hk,
                                                int page, int lane, uint32_t (&bits)[D / 32]) {
  const int pg = __ldg(pt + page);
  const bool in = static_cast<unsigned>(pg) < static_cast<unsigned>(a.num_pages);
  const uint4* src = reinterpret_cast<const uint4*>(
      a.v + (static_cast<size_t>(in ? pg : 0) * a.hkv + hk) * (16 * D)) + lane;
#pragma unroll
  for (int l = 0; l < D / 32; ++l) {
    const uint4 v = in ? __ldg(src + 32 * l) : make_uint4(0u, 0u, 0u, 0u);
    bits[l] = e4m3_nan_bits(e4m3_nan(v.x)) | e4m3_nan_bits(e4m3_nan(v.y)) << 4 |
              e4m3_nan_bits(e4m3_nan(v.z)) << 8 | e4m3_nan_bits(e4m3_nan(v.w)) << 12;
  }
}

// All of them, by every thread of the CTA after its first output.  It finds its tile from the
// block's index by itself (TILE::at): the kernels hold no register for it.
template <int D, class TILE>
__device__ __noinline__ void quant_redo_tile(const QuantChunkLaunch& a) {
  QuantRedo& set = quant_redo();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  int bpos, hk, t0;
  TILE::at(a, bpos, hk, t0);
  const int b = a.order != nullptr ? __ldg(a.order + bpos) : bpos;
  const int lg = a.group_log2, n = a.q_len[b], P = a.prompt_len[b], W = a.window[b];
  const int first = a.seq_len[b] - n + t0;
  const int last = min(first + ((TILE::kColumns - 1) >> lg), a.seq_len[b] - 1);
  const int pa = (min(P, last + 1) + 15) >> 4;
  const int pb = max(pa, max(first - W, 0) >> 4), pages = pa + max(0, (last >> 4) - pb + 1);
  auto page_of = [&](int x) { return x < pa ? x : pb + (x - pa); };
  const int32_t* pt = a.page_table + static_cast<size_t>(b) * a.max_pages;
  uint32_t bits[D / 32];
  if (threadIdx.x == 0) {
    set.lo = pages;
    set.hi = -1;
  }
  __syncthreads();
  for (int x = warp; x < pages; x += warps) {
    quant_nan_codes<D>(a, pt, hk, page_of(x), lane, bits);
    uint32_t any = 0u;
#pragma unroll
    for (int l = 0; l < D / 32; ++l) any |= bits[l];
    if (__any_sync(0xffffffffu, any != 0u) && lane == 0) {
      atomicMin(&set.lo, x);
      atomicMax(&set.hi, x);
    }
  }
  __syncthreads();
  // Of the columns (one to a lane), those that need it: some row that the query does not keep
  // holds a NaN where no row does that it keeps; or the sum went wrong.
  const unsigned outs = warp < 4 ? set.out[warp] : 0u;
  if (outs != 0u) {
    constexpr int kPieces = D / 16, kRows = 32 / kPieces;
    const int i = first + ((32 * warp + lane) >> lg);
    const uint32_t* mrow = a.keep_mask + (static_cast<size_t>(b) * a.hkv + hk) * a.mask_words;
    uint32_t kept[D / 32], other[D / 32];
#pragma unroll
    for (int k = 0; k < D / 32; ++k) kept[k] = other[k] = 0u;
    for (int x = set.lo; x <= set.hi; ++x) {
      quant_nan_codes<D>(a, pt, hk, page_of(x), lane, bits);
#pragma unroll
      for (int l = 0; l < D / 32; ++l) {
        unsigned left = __ballot_sync(0xffffffffu, bits[l] != 0u);
        while (left != 0u) {
          const int src = __ffs(left) - 1;
          left &= left - 1u;
          const uint32_t got = __shfl_sync(0xffffffffu, bits[l], src) << (16 * (src & 1));
          const int j = page_of(x) * 16 + l * kRows + src / kPieces, o = i - j;
          bool keeps = o >= 0;
          if (o > 0 && j >= P) keeps = o <= W && ((__ldg(mrow + ((o - 1) >> 5)) >> ((o - 1) & 31)) & 1u);
#pragma unroll
          for (int k = 0; k < D / 32; ++k)
            if (src % kPieces / 2 == k) (keeps ? kept[k] : other[k]) |= got;
        }
      }
    }
    bool need = (set.sum[warp] >> lane) & 1u;
#pragma unroll
    for (int k = 0; k < D / 32; ++k) need |= (other[k] & ~kept[k]) != 0u;
    const unsigned needs = __ballot_sync(0xffffffffu, need);
    if (lane == 0) set.out[warp] = outs & needs;
  }
  __syncthreads();
  for (int x = warp; x < 16; x += warps) {  // eight columns a warp
    const unsigned eight = (set.out[x >> 2] >> (8 * (x & 3))) & 0xffu;
    if (eight != 0u)
      quant_redo_columns<D>(a, b, hk, t0, 8 * x, eight, set.sum[x >> 2] >> (8 * (x & 3)));
  }
}

}  // namespace dsa
