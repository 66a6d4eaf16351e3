// quant_redo.cuh -- one query of a chunk over the 8-bit cache, row by row.
//
// The chunk kernels multiply a tile of rows with the weights of many queries at once; a
// row that a query does not keep has weight 0 there, which is right for every finite V
// and not for NaN (0 x NaN).  A tile whose output holds a NaN is done again by this
// function, which reads the rows the query keeps and no others.  It is never on the path
// of finite data, so it is written for its result alone: a warp per query and head, one
// row at a time, running maximum and sum in fp32.
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

// Query token at row i of request b, head row qh of q and out.
template <int D>
__device__ __noinline__ void quant_redo_query(const QuantChunkLaunch& a, int b, int hk, int i, int P,
                                              int W, size_t qh, int lane) {
  constexpr int E = D / 32;  // elements per lane
  const int32_t* pt = a.page_table + static_cast<size_t>(b) * a.max_pages;
  const uint32_t* mrow = a.keep_mask + (static_cast<size_t>(b) * a.hkv + hk) * a.mask_words;
  float q[E], acc[E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = bf16_lo(a.q[qh * D + lane * E + e]);
    acc[e] = 0.f;
  }
  auto codes = [&](const uint8_t* p, float (&x)[E]) {
#pragma unroll
    for (int e = 0; e < E; e += 2) {
      const float2 v = f16x2_f32x2(e4m3x2_f16x2(*reinterpret_cast<const uint16_t*>(p + lane * E + e)));
      x[e] = v.x;
      x[e + 1] = v.y;
    }
  };
  const int np = min(P, i + 1);
  const int first = i >= P ? max(np, i - W) : i + 1;  // first row of the window
  for (int x = 0; x < np + max(0, i - first + 1); ++x) {
    const int j = x < np ? x : first + (x - np), o = i - j;
    if (x >= np && o > 0 && !((__ldg(mrow + ((o - 1) >> 5)) >> ((o - 1) & 31)) & 1u)) continue;
    const int pg = __ldg(pt + (j >> 4));
    if (static_cast<unsigned>(pg) >= static_cast<unsigned>(a.num_pages)) continue;
    const size_t ph = static_cast<size_t>(pg) * a.hkv + hk, at = (ph * 16 + (j & 15)) * D;
    float k[E], v[E], dot = 0.f;
    codes(a.k + at, k);
    codes(a.v + at, v);
#pragma unroll
    for (int e = 0; e < E; ++e) dot = fmaf(q[e], k[e], dot);
    const float y = warp_sum(dot) * (a.scale_log2 * __ldg(a.k_scale + ph));
    const float to = fmaxf(m, y);  // a NaN score leaves m and makes its weight NaN
    const float down = to == m ? 1.f : exp2f(m - to), w = exp2f(y - to);
    const float wv = w * __ldg(a.v_scale + ph);
    m = to;
    l = l * down + w;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = acc[e] * down + wv * v[e];
  }
#pragma unroll
  for (int e = 0; e < E; ++e) a.out[qh * D + lane * E + e] = f32_to_bf16_rn(acc[e] / l);
  if (a.lse != nullptr && lane == 0) a.lse[qh] = (m + log2f(l)) * kLn2;
}

}  // namespace dsa
