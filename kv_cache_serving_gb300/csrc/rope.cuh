// rope.cuh -- what the kernels that turn heads to their positions share (rope.cu,
// qk_norm.cu): the table of cosines and sines of a token, and the turning of 8 pairs held in
// registers.
#pragma once

#include "common.cuh"
#include "internal.h"
#include "mma.cuh"

namespace dsa {

// Cosine of a pair that does not turn at any position: its elements stay what they are, where
// x 1 - y 0 would carry an infinity or a NaN from one to the other.
constexpr float kStill = 2.f;

template <bool BF16>
__device__ __forceinline__ void load8(const void* p, size_t at, float (&x)[8]) {
  if constexpr (BF16) {
    const uint4 v = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p) + at);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = bf16_lo(w[i]);
      x[2 * i + 1] = bf16_hi(w[i]);
    }
  } else {
    const float4* f = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p) + at);
    const float4 u = f[0], v = f[1];
    x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w;
    x[4] = v.x, x[5] = v.y, x[6] = v.z, x[7] = v.w;
  }
}
template <bool BF16>
__device__ __forceinline__ void store8(void* p, size_t at, const float (&x)[8]) {
  if constexpr (BF16) {
    *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p) + at) =
        make_uint4(bf16x2_rn(x[0], x[1]), bf16x2_rn(x[2], x[3]), bf16x2_rn(x[4], x[5]),
                   bf16x2_rn(x[6], x[7]));
  } else {
    float4* f = reinterpret_cast<float4*>(reinterpret_cast<float*>(p) + at);
    f[0] = make_float4(x[0], x[1], x[2], x[3]);
    f[1] = make_float4(x[4], x[5], x[6], x[7]);
  }
}

// Place of 16-byte unit u (the cosines and sines of two pairs) in a token's table: 8 lanes
// that read units 4 l + j, or 2 l + j, then find 8 different banks.
__device__ __forceinline__ int table_unit(int u) { return u ^ ((u >> 3) & 3); }

// Cosine and sine of pair i of token t: its angle as a fixed-point fraction of a turn.
__device__ __forceinline__ float2 rope_turn(const RopeLaunch& a, int t, int i) {
  const int64_t pos = a.positions[static_cast<size_t>(t) * a.axes + a.pair_axis[i]];
  const uint64_t turn = static_cast<uint64_t>(pos) * a.turn[i];
  const uint32_t quarter = static_cast<uint32_t>((turn + (1ull << 61)) >> 62);  // the nearest, 0 .. 3
  const int64_t rest = static_cast<int64_t>(turn - (static_cast<uint64_t>(quarter) << 62));
  float s, c;  // of half turns in [-1/4, 1/4)
  sincospif(static_cast<float>(static_cast<int32_t>(rest >> 30)) * 0x1p-33f, &s, &c);
  const float cq = quarter & 1 ? s : c, sq = quarter & 1 ? c : s;
  const float co = a.turn[i] == 0 ? kStill : quarter == 1 || quarter == 2 ? -cq : cq;
  return make_float2(co, quarter >= 2 ? -sq : sq);
}

// Turns the l-th 8 pairs of a head, held as elements 8 l .. (u) and 8 l + D / 2 .. (v): pairs
// 8 l .., or (NEAR) 4 l .. and D / 4 + 4 l ..; cs is the token's table.
template <int D, bool NEAR>
__device__ __forceinline__ void turn8(float (&u)[8], float (&v)[8], int l, const float4* cs) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // pairs 2 i and 2 i + 1 of the eight
    const float4 t = cs[table_unit(!NEAR ? 4 * l + i : i < 2 ? 2 * l + i : D / 8 + 2 * l + i - 2)];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float c = k ? t.z : t.x, n = k ? t.w : t.y;
      float& x = !NEAR ? u[2 * i + k] : i < 2 ? u[4 * i + 2 * k] : v[4 * i - 8 + 2 * k];
      float& y = !NEAR ? v[2 * i + k] : i < 2 ? u[4 * i + 2 * k + 1] : v[4 * i - 7 + 2 * k];
      const float rx = x * c - y * n, ry = y * c + x * n;
      x = c == kStill ? x : rx;
      y = c == kStill ? y : ry;
    }
  }
}

}  // namespace dsa
