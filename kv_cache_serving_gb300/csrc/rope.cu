// rope.cu -- rotary positions with several axes on the query and key heads of a batch
// of tokens, q and k in one launch.
//
// Pair i of every head of a token turns by positions[axis(i)] * inv_freq[i].  The angle
// is a fixed-point fraction of a turn: the host gives pair i's turns per position as a
// 64-bit fraction (2^-65), the kernel multiplies by the position modulo 2^64 -- which is the
// reduction to one turn, good to 2^-34 turns at the farthest position -- and takes the rest to
// the nearest quarter turn as an fp32, at most an eighth of a turn and so good to 2^-28, for
// sincospi; the quarters swap and negate the two.
//
// Bound by HBM: each element is read and written once.  A CTA computes the table of
// its tokens' cosines and sines in shared memory once for all heads, then streams the
// heads; a thread handles 8 pairs (two 16-byte loads and stores with bf16, each in a line
// of its lanes' own; the table is swizzled against bank conflicts).  Measured: q and k of
// 65 K tokens, 32/8 heads of 128, two axes: 195 us, the copy rate (223 with 8 pairs
// side by side and a plain table, whose conflicts kept the L1 pipe 91% busy).
#include <math.h>

#include "common.cuh"
#include "internal.h"
#include "mma.cuh"

namespace dsa {
namespace {

constexpr int kRopeThreads = 256;
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

// The l-th 8 pairs of the head at element `at`: pairs 8 l .., or (NEAR) 4 l .. and
// D / 4 + 4 l .., so that either way 8 lanes read and write whole lines.
template <int D, bool BF16, bool NEAR>
__device__ __forceinline__ void rotate8(const void* in, size_t at_in, void* out, size_t at_out,
                                        int l, const float4* cs) {
  const int lo = 8 * l, hi = 8 * l + D / 2;
  float u[8], v[8];
  load8<BF16>(in, at_in + lo, u);
  load8<BF16>(in, at_in + hi, v);
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
  store8<BF16>(out, at_out + lo, u);
  store8<BF16>(out, at_out + hi, v);
}

template <int D, bool QBF, bool KBF, bool NEAR, int TT>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeLaunch a) {
  constexpr int kPairs = D / 2, kGroups = kPairs / 8;
  __shared__ float4 cs[TT][kPairs / 2];
  griddep_wait();
  griddep_launch_dependents();
  const int t0 = blockIdx.x * TT, nt = min(TT, a.tokens - t0);
  for (int x = threadIdx.x; x < nt * kPairs; x += kRopeThreads) {
    const int t = x / kPairs, i = x % kPairs;
    const int64_t pos = a.positions[static_cast<size_t>(t0 + t) * a.axes + a.pair_axis[i]];
    const uint64_t turn = static_cast<uint64_t>(pos) * a.turn[i];
    const uint32_t quarter = static_cast<uint32_t>((turn + (1ull << 61)) >> 62);  // the nearest, 0 .. 3
    const int64_t rest = static_cast<int64_t>(turn - (static_cast<uint64_t>(quarter) << 62));
    float s, c;  // of half turns in [-1/4, 1/4)
    sincospif(static_cast<float>(static_cast<int32_t>(rest >> 30)) * 0x1p-33f, &s, &c);
    const float cq = quarter & 1 ? s : c, sq = quarter & 1 ? c : s;
    const float co = a.turn[i] == 0 ? kStill : quarter == 1 || quarter == 2 ? -cq : cq;
    reinterpret_cast<float2*>(&cs[t][table_unit(i >> 1)])[i & 1] =
        make_float2(co, quarter >= 2 ? -sq : sq);
  }
  __syncthreads();
  const int nq = a.q != nullptr ? a.hq : 0, nk = a.k != nullptr ? a.hkv : 0;
  const int per = (nq + nk) * kGroups;
  for (int x = threadIdx.x; x < nt * per; x += kRopeThreads) {
    const int t = x / per, y = x % per;
    const int h = y / kGroups, l = y % kGroups;
    const size_t tok = static_cast<size_t>(t0 + t);
    if (h < nq)
      rotate8<D, QBF, NEAR>(a.q, tok * a.q_stride + static_cast<size_t>(h) * D, a.q_out,
                            tok * a.q_out_stride + static_cast<size_t>(h) * D, l, cs[t]);
    else
      rotate8<D, KBF, NEAR>(a.k, tok * a.k_stride + static_cast<size_t>(h - nq) * D, a.k_out,
                            tok * a.k_out_stride + static_cast<size_t>(h - nq) * D, l, cs[t]);
  }
}

template <int D, bool QBF, bool KBF, bool NEAR>
cudaError_t launch_tokens(const RopeLaunch& a, int sms, cudaStream_t s) {
  // four tokens per CTA once that still fills the GPU (the table then costs each
  // thread one sine), else one
  if (a.tokens >= 16 * sms)
    return launch_pdl(rope_kernel<D, QBF, KBF, NEAR, 4>, dim3((a.tokens + 3) / 4),
                      dim3(kRopeThreads), 0, s, a);
  return launch_pdl(rope_kernel<D, QBF, KBF, NEAR, 1>, dim3(a.tokens), dim3(kRopeThreads), 0, s, a);
}
template <int D, bool QBF, bool KBF>
cudaError_t launch_pairing(const RopeLaunch& a, int sms, cudaStream_t s) {
  return a.neighbours ? launch_tokens<D, QBF, KBF, true>(a, sms, s)
                      : launch_tokens<D, QBF, KBF, false>(a, sms, s);
}
template <int D>
cudaError_t launch_types(const RopeLaunch& a, int sms, cudaStream_t s) {
  if (a.q_bf16)
    return a.k_bf16 ? launch_pairing<D, true, true>(a, sms, s)
                    : launch_pairing<D, true, false>(a, sms, s);
  return a.k_bf16 ? launch_pairing<D, false, true>(a, sms, s)
                  : launch_pairing<D, false, false>(a, sms, s);
}

}  // namespace

cudaError_t launch_rope(const RopeLaunch& a, int sms, cudaStream_t s) {
  return a.head_dim == 128 ? launch_types<128>(a, sms, s) : launch_types<64>(a, sms, s);
}

}  // namespace dsa
