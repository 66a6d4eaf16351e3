// qk_norm.cu -- query and key heads normed, each head for itself, and turned to their
// positions in the same pass, q and k in one launch.
//
//   y = (x - mu) / sqrt(mean((x - mu)^2) + eps) * w + b,   mu = mean(x) or 0,
// then the rotation of rope.cu on y: statistics, norm and rotation in fp32, one rounding at
// the end.
//
// A head lies in the registers of 8 lanes (4 with head_dim 64), 16 elements each, so the
// statistics are shuffles among them and nothing is read twice; mean and squares one after the
// other, which a single pass over sum and sum of squares would lose to cancellation where the
// mean is large.  A head whose squares leave fp32 (elements past 2^61, or a sum so small that
// squares are subnormal) is scaled by a power of two first.
//
// Bound by HBM: each element is read and written once, as without the norm (rope.cu).
#include <math.h>

#include "common.cuh"
#include "internal.h"
#include "rope.cuh"

namespace dsa {
namespace {

constexpr int kNormThreads = 256;

// Sum over the kGroups lanes of a head (the whole warp takes part).
template <int kGroups>
__device__ __forceinline__ float head_sum(float x) {
#pragma unroll
  for (int o = kGroups / 2; o >= 1; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
template <int kGroups>
__device__ __forceinline__ float head_max(float x) {
#pragma unroll
  for (int o = kGroups / 2; o >= 1; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}

// Centres u, v (LAYER) and returns the mean of the squares of what is left.
template <int kGroups>
__device__ __forceinline__ float centre(float (&u)[8], float (&v)[8], bool layer) {
  constexpr float kInv = 1.f / (16 * kGroups);
  if (layer) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += u[i] + v[i];
    const float mu = head_sum<kGroups>(s) * kInv;
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] -= mu, v[i] -= mu;
  }
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) s = fmaf(u[i], u[i], fmaf(v[i], v[i], s));
  return head_sum<kGroups>(s) * kInv;
}

__device__ __forceinline__ void load8_as(const void* p, bool bf16, size_t at, float (&x)[8]) {
  if (bf16) load8<true>(p, at, x);
  else load8<false>(p, at, x);
}

// Head h of kind K (0: q, 1: k) of token tok, its l-th 8 pairs; `live` lanes load and store,
// all lanes of the warp take part in the sums.
template <int D, bool BF16, bool NEAR, int K>
__device__ __forceinline__ void norm8(const NormLaunch& a, bool live, size_t tok, int h, int l,
                                      const float4* cs) {
  constexpr int kGroups = D / 16;
  const void* in = K == 0 ? a.rope.q : a.rope.k;
  void* out = K == 0 ? a.rope.q_out : a.rope.k_out;
  const size_t at = tok * (K == 0 ? a.rope.q_stride : a.rope.k_stride) + static_cast<size_t>(h) * D;
  const int lo = 8 * l, hi = 8 * l + D / 2;
  float u[8], v[8];
  if (live) {
    load8<BF16>(in, at + lo, u);
    load8<BF16>(in, at + hi, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = v[i] = 0.f;
  }
  const size_t wat = a.per_head != 0 ? static_cast<size_t>(h) * D : 0;
  float wu[8], wv[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) wu[i] = wv[i] = 1.f;
  if (a.weight[K] != nullptr && live) {
    load8_as(a.weight[K], a.weight_bf16 != 0, wat + lo, wu);
    load8_as(a.weight[K], a.weight_bf16 != 0, wat + hi, wv);
  }
  const bool layer = a.layer != 0;
  float xu[8], xv[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) xu[i] = u[i], xv[i] = v[i];
  float ms = centre<kGroups>(xu, xv, layer), eps = a.eps;
  // squares that overflow, or are too small to be exact: once more, scaled by a power of two
  const bool odd = !(ms < 1e36f) || ms < 1e-30f;
  if (__any_sync(0xffffffffu, odd)) {
    float top = sqrtf(eps);
#pragma unroll
    for (int i = 0; i < 8; ++i) top = fmaxf(top, fmaxf(fabsf(u[i]), fabsf(v[i])));
    top = head_max<kGroups>(top);
    float f = 1.f;  // 2^-e of the larger of the largest element's binade and of sqrt(eps)'s
    if (odd && top < INFINITY) {
      const int e = static_cast<int>(__float_as_uint(top) >> 23) - 127;
      f = __uint_as_float(static_cast<uint32_t>(127 - min(max(e, -126), 126)) << 23);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) xu[i] = u[i] * f, xv[i] = v[i] * f;
    eps = (eps * f) * f;
    ms = centre<kGroups>(xu, xv, layer);
  }
  const float r = rsqrtf(ms + eps);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    xu[i] = xu[i] * r * wu[i];
    xv[i] = xv[i] * r * wv[i];
  }
  if (a.bias[K] != nullptr && live) {
    load8_as(a.bias[K], a.weight_bf16 != 0, wat + lo, wu);
    load8_as(a.bias[K], a.weight_bf16 != 0, wat + hi, wv);
#pragma unroll
    for (int i = 0; i < 8; ++i) xu[i] += wu[i], xv[i] += wv[i];
  }
  if (live) {
    turn8<D, NEAR>(xu, xv, l, cs);
    const size_t to =
        tok * (K == 0 ? a.rope.q_out_stride : a.rope.k_out_stride) + static_cast<size_t>(h) * D;
    store8<BF16>(out, to + lo, xu);
    store8<BF16>(out, to + hi, xv);
  }
}

template <int D, bool QBF, bool KBF, bool NEAR, int TT>
__global__ void __launch_bounds__(kNormThreads) qk_norm_kernel(const __grid_constant__ NormLaunch a) {
  constexpr int kPairs = D / 2, kGroups = kPairs / 8;
  __shared__ float4 cs[TT][kPairs / 2];
  griddep_wait();
  griddep_launch_dependents();
  const int t0 = blockIdx.x * TT, nt = min(TT, a.rope.tokens - t0);
  for (int x = threadIdx.x; x < nt * kPairs; x += kNormThreads) {
    const int t = x / kPairs, i = x % kPairs;
    reinterpret_cast<float2*>(&cs[t][table_unit(i >> 1)])[i & 1] = rope_turn(a.rope, t0 + t, i);
  }
  __syncthreads();
  const int l = threadIdx.x % kGroups;
  if (a.rope.q != nullptr) {
    const int n = nt * a.rope.hq;
    for (int x = threadIdx.x / kGroups; x - (threadIdx.x & 31) / kGroups < n; x += kNormThreads / kGroups) {
      const bool live = x < n;
      const int t = live ? x / a.rope.hq : 0, h = live ? x % a.rope.hq : 0;
      norm8<D, QBF, NEAR, 0>(a, live, static_cast<size_t>(t0 + t), h, l, cs[t]);
    }
  }
  if (a.rope.k != nullptr) {
    const int n = nt * a.rope.hkv;
    for (int x = threadIdx.x / kGroups; x - (threadIdx.x & 31) / kGroups < n; x += kNormThreads / kGroups) {
      const bool live = x < n;
      const int t = live ? x / a.rope.hkv : 0, h = live ? x % a.rope.hkv : 0;
      norm8<D, KBF, NEAR, 1>(a, live, static_cast<size_t>(t0 + t), h, l, cs[t]);
    }
  }
}

template <int D, bool QBF, bool KBF, bool NEAR>
cudaError_t launch_tokens(const NormLaunch& a, int sms, cudaStream_t s) {
  // as in rope.cu: four tokens per CTA once that still fills the GPU
  const int n = a.rope.tokens;
  if (n >= 16 * sms)
    return launch_pdl(qk_norm_kernel<D, QBF, KBF, NEAR, 4>, dim3((n + 3) / 4), dim3(kNormThreads), 0, s, a);
  return launch_pdl(qk_norm_kernel<D, QBF, KBF, NEAR, 1>, dim3(n), dim3(kNormThreads), 0, s, a);
}
template <int D, bool QBF, bool KBF>
cudaError_t launch_pairing(const NormLaunch& a, int sms, cudaStream_t s) {
  return a.rope.neighbours ? launch_tokens<D, QBF, KBF, true>(a, sms, s)
                           : launch_tokens<D, QBF, KBF, false>(a, sms, s);
}
template <int D>
cudaError_t launch_types(const NormLaunch& a, int sms, cudaStream_t s) {
  if (a.rope.q_bf16)
    return a.rope.k_bf16 ? launch_pairing<D, true, true>(a, sms, s)
                         : launch_pairing<D, true, false>(a, sms, s);
  return a.rope.k_bf16 ? launch_pairing<D, false, true>(a, sms, s)
                       : launch_pairing<D, false, false>(a, sms, s);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const NormLaunch& a, int sms, cudaStream_t s) {
  return a.rope.head_dim == 128 ? launch_types<128>(a, sms, s) : launch_types<64>(a, sms, s);
}

}  // namespace dsa
