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
// mean is large.  A head whose squares leave fp32 (elements past 2^60, or a sum so small that
// squares are subnormal) is scaled by a power of two first.
//
// Bound by HBM: each element is read and written once, as without the norm (rope.cu).  What
// stands in the way is issue and the latency of loads with few warps (96 registers): a thread
// keeps its place in a head, and with it weight and bias in registers, over the tokens of its
// CTA, computes on two fp32 at once, has the next two tokens' elements on their way and asks
// the L2 for those of the fourth.  Measured: q and k of 65 K tokens, 32/8 heads of 128, bf16,
// mean, weight and bias of every head's own, 225 us (0.87 of the copy rate): 370 us with a
// thread's place changing from head to head, 252 without the L2's part; 8 elements per thread
// instead of 16 took 298 us, 80 registers (more warps, spills) 293.
#include <math.h>

#include "common.cuh"
#include "f32x2.cuh"
#include "host.h"
#include "internal.h"
#include "rope.cuh"

namespace dsa {
namespace {

constexpr int kNormThreads = 512;  // at most
constexpr int kNormTurns = 16;     // tokens of a thread at most
constexpr int kNormPrefetch = 4;   // tokens ahead that the L2 is asked for

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
__device__ __forceinline__ float both(f32x2 a) {
  float lo, hi;
  unpack2(a, lo, hi);
  return lo + hi;
}

// Centres x (layer) and returns the mean of the squares of what is left.
template <int kGroups>
__device__ __forceinline__ float centre(f32x2 (&x)[8], bool layer) {
  constexpr float kInv = 1.f / (16 * kGroups);
  if (layer) {
    f32x2 s = add2(x[0], x[1]), t = add2(x[2], x[3]);
    s = add2(s, add2(x[4], x[5]));
    t = add2(t, add2(x[6], x[7]));
    const float mu = head_sum<kGroups>(both(add2(s, t))) * kInv;
    const f32x2 minus = pack2(-mu, -mu);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = add2(x[i], minus);
  }
  f32x2 s = mul2(x[0], x[0]), t = mul2(x[1], x[1]);
#pragma unroll
  for (int i = 2; i < 8; i += 2) {
    s = fma2(x[i], x[i], s);
    t = fma2(x[i + 1], x[i + 1], t);
  }
  return head_sum<kGroups>(both(add2(s, t))) * kInv;
}

// 16 elements of a head as they are in memory: 8 l .. and D / 2 + 8 l ...
template <bool BF16>
struct Raw {
  uint4 v[BF16 ? 2 : 4];
  __device__ __forceinline__ void load(const unsigned char* p, int apart) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < (BF16 ? 1 : 2); ++i)
        v[(BF16 ? 1 : 2) * h + i] = *reinterpret_cast<const uint4*>(p + h * apart + 16 * i);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < (BF16 ? 2 : 4); ++i) v[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  // As 8 pairs of neighbours: 0 .. 3 the first eight elements, 4 .. 7 the others.
  __device__ __forceinline__ void pairs(f32x2 (&x)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (BF16) {
        const uint32_t w = i % 4 == 0   ? v[i / 4].x
                           : i % 4 == 1 ? v[i / 4].y
                           : i % 4 == 2 ? v[i / 4].z
                                        : v[i / 4].w;
        x[i] = pack2(bf16_lo(w), bf16_hi(w));
      } else {
        const uint4 q = v[i / 2];
        x[i] = i % 2 == 0 ? pack2(__uint_as_float(q.x), __uint_as_float(q.y))
                          : pack2(__uint_as_float(q.z), __uint_as_float(q.w));
      }
    }
  }
};

// Weight or bias of this thread's 16 elements.
template <int D>
__device__ __forceinline__ void load_vector(const void* p, bool bf16, size_t at, float none,
                                            f32x2 (&w)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = pack2(none, none);
  if (p == nullptr) return;
  if (bf16) {
    Raw<true> r;
    r.load(static_cast<const unsigned char*>(p) + 2 * at, D);
    r.pairs(w);
  } else {
    Raw<false> r;
    r.load(static_cast<const unsigned char*>(p) + 4 * at, 2 * D);
    r.pairs(w);
  }
}

// Turns the pairs of this thread's 16 elements; STILL: pairs that do not turn stay what they are.
template <int D, bool NEAR, bool STILL>
__device__ __forceinline__ void turn(f32x2 (&x)[8], int l, const float4* cs) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (!NEAR) {  // pairs 8 l ..: x[i] with x[i + 4]
      const float4 q = cs[table_unit(4 * l + i)];
      const f32x2 c = pack2(q.x, q.y), s = pack2(q.z, q.w), ns = pack2(-q.z, -q.w);
      f32x2 rx = fma2(x[i + 4], ns, mul2(x[i], c)), ry = fma2(x[i], s, mul2(x[i + 4], c));
      if constexpr (STILL) {
        float x0, x1, y0, y1, u0, u1, v0, v1;
        unpack2(x[i], x0, x1);
        unpack2(x[i + 4], y0, y1);
        unpack2(rx, u0, u1);
        unpack2(ry, v0, v1);
        rx = pack2(q.x == kStill ? x0 : u0, q.y == kStill ? x1 : u1);
        ry = pack2(q.x == kStill ? y0 : v0, q.y == kStill ? y1 : v1);
      }
      x[i] = rx;
      x[i + 4] = ry;
    } else {  // pairs 4 l .. and D / 4 + 4 l ..: the two elements of x[2 i] and x[2 i + 1]
      const float4 q = cs[table_unit(i < 2 ? 2 * l + i : D / 8 + 2 * l + i - 2)];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float c = k ? q.y : q.x, s = k ? q.w : q.z;
        float u, v;
        unpack2(x[2 * i + k], u, v);
        const float ru = fmaf(-v, s, u * c), rv = fmaf(u, s, v * c);
        x[2 * i + k] = STILL && c == kStill ? x[2 * i + k] : pack2(ru, rv);
      }
    }
  }
}

// The tokens' table: unit u of a token (table_unit) holds the cosines of pairs 2 u and 2 u + 1,
// then their sines.
template <int D, bool BF16, bool NEAR>
__global__ void __maxnreg__(96) qk_norm_kernel(const __grid_constant__ NormLaunch a) {
  constexpr int kPairs = D / 2, kGroups = kPairs / 8, kElt = BF16 ? 2 : 4;
  extern __shared__ float4 table[];  // [a.tile][kPairs / 2]
  griddep_wait();
  griddep_launch_dependents();
  // this thread's place: a head's eighth (or fourth), the same for every token it takes
  const int t0 = blockIdx.x * a.tile, nt = min(a.tile, a.rope.tokens - t0);
  const int sub = threadIdx.x / a.lanes;  // of the tokens side by side
  const int place = threadIdx.x % a.lanes + blockIdx.y * a.lanes;
  const int head = place / kGroups, l = place % kGroups;
  const bool is_q = head < a.q_heads;
  const int h = is_q ? head : head - a.q_heads;
  const bool live = sub < a.subs && head < a.q_heads + a.k_heads;
  int64_t in_step = (is_q ? a.rope.q_stride : a.rope.k_stride) * kElt;
  int64_t out_step = (is_q ? a.rope.q_out_stride : a.rope.k_out_stride) * kElt;
  const int64_t off = (static_cast<int64_t>(h) * D + 8 * l) * kElt;
  const unsigned char* in =
      static_cast<const unsigned char*>(is_q ? a.rope.q : a.rope.k) + off + (t0 + sub) * in_step;
  unsigned char* out =
      static_cast<unsigned char*>(is_q ? a.rope.q_out : a.rope.k_out) + off + (t0 + sub) * out_step;
  in_step *= a.subs;  // from one of this thread's tokens to the next
  out_step *= a.subs;
  // the next tokens' elements, 64 bytes of a thread on their way
  constexpr int kAhead = BF16 ? 2 : 1;
  Raw<BF16> next[kAhead];
#pragma unroll
  for (int y = 0; y < kAhead; ++y) {
    next[y].zero();
    if (live && sub + y * a.subs < nt) next[y].load(in + y * in_step, D / 2 * kElt);
  }
  f32x2 w[8], bias[8];
  {
    const size_t at = (a.per_head != 0 ? static_cast<size_t>(h) * D : 0) + 8 * l;
    const int k = is_q ? 0 : 1;
    load_vector<D>(live ? a.weight[k] : nullptr, a.weight_bf16 != 0, at, 1.f, w);
    load_vector<D>(live ? a.bias[k] : nullptr, a.weight_bf16 != 0, at, 0.f, bias);
  }
  for (int x = threadIdx.x; x < nt * kPairs; x += blockDim.x) {
    const int t = x / kPairs, i = x % kPairs;
    const float2 c = rope_turn(a.rope, t0 + t, i);
    float* unit = reinterpret_cast<float*>(table + t * (kPairs / 2) + table_unit(i >> 1));
    unit[i & 1] = c.x;
    unit[2 + (i & 1)] = c.y;
  }
  __syncthreads();
  const bool layer = a.layer != 0;
  const int ahead = a.rope.tokens - t0 - kNormPrefetch * a.subs;
  for (int t = sub; t - sub < nt; t += a.subs, in += in_step, out += out_step) {
    const bool now = live && t < nt;
    f32x2 x[8];
    next[0].pairs(x);
#pragma unroll
    for (int y = 1; y < kAhead; ++y) next[y - 1] = next[y];
    if (live && t + kAhead * a.subs < nt)
      next[kAhead - 1].load(in + kAhead * in_step, D / 2 * kElt);
    // the lines of the head a few tokens on into the L2
    if (l == 0 && live && t < ahead) {
#pragma unroll
      for (int y = 0; y < D * kElt; y += 128)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(in + kNormPrefetch * in_step + y));
    }
    float eps = a.eps;
    float ms = centre<kGroups>(x, layer);
    // squares that overflow, or are too small to be exact: once more, scaled by a power of two
    const bool odd = !(ms < 1e36f) || ms < 1e-30f;
    if (__any_sync(0xffffffffu, odd)) {
      Raw<BF16> raw;
      raw.zero();
      if (now) raw.load(in, D / 2 * kElt);
      raw.pairs(x);
      float top = sqrtf(eps);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float u, v;
        unpack2(x[i], u, v);
        top = fmaxf(top, fmaxf(fabsf(u), fabsf(v)));
      }
      top = head_max<kGroups>(top);
      float f = 1.f;  // 2^-e of the larger of the largest element's binade and of sqrt(eps)'s
      if (odd && top < INFINITY) {
        const int e = static_cast<int>(__float_as_uint(top) >> 23) - 127;
        f = __uint_as_float(static_cast<uint32_t>(127 - min(max(e, -126), 126)) << 23);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = mul2(x[i], pack2(f, f));
      eps = (eps * f) * f;
      ms = centre<kGroups>(x, layer);
    }
    const float r = rsqrtf(ms + eps);
    const f32x2 r2 = pack2(r, r);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = fma2(mul2(x[i], r2), w[i], bias[i]);
    // the rotation
    const float4* cs = table + (now ? t : 0) * (kPairs / 2);
    if (a.still == 0) turn<D, NEAR, false>(x, l, cs);
    else turn<D, NEAR, true>(x, l, cs);
    if (now) {
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        float e[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) unpack2(x[4 * g + i], e[2 * i], e[2 * i + 1]);
        store8<BF16>(out + g * (D / 2) * kElt, 0, e);
      }
    }
  }
}

template <int D, bool BF16, bool NEAR>
cudaError_t launch_one(NormLaunch a, int sms, cudaStream_t s) {
  constexpr int kGroups = D / 16;
  // All heads of a token side by side in a CTA, or an even share of them where they are too
  // many; several tokens side by side where they are few.
  const int64_t places = static_cast<int64_t>(a.q_heads + a.k_heads) * kGroups;
  const int64_t parts = ceil_div(places, kNormThreads);
  a.lanes = static_cast<int32_t>(ceil_div(ceil_div(places, parts), kGroups) * kGroups);
  const int tokens = a.rope.tokens;
  a.subs = 256 / a.lanes > 1 ? 256 / a.lanes : 1;
  // Tokens of a CTA: weights are loaded and the table's latency is waited for once, so as many as
  // leave some CTAs for every SM, at most 16 in turn.
  int turns = static_cast<int>(tokens / (static_cast<int64_t>(a.subs) * sms * 8));
  turns = turns < 1 ? 1 : turns > kNormTurns ? kNormTurns : turns;
  a.tile = a.subs * turns;
  while (a.tile * (D / 4) * 16 > 32768) a.tile -= a.subs;  // the table in the default shared memory
  const int threads = static_cast<int>(ceil_div(static_cast<int64_t>(a.lanes) * a.subs, 32) * 32);
  if (parts > 65535) return cudaErrorInvalidValue;
  return launch_pdl(qk_norm_kernel<D, BF16, NEAR>,
                    dim3(static_cast<unsigned>(ceil_div(tokens, a.tile)), static_cast<unsigned>(parts)),
                    dim3(threads), static_cast<size_t>(a.tile) * (D / 4) * 16, s, a);
}

template <int D>
cudaError_t launch_type(const NormLaunch& a, bool bf16, int sms, cudaStream_t s) {
  if (bf16)
    return a.rope.neighbours ? launch_one<D, true, true>(a, sms, s) : launch_one<D, true, false>(a, sms, s);
  return a.rope.neighbours ? launch_one<D, false, true>(a, sms, s) : launch_one<D, false, false>(a, sms, s);
}

cudaError_t launch_heads(const NormLaunch& a, bool bf16, int sms, cudaStream_t s) {
  if (a.q_heads + a.k_heads == 0) return cudaSuccess;
  return a.rope.head_dim == 128 ? launch_type<128>(a, bf16, sms, s) : launch_type<64>(a, bf16, sms, s);
}

}  // namespace

cudaError_t launch_qk_norm_rope(NormLaunch a, int sms, cudaStream_t s) {
  const int nq = a.rope.q != nullptr ? a.rope.hq : 0, nk = a.rope.k != nullptr ? a.rope.hkv : 0;
  a.still = 0;
  for (int i = 0; i < a.rope.head_dim / 2; ++i) a.still |= a.rope.turn[i] == 0;
  if (a.rope.q_bf16 == a.rope.k_bf16 || nq == 0 || nk == 0) {
    a.q_heads = nq;
    a.k_heads = nk;
    return launch_heads(a, nq != 0 ? a.rope.q_bf16 != 0 : a.rope.k_bf16 != 0, sms, s);
  }
  // q and k of different types: one launch each
  a.q_heads = nq;
  a.k_heads = 0;
  const cudaError_t e = launch_heads(a, a.rope.q_bf16 != 0, sms, s);
  if (e != cudaSuccess) return e;
  a.q_heads = 0;
  a.k_heads = nk;
  return launch_heads(a, a.rope.k_bf16 != 0, sms, s);
}

}  // namespace dsa
