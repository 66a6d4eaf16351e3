// quant_rows.cu -- rows into and out of the 8-bit paged K/V cache.
//
// Write: for the rows that one call brings to a (page, kv head),
//   e = the smallest exponent with max |x| <= 448 * 2^e (-40 <= e <= 40; at least the
//       page's present one if rows before them stay), code = e4m3(x * 2^-e)
// A power of two makes the division exact, so the code depends on x alone and the
// exponent is read off the largest magnitude's bits.  The rows the page already holds
// move to the new exponent only when it grows.
// Read: code * 2^e, exact in bf16.
//
// Both are bound by HBM (3 bytes per element with bf16 rows), so what counts is bytes in
// flight and whole sectors.  Write: one warp takes one page of one kv head, K and V (bf16
// rows: both in flight at once, 8 KB per warp at D = 128; the rows are asked for together
// with the page id, not after it); the maximum is a warp reduction; the codes of a row
// leave in 8-byte pieces, contiguous over the lanes.  Read: one warp takes one page of one
// kv head, K or V, and a lane as many codes as make 16 bytes of output, so that every store
// instruction covers 512 contiguous bytes of a row or two.  Measured, of the copy rate:
// prompts of 64 requests written in 48 us = 0.87, read back in 36 us = 0.91.
#include <math.h>

#include "common.cuh"
#include "internal.h"
#include "mma.cuh"
#include "quant.cuh"

namespace dsa {
namespace {

constexpr int kRowWarps = 4;

// 8 consecutive elements of a row: their largest magnitude (an infinity counts, a NaN does
// not), and their codes.  With bf16 both work on pairs: multiplying by a power of two is
// exact in bf16 too (what falls below its range is zero as a code anyway).
template <bool BF16>
struct Row8;
template <>
struct Row8<true> {
  uint32_t w[4];
  __device__ __forceinline__ void load(const void* base, size_t elem) {
    const uint4 v =
        __ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(base) + elem));
    w[0] = v.x;
    w[1] = v.y;
    w[2] = v.z;
    w[3] = v.w;
  }
  __device__ __forceinline__ void zero() { w[0] = w[1] = w[2] = w[3] = 0u; }
  using Max = uint32_t;
  __device__ __forceinline__ void max_into(uint32_t& m) const {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      asm("max.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(w[k] & 0x7fff7fffu));
  }
  __device__ __forceinline__ static float value(uint32_t m) { return fmaxf(bf16_lo(m), bf16_hi(m)); }
  __device__ __forceinline__ uint2 codes(float down) const {
    const uint32_t d = __float_as_uint(down), dd = (d >> 16) | (d & 0xffff0000u);
    uint32_t c[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint32_t p;
      asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(p) : "r"(w[k]), "r"(dd));
      c[k] = f32x2_e4m3x2(bf16_lo(p), bf16_hi(p));
    }
    return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
  }
  // NaN for every infinity; the largest finite magnitude joins m.
  __device__ __forceinline__ void drop_infinite(float& m) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if ((w[k] & 0x7f80u) == 0x7f80u) w[k] |= 0x7fffu;
      else m = fmaxf(m, fabsf(bf16_lo(w[k])));
      if ((w[k] & 0x7f800000u) == 0x7f800000u) w[k] |= 0x7fff0000u;
      else m = fmaxf(m, fabsf(bf16_hi(w[k])));
    }
  }
};
template <>
struct Row8<false> {
  float x[8];
  __device__ __forceinline__ void load(const void* base, size_t elem) {
    const float4* p = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(base) + elem);
    const float4 a = __ldg(p), b = __ldg(p + 1);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = 0.f;
  }
  using Max = float;
  __device__ __forceinline__ void max_into(float& m) const {
#pragma unroll
    for (int k = 0; k < 8; ++k) m = fmaxf(m, fabsf(x[k]));
  }
  __device__ __forceinline__ static float value(float m) { return m; }
  __device__ __forceinline__ uint2 codes(float down) const {
    uint32_t c[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) c[k] = f32x2_e4m3x2(x[2 * k] * down, x[2 * k + 1] * down);
    return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
  }
  __device__ __forceinline__ void drop_infinite(float& m) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (fabsf(x[k]) < INFINITY) m = fmaxf(m, fabsf(x[k]));
      else x[k] = __int_as_float(0x7fc00000);
    }
  }
};

// The smallest e in -40..40 with amax <= 448 * 2^e = 1.75 * 2^(e + 8).
__device__ __forceinline__ int exponent_for(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return min(max(e, kScaleExpMin), kScaleExpMax);
}

// A warp's page: which request, page slot, item (kv head, and for reading K or V).
struct Task {
  int b, slot, item;
};
__device__ __forceinline__ bool task_of(const QuantRowsLaunch& a, int items, Task& t) {
  const int64_t id = static_cast<int64_t>(blockIdx.x) * kRowWarps + (threadIdx.x >> 5);
  if (id >= static_cast<int64_t>(a.batch) * a.slots * items) return false;
  const uint32_t u = static_cast<uint32_t>(id);  // the host keeps ids within 31 bits
  t.item = static_cast<int>(u % items);
  t.slot = static_cast<int>(u / items % a.slots);
  t.b = static_cast<int>(u / items / a.slots);
  return true;
}

// The new rows r0 .. r1 - 1 of one page of one kv head, K or V, in registers.
template <int D, bool BF16>
struct NewRows {
  static constexpr int kLpr = D / 8;      // lanes per row
  static constexpr int kRpp = 32 / kLpr;  // rows per pass
  static constexpr int kPasses = 16 / kRpp;
  Row8<BF16> x[kPasses];

  __device__ __forceinline__ void load(const void* src, size_t row0, int64_t stride, size_t at,
                                       int r0, int r1, int lane) {
    const int d0 = 8 * (lane % kLpr), lr = lane / kLpr;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int r = i * kRpp + lr;
      if (r >= r0 && r < r1) x[i].load(src, (row0 + (r - r0)) * stride + at + d0);
      else x[i].zero();
    }
  }

  // Quantises into `codes` / `scale` of the (page, kv head); was: the scale's bits before.
  __device__ __forceinline__ void store(uint8_t* codes, float* scale, uint32_t was, int r0, int r1,
                                        int32_t* err, int lane) {
    const int d0 = 8 * (lane % kLpr), lr = lane / kLpr;
    typename Row8<BF16>::Max top{};
#pragma unroll
    for (int i = 0; i < kPasses; ++i) x[i].max_into(top);
    float amax = warp_max(Row8<BF16>::value(top));
    if (amax == INFINITY) {  // infinities become NaN and do not set the scale
      amax = 0.f;
#pragma unroll
      for (int i = 0; i < kPasses; ++i) x[i].drop_infinite(amax);
      amax = warp_max(amax);
    }
    int e = exponent_for(amax);
    if (r0 > 0) {
      if (!scale_ok(was)) {
        if (lane == 0) set_error(err, DSA_DEV_BAD_SCALE);
        return;
      }
      const int e_was = scale_exp(was);
      if (e > e_was) {
        // the rows that stay move to the larger exponent
        const float down = pow2i(e_was - e);
        for (int r = lr; r < r0; r += kRpp) {
          uint2* p = reinterpret_cast<uint2*>(codes + r * D + d0);
          const uint2 v = *p;
          uint32_t w[2] = {v.x, v.y};
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float2 lo = f16x2_f32x2(e4m3x2_f16x2(w[h]));
            const float2 hi = f16x2_f32x2(e4m3x2_f16x2_hi(w[h]));
            w[h] = f32x2_e4m3x2(lo.x * down, lo.y * down) |
                   (f32x2_e4m3x2(hi.x * down, hi.y * down) << 16);
          }
          *p = make_uint2(w[0], w[1]);
        }
      } else {
        e = e_was;
      }
    }
    const float down = pow2i(-e);
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int r = i * kRpp + lr;
      if (r >= r0 && r < r1) *reinterpret_cast<uint2*>(codes + r * D + d0) = x[i].codes(down);
    }
    __syncwarp();  // behind the other lanes' reads of the old scale
    if (lane == 0) *scale = pow2i(e);
  }
};

template <int D, bool BF16>
__global__ void __launch_bounds__(kRowWarps * 32) quant_write_kernel(const QuantRowsLaunch a) {
  griddep_wait();
  griddep_launch_dependents();
  Task t;
  if (!task_of(a, a.hkv, t)) return;
  const int lane = threadIdx.x & 31, hk = t.item;
  const int L = __ldg(a.seq_len + t.b);
  const int n = a.count != nullptr ? __ldg(a.count + t.b) : a.max_rows;
  if (L < 1 || L > a.max_pages * kPage) {
    if (lane == 0) set_error(a.err, DSA_DEV_BAD_SEQ_LEN);
    return;
  }
  if (n < 0 || n > L || n > a.max_rows) {
    if (lane == 0) set_error(a.err, DSA_DEV_BAD_QLEN);
    return;
  }
  const int first = L - n;                    // logical row of new row 0
  const int page_no = first / kPage + t.slot;
  if (n == 0 || page_no > (L - 1) / kPage) return;
  const int r0 = max(first - page_no * kPage, 0);
  const int r1 = min(L - page_no * kPage, kPage);  // rows r0 .. r1 - 1 of the page
  const int pg = __ldg(a.page_table + static_cast<size_t>(t.b) * a.max_pages + page_no);
  const size_t row0 = static_cast<size_t>(t.b) * a.max_rows + (page_no * kPage + r0 - first);
  const size_t at = static_cast<size_t>(hk) * D;
  constexpr bool kBoth = BF16 || D == 64;  // K and V in flight together
  NewRows<D, BF16> k, v;
  k.load(a.k_rows, row0, a.stride, at, r0, r1, lane);
  if (kBoth) v.load(a.v_rows, row0, a.stride, at, r0, r1, lane);
  if (static_cast<unsigned>(pg) >= static_cast<unsigned>(a.num_pages)) {
    if (lane == 0) set_error(a.err, DSA_DEV_BAD_PAGE);
    return;
  }
  const size_t ph = static_cast<size_t>(pg) * a.hkv + hk;
  // every lane has the old scales before lane 0 writes the new ones (store())
  const uint32_t ks = r0 > 0 ? __float_as_uint(a.k_scale[ph]) : 0u;
  const uint32_t vs = r0 > 0 ? __float_as_uint(a.v_scale[ph]) : 0u;
  k.store(a.k + ph * (16 * D), a.k_scale + ph, ks, r0, r1, a.err, lane);
  if (!kBoth) v.load(a.v_rows, row0, a.stride, at, r0, r1, lane);
  v.store(a.v + ph * (16 * D), a.v_scale + ph, vs, r0, r1, a.err, lane);
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kRowWarps * 32) quant_read_kernel(const QuantRowsLaunch a) {
  constexpr int kE = BF16 ? 8 : 4;      // elements per lane: 16 bytes of output
  constexpr int kLpr = D / kE;          // lanes per row
  constexpr int kRpp = 32 / kLpr;       // rows per pass
  constexpr int kPasses = 16 / kRpp;
  griddep_wait();
  griddep_launch_dependents();
  Task t;
  if (!task_of(a, 2 * a.hkv, t)) return;
  const bool is_v = t.item >= a.hkv;
  const int hk = is_v ? t.item - a.hkv : t.item;
  void* dst = is_v ? a.v_out : a.k_out;
  if (dst == nullptr) return;
  const int lane = threadIdx.x & 31;
  const int L = __ldg(a.seq_len + t.b), first = __ldg(a.start + t.b), n = __ldg(a.count + t.b);
  if (L < 1 || L > a.max_pages * kPage) {
    if (lane == 0) set_error(a.err, DSA_DEV_BAD_SEQ_LEN);
    return;
  }
  if (first < 0 || n < 0 || n > a.max_rows || first > L - n) {
    if (lane == 0) set_error(a.err, DSA_DEV_BAD_QLEN);
    return;
  }
  const int page_no = first / kPage + t.slot;
  if (n == 0 || page_no > (first + n - 1) / kPage) return;
  const int r0 = max(first - page_no * kPage, 0), r1 = min(first + n - page_no * kPage, kPage);
  const int pg = __ldg(a.page_table + static_cast<size_t>(t.b) * a.max_pages + page_no);
  if (static_cast<unsigned>(pg) >= static_cast<unsigned>(a.num_pages)) {
    if (lane == 0) set_error(a.err, DSA_DEV_BAD_PAGE);
    return;
  }
  const size_t ph = static_cast<size_t>(pg) * a.hkv + hk;
  const uint8_t* codes = (is_v ? a.v : a.k) + ph * (16 * D);
  const uint32_t sc = __float_as_uint(__ldg((is_v ? a.v_scale : a.k_scale) + ph));
  const int d0 = kE * (lane % kLpr), lr = lane / kLpr;
  uint32_t x[kPasses][kE / 4];
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int r = i * kRpp + lr;
    if (r >= r0 && r < r1) {
      if constexpr (BF16) {
        const uint2 w = __ldg(reinterpret_cast<const uint2*>(codes + r * D + d0));
        x[i][0] = w.x;
        x[i][kE / 4 - 1] = w.y;
      } else {
        x[i][0] = __ldg(reinterpret_cast<const uint32_t*>(codes + r * D + d0));
      }
    }
  }
  if (!scale_ok(sc)) {
    if (lane == 0) set_error(a.err, DSA_DEV_BAD_SCALE);
    return;
  }
  const float s = __uint_as_float(sc);
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int r = i * kRpp + lr;
    if (r < r0 || r >= r1) continue;
    const size_t slot = static_cast<size_t>(t.b) * a.max_rows + (page_no * kPage + r - first);
    const size_t at = (slot * a.hkv + hk) * D + d0;
    float f[kE];
#pragma unroll
    for (int k = 0; k < kE / 4; ++k) {
      const float2 lo = f16x2_f32x2(e4m3x2_f16x2(x[i][k])), hi = f16x2_f32x2(e4m3x2_f16x2_hi(x[i][k]));
      f[4 * k] = lo.x * s;
      f[4 * k + 1] = lo.y * s;
      f[4 * k + 2] = hi.x * s;
      f[4 * k + 3] = hi.y * s;
    }
    if constexpr (BF16)
      *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(dst) + at) =
          make_uint4(bf16x2_rn(f[0], f[1]), bf16x2_rn(f[2], f[3]), bf16x2_rn(f[4], f[5]),
                     bf16x2_rn(f[6], f[7]));
    else
      *reinterpret_cast<float4*>(reinterpret_cast<float*>(dst) + at) =
          make_float4(f[0], f[1], f[2], f[3]);
  }
}

dim3 rows_grid(const QuantRowsLaunch& a, int items) {
  const int64_t tasks = static_cast<int64_t>(a.batch) * a.slots * items;
  return dim3(static_cast<unsigned>((tasks + kRowWarps - 1) / kRowWarps));
}

}  // namespace

cudaError_t launch_quant_write(const QuantRowsLaunch& a, cudaStream_t s) {
  auto kern = a.head_dim == 128
                  ? (a.rows_bf16 ? quant_write_kernel<128, true> : quant_write_kernel<128, false>)
                  : (a.rows_bf16 ? quant_write_kernel<64, true> : quant_write_kernel<64, false>);
  return launch_pdl(kern, rows_grid(a, a.hkv), dim3(kRowWarps * 32), 0, s, a);
}

cudaError_t launch_quant_read(const QuantRowsLaunch& a, cudaStream_t s) {
  auto kern = a.head_dim == 128
                  ? (a.rows_bf16 ? quant_read_kernel<128, true> : quant_read_kernel<128, false>)
                  : (a.rows_bf16 ? quant_read_kernel<64, true> : quant_read_kernel<64, false>);
  return launch_pdl(kern, rows_grid(a, 2 * a.hkv), dim3(kRowWarps * 32), 0, s, a);
}

}  // namespace dsa
