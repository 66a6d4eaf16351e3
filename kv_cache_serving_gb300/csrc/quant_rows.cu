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
// Both are bound by HBM (3 bytes per element with bf16 rows).  One warp takes one
// page of one kv head, K or V: its rows (4 KB of bf16 at D = 128) are loaded with all
// 16-byte loads in flight before the first is used, the maximum is a warp reduction,
// and the codes of a row leave in 8-byte pieces, contiguous over the 16 rows.
#include "common.cuh"
#include "internal.h"
#include "mma.cuh"
#include "quant.cuh"

namespace dsa {
namespace {

constexpr int kRowWarps = 4;

// 8 consecutive elements of a row as fp32.
template <bool BF16>
struct Row8;
template <>
struct Row8<true> {
  uint4 v;
  __device__ __forceinline__ void load(const void* base, size_t elem) {
    v = __ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(base) + elem));
  }
  __device__ __forceinline__ void zero() { v = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ float get(int i) const {
    const uint32_t w = i < 2 ? v.x : i < 4 ? v.y : i < 6 ? v.z : v.w;
    return (i & 1) ? bf16_hi(w) : bf16_lo(w);
  }
};
template <>
struct Row8<false> {
  float4 a, b;
  __device__ __forceinline__ void load(const void* base, size_t elem) {
    const float4* p = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(base) + elem);
    a = __ldg(p);
    b = __ldg(p + 1);
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ float get(int i) const {
    const float4& w = i < 4 ? a : b;
    return (i & 3) == 0 ? w.x : (i & 3) == 1 ? w.y : (i & 3) == 2 ? w.z : w.w;
  }
};

// The smallest e in -40..40 with amax <= 448 * 2^e = 1.75 * 2^(e + 8).
__device__ __forceinline__ int exponent_for(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return min(max(e, kScaleExpMin), kScaleExpMax);
}

// x * down as a code: an infinity becomes NaN like NaN itself.
__device__ __forceinline__ float to_code_range(float x, float down) {
  const bool finite = (__float_as_uint(x) & 0x7f800000u) != 0x7f800000u;
  return finite ? x * down : __int_as_float(0x7fc00000);
}

// A warp's page: which request, page slot, kv head, K or V.
struct Task {
  int b, slot, hk;
  bool is_v;
};
__device__ __forceinline__ bool task_of(const QuantRowsLaunch& a, Task& t) {
  const int64_t id = static_cast<int64_t>(blockIdx.x) * kRowWarps + (threadIdx.x >> 5);
  const int64_t per_slot = 2 * a.hkv;
  if (id >= static_cast<int64_t>(a.batch) * a.slots * per_slot) return false;
  const int x = static_cast<int>(id % per_slot);
  t.is_v = x >= a.hkv;
  t.hk = t.is_v ? x - a.hkv : x;
  t.slot = static_cast<int>(id / per_slot % a.slots);
  t.b = static_cast<int>(id / (per_slot * a.slots));
  return true;
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kRowWarps * 32) quant_write_kernel(const QuantRowsLaunch a) {
  constexpr int kLpr = D / 8;           // lanes per row
  constexpr int kRpp = 32 / kLpr;       // rows per pass
  constexpr int kPasses = 16 / kRpp;
  griddep_wait();
  griddep_launch_dependents();
  Task t;
  if (!task_of(a, t)) return;
  const int lane = threadIdx.x & 31;
  const int L = a.seq_len[t.b];
  const int n = a.count != nullptr ? a.count[t.b] : a.max_rows;
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
  if (static_cast<unsigned>(pg) >= static_cast<unsigned>(a.num_pages)) {
    if (lane == 0) set_error(a.err, DSA_DEV_BAD_PAGE);
    return;
  }
  const size_t ph = static_cast<size_t>(pg) * a.hkv + t.hk;
  uint8_t* codes = (t.is_v ? a.v : a.k) + ph * (16 * D);
  float* scale = (t.is_v ? a.v_scale : a.k_scale) + ph;
  const void* src = t.is_v ? a.v_rows : a.k_rows;
  const int d0 = 8 * (lane % kLpr), lr = lane / kLpr;
  Row8<BF16> x[kPasses];
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int r = i * kRpp + lr;
    if (r >= r0 && r < r1) {
      const size_t slot = static_cast<size_t>(t.b) * a.max_rows + (page_no * kPage + r - first);
      x[i].load(src, slot * a.stride + static_cast<size_t>(t.hk) * D + d0);
    } else {
      x[i].zero();
    }
  }
  const uint32_t was = r0 > 0 ? __float_as_uint(*scale) : 0u;
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < kPasses; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float m = fabsf(x[i].get(k));
      amax = m < INFINITY ? fmaxf(amax, m) : amax;  // finite ones only
    }
  amax = warp_max(amax);
  int e = exponent_for(amax);
  if (r0 > 0) {
    if (!scale_ok(was)) {
      if (lane == 0) set_error(a.err, DSA_DEV_BAD_SCALE);
      return;
    }
    const int e_was = scale_exp(was);
    if (e > e_was) {
      // the rows that stay move to the larger exponent
      const float down = pow2i(e_was - e);
      for (int r = lr; r < r0; r += kRpp) {
        uint2* p = reinterpret_cast<uint2*>(codes + r * D + d0);
        uint2 v = *p;
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
    if (r >= r0 && r < r1) {
      uint32_t c[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        c[k] = f32x2_e4m3x2(to_code_range(x[i].get(2 * k), down),
                            to_code_range(x[i].get(2 * k + 1), down));
      *reinterpret_cast<uint2*>(codes + r * D + d0) =
          make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
    }
  }
  __syncwarp();  // every lane has read the old scale
  if (lane == 0) *scale = pow2i(e);
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kRowWarps * 32) quant_read_kernel(const QuantRowsLaunch a) {
  constexpr int kLpr = D / 16;          // lanes per row
  constexpr int kRpp = 32 / kLpr;       // rows per pass
  constexpr int kPasses = 16 / kRpp;
  griddep_wait();
  griddep_launch_dependents();
  Task t;
  if (!task_of(a, t)) return;
  void* dst = t.is_v ? a.v_out : a.k_out;
  if (dst == nullptr) return;
  const int lane = threadIdx.x & 31;
  const int L = a.seq_len[t.b], first = a.start[t.b], n = a.count[t.b];
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
  const size_t ph = static_cast<size_t>(pg) * a.hkv + t.hk;
  const uint8_t* codes = (t.is_v ? a.v : a.k) + ph * (16 * D);
  const uint32_t sc = __float_as_uint(__ldg((t.is_v ? a.v_scale : a.k_scale) + ph));
  const int ch = lane % kLpr, lr = lane / kLpr;
  uint4 x[kPasses];
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int r = i * kRpp + lr;
    if (r >= r0 && r < r1) x[i] = __ldg(reinterpret_cast<const uint4*>(codes + r * D) + ch);
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
    const size_t at = (slot * a.hkv + t.hk) * D + 16 * ch;
    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
    float f[16];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 lo = f16x2_f32x2(e4m3x2_f16x2(w[k])), hi = f16x2_f32x2(e4m3x2_f16x2_hi(w[k]));
      f[4 * k] = lo.x * s;
      f[4 * k + 1] = lo.y * s;
      f[4 * k + 2] = hi.x * s;
      f[4 * k + 3] = hi.y * s;
    }
    if constexpr (BF16) {
      uint4* p = reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(dst) + at);
#pragma unroll
      for (int h = 0; h < 2; ++h)
        p[h] = make_uint4(bf16x2_rn(f[8 * h], f[8 * h + 1]), bf16x2_rn(f[8 * h + 2], f[8 * h + 3]),
                          bf16x2_rn(f[8 * h + 4], f[8 * h + 5]),
                          bf16x2_rn(f[8 * h + 6], f[8 * h + 7]));
    } else {
      float4* p = reinterpret_cast<float4*>(reinterpret_cast<float*>(dst) + at);
#pragma unroll
      for (int h = 0; h < 4; ++h)
        p[h] = make_float4(f[4 * h], f[4 * h + 1], f[4 * h + 2], f[4 * h + 3]);
    }
  }
}

dim3 rows_grid(const QuantRowsLaunch& a) {
  const int64_t tasks = static_cast<int64_t>(a.batch) * a.slots * 2 * a.hkv;
  return dim3(static_cast<unsigned>((tasks + kRowWarps - 1) / kRowWarps));
}

}  // namespace

cudaError_t launch_quant_write(const QuantRowsLaunch& a, cudaStream_t s) {
  auto kern = a.head_dim == 128
                  ? (a.rows_bf16 ? quant_write_kernel<128, true> : quant_write_kernel<128, false>)
                  : (a.rows_bf16 ? quant_write_kernel<64, true> : quant_write_kernel<64, false>);
  return launch_pdl(kern, rows_grid(a), dim3(kRowWarps * 32), 0, s, a);
}

cudaError_t launch_quant_read(const QuantRowsLaunch& a, cudaStream_t s) {
  auto kern = a.head_dim == 128
                  ? (a.rows_bf16 ? quant_read_kernel<128, true> : quant_read_kernel<128, false>)
                  : (a.rows_bf16 ? quant_read_kernel<64, true> : quant_read_kernel<64, false>);
  return launch_pdl(kern, rows_grid(a), dim3(kRowWarps * 32), 0, s, a);
}

}  // namespace dsa
