// quant.cuh -- device helpers of the 8-bit K/V cache (e4m3 codes, one power-of-two
// scale per page and kv head): conversions, the layout of a 16-row tile in shared
// memory, and the tensor-core fragments read from it.
//
// Scores and output are two chains of mma.sync m16n8k16 with fp16 operands (an
// e4m3 value is an fp16 value, so a code enters exactly):
//   S  (16 rows x 8 columns)   = K (16 x D) * Q^T (D x 8),   K as the A operand
//   O^T (16 dims x 8 columns) += V^T (16 x 16 rows) * P (16 x 8)
// where a column is a query head (or a query token and head).  Both contractions
// leave the order of their inner index free, so every thread reads whole 16-byte
// pieces of a row instead of the pairs the fragment layout names:
//   K: thread (g = lane / 4, c = lane % 4) takes dims c*D/4 .. (c+1)*D/4 - 1 of rows g
//      and g + 8; inner step i of the product is its 4-byte word i.
//   V: it takes dims g*D/8 .. (g+1)*D/8 - 1 of rows 2c, 2c+1, 2c+8, 2c+9; rows 2c and
//      2c+1 are interleaved byte by byte (prmt) into the row pairs the A operand
//      wants, and output tile mt holds dims g*D/8 + 2mt, + 2mt + 1 (its rows g, g + 8).
#pragma once

#include <math.h>

#include "common.cuh"
#include "mma.cuh"

namespace dsa {

constexpr int kScaleExpMin = -40, kScaleExpMax = 40;

// 2^e for e in -126..127.
__device__ __forceinline__ float pow2i(int e) {
  return __int_as_float((e + 127) << 23);
}
// Whether the bits of a scale are those of 2^e, e in -40..40.
__device__ __forceinline__ bool scale_ok(uint32_t bits) {
  return (bits & 0x7fffffu) == 0 &&
         (bits >> 23) - static_cast<uint32_t>(127 + kScaleExpMin) <=
             static_cast<uint32_t>(kScaleExpMax - kScaleExpMin);
}
__device__ __forceinline__ int scale_exp(uint32_t bits) { return static_cast<int>(bits >> 23) - 127; }

// Two e4m3 codes (low 16 bits) as packed fp16, exact.
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t codes) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}"
      : "=r"(r)
      : "r"(codes));
  return r;
}
// The same for the high 16 bits.
__device__ __forceinline__ uint32_t e4m3x2_f16x2_hi(uint32_t codes) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}"
      : "=r"(r)
      : "r"(codes));
  return r;
}
// Two floats as e4m3 codes (x in the low byte): nearest even, saturated at +-448,
// NaN stays NaN.
__device__ __forceinline__ uint32_t f32x2_e4m3x2(float x, float y) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(y), "f"(x));
  return r;
}
// Two floats as packed fp16 (lo in the low half), nearest even.
__device__ __forceinline__ uint32_t f16x2_rn(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 f16x2_f32x2(uint32_t v) {
  float2 r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.f32.f16 %0, lo;\n\t"
      "cvt.f32.f16 %1, hi;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "r"(v));
  return r;
}
// What rounding (lo, hi) to fp16 lost, as fp16 again.
__device__ __forceinline__ uint32_t f16x2_rest(float lo, float hi, uint32_t rounded) {
  const float2 h = f16x2_f32x2(rounded);
  return f16x2_rn(lo - h.x, hi - h.y);
}

// d (16x8, fp32) += a (16x16, fp16, row) * b (16x8, fp16, col)
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// cp.async of 16 (or 4) bytes; with ok false nothing is read and zeros are written.
__device__ __forceinline__ void cp_async16_zfill(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(ok ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async4_zfill(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(ok ? 4 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
// At most N of this thread's latest groups still in flight.
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// A tile of 16 rows of codes in shared memory.  The 16-byte pieces of the rows are
// permuted inside 128-byte lines so that the fragment reads above hit every bank
// once: with D = 128 a line is a row and piece ch sits at ch ^ (row & 7); with
// D = 64 a line is two rows and piece (row & 1) * 4 + ch sits at that ^ 2 (row / 2 & 3).
template <int D>
struct QuantTile {
  static constexpr int kPieces = D / 16;         // 16-byte pieces of a row
  static constexpr int kBytes = 16 * D;          // one tile of K or of V
  static constexpr int kScaleOff = 2 * kBytes;   // K tile, V tile, 16 K scales, 16 V scales
  static constexpr int kStage = 2 * kBytes + 128;
  static constexpr int kCopies = 16 * kPieces / 32;  // cp.async per lane and tile
  static constexpr int kKW = D / 16;             // words of a K row per thread
  static constexpr int kVW = D / 32;             // words of a V row per thread

  __device__ __forceinline__ static int offset(int row, int ch) {
    if (D == 128) return row * 128 + ((ch ^ (row & 7)) << 4);
    return (row >> 1) * 128 + (((((row & 1) << 2) | ch) ^ (((row >> 1) & 3) << 1)) << 4);
  }
  // Row and piece of the i-th of a lane's kCopies copies.
  __device__ __forceinline__ static int copy_row(int i, int lane) {
    return i * (32 / kPieces) + lane / kPieces;
  }
  __device__ __forceinline__ static int copy_piece(int lane) { return lane % kPieces; }

  // Words of rows g (w[0]) and g + 8 (w[1]).
  __device__ __forceinline__ static void load_k(uint32_t tile, int lane, uint32_t (&w)[2][kKW]) {
    const int g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int p = 0; p < kKW / 4; ++p) {
      const uint32_t at = tile + offset(g, c * (kKW / 4) + p);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const uint4 v = lds128(at + r * (8 * D));
        w[r][4 * p] = v.x;
        w[r][4 * p + 1] = v.y;
        w[r][4 * p + 2] = v.z;
        w[r][4 * p + 3] = v.w;
      }
    }
  }
  // Words of rows 2c, 2c+1, 2c+8, 2c+9.
  __device__ __forceinline__ static void load_v(uint32_t tile, int lane, uint32_t (&w)[4][kVW]) {
    const int g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = 2 * c + (r & 1);
      if constexpr (D == 128) {
        const uint4 v = lds128(tile + offset(row, g) + (r >> 1) * (8 * D));
        w[r][0] = v.x;
        w[r][1] = v.y;
        w[r][2] = v.z;
        w[r][3] = v.w;
      } else {
        const uint2 v = lds64(tile + offset(row, g >> 1) + 8 * (g & 1) + (r >> 1) * (8 * D));
        w[r][0] = v.x;
        w[r][1] = v.y;
      }
    }
  }
  // A operand of output tile mt (0 .. D/16 - 1) from the words of load_v.
  __device__ __forceinline__ static void frag_v(const uint32_t (&w)[4][kVW], int mt,
                                                uint32_t (&a)[4]) {
    const uint32_t sel = (mt & 1) ? 0x7362u : 0x5140u;
    const uint32_t lo = __byte_perm(w[0][mt >> 1], w[1][mt >> 1], sel);
    const uint32_t hi = __byte_perm(w[2][mt >> 1], w[3][mt >> 1], sel);
    a[0] = e4m3x2_f16x2(lo);
    a[1] = e4m3x2_f16x2_hi(lo);
    a[2] = e4m3x2_f16x2(hi);
    a[3] = e4m3x2_f16x2_hi(hi);
  }
};

// Exponent by which a q row of largest magnitude amax is divided before it enters
// the product as fp16: amax lands in [2^8, 2^9), far from fp16's ends; rows of
// zeros or with an infinity or NaN are left alone.
__device__ __forceinline__ int q_exponent(float amax) {
  const int e = static_cast<int>(__float_as_uint(amax) >> 23) - 127;
  if (!(amax > 0.f) || e > 127) return 0;
  return max(e, -110) - 8;
}

}  // namespace dsa
