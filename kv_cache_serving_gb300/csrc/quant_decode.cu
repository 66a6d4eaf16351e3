// quant_decode.cu -- decode attention over the 8-bit paged K/V cache: one query token
// per request, dense rows or the kept set of the method's mask.
//
// Mathematics.  With codes k_j, v_j and scales s_j, t_j (powers of two), per head:
//   x_j = log2(e) * scale * s_j (q . k_j)
//   out = sum_j 2^x_j t_j v_j / sum_j 2^x_j,     lse = ln 2 * log2 sum_j 2^x_j
// The V scale joins the exponent: with y_j = x_j + log2 t_j (exact) and a reference
// r, p_j = 2^(y_j - r) multiplies the bare code in the tensor-core product and
// p_j / t_j (exact) enters the sum.  So the weights of that product share one range
// however much the pages' scales differ, and no V element is ever scaled.  r follows
// the running maximum with a slack of 2^10: one vote per tile instead of a reduction
// over its rows, and the accumulators are rescaled only when it moves.
// bf16 q: p_j <= 2^14 is rounded to fp16 (2^-11 relative, below the bf16 output's own 2^-8;
// the largest is 2^4 or more, so below 2^-18 of it, where fp16's normal range ends, by steps of
// 2^-28 of the largest).  fp32 q: q in two fp16 halves (2^-22 relative, 2^-33 of the row's
// largest), p_j <= 2^15 likewise (2^-22), or, in a tile with weights below 2^-2, which halves
// hold worse and lose 2^-24 below a sink, in three bf16 thirds (2^-24 relative, down to 2^-100
// of the largest), V widened to bf16 for them.  The dense batch below with fp32 q: 126 us, 132
// with thirds throughout.
//
// What bounds it: HBM, and for short calls the chain of dependent loads at a CTA's start.  A
// row is 2 D bytes for 4 D G flops (<= 8 flops per byte; the 8 columns of an mma cost the
// same for G = 1 .. 8), so the design keeps bytes in flight: each warp owns a ring of two
// 16-row tiles filled by cp.async (4 KB of K and V each at D = 128; 16 warps per SM hold 128
// KB; a third stage measured 2% slower, more warps with fewer registers 8%), and nothing
// but its own copies ever stops a warp.  q, the page ids of a kept set's first tiles and the
// sizes are asked for together.
// Measured (GB300, back-to-back calls): 128 requests of 33 .. 4608 rows, 32/8 heads, dense 102
// us = 5.7 TB/s, 0.83 of the copy rate; 8 requests of 8000 rows 32 us (10 us of it start and
// joining); 2048 units of 290 kept rows 33 us.  The copies alone, without the arithmetic,
// take 99.5, 30.8 and 29.4 us.
//
// Work split.  Dense rows: a persistent grid of one CTA per resident slot takes equal
// shares of all tiles of the batch, in unit order (a unit is a request and kv head); the
// shares' borders come from a prefix sum over seq_len that every warp makes itself (handing
// out the last quarter in small pieces as CTAs get done measured 2-5% slower: a piece's start
// costs what the balance gains).  Sparse rows: one CTA per unit, or a few when there are
// too few units.  A unit cut over several CTAs leaves partial states in the workspace, and
// the last one to arrive sums them in order.
#include <math.h>

#include "common.cuh"
#include "host.h"
#include "internal.h"
#include "mma.cuh"
#include "quant.cuh"
#include "rows.cuh"

namespace dsa {
namespace {

// Weights are 2^(y - ref).  ref follows the largest y so that it stands for 2^kHead, once
// a y passes it by kSlack; before the first row it is far below every score, and finite.
constexpr float kNoRef = -3e38f;

template <int D, int NW>
struct QuantRing {
  static constexpr int kStages = 2;
  static constexpr int kWarp = kStages * QuantTile<D>::kStage;
  static constexpr int kSmem = NW * kWarp;
  // a warp's end state, 8 heads of [acc(D), m, l], fits the start of its ring
  static_assert(8 * (D + 2) * 4 <= kWarp, "state fits the ring");
};

// One warp's state over the rows it has seen, for the 8 columns of a kv head.
template <int D, bool XQ>
struct QuantWarp {
  using Tile = QuantTile<D>;
  static constexpr int NK = D / 16;
  // fp32 q: high, so that most weights lie where fp16 halves hold them (2^15 is still one)
  static constexpr float kHead = XQ ? 13.f : 4.f, kSlack = XQ ? 2.f : 10.f;
  uint32_t qh[NK][2], ql[XQ ? NK : 1][2];  // B operand: head lane / 4
  float f[2];                                // score factor of heads 2c, 2c + 1
  float ref[2], l[2], acc[NK][4];
  bool bad;

  __device__ __forceinline__ void reset() {
    ref[0] = ref[1] = kNoRef;
    l[0] = l[1] = 0.f;
#pragma unroll
    for (int mt = 0; mt < NK; ++mt)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[mt][e] = 0.f;
  }

  // This thread's part (dims c*D/4 .. of head g) of heads qrow0 .. qrow0 + group - 1, as it
  // is in memory: asked for before anything else, converted when the copies are out.
  // Columns past the group are zero.
  static constexpr int kQV = D / (XQ ? 16 : 32);
  __device__ __forceinline__ static void fetch_q(const void* q, size_t qrow0, int group, int lane,
                                                 uint4 (&v)[kQV]) {
    const int g = lane >> 2, c = lane & 3;
    const size_t at = (qrow0 + g) * D + c * (D / 4);
    const uint4* p = reinterpret_cast<const uint4*>(
        reinterpret_cast<const unsigned char*>(q) + at * (XQ ? 4 : 2));
#pragma unroll
    for (int i = 0; i < kQV; ++i) v[i] = g < group ? __ldg(p + i) : make_uint4(0u, 0u, 0u, 0u);
  }
  __device__ __forceinline__ void take_q(const uint4 (&v)[kQV], float scale_log2, int lane) {
    const int c = lane & 3;
    float x[D / 4];
#pragma unroll
    for (int i = 0; i < kQV; ++i) {
      const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (XQ) {
          x[4 * i + k] = __uint_as_float(w[k]);
        } else {
          x[8 * i + 2 * k] = bf16_lo(w[k]);
          x[8 * i + 2 * k + 1] = bf16_hi(w[k]);
        }
      }
    }
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < D / 4; ++i) amax = fmaxf(amax, fabsf(x[i]));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    const int e = q_exponent(amax);
    const float down = pow2i(-e);
#pragma unroll
    for (int i = 0; i < NK; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float a = x[4 * i + 2 * h] * down, b = x[4 * i + 2 * h + 1] * down;
        qh[i][h] = f16x2_rn(a, b);
        if constexpr (XQ) ql[i][h] = f16x2_rest(a, b, qh[i][h]);
      }
    const float up = scale_log2 * pow2i(e);
    f[0] = __shfl_sync(0xffffffffu, up, (2 * c) * 4);
    f[1] = __shfl_sync(0xffffffffu, up, (2 * c + 1) * 4);
  }

  // Rows 0 .. nrows - 1 of the tile at shared address `tile`.  PAGE: the rows are those of
  // one page (one K and one V scale), else every row has its own.
  template <bool PAGE>
  __device__ __forceinline__ void tile(uint32_t tile, int nrows, int lane) {
    const int g = lane >> 2;
    float s[4] = {0.f, 0.f, 0.f, 0.f}, s2[4] = {0.f, 0.f, 0.f, 0.f};
    {
      uint32_t w[2][Tile::kKW];
      Tile::load_k(tile, lane, w);
#pragma unroll
      for (int i = 0; i < NK; ++i) {
        const uint32_t a0 = e4m3x2_f16x2(w[0][i]), a1 = e4m3x2_f16x2(w[1][i]);
        const uint32_t a2 = e4m3x2_f16x2_hi(w[0][i]), a3 = e4m3x2_f16x2_hi(w[1][i]);
        mma_f16((i & 1) ? s2 : s, a0, a1, a2, a3, qh[i][0], qh[i][1]);
        if constexpr (XQ) mma_f16((i & 1) ? s : s2, a0, a1, a2, a3, ql[i][0], ql[i][1]);
      }
    }
    const uint32_t sc = tile + Tile::kScaleOff;
    float y[4];  // rows g (0, 1) and g + 8 (2, 3), heads 2c and 2c + 1
    float inv[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const uint32_t ks = lds32(sc + (PAGE ? 0 : 4 * g + 32 * r));
      const uint32_t vs = lds32(sc + 64 + (PAGE ? 0 : 4 * g + 32 * r));
      bad |= (PAGE || g + 8 * r < nrows) && !(scale_ok(ks) && scale_ok(vs));
      inv[r] = __uint_as_float((254u << 23) - vs);
      const float lv = static_cast<float>(scale_exp(vs));
#pragma unroll
      for (int j = 0; j < 2; ++j)
        y[2 * r + j] = fmaf(s[2 * r + j] + s2[2 * r + j], f[j] * __uint_as_float(ks), lv);
    }
    if (nrows < 16) {  // rows that are not there: no weight, and finite in the sum
#pragma unroll
      for (int r = 0; r < 2; ++r)
        if (g + 8 * r >= nrows) {
          y[2 * r] = y[2 * r + 1] = -INFINITY;
          inv[r] = 0.f;
        }
    }
    // (the difference is exact where it counts; ref + 14 rounds to as much as ref + 16 from 2^25
    // on, and 2^16 is no fp16)
    const bool over = fmaxf(y[0], y[2]) - ref[0] > kHead + kSlack ||
                      fmaxf(y[1], y[3]) - ref[1] > kHead + kSlack;
    if (__any_sync(0xffffffffu, over)) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float mx = fmaxf(y[j], y[2 + j]);
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
        // (mx - 13 rounds to mx - 16 from 2^26 on)
        const float to = fmaxf(ref[j], fabsf(mx) < 0x1p20f ? mx - kHead : mx);
        const float down = ex2_approx(ref[j] - to);
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
      l[e & 1] = fmaf(y[e], inv[e >> 1], l[e & 1]);
    }
    uint32_t w[4][Tile::kVW];
    // fp32 q: fp16 halves are good to 2^-22 from 2^-2 on (the second one's last step is 2^-24);
    // a tile with smaller weights takes thirds
    bool thirds = false;
    if constexpr (XQ) {
#pragma unroll
      for (int e = 0; e < 4; ++e) thirds |= y[e] < 0.25f && y[e] != 0.f;
      thirds = __any_sync(0xffffffffu, thirds);
    }
    if (!thirds) {
      const uint32_t p0 = f16x2_rn(y[0], y[1]), p1 = f16x2_rn(y[2], y[3]);
      const uint32_t b0 = movmatrix_trans(p0), b1 = movmatrix_trans(p1);
      uint32_t c0 = 0, c1 = 0;
      if constexpr (XQ) {
        c0 = movmatrix_trans(f16x2_rest(y[0], y[1], p0));
        c1 = movmatrix_trans(f16x2_rest(y[2], y[3], p1));
      }
      Tile::load_v(tile + Tile::kBytes, lane, w);
#pragma unroll
      for (int mt = 0; mt < NK; ++mt) {
        uint32_t a[4];
        Tile::frag_v(w, mt, a);
        mma_f16(acc[mt], a[0], a[1], a[2], a[3], b0, b1);
        if constexpr (XQ) mma_f16(acc[mt], a[0], a[1], a[2], a[3], c0, c1);
      }
    } else {
      // of 8 bits; what bf16 took off a float is a float, so the thirds add up
      uint32_t b[3][2];
#pragma unroll
      for (int k = 0; k < 3; ++k)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint32_t part = bf16x2_rn(y[2 * r], y[2 * r + 1]);
          y[2 * r] -= bf16_lo(part);
          y[2 * r + 1] -= bf16_hi(part);
          b[k][r] = movmatrix_trans(part);
        }
      Tile::load_v(tile + Tile::kBytes, lane, w);
#pragma unroll
      for (int mt = 0; mt < NK; ++mt) {
        uint32_t a[4];
        Tile::frag_v(w, mt, a);
#pragma unroll
        for (int k = 0; k < 4; ++k) {  // 4 bits: exact in bf16 too
          const float2 v = f16x2_f32x2(a[k]);
          a[k] = bf16x2_rn(v.x, v.y);
        }
#pragma unroll
        for (int k = 2; k >= 0; --k) mma_bf16(acc[mt], a, b[k][0], b[k][1]);
      }
    }
  }

  // State as [head][acc(D), m, l] for the heads of the group; m is the reference the
  // weights were taken against.
  __device__ __forceinline__ void flush(float* to, int group, int lane) {
    const int g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float sum = l[j];
      sum += __shfl_xor_sync(0xffffffffu, sum, 4);
      sum += __shfl_xor_sync(0xffffffffu, sum, 8);
      sum += __shfl_xor_sync(0xffffffffu, sum, 16);
      const int h = 2 * c + j;
      if (h < group) {
        float* row = to + h * (D + 2);
#pragma unroll
        for (int mt = 0; mt < NK; ++mt) {
          row[g * (D / 8) + 2 * mt] = acc[mt][j];
          row[g * (D / 8) + 2 * mt + 1] = acc[mt][2 + j];
        }
        if (g == 0) {
          row[D] = ref[j];
          row[D + 1] = sum;
        }
      }
    }
  }
};

__device__ __forceinline__ int arrive(int32_t* p) {
  int v;
  asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(v) : "l"(p) : "memory");
  return v;
}

// x / d; tile counts almost always fit 32 bits, where a division costs a third.
__device__ __forceinline__ uint64_t div(uint64_t x, uint64_t d) {
  return ((x | d) >> 32) == 0 ? static_cast<uint32_t>(x) / static_cast<uint32_t>(d) : x / d;
}

// One CTA's piece of a unit: tiles t0 .. t1 - 1 of the unit's row list.
struct Segment {
  int b, hk, L, n, t0, t1;
};

template <int D, int MODE, bool XQ, int NW>
struct QuantDecode {
  using Tile = QuantTile<D>;
  using Ring = QuantRing<D, NW>;
  using Warp = QuantWarp<D, XQ>;
  static constexpr int S = Ring::kStages;
  const QuantDecodeLaunch& a;
  unsigned char* smem;
  int lane, warp;
  MaskRows rows;  // kModeMask: the unit's kept set

  __device__ QuantDecode(const QuantDecodeLaunch& args, unsigned char* sm)
      : a(args), smem(sm), lane(threadIdx.x & 31), warp(threadIdx.x >> 5) {}

  __device__ __forceinline__ float* state(int w) {
    return reinterpret_cast<float*>(smem + w * Ring::kWarp);
  }

  // NaN into every output of unit (b, hk).
  __device__ void poison(int b, int hk) {
    for (int x = threadIdx.x; x < a.group * D; x += NW * 32) {
      const size_t qh = static_cast<size_t>(b) * a.hq + hk * a.group + x / D;
      if (XQ)
        reinterpret_cast<float*>(a.out)[qh * D + x % D] = __int_as_float(0x7fc00000);
      else
        reinterpret_cast<uint16_t*>(a.out)[qh * D + x % D] = 0x7fc0;
      if (a.lse != nullptr && x % D == 0) a.lse[qh] = __int_as_float(0x7fc00000);
    }
  }

  // Every warp's state over its tiles of the segment, in shared memory; ends with
  // a barrier.
  // spec[t]: page ids loaded before the row set was known, as if tile t were rows of the
  // prompt (kModeMask; they are used where that turns out so).
  __device__ __forceinline__ void scan(const Segment& sg, const int (&spec)[S],
                                       const uint4 (&qv)[Warp::kQV]) {
    Warp w;
    const int nt = sg.t1 - sg.t0;
    const int my_tiles = warp < nt ? (nt - warp + NW - 1) / NW : 0;
    const int32_t* pt = a.page_table + static_cast<size_t>(sg.b) * a.max_pages;
    const int32_t* list =
        MODE == kModeList ? a.kept_idx + (static_cast<size_t>(sg.b) * a.hkv + sg.hk) * a.max_kept
                          : nullptr;
    const uint32_t ring = smem_addr(smem + warp * Ring::kWarp);
    const int my_r = lane & 15;
    auto tile_of = [&](int t) { return sg.t0 + warp + t * NW; };
    auto rows_of = [&](int t) { return min(16, sg.n - 16 * tile_of(t)); };

    // Logical row of this lane's row (lane % 16) of local tile t.
    auto load_j = [&](int t) -> int {
      if (t >= my_tiles) return 0;
      const int p = 16 * tile_of(t) + my_r;
      if constexpr (MODE == kModeMask) {
        if (16 * tile_of(t) + rows_of(t) > rows.np) {  // warp-uniform: reaches window rows
          const int jw = rows.window_row(p - rows.np);
          return my_r >= rows_of(t) ? 0 : (p < rows.np ? p : jw);
        }
      }
      if (my_r >= rows_of(t)) return 0;
      if constexpr (MODE == kModeList) return __ldg(list + p);
      return p;
    };
    auto load_page = [&](int t, int& j) -> int {
      if (t >= my_tiles || my_r >= rows_of(t)) return 0;
      if (MODE == kModeList && static_cast<unsigned>(j) >= static_cast<unsigned>(sg.L)) {
        set_error(a.err, DSA_DEV_BAD_INDEX);
        j = 0;
      }
      return __ldg(pt + (j >> 4));
    };
    // Copies of local tile t into stage s: this lane's row (lane % 16) is row j, in page pg.
    auto issue = [&](int t, int s, int j, int pg) {
      if (t < my_tiles) {
        const int nrows = rows_of(t);
        bool ok = my_r < nrows;
        if (static_cast<unsigned>(pg) >= static_cast<unsigned>(a.num_pages)) {
          set_error(a.err, DSA_DEV_BAD_PAGE);  // lanes without a row hold page 0, or the tile's
          ok = false;
          pg = 0;
        }
        const uint32_t ph = static_cast<uint32_t>(pg) * a.hkv + sg.hk;
        const uint32_t dst = ring + s * Tile::kStage;
        const unsigned okm = __ballot_sync(0xffffffffu, ok);
        if constexpr (MODE == kModeDense) {
          const size_t at = static_cast<size_t>(ph) * (16 * D) + 16 * lane;
          const uint8_t *kp = a.k + at, *vp = a.v + at;
#pragma unroll
          for (int i = 0; i < Tile::kCopies; ++i) {
            const int r = Tile::copy_row(i, lane);
            const uint32_t to = dst + Tile::offset(r, Tile::copy_piece(lane));
            const bool in = (okm >> r) & 1u;
            cp_async16_zfill(to, kp + 512 * i, in);
            cp_async16_zfill(to + Tile::kBytes, vp + 512 * i, in);
          }
          if (lane < 2)  // the page's scales
            cp_async4_zfill(dst + Tile::kScaleOff + 64 * lane,
                            (lane == 0 ? a.k_scale : a.v_scale) + ph, okm != 0u);
        } else {
          const uint32_t row = ph * 16u + (j & 15);
#pragma unroll
          for (int i = 0; i < Tile::kCopies; ++i) {
            const int r = Tile::copy_row(i, lane);
            const uint32_t gr = __shfl_sync(0xffffffffu, row, r);
            const size_t off = static_cast<size_t>(gr) * D + 16 * Tile::copy_piece(lane);
            const uint32_t to = dst + Tile::offset(r, Tile::copy_piece(lane));
            const bool in = (okm >> r) & 1u;
            cp_async16_zfill(to, a.k + off, in);
            cp_async16_zfill(to + Tile::kBytes, a.v + off, in);
          }
          cp_async4_zfill(dst + Tile::kScaleOff + 4 * lane,
                          (lane < 16 ? a.k_scale : a.v_scale) + ph, ok);
        }
      }
      cp_async_commit();
    };

    // Dense rows: a tile is a page, the same for every lane, so a lane holds the page
    // id of one of the warp's next 32 tiles (and of one of the 32 after them).
    int held = 0, held_next = 0;
    auto dense_pages = [&](int t) -> int {
      const int x = tile_of(t + lane);
      return t + lane < my_tiles ? __ldg(pt + x) : 0;
    };
    int jn = 0, pn = 0, jn2 = 0;
    if constexpr (MODE == kModeDense) {
      held = dense_pages(0);
      held_next = dense_pages(32);
    } else {
      int js[S], ps[S];
#pragma unroll
      for (int t = 0; t < S; ++t) js[t] = load_j(t);
      jn2 = load_j(S);
#pragma unroll
      for (int t = 0; t < S; ++t)
        ps[t] = MODE == kModeMask && my_r < rows_of(t) && js[t] == 16 * (warp + t * NW) + my_r
                    ? spec[t]
                    : load_page(t, js[t]);
#pragma unroll
      for (int t = 0; t < S - 1; ++t) issue(t, t, js[t], ps[t]);
      jn = js[S - 1];
      pn = ps[S - 1];
    }
    if constexpr (MODE == kModeDense) {
#pragma unroll
      for (int t = 0; t < S - 1; ++t)
        issue(t, t, my_r, __shfl_sync(0xffffffffu, held, t));
    }
    w.reset();
    w.bad = false;
    w.take_q(qv, a.scale_log2, lane);
    int s = 0, s_fill = S - 1;
    for (int t = 0; t < my_tiles; ++t) {
      const int tf = t + S - 1;  // tile whose copies go out now
      if constexpr (MODE == kModeDense) {
        if ((tf & 31) == 0) {
          held = held_next;
          held_next = dense_pages(tf + 32);
        }
        issue(tf, s_fill, my_r, __shfl_sync(0xffffffffu, held, tf & 31));
      } else {
        issue(tf, s_fill, jn, pn);
        jn = jn2;
        pn = load_page(tf + 1, jn);
        jn2 = load_j(tf + 2);
      }
      cp_async_wait<S - 1>();
      __syncwarp();
      w.template tile<MODE == kModeDense>(ring + s * Tile::kStage, rows_of(t), lane);
      __syncwarp();  // every lane has read the stage before it is refilled
      s = s + 1 == S ? 0 : s + 1;
      s_fill = s_fill + 1 == S ? 0 : s_fill + 1;
    }
    cp_async_wait<0>();
    if (w.bad) set_error(a.err, DSA_DEV_BAD_SCALE);
    __syncwarp();
    w.flush(state(warp), a.group, lane);
    __syncthreads();
  }

  // The CTA's state (summed over its warps) of head h: weight of each warp's state,
  // and the combined m and l.
  __device__ __forceinline__ void weights(int h, float (&wt)[NW], float& m, float& l) {
    m = -INFINITY;
#pragma unroll
    for (int w = 0; w < NW; ++w) m = fmaxf(m, state(w)[h * (D + 2) + D]);
    l = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      wt[w] = ex2_approx(state(w)[h * (D + 2) + D] - m);
      l += state(w)[h * (D + 2) + D + 1] * wt[w];
    }
  }

  __device__ __forceinline__ void store(size_t qh, int d, float4 v) {
    if (XQ) {
      *reinterpret_cast<float4*>(reinterpret_cast<float*>(a.out) + qh * D + d) = v;
    } else {
      uint2 r;
      r.x = bf16x2_rn(v.x, v.y);
      r.y = bf16x2_rn(v.z, v.w);
      *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(a.out) + qh * D + d) = r;
    }
  }

  // After scan(): write the unit's output (slot < 0), or leave the partial state in
  // `slot` and, as the last of `nparts` CTAs to arrive at counter `cnt`, sum the
  // parts: part 0 in slot `first`, part p > 0 in slot `later + p * stride`.
  __device__ __forceinline__ void finish(const Segment& sg, int slot, int cnt, int nparts,
                                         int first, int later, int stride) {
    const size_t qh0 = static_cast<size_t>(sg.b) * a.hq + sg.hk * a.group;
    const int part_floats = quant_part_floats(a.group, D);
    float* part = slot < 0 ? nullptr : a.part + static_cast<size_t>(slot) * part_floats;
    for (int x = threadIdx.x; x < a.group * (D / 4); x += NW * 32) {
      const int h = x / (D / 4), d = 4 * (x % (D / 4));
      float wt[NW], m, l;
      weights(h, wt, m, l);
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const float2 u = *reinterpret_cast<const float2*>(state(w) + h * (D + 2) + d);
        const float2 v = *reinterpret_cast<const float2*>(state(w) + h * (D + 2) + d + 2);
        o.x = fmaf(u.x, wt[w], o.x);
        o.y = fmaf(u.y, wt[w], o.y);
        o.z = fmaf(v.x, wt[w], o.z);
        o.w = fmaf(v.y, wt[w], o.w);
      }
      if (part == nullptr) {
        const float r = 1.f / l;
        store(qh0 + h, d, make_float4(o.x * r, o.y * r, o.z * r, o.w * r));
        if (d == 0 && a.lse != nullptr) a.lse[qh0 + h] = (m + log2f(l)) * kLn2;
      } else {
        // [acc of every head], then [m, l of every head]: 16-byte aligned rows
        *reinterpret_cast<float4*>(part + h * D + d) = o;
        if (d == 0)
          *reinterpret_cast<float2*>(part + a.group * D + 2 * h) = make_float2(m, l);
      }
    }
    if (part == nullptr) {
      __syncthreads();  // the states are read before the rings are refilled
      return;
    }
    // the CTA's stores, ordered by the barrier, are released by one thread's arrival; the
    // last arrival acquires those of the others
    __shared__ int last;
    __syncthreads();
    if (threadIdx.x == 0) {
      last = arrive(a.count + cnt) == nparts - 1;
      if (last) a.count[cnt] = 0;  // every part has arrived
    }
    __syncthreads();
    if (!last) return;
    auto slot_of = [&](int p) {
      return a.part + static_cast<size_t>(p == 0 ? first : later + p * stride) * part_floats;
    };
    // one pass over the parts in order, eight in flight: running maximum, sum and
    // accumulator of this thread's head and dims
    for (int x = threadIdx.x; x < a.group * (D / 4); x += NW * 32) {
      const int h = x / (D / 4), d = 4 * (x % (D / 4));
      float m = kNoRef, l = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int p0 = 0; p0 < nparts; p0 += 8) {
        float2 ml[8];
        float4 v[8];
#pragma unroll
        for (int p = 0; p < 8; ++p) {
          const float* src = slot_of(min(p0 + p, nparts - 1));
          ml[p] = __ldcg(reinterpret_cast<const float2*>(src + a.group * D + 2 * h));
          v[p] = __ldcg(reinterpret_cast<const float4*>(src + h * D + d));
        }
        float to = m;
#pragma unroll
        for (int p = 0; p < 8; ++p) to = fmaxf(to, ml[p].x);
        const float keep = ex2_approx(m - to);
        m = to;
        l *= keep;
        o.x *= keep;
        o.y *= keep;
        o.z *= keep;
        o.w *= keep;
#pragma unroll
        for (int p = 0; p < 8; ++p) {
          if (p0 + p >= nparts) break;
          const float wt = ex2_approx(ml[p].x - m);
          l = fmaf(ml[p].y, wt, l);
          o.x = fmaf(v[p].x, wt, o.x);
          o.y = fmaf(v[p].y, wt, o.y);
          o.z = fmaf(v[p].z, wt, o.z);
          o.w = fmaf(v[p].w, wt, o.w);
        }
      }
      const float r = 1.f / l;
      store(qh0 + h, d, make_float4(o.x * r, o.y * r, o.z * r, o.w * r));
      if (d == 0 && a.lse != nullptr) a.lse[qh0 + h] = (m + log2f(l)) * kLn2;
    }
    __syncthreads();
  }

  // Dense rows: this CTA's share of all tiles of the batch, in unit order.  Every warp finds
  // the share by itself, from a prefix sum over the requests' tiles (lane l: requests
  // l * per .. l * per + per - 1).
  __device__ __forceinline__ void run_dense() {
    auto valid = [&](int L) { return L >= 1 && L <= a.max_pages * kPage; };
    auto tiles_of = [&](int L) { return valid(L) ? (L + 15) >> 4 : 0; };
    const int per = (a.batch + 31) / 32;
    const int b0 = min(a.batch, lane * per), b1 = min(a.batch, b0 + per);
    int64_t mine = 0;
    bool any_bad = false;
#pragma unroll 4
    for (int b = b0; b < b1; ++b) {
      const int L = __ldg(a.seq_len + b);
      mine += tiles_of(L);
      any_bad |= !valid(L);
    }
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (__any_sync(0xffffffffu, any_bad)) {
      // requests with a bad length are flagged and get NaN (by one CTA each)
      for (int b = blockIdx.x; b < a.batch; b += gridDim.x)
        if (!valid(a.seq_len[b])) {
          if (threadIdx.x == 0) set_error(a.err, DSA_DEV_BAD_SEQ_LEN);
          for (int hk = 0; hk < a.hkv; ++hk) poison(b, hk);
        }
    }
    // T tiles over N CTAs (no more than leave each its least share, or a unit): CTA i takes
    // tiles floor(i T / N) .. floor((i+1) T / N) - 1
    const uint64_t T = static_cast<uint64_t>(__shfl_sync(0xffffffffu, incl, 31)) * a.hkv;
    const uint64_t units = static_cast<uint64_t>(a.batch) * a.hkv;
    uint64_t most = div(T + a.min_tiles - 1, a.min_tiles);
    if (most < units) most = units < T ? units : T;
    const uint64_t N = most < gridDim.x ? most : gridDim.x;
    if (blockIdx.x >= N) return;
    auto owner = [&](uint64_t x) { return static_cast<int>(div((x + 1) * N + T - 1, T) - 1); };
    uint64_t x = div(blockIdx.x * T, N);
    const uint64_t x1 = div((blockIdx.x + 1) * T, N);
    // the request of tile x: its lane by vote, then that lane's walk over its requests
    uint64_t base = static_cast<uint64_t>(incl - mine) * a.hkv;
    int b = b0;
    const bool have = x >= base && x < base + static_cast<uint64_t>(mine) * a.hkv;
    if (have)
      for (; b < b1; ++b) {
        const uint64_t nb = static_cast<uint64_t>(tiles_of(__ldg(a.seq_len + b))) * a.hkv;
        if (x < base + nb) break;
        base += nb;
      }
    const int src = __ffs(__ballot_sync(0xffffffffu, have)) - 1;
    b = __shfl_sync(0xffffffffu, b, src);
    base = __shfl_sync(0xffffffffu, base, src);
    while (x < x1) {
      int L = __ldg(a.seq_len + b);
      while (!valid(L)) L = __ldg(a.seq_len + ++b);  // a tile x < T lies ahead
      const int nb = tiles_of(L);
      const int hk = static_cast<int>(div(x - base, nb));
      const int tl = static_cast<int>(x - base - static_cast<uint64_t>(hk) * nb);
      const uint64_t left = x1 - x;
      const int t1 = left < static_cast<uint64_t>(nb - tl) ? tl + static_cast<int>(left) : nb;
      const Segment sg{b, hk, L, L, tl, t1};
      uint4 qv[Warp::kQV];
      Warp::fetch_q(a.q, static_cast<size_t>(b) * a.hq + hk * a.group, a.group, lane, qv);
      scan(sg, {}, qv);
      // CTA i leaves the unit it began before i's share in slot 2i, the unit that goes on
      // after it in slot 2i + 1; the counter is that of the unit's first CTA
      int slot = -1, i0 = 0, nparts = 1;
      if (tl != 0 || t1 != nb) {
        const uint64_t u0 = x - tl;
        i0 = owner(u0);
        nparts = owner(u0 + nb - 1) - i0 + 1;
        slot = 2 * static_cast<int>(blockIdx.x) + (static_cast<int>(blockIdx.x) == i0);
      }
      finish(sg, slot, i0, nparts, 2 * i0 + 1, 2 * i0, 2);
      x += t1 - tl;
      if (t1 == nb && hk == a.hkv - 1) {
        base += static_cast<uint64_t>(nb) * a.hkv;
        ++b;
      }
    }
  }

  // Sparse rows: part `part` of a.parts of one unit.
  __device__ __forceinline__ void run_sparse() {
    const int part = blockIdx.x % a.parts, unit = blockIdx.x / a.parts;
    const int hk = unit % a.hkv, bpos = unit / a.hkv;
    int b = a.order != nullptr ? __ldg(a.order + bpos) : bpos;
    if (MODE == kModeList && a.sched != nullptr) {
      const int tag = a.sched_tag[0], sb = a.sched[bpos];
      if (tag == a.sched_expect) b = sb;
    }
    if (static_cast<unsigned>(b) >= static_cast<unsigned>(a.batch)) {
      if (part == 0 && hk == 0 && threadIdx.x == 0) set_error(a.err, DSA_DEV_BAD_ORDER);
      return;
    }
    uint4 qv[Warp::kQV];
    Warp::fetch_q(a.q, static_cast<size_t>(b) * a.hq + hk * a.group, a.group, lane, qv);
    const int L = a.seq_len[b];
    int spec[S] = {};
    if constexpr (MODE == kModeMask) {
#pragma unroll
      for (int t = 0; t < S; ++t)
        if (warp + t * NW < a.max_pages)
          spec[t] = __ldg(a.page_table + static_cast<size_t>(b) * a.max_pages + warp + t * NW);
    }
    int n;
    if constexpr (MODE == kModeMask) {
      const uint32_t* mrow = a.keep_mask + (static_cast<size_t>(b) * a.hkv + hk) * a.mask_words;
      const unsigned raw = lane < a.mask_words ? __ldg(mrow + lane) : 0u;
      n = rows.init(raw, L, a.prompt_len[b], a.window[b], a.max_pages, a.max_window, a.max_kept,
                    lane);
    } else {
      n = a.kept_cnt[static_cast<size_t>(b) * a.hkv + hk];
      if (L < 1 || L > a.max_pages * kPage) n = -DSA_DEV_BAD_SEQ_LEN;
      else if (n < 1 || n > a.max_kept || n > L) n = -DSA_DEV_BAD_COUNT;
    }
    if (n < 0) {
      if (part == 0) {
        if (threadIdx.x == 0) set_error(a.err, -n);
        poison(b, hk);
      }
      return;
    }
    const int nt = (n + 15) >> 4;
    const int per = (nt + a.parts - 1) / a.parts, nparts = (nt + per - 1) / per;
    if (part >= nparts) return;
    const Segment sg{b, hk, L, n, part * per, min(nt, (part + 1) * per)};
    scan(sg, spec, qv);
    const int slot0 = unit * a.parts;
    finish(sg, nparts == 1 ? -1 : slot0 + part, unit, nparts, slot0, slot0, 1);
  }
};

// Resident CTAs per SM the register budget allows for: 16 warps of the bf16 builds at D = 128
// (128 registers a thread), 12 with fp32 q (its second halves), more at D = 64.
constexpr int resident_ctas(int d, bool xq, int nw) {
  return (d == 128 ? (xq ? 12 : 16) : (xq ? 16 : 24)) / nw;
}

template <int D, int MODE, bool XQ, int NW>
__global__ void __launch_bounds__(NW * 32, (resident_ctas(D, XQ, NW)))
    quant_decode_kernel(const QuantDecodeLaunch a) {
  extern __shared__ __align__(128) unsigned char smem[];
  griddep_wait();
  griddep_launch_dependents();
  QuantDecode<D, MODE, XQ, NW> k(a, smem);
  if constexpr (MODE == kModeDense) k.run_dense();
  else k.run_sparse();
}

// Parts of a unit of sparse rows: one CTA per unit unless the batch would leave
// more than half of the resident slots empty; a part keeps a tile for each warp.
int sparse_parts(int64_t units, int64_t slots, int max_kept) {
  if (units < 1 || units * 2 > slots || units > kMultiCounters) return 1;
  int64_t parts = slots / units;
  const int64_t most = (max_kept + 63) / 64;
  if (parts > most) parts = most;
  if (parts > kQuantMaxParts) parts = kQuantMaxParts;
  return parts < 1 ? 1 : static_cast<int>(parts);
}

template <int D, int MODE, bool XQ, int NW>
cudaError_t launch_one(QuantDecodeLaunch a, cudaStream_t s) {
  auto kern = quant_decode_kernel<D, MODE, XQ, NW>;
  constexpr int smem = QuantRing<D, NW>::kSmem;
  static KernelSlots cache;
  int per_sm = 0;
  const cudaError_t e = cache.get(reinterpret_cast<const void*>(kern), NW * 32, smem, &per_sm);
  if (e != cudaSuccess) return e;
  const int64_t slots = static_cast<int64_t>(per_sm) * a.sms;
  const int64_t units = static_cast<int64_t>(a.batch) * a.hkv;
  int64_t grid;
  if (MODE == kModeDense) {
    a.min_tiles = kQuantMinTiles;
    int64_t most = (units * a.max_pages + kQuantMinTiles - 1) / kQuantMinTiles;
    if (most < units) most = units;
    grid = slots < most ? slots : most;
    // two slots of partials and one counter for each CTA
    const int64_t fit = a.part_cap / (2 * quant_part_floats(a.group, D));
    if (grid > fit) grid = fit;
    if (grid > kMultiCounters) grid = kMultiCounters;
    if (grid < 1) grid = 1;
  } else {
    a.parts = sparse_parts(units, slots, a.max_kept);
    if (units * a.parts * quant_part_floats(a.group, D) > a.part_cap) a.parts = 1;
    grid = units * a.parts;
  }
  return launch_pdl(kern, dim3(static_cast<unsigned>(grid)), dim3(NW * 32),
                    static_cast<size_t>(smem), s, a);
}

// Warps per CTA: 2 once there are units enough, else 4.  A unit's start and end (sizes, mask,
// first pages, the join of the warps: 3 us under load) are then paid by half as many warps,
// but a unit cut over CTAs leaves twice the partial states.  Sparse rows, a unit per CTA:
// enough is half of the resident slots; 2048 units of 290 rows 33.3 us against 36.5, 640
// units of 140 rows 9.1 against 9.9.  Dense rows, equal shares: all of the slots; 960 units
// of 1 .. 165 rows 15.4 us against 20.8, 2048 of 100 .. 300 24.0 against 28.6, the mixed
// batch's 1024 of 33 .. 4608 100.5 either way -- but 512 of 1 .. 40 11.5 against 10.5, 256 of
// 200 .. 600 15.3 against 13.8, 64 of 8000 39 against 30.  (8 warps: 106 on the mixed batch.)
template <int D, int MODE, bool XQ>
cudaError_t launch_warps(const QuantDecodeLaunch& a, cudaStream_t s) {
  const int64_t units = static_cast<int64_t>(a.batch) * a.hkv;
  return units * (MODE == kModeDense ? 1 : 2) > static_cast<int64_t>(resident_ctas(D, XQ, 4)) * a.sms
             ? launch_one<D, MODE, XQ, 2>(a, s)
             : launch_one<D, MODE, XQ, 4>(a, s);
}

template <int D, bool XQ>
cudaError_t launch_mode(const QuantDecodeLaunch& a, int mode, cudaStream_t s) {
  if (mode == kModeDense) return launch_warps<D, kModeDense, XQ>(a, s);
  if (mode == kModeList) return launch_warps<D, kModeList, XQ>(a, s);
  return launch_warps<D, kModeMask, XQ>(a, s);
}

}  // namespace

cudaError_t launch_quant_decode(const QuantDecodeLaunch& a, int mode, cudaStream_t s) {
  if (a.head_dim == 128)
    return a.q_bf16 ? launch_mode<128, false>(a, mode, s) : launch_mode<128, true>(a, mode, s);
  if (a.head_dim == 64)
    return a.q_bf16 ? launch_mode<64, false>(a, mode, s) : launch_mode<64, true>(a, mode, s);
  return cudaErrorInvalidValue;
}

}  // namespace dsa
