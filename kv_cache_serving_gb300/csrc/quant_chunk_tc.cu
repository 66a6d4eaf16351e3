// quant_chunk_tc.cu -- several query tokens per request over the 8-bit paged K/V cache
// on the 5th-generation tensor cores (head_dim 128).
//
// Mathematics as in quant_chunk.cu.  A CTA holds N = 32 or 64 columns (query token,
// head of the kv head's group) of one (request, kv head) and walks its pages in blocks
// of 8 (128 rows).  Per block, both products have the rows or the head's dims on the 128
// lanes of tensor memory and the columns along it:
//   S  (128 rows x N) = K (128 x 128) Q^T,      O^T (128 dims x N) += V^T (128 x 128 rows) P
// so any number of columns fits without waste, a row's scales and its place in the
// mask are constants of a thread, and the weights (rows x columns) are written as they
// are held: a thread stores its row's columns side by side, which is the B operand with
// the contraction in the rows.
//
// K and V become fp16 on the way into shared memory (a warp converts one page: 4 loads
// of 512 bytes, swizzled 16-byte stores), once for all N columns.  q enters as fp16
// scaled by one power of two per CTA.  The softmax of a block is 128 N elements over 256
// threads: z = s * (q and K scale) + (log2 of the V scale - reference), weight 2^z, sum +=
// weight / V scale.  The reference of a column moves only when a weight would pass 2^15
// (a vote at the barrier the block has anyway); then the sums and the accumulators in
// tensor memory are rescaled.
//
// What bounds it: instruction issue in the conversion and the softmax (about 2100
// instructions per block of 128 rows x 64 columns against 512 cycles of MMA).  Two CTAs
// per SM, so that one converts while the other's products run; loads of the next block
// are in flight during the softmax.
#include <math.h>

#include "common.cuh"
#include "host.h"
#include "internal.h"
#include "mma.cuh"
#include "quant.cuh"
#include "tcgen05.cuh"

namespace dsa {
namespace {

constexpr int kTD = 128;           // head_dim
constexpr int kTRows = 128;        // rows per block
constexpr int kTPages = 8;         // pages per block: one per warp
constexpr int kTThreads = 256;
constexpr float kTHead = 4.f;      // the reference stands for 2^4

template <int N>
struct TcShape {
  static constexpr int kHalf = kTRows * 128;             // 64 dims of a block, fp16
  static constexpr int kK = 0, kV = 2 * kHalf;
  static constexpr int kPRow = N * 2;                      // bytes of a row of weights
  static constexpr int kP = 4 * kHalf;
  static constexpr int kQ = kP + kTRows * kPRow;           // two halves of N rows x 128 B
  static constexpr int kInfo = kQ + 2 * N * 128;           // 2 x 8 int4: needed rows, scales
  static constexpr int kRef = kInfo + 2 * kTPages * 16;    // ref, head - ref, factor: N each
  static constexpr int kMax = kRef + 3 * N * 4;            // 4 x N column maxima / sums
  static constexpr int kRed = kMax + 4 * N * 4;            // 8 floats
  static constexpr int kBar = kRed + 32;                   // two barriers, address, flag
  static constexpr int kMask = kBar + 32;
  static constexpr int kSlack = 1024;                      // the base is rounded up to 1024
  static constexpr int kTmem = 2 * N;                      // S, then O^T
  static int smem(int words) { return kSlack + kMask + 4 * words; }
};

__device__ __forceinline__ void sts128(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y),
               "r"(v.z), "r"(v.w)
               : "memory");
}

// 16 codes as two 16-byte pieces of fp16.
__device__ __forceinline__ void codes16(const uint4& v, uint4& lo, uint4& hi) {
  lo = make_uint4(e4m3x2_f16x2(v.x), e4m3x2_f16x2_hi(v.x), e4m3x2_f16x2(v.y), e4m3x2_f16x2_hi(v.y));
  hi = make_uint4(e4m3x2_f16x2(v.z), e4m3x2_f16x2_hi(v.z), e4m3x2_f16x2(v.w), e4m3x2_f16x2_hi(v.w));
}

// Maximum over the warp of each of W values: lane l ends with value l * W / 32.
template <int W>
__device__ __forceinline__ float scatter_max(float (&v)[W], int lane) {
#pragma unroll
  for (int n = W, off = 16; n > 1; n >>= 1, off >>= 1) {
    const bool hi = (lane & off) != 0;
#pragma unroll
    for (int i = 0; i < n / 2; ++i) {
      const float send = hi ? v[i] : v[i + n / 2], keep = hi ? v[i + n / 2] : v[i];
      v[i] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, send, off));
    }
  }
  float m = v[0];
#pragma unroll
  for (int off = 32 / W / 2; off >= 1; off >>= 1)
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
  return m;
}

template <int N>
__global__ void __launch_bounds__(kTThreads, 2) quant_chunk_tc_kernel(const QuantChunkLaunch a) {
  using Sh = TcShape<N>;
  constexpr int W = N / 2;  // columns per warp
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  const uint32_t sm = smem_addr(smem);
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int wq = warp & 3, cg = warp >> 2;  // lane quarter of tensor memory, column half
  const int unit = blockIdx.x;
  const int qt = a.q_tiles - 1 - unit % a.q_tiles;
  const int hk = unit / a.q_tiles % a.hkv, bpos = unit / (a.q_tiles * a.hkv);
  const int b = a.order != nullptr ? __ldg(a.order + bpos) : bpos;
  if (static_cast<unsigned>(b) >= static_cast<unsigned>(a.batch)) {
    if (qt == 0 && hk == 0 && tid == 0) set_error(a.err, DSA_DEV_BAD_ORDER);
    return;
  }
  const int lg = a.group_log2, per_cta = N >> lg, t0 = qt * per_cta;
  const int L = a.seq_len[b], n = a.q_len[b], P = a.prompt_len[b], Wn = a.window[b];
  int code = 0;
  if (L < 1 || L > a.max_pages * kPage) code = DSA_DEV_BAD_SEQ_LEN;
  else if (n < 0 || n > L || n > a.max_q) code = DSA_DEV_BAD_QLEN;
  else if (P < 0) code = DSA_DEV_BAD_PROMPT;
  else if (Wn < 0 || Wn > a.max_window) code = DSA_DEV_BAD_WINDOW;
  if (code != 0) {
    // q_len is not trusted: NaN into every slot of the unit
    if (qt == 0 && hk == 0 && tid == 0) set_error(a.err, code);
    const int heads = 1 << lg;
    for (int x = tid; x < N * kTD; x += kTThreads) {
      const int t = t0 + x / (heads * kTD);
      if (t >= a.max_q) break;
      const size_t qh =
          (static_cast<size_t>(b) * a.max_q + t) * a.hq + hk * heads + x / kTD % heads;
      a.out[qh * kTD + x % kTD] = 0x7fc0;
      if (a.lse != nullptr && x % kTD == 0) a.lse[qh] = __int_as_float(0x7fc00000);
    }
    return;
  }
  if (t0 >= n) return;
  const int t1 = min(t0 + per_cta, n);
  const int i_first = L - n + t0, i_last = L - n + t1 - 1;
  const int n_prompt = min(P, i_last + 1);
  const int pa = (n_prompt + 15) >> 4;
  const int pb = max(pa, max(i_first - Wn, 0) >> 4), pe = i_last >> 4;
  const int pages = pa + max(0, pe - pb + 1);
  const int nblocks = (pages + kTPages - 1) / kTPages;
  auto page_of = [&](int x) { return x < pa ? x : pb + (x - pa); };

  int4* info = reinterpret_cast<int4*>(smem + Sh::kInfo);
  float* ref = reinterpret_cast<float*>(smem + Sh::kRef);
  float* nref = ref + N;
  float* fac = ref + 2 * N;
  float* cmax = reinterpret_cast<float*>(smem + Sh::kMax);
  float* red = reinterpret_cast<float*>(smem + Sh::kRed);
  uint64_t* s_done = reinterpret_cast<uint64_t*>(smem + Sh::kBar);
  uint64_t* o_done = s_done + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(s_done + 2);
  volatile int* failed = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint32_t* msk = reinterpret_cast<uint32_t*>(smem + Sh::kMask);
  if (warp == 0) tmem_alloc<Sh::kTmem>(tmem_slot);
  if (tid == 0) {
    mbar_init(s_done, 1);
    mbar_init(o_done, 1);
    fence_mbar_init();
    *failed = 0;
  }
  // the mask shifted by one: bit o keeps offset o, 0 (the query itself) and 1 .. window
  {
    const uint32_t* mrow = a.keep_mask + (static_cast<size_t>(b) * a.hkv + hk) * a.mask_words;
    for (int x = tid; x < a.max_window / 32 + 1; x += kTThreads) {
      const uint32_t lo = x == 0 ? 0x80000000u : __ldg(mrow + x - 1);
      const uint32_t hi = x < a.mask_words ? __ldg(mrow + x) : 0u;
      uint32_t v = (hi << 1) | (lo >> 31);
      const int live = Wn + 1 - 32 * x;
      if (live < 32) v = live <= 0 ? 0u : v & ((1u << live) - 1u);
      msk[x] = v;
    }
  }
  if (tid < N) {
    ref[tid] = -INFINITY;
    nref[tid] = INFINITY;
  }

  // q: a thread holds 128 N / 256 elements of one column
  constexpr int kTpc = kTThreads / N;       // threads per column
  constexpr int kQE = kTD / kTpc;           // elements per thread
  const int qcol = tid / kTpc, qd0 = (tid % kTpc) * kQE;
  uint4 qv[kQE / 8];
  {
    const int t = t0 + (qcol >> lg);
    const size_t qh =
        (static_cast<size_t>(b) * a.max_q + t) * a.hq + (hk << lg) + (qcol & ((1 << lg) - 1));
    const uint4* p = reinterpret_cast<const uint4*>(a.q + qh * kTD + qd0);
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < kQE / 8; ++i) {
      qv[i] = t < t1 ? __ldg(p + i) : make_uint4(0u, 0u, 0u, 0u);
      const uint32_t w[4] = {qv[i].x, qv[i].y, qv[i].z, qv[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k)
        amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(w[k])), fabsf(bf16_hi(w[k]))));
    }
    amax = warp_max(amax);
    if (lane == 0) red[warp] = amax;
  }
  __syncthreads();  // mask, references, maxima, tensor-memory address
  const uint32_t tmem = *tmem_slot;
  float amax = red[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) amax = fmaxf(amax, red[i]);
  const int qe = q_exponent(amax);
  const float f = a.scale_log2 * pow2i(qe);
  {
    const float down = pow2i(-qe);
#pragma unroll
    for (int i = 0; i < kQE / 8; ++i) {
      const uint32_t w[4] = {qv[i].x, qv[i].y, qv[i].z, qv[i].w};
      uint32_t h[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) h[k] = f16x2_rn(bf16_lo(w[k]) * down, bf16_hi(w[k]) * down);
      const int d = qd0 + 8 * i, piece = (d & 63) >> 3;
      sts128(sm + Sh::kQ + (d >> 6) * (N * 128) + qcol * 128 + ((piece ^ (qcol & 7)) << 4),
             make_uint4(h[0], h[1], h[2], h[3]));
    }
  }

  const int32_t* pt = a.page_table + static_cast<size_t>(b) * a.max_pages;
  auto load_page = [&](int blk) {
    const int x = blk * kTPages + warp;
    return x < pages ? __ldg(pt + page_of(x)) : 0;
  };
  // Rows of this warp's page of block blk that some query of the CTA keeps.
  auto rows_needed = [&](int blk) -> unsigned {
    const int x = blk * kTPages + warp;
    if (x >= pages) return 0u;
    const int j = page_of(x) * 16 + (lane & 15);
    bool need = j <= i_last;
    if (need && j >= P && j < i_first) {
      const int lo = i_first - j, hi = min(Wn, i_last - j);
      need = false;
      for (int w = lo >> 5; w <= (hi >> 5) && lo <= hi; ++w) {
        uint32_t v = msk[w];
        if (w == (lo >> 5)) v &= 0xffffffffu << (lo & 31);
        if (w == (hi >> 5) && (hi & 31) != 31) v &= (2u << (hi & 31)) - 1u;
        need |= v != 0u;
      }
    }
    return __ballot_sync(0xffffffffu, need) & 0xffffu;
  };
  const int ch = lane & 7, r8 = lane >> 3;
  // Codes of this lane: rows 4 i + lane / 8 of the page, piece lane % 8.
  auto load_codes = [&](const uint8_t* base, size_t ph, unsigned need, uint4 (&v)[4]) {
    const uint4* p = reinterpret_cast<const uint4*>(base + ph * (16 * kTD)) + lane;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = (need >> (4 * i + r8)) & 1u ? __ldg(p + 32 * i) : make_uint4(0u, 0u, 0u, 0u);
  };
  // The same as fp16 into a block's tile (rows 16 warp .. + 15): 64-dim halves of 128
  // rows, 16-byte pieces swizzled by the row.  The lanes of the second half write their
  // odd piece first, so that the 8 lanes of a row cover all banks.
  auto store_f16 = [&](uint32_t tile, const uint4 (&v)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint4 lo, hi;
      codes16(v[i], lo, hi);
      const int r = 16 * warp + 4 * i + r8, c16 = 2 * (ch & 3);
      const uint32_t row = tile + (ch >> 2) * Sh::kHalf + r * 128;
      const uint32_t at0 = row + ((c16 ^ (r & 7)) << 4), at1 = row + (((c16 + 1) ^ (r & 7)) << 4);
      const bool odd = ch >= 4;
      sts128(odd ? at1 : at0, odd ? hi : lo);
      sts128(odd ? at0 : at1, odd ? lo : hi);
    }
  };
  auto check_page = [&](unsigned& need, int pg) -> size_t {
    if (need != 0u && static_cast<unsigned>(pg) >= static_cast<unsigned>(a.num_pages)) {
      set_error(a.err, DSA_DEV_BAD_PAGE);
      need = 0u;
    }
    return need != 0u ? static_cast<size_t>(pg) * a.hkv + hk : 0;
  };
  auto put_info = [&](int blk, unsigned need, size_t ph) {
    if (lane == 0) {
      // rows nobody needs: scales of one
      uint32_t ks = 0x3f800000u, vs = 0x3f800000u;
      if (need != 0u) {
        ks = __float_as_uint(__ldg(a.k_scale + ph));
        vs = __float_as_uint(__ldg(a.v_scale + ph));
        if (!scale_ok(ks) || !scale_ok(vs)) set_error(a.err, DSA_DEV_BAD_SCALE);
      }
      info[(blk & 1) * kTPages + warp] =
          make_int4(static_cast<int>(need), static_cast<int>(ks), static_cast<int>(vs), 0);
    }
  };
  constexpr uint32_t kIdS = tc_idesc(128, N, false), kIdO = tc_idesc(128, N, true);
  auto issue_s = [&]() {  // S = K Q^T
#pragma unroll
    for (int k = 0; k < 8; ++k)
      tc_mma_f16(tmem,
                 tc_desc(sm + Sh::kK + (k >> 2) * Sh::kHalf + (k & 3) * 32, 16, 1024, kSwizzle128),
                 tc_desc(sm + Sh::kQ + (k >> 2) * (N * 128) + (k & 3) * 32, 16, 1024, kSwizzle128),
                 kIdS, k > 0);
    tc_commit(s_done);
  };
  auto issue_o = [&](bool first) {  // O^T += V^T P
#pragma unroll
    for (int k = 0; k < 8; ++k)
      tc_mma_f16(tmem + N, tc_desc(sm + Sh::kV + k * 2048, Sh::kHalf, 1024, kSwizzle128),
                 tc_desc(sm + Sh::kP + k * (16 * Sh::kPRow), 16, 8 * Sh::kPRow,
                         N == 64 ? kSwizzle128 : kSwizzle64),
                 kIdO, !first || k > 0);
    tc_commit(o_done);
  };

  uint4 kreg[4], vreg[4];
  int pg = load_page(0);
  {
    unsigned need = rows_needed(0);
    const size_t ph = check_page(need, pg);
    load_codes(a.k, ph, need, kreg);
    load_codes(a.v, ph, need, vreg);
    put_info(0, need, ph);
  }
  pg = load_page(1);
  store_f16(sm + Sh::kK, kreg);
  fence_proxy_async_smem();
  __syncthreads();
  if (tid == 0) {
    tc_fence_after();
    issue_s();
  }

  // this thread's row of a block: lane 32 wq + lane of tensor memory
  const int row = 32 * wq + lane;
  const uint32_t t_lane = tmem + (static_cast<uint32_t>(32 * wq) << 16) + cg * W;
  f32x2 l[W / 2];
#pragma unroll
  for (int i = 0; i < W / 2; ++i) l[i] = pack2(0.f, 0.f);
  bool ok = true;
  for (int blk = 0; blk < nblocks && ok; ++blk) {
    // next block's K on its way, then this block's V into shared memory
    unsigned need = 0;
    size_t ph = 0;
    if (blk + 1 < nblocks) {
      need = rows_needed(blk + 1);
      ph = check_page(need, pg);
      load_codes(a.k, ph, need, kreg);
    }
    if (blk > 0) ok = mbar_wait(o_done, (blk - 1) & 1);
    store_f16(sm + Sh::kV, vreg);
    if (blk + 1 < nblocks) {
      load_codes(a.v, ph, need, vreg);
      put_info(blk + 1, need, ph);
      pg = load_page(blk + 2);
    }
    ok = mbar_wait(s_done, blk & 1) && ok;
    if (!ok) *failed = 1;
    tc_fence_after();

    // softmax of the block: this thread's row, W columns
    const int x = blk * kTPages + (row >> 4);
    const int4 in = info[(blk & 1) * kTPages + (row >> 4)];
    const int j = x < pages ? page_of(x) * 16 + (row & 15) : 0;
    const bool here = (in.x >> (row & 15)) & 1;
    const float c1 = f * __uint_as_float(static_cast<uint32_t>(in.y));
    const float lv = static_cast<float>(scale_exp(static_cast<uint32_t>(in.z)));
    const float inv = __uint_as_float((254u << 23) - static_cast<uint32_t>(in.z));
    const int tok0 = (cg * W) >> lg;  // token of the warp's first column
    uint32_t keep = here ? 0xffffffffu : 0u;  // bit c: column cg W + c keeps this row
    const bool all = __all_sync(0xffffffffu, here && j < P && j <= i_first);
    if (!all && here) {
      // bit t of `win`: token tok0 + t keeps the row, for the tokens of W columns
      const int o0 = i_first + tok0 - j;  // offset of the first of them
      uint32_t win;
      if (j < P) {
        win = 0xffffffffu;
      } else {
        const int w0 = max(o0, 0) >> 5, sh = max(o0, 0) & 31, last = a.max_window / 32;
        const uint32_t lo = w0 <= last ? msk[w0] : 0u, hi = w0 < last ? msk[w0 + 1] : 0u;
        win = __funnelshift_r(lo, hi, sh);
      }
      if (o0 < 0) win = o0 <= -32 ? 0u : win << -o0;
      if (lg == 0) {
        keep = win;
      } else {
        keep = 0u;
        const uint32_t ones = (1u << (1 << lg)) - 1u;
#pragma unroll
        for (int t = 0; t < W / 2; ++t)
          if (t < (W >> lg)) keep |= ((win >> t) & 1u) ? ones << (t << lg) : 0u;
      }
    }
    float p[W];
    uint32_t h[W / 2];
    auto softmax = [&]() -> bool {
      uint32_t s[W];
      tmem_load<W>(t_lane, s);
      tc_wait_ld();
      const f32x2 c2 = pack2(c1, c1), lv2 = pack2(lv, lv);
      uint32_t top = 0u;
#pragma unroll
      for (int i = 0; i < W / 2; i += 2) {
        const float4 r = *reinterpret_cast<const float4*>(nref + cg * W + 2 * i);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int c = 2 * (i + k);
          const f32x2 z2 = fma2(pack2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), c2,
                                add2(k == 0 ? pack2(r.x, r.y) : pack2(r.z, r.w), lv2));
          unpack2(z2, p[c], p[c + 1]);
        }
      }
      if (!all) {
#pragma unroll
        for (int c = 0; c < W; ++c) p[c] = (keep >> c) & 1u ? p[c] : -INFINITY;
      }
#pragma unroll
      for (int i = 0; i < W / 2; ++i) {
        p[2 * i] = ex2_approx(p[2 * i]);
        p[2 * i + 1] = ex2_approx(p[2 * i + 1]);
        h[i] = f16x2_rn(p[2 * i], p[2 * i + 1]);
        top = hmax2(top, h[i]);
      }
      // weights of 2^15 and more (0x7800 as fp16): the reference has to move
      return (top & 0xffffu) >= 0x7800u || (top >> 16) >= 0x7800u;
    };
    auto store_p = [&]() {
      const uint32_t at = sm + Sh::kP + row * Sh::kPRow;
#pragma unroll
      for (int i = 0; i < W / 8; ++i) {
        const int piece = cg * (W / 8) + i;
        const int sw = N == 64 ? piece ^ (row & 7) : piece ^ ((row >> 1) & 3);
        sts128(at + (sw << 4), make_uint4(h[4 * i], h[4 * i + 1], h[4 * i + 2], h[4 * i + 3]));
      }
    };
    const bool over = softmax();
    store_p();
    if (blk + 1 < nblocks) store_f16(sm + Sh::kK, kreg);  // S of this block is done with K
    fence_proxy_async_smem();
    tc_fence_before();
    if (__syncthreads_or(over)) {
      // column maxima over the block, new references, everything so far rescaled
      tc_fence_after();
      {
        uint32_t s[W];
        tmem_load<W>(t_lane, s);
        tc_wait_ld();
        float y[W];
#pragma unroll
        for (int c = 0; c < W; ++c)
          y[c] = (keep >> c) & 1u ? fmaf(__uint_as_float(s[c]), c1, lv) : -INFINITY;
        const float m = scatter_max<W>(y, lane);
        if (lane % (32 / W) == 0) cmax[wq * N + cg * W + lane / (32 / W)] = m;
      }
      __syncthreads();
      if (tid < N) {
        float m = ref[tid];
        const float was = m;
#pragma unroll
        for (int q = 0; q < 4; ++q) m = fmaxf(m, cmax[q * N + tid]);
        fac[tid] = m == was ? 1.f : ex2_approx(was - m);
        ref[tid] = m;
        nref[tid] = kTHead - m;
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < W / 2; ++i)
        l[i] = mul2(l[i], *reinterpret_cast<const f32x2*>(fac + cg * W + 2 * i));
      if (blk > 0) {
        uint32_t o[W];
        tmem_load<W>(t_lane + N, o);
        tc_wait_ld();
#pragma unroll
        for (int c = 0; c < W; ++c)
          o[c] = __float_as_uint(__uint_as_float(o[c]) * fac[cg * W + c]);
#pragma unroll
        for (int c = 0; c < W; c += 16) tmem_store16(t_lane + N + c, o + c);
        tc_wait_st();
      }
      softmax();
      store_p();
      fence_proxy_async_smem();
      tc_fence_before();
      __syncthreads();
    }
    const f32x2 inv2 = pack2(here ? inv : 0.f, here ? inv : 0.f);
#pragma unroll
    for (int i = 0; i < W / 2; ++i) l[i] = fma2(pack2(p[2 * i], p[2 * i + 1]), inv2, l[i]);
    ok = *failed == 0;
    if (tid == 0 && ok) {
      tc_fence_after();
      issue_o(blk == 0);
      if (blk + 1 < nblocks) issue_s();
    }
  }
  if (ok) ok = mbar_wait(o_done, (nblocks - 1) & 1);
  if (!ok) *failed = 1;
  // sums of the columns over all rows
  {
    float v[W];
#pragma unroll
    for (int i = 0; i < W / 2; ++i) unpack2(l[i], v[2 * i], v[2 * i + 1]);
    const float t = reduce_scatter<W>(v, lane);
    if (lane % (32 / W) == 0) cmax[wq * N + cg * W + lane / (32 / W)] = t;
  }
  __syncthreads();
  ok = *failed == 0;
  if (ok) {
    if (tid < N) {
      const float t = cmax[tid] + cmax[N + tid] + cmax[2 * N + tid] + cmax[3 * N + tid];
      fac[tid] = 1.f / t;
      const int tk = t0 + (tid >> lg);
      if (a.lse != nullptr && tk < t1)
        a.lse[(static_cast<size_t>(b) * a.max_q + tk) * a.hq + (hk << lg) +
              (tid & ((1 << lg) - 1))] = (ref[tid] - kTHead + log2f(t)) * kLn2;
    }
    __syncthreads();
    tc_fence_after();
    uint32_t o[W];
    tmem_load<W>(t_lane + N, o);
    tc_wait_ld();
    // lane pairs exchange columns: an even lane stores column c, dims row and row + 1,
    // its neighbour column c + 1
    const int odd = lane & 1;
#pragma unroll
    for (int c = 0; c < W; c += 2) {
      const float u = __uint_as_float(o[c]) * fac[cg * W + c];
      const float v = __uint_as_float(o[c + 1]) * fac[cg * W + c + 1];
      const float got = __shfl_xor_sync(0xffffffffu, odd ? u : v, 1);
      const uint32_t w = odd ? bf16x2_rn(got, v) : bf16x2_rn(u, got);
      const int col = cg * W + c + odd, tk = t0 + (col >> lg);
      if (tk < t1) {
        const size_t qh =
            (static_cast<size_t>(b) * a.max_q + tk) * a.hq + (hk << lg) + (col & ((1 << lg) - 1));
        *reinterpret_cast<uint32_t*>(a.out + qh * kTD + (row & ~1)) = w;
      }
    }
    tc_fence_before();
  } else {
    // give products in flight a bounded time to finish before the memory goes back
    if (tid == 0) set_error(a.err, DSA_DEV_TIMEOUT);
    mbar_wait(o_done, (nblocks - 1) & 1);
    tc_fence_before();
  }
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc<Sh::kTmem>(tmem);
  }
}

template <int N>
cudaError_t launch_one(QuantChunkLaunch a, cudaStream_t s) {
  auto kern = quant_chunk_tc_kernel<N>;
  const int smem = TcShape<N>::smem(a.max_window / 32 + 1);
  static KernelSlots cache;
  int per_sm = 0;
  const cudaError_t e =
      cache.get(reinterpret_cast<const void*>(kern), kTThreads, smem, &per_sm);
  if (e != cudaSuccess) return e;
  const int per_cta = N >> a.group_log2;
  a.q_tiles = (a.max_q + per_cta - 1) / per_cta;
  a.parts = 1;
  const int64_t units = static_cast<int64_t>(a.q_tiles) * a.hkv * a.batch;
  if (units > INT32_MAX) return cudaErrorInvalidValue;
  return launch_pdl(kern, dim3(static_cast<unsigned>(units)), dim3(kTThreads),
                    static_cast<size_t>(smem), s, a);
}

// Columns per CTA, and the CTAs of a call.
int columns(const QuantChunkLaunch& a) {
  return (static_cast<int64_t>(a.max_q) << a.group_log2) <= 32 ? 32 : 64;
}

}  // namespace

// A unit here is never cut along its pages, so this kernel needs as many units as
// fill the GPU at least in part.
bool quant_chunk_tc_fits(const QuantChunkLaunch& a) {
  if (a.split_setting != 0) return a.split_setting == 1;
  const int per_cta = columns(a) >> a.group_log2;
  const int64_t units =
      static_cast<int64_t>((a.max_q + per_cta - 1) / per_cta) * a.hkv * a.batch;
  return units * 2 >= a.sms;
}

cudaError_t launch_quant_chunk_tc(const QuantChunkLaunch& a, cudaStream_t s) {
  return columns(a) == 32 ? launch_one<32>(a, s) : launch_one<64>(a, s);
}

}  // namespace dsa
