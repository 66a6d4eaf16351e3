// quant_chunk_tc.cu -- several query tokens per request over the 8-bit paged K/V cache
// on the 5th-generation tensor cores (head_dim 128), for chunks of up to 32 (query token,
// head) columns: speculative steps, the rows of an image.
//
// Mathematics as in quant_chunk.cu.  A CTA holds the 32 columns of one (request, kv head)
// and walks its pages in blocks of 8 (128 rows).  Per block, both products have the rows
// or the head's dims on the 128 lanes of tensor memory and the columns along it:
//   S  (128 rows x 32) = K (128 x 128) Q^T,    O^T (128 dims x 32) += V^T (128 x 128 rows) P
// so few columns fit without the waste of queries on 128 lanes, a row's scales and its
// place in the mask are constants of a thread, and the weights (rows x columns) are written
// as they are held: a thread stores its row's columns side by side, which is the B operand
// with the contraction in the rows.
//
// K and V become fp16 on the way into shared memory (a warp converts one page: 4 loads
// of 512 bytes, swizzled 16-byte stores), once for all columns.  q enters as fp16, a column
// scaled by its own power of two.  The softmax of a block is 128 x 32 elements over 256
// threads: z = s * (q and K scale) + (log2 of the V scale - reference), weight 2^z, sum +=
// weight / V scale.  The reference of a column moves only when a weight would pass 2^15
// (a vote at the barrier the block has anyway); then the sums and the accumulators in
// tensor memory are rescaled.
//
// What bounds it: latency and instruction issue between the products, not the products (6%
// of the tensor pipe): a block's chain is V into shared memory, S awaited, K, softmax,
// barrier, products, about 700 instructions per warp at 16 warps per SM, of which the
// conversions are 130 and the softmax 300.  Two CTAs per SM, so that one converts while the
// other's products run; the next block's K and V are loaded an iteration ahead, past the
// L1 (whose 20 KB keep page ids, masks and spills).  Measured: 32 tokens of 64 requests of 320 ..
// 1280 rows under the mask, 32/32 heads: 91 us with a flushed L2 (136 with quant_chunk.cu).  A
// persistent form (tiles of several units in one CTA, the next tile's q and first block ahead)
// measured slower: 141 us, its second set of tile values spills.
#include <math.h>

#include "common.cuh"
#include "host.h"
#include "internal.h"
#include "mma.cuh"
#include "quant.cuh"
#include "quant_redo.cuh"
#include "tcgen05.cuh"

namespace dsa {
namespace {

constexpr int kTD = 128;           // head_dim
constexpr int kTRows = 128;        // rows per block
constexpr int kTPages = 8;         // pages per block: one per warp
constexpr int kTCols = 32;         // columns: (query token, head of the group)
constexpr int kTThreads = 256;
constexpr float kTHead = 4.f;      // the reference stands for 2^4

struct TcShape {
  static constexpr int kHalf = kTRows * 128;             // 64 dims of a block, fp16
  static constexpr int kK = 0, kV = 2 * kHalf;
  static constexpr int kPRow = kTCols * 2;                      // bytes of a row of weights
  static constexpr int kP = 4 * kHalf;
  static constexpr int kQ = kP + kTRows * kPRow;           // two halves of kTCols rows x 128 B
  static constexpr int kInfo = kQ + 2 * kTCols * 128;           // 2 x 8 int4: needed rows, scales
  static constexpr int kRef = kInfo + 2 * kTPages * 16;    // ref, head - ref, factor: kTCols each
  static constexpr int kMax = kRef + 3 * kTCols * 4;            // 4 x kTCols column maxima / sums
  static constexpr int kUp = kMax + 4 * kTCols * 4;             // score factor of a column: kTCols floats
  static constexpr int kBar = kUp + 4 * kTCols;                  // two barriers, address, flags
  static constexpr int kMask = kBar + 32;
  static constexpr int kSlack = 1024;                      // the base is rounded up to 1024
  // tensor memory: S, O^T, and two copies of every row's part of the columns' sums
  static constexpr int kS = 0, kO = kTCols, kL = 2 * kTCols, kTmem = 4 * kTCols;
  static int smem(int words) { return kSlack + kMask + 4 * words; }
};

__device__ __forceinline__ void sts128(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y),
               "r"(v.z), "r"(v.w)
               : "memory");
}

// Read once: past the L1, whose few kilobytes beside the tiles hold the page ids and masks.
__device__ __forceinline__ uint2 ld_stream(const uint2* p) {
  uint2 v;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}

// Maximum over the warp of each of 16 values: lane l ends with value l / 2.
__device__ __forceinline__ float scatter_max(float (&v)[16], int lane) {
#pragma unroll
  for (int n = 16, off = 16; n > 1; n >>= 1, off >>= 1) {
    const bool hi = (lane & off) != 0;
#pragma unroll
    for (int i = 0; i < n / 2; ++i) {
      const float send = hi ? v[i] : v[i + n / 2], keep = hi ? v[i + n / 2] : v[i];
      v[i] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, send, off));
    }
  }
  return fmaxf(v[0], __shfl_xor_sync(0xffffffffu, v[0], 1));
}

template <int LG>
struct TcTile {
  static constexpr int kColumns = kTCols;
  __device__ __forceinline__ static void at(const QuantChunkLaunch&, int& bpos, int& hk, int& t0) {
    bpos = blockIdx.z;
    hk = blockIdx.y;
    t0 = blockIdx.x * (kTCols >> LG);
  }
};

template <int LG>
__global__ void __launch_bounds__(kTThreads, 2) quant_chunk_tc_kernel(const QuantChunkLaunch a) {
  using Sh = TcShape;
  constexpr int W = kTCols / 2;              // columns per warp ...
  constexpr int kChunks = W / 16;       // ... in pieces of 16
  constexpr int per_cta = kTCols >> LG;      // query tokens per CTA
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  const uint32_t sm = smem_addr(smem);
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // known to be the warp's
  const int wq = warp & 3, cg = warp >> 2;  // lane quarter of tensor memory, column half
  const int qt = blockIdx.x, hk = blockIdx.y, bpos = blockIdx.z;
  const int b = a.order != nullptr ? __ldg(a.order + bpos) : bpos;
  if (static_cast<unsigned>(b) >= static_cast<unsigned>(a.batch)) {
    if (qt == 0 && hk == 0 && tid == 0) set_error(a.err, DSA_DEV_BAD_ORDER);
    return;
  }
  const int t0 = qt * per_cta;
  const int L = a.seq_len[b], n = a.q_len[b], P = a.prompt_len[b], Wn = a.window[b];
  const int32_t* pt = a.page_table + static_cast<size_t>(b) * a.max_pages;
  // page ids of the first two blocks, should they be the request's first pages
  const int spec0 = warp < a.max_pages ? __ldg(pt + warp) : 0;
  const int spec1 = warp + kTPages < a.max_pages ? __ldg(pt + warp + kTPages) : 0;
  int code = 0;
  if (L < 1 || L > a.max_pages * kPage) code = DSA_DEV_BAD_SEQ_LEN;
  else if (n < 0 || n > L || n > a.max_q) code = DSA_DEV_BAD_QLEN;
  else if (P < 0) code = DSA_DEV_BAD_PROMPT;
  else if (Wn < 0 || Wn > a.max_window) code = DSA_DEV_BAD_WINDOW;
  if (code != 0) {
    // q_len is not trusted: NaN into every slot of the unit
    if (qt == 0 && hk == 0 && tid == 0) set_error(a.err, code);
    for (int x = tid; x < kTCols * kTD; x += kTThreads) {
      const int t = t0 + x / (kTD << LG);
      if (t >= a.max_q) break;
      const size_t qh = (static_cast<size_t>(b) * a.max_q + t) * a.hq + (hk << LG) +
                        (x / kTD & ((1 << LG) - 1));
      a.out[qh * kTD + x % kTD] = 0x7fc0;
      if (a.lse != nullptr && x % kTD == 0) a.lse[qh] = __int_as_float(0x7fc00000);
    }
    return;
  }
  if (t0 >= n) return;
  const int t1 = min(t0 + per_cta, n);
  const int i_first = L - n + t0, i_last = L - n + t1 - 1;
  // pages scanned: those of the prompt rows [0, pa), then those from the window's start
  const int n_prompt = min(P, i_last + 1);
  const int pa = (n_prompt + 15) >> 4;
  const int pb = max(pa, max(i_first - Wn, 0) >> 4), pe = i_last >> 4;
  const int pages = pa + max(0, pe - pb + 1);
  const int nblocks = (pages + kTPages - 1) / kTPages;
  auto page_of = [&](int x) { return x < pa ? x : pb + (x - pa); };
  // row of q and out of column c
  const size_t qh0 = (static_cast<size_t>(b) * a.max_q + t0) * a.hq + (hk << LG);
  auto qh_of = [&](int c) {
    return qh0 + static_cast<size_t>(c >> LG) * a.hq + (c & ((1 << LG) - 1));
  };

  int4* info = reinterpret_cast<int4*>(smem + Sh::kInfo);
  float* ref = reinterpret_cast<float*>(smem + Sh::kRef);
  float* nref = ref + kTCols;
  float* fac = ref + 2 * kTCols;
  float* cmax = reinterpret_cast<float*>(smem + Sh::kMax);
  float* up = reinterpret_cast<float*>(smem + Sh::kUp);
  uint64_t* s_done = reinterpret_cast<uint64_t*>(smem + Sh::kBar);
  uint64_t* o_done = s_done + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(s_done + 2);
  volatile int* failed = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint32_t* msk = reinterpret_cast<uint32_t*>(smem + Sh::kMask);

  // q: a thread holds 128 kTCols / 256 elements of one column
  constexpr int kTpc = kTThreads / kTCols;       // threads per column
  constexpr int kQE = kTD / kTpc;           // elements per thread
  const int qcol = tid / kTpc, qd0 = (tid % kTpc) * kQE;
  uint4 qv[kQE / 8];
  {
    const bool in = t0 + (qcol >> LG) < t1;
    const uint4* p = reinterpret_cast<const uint4*>(a.q + qh_of(qcol) * kTD + qd0);
#pragma unroll
    for (int i = 0; i < kQE / 8; ++i) qv[i] = in ? __ldg(p + i) : make_uint4(0u, 0u, 0u, 0u);
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
  if (warp == 0) tmem_alloc<Sh::kTmem>(tmem_slot);
  if (tid == 0) {
    mbar_init(s_done, 1);
    mbar_init(o_done, 1);
    fence_mbar_init();
    *failed = 0;
  }
  if (tid < 4) quant_redo_clear();
  if (tid < kTCols) {
    ref[tid] = -INFINITY;
    nref[tid] = INFINITY;
  }

  auto load_page = [&](int blk) {
    const int x = blk * kTPages + warp;
    return x < pages ? __ldg(pt + page_of(x)) : 0;
  };
  // Rows of this warp's page of block blk that some query of the CTA keeps.
  auto rows_needed = [&](int blk) -> unsigned {
    const int x = blk * kTPages + warp;
    if (x >= pages) return 0u;
    const int j0 = page_of(x) * 16;
    if (j0 + 15 <= i_last && (j0 + 15 < P || j0 >= i_first)) return 0xffffu;
    const int j = j0 + (lane & 15);
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
  // One page of a block on its way to a warp: the rows needed, the page's index in the
  // pool, its scales (lane 0).
  struct Page {
    unsigned need;
    size_t ph;
    float ks, vs;
  };
  auto open_page = [&](int blk, int pg) -> Page {
    Page p{rows_needed(blk), 0, 1.f, 1.f};
    if (p.need != 0u && static_cast<unsigned>(pg) >= static_cast<unsigned>(a.num_pages)) {
      set_error(a.err, DSA_DEV_BAD_PAGE);
      p.need = 0u;
    }
    if (p.need != 0u) {
      p.ph = static_cast<size_t>(pg) * a.hkv + hk;
      p.ks = __ldg(a.k_scale + p.ph);
      p.vs = __ldg(a.v_scale + p.ph);
    }
    return p;
  };
  // Its codes: this lane's 8 of rows 2 i + lane / 16, piece lane % 16.
  auto load_codes = [&](const uint8_t* base, const Page& p, uint2 (&v)[8]) {
    const uint2* src = reinterpret_cast<const uint2*>(base + p.ph * (16 * kTD)) + lane;
    if (p.need == 0xffffu) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = ld_stream(src + 32 * i);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        v[i] = (p.need >> (2 * i + (lane >> 4))) & 1u ? ld_stream(src + 32 * i) : make_uint2(0u, 0u);
    }
  };
  // The same as fp16 into a block's tile (rows 16 warp .. + 15): 64-dim halves of 128
  // rows of 128 bytes, 16-byte pieces swizzled by the row (conflict-free: 8 lanes write
  // the 8 pieces of one line).
  uint32_t f16_at[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 2 * i + (lane >> 4);
    f16_at[i] = sm + ((lane >> 3) & 1) * Sh::kHalf + (16 * warp + r) * 128 +
                (((lane & 7) ^ r) << 4);
  }
  auto store_f16 = [&](int tile, const uint2 (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      sts128(f16_at[i & 3] + tile + (i >> 2) * 1024,
             make_uint4(e4m3x2_f16x2(v[i].x), e4m3x2_f16x2_hi(v[i].x), e4m3x2_f16x2(v[i].y),
                        e4m3x2_f16x2_hi(v[i].y)));
  };
  auto put_info = [&](int blk, const Page& p) {
    if (lane == 0) {
      const uint32_t ks = __float_as_uint(p.ks), vs = __float_as_uint(p.vs);
      if (!scale_ok(ks) || !scale_ok(vs)) set_error(a.err, DSA_DEV_BAD_SCALE);
      info[(blk & 1) * kTPages + warp] =
          make_int4(static_cast<int>(p.need), static_cast<int>(ks), static_cast<int>(vs), 0);
    }
  };

  // q as fp16, a column (query token, head) scaled by its own power of two: a query's result
  // does not hang on the others of its tile.
  {
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < kQE / 8; ++i) {
      const uint32_t w[4] = {qv[i].x, qv[i].y, qv[i].z, qv[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k)
        amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(w[k])), fabsf(bf16_hi(w[k]))));
    }
#pragma unroll
    for (int o = kTpc / 2; o >= 1; o >>= 1)
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const int qe = q_exponent(amax);
    const float down = pow2i(-qe);
    if (tid % kTpc == 0) up[qcol] = a.scale_log2 * pow2i(qe);
#pragma unroll
    for (int i = 0; i < kQE / 8; ++i) {
      const uint32_t w[4] = {qv[i].x, qv[i].y, qv[i].z, qv[i].w};
      uint32_t h[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) h[k] = f16x2_rn(bf16_lo(w[k]) * down, bf16_hi(w[k]) * down);
      const int d = qd0 + 8 * i, piece = (d & 63) >> 3;
      sts128(sm + Sh::kQ + (d >> 6) * (kTCols * 128) + qcol * 128 + ((piece ^ (qcol & 7)) << 4),
             make_uint4(h[0], h[1], h[2], h[3]));
    }
  }
  __syncthreads();  // mask, references, tensor-memory address
  uint2 kreg[8], vreg[8];
  Page cur = open_page(0, page_of(warp) == warp ? spec0 : load_page(0));
  load_codes(a.k, cur, kreg);
  load_codes(a.v, cur, vreg);
  int pg = page_of(kTPages + warp) == kTPages + warp ? spec1 : load_page(1);
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  constexpr uint32_t kIdS = tc_idesc(128, kTCols, false), kIdO = tc_idesc(128, kTCols, true);
  // Operand descriptors differ by whole multiples of their address unit (16 bytes) from one
  // step of a product to the next, so a step is an addition.
  const uint64_t k_desc = tc_desc(sm + Sh::kK, 16, 1024, kSwizzle128);
  const uint64_t q_desc = tc_desc(sm + Sh::kQ, 16, 1024, kSwizzle128);
  const uint64_t v_desc = tc_desc(sm + Sh::kV, Sh::kHalf, 1024, kSwizzle128);
  const uint64_t p_desc =
      tc_desc(sm + Sh::kP, 16, 8 * Sh::kPRow, kSwizzle64);
  auto issue_s = [&]() {  // S = K Q^T
#pragma unroll
    for (int k = 0; k < 8; ++k)
      tc_mma_f16(tmem + Sh::kS, k_desc + (((k >> 2) * Sh::kHalf + (k & 3) * 32) >> 4),
                 q_desc + (((k >> 2) * (kTCols * 128) + (k & 3) * 32) >> 4), kIdS, k > 0);
    tc_commit(s_done);
  };
  auto issue_o = [&](bool first, int present) {  // O^T += V^T P, a step for each page
#pragma unroll
    for (int k = 0; k < kTPages; ++k)
      if (k < present)
        tc_mma_f16(tmem + Sh::kO, v_desc + (k * 2048 >> 4), p_desc + (k * (16 * Sh::kPRow) >> 4),
                   kIdO, !first || k > 0);
    tc_commit(o_done);
  };

  if (warp < pages) store_f16(Sh::kK, kreg);
  put_info(0, cur);
  // the next block's K and V leave as soon as their registers are free, an iteration
  // before they are wanted
  Page nxt = cur;
  if (nblocks > 1) {
    nxt = open_page(1, pg);
    load_codes(a.k, nxt, kreg);
    pg = load_page(2);
  }
  fence_proxy_async_smem();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    if (elect_one()) issue_s();
    __syncwarp();
  }

  // this thread's row of a block: lane 32 wq + lane of tensor memory
  const int row = 32 * wq + lane;
  const uint32_t t_lane = tmem + (static_cast<uint32_t>(32 * wq) << 16) + cg * W;
  bool ok = true;
  for (int blk = 0; blk < nblocks && ok; ++blk) {
    if (blk > 0) ok = mbar_wait(o_done, (blk - 1) & 1);  // V and the weights are free
    if (blk * kTPages + warp < pages) store_f16(Sh::kV, vreg);
    if (blk + 1 < nblocks) load_codes(a.v, nxt, vreg);
    ok = mbar_wait(s_done, blk & 1) && ok;               // S is there, K is free
    if (!ok) *failed = 1;
    tc_fence_after();
    if (blk + 1 < nblocks) {
      if ((blk + 1) * kTPages + warp < pages) store_f16(Sh::kK, kreg);
      put_info(blk + 1, nxt);
      if (blk + 2 < nblocks) {
        nxt = open_page(blk + 2, pg);
        load_codes(a.k, nxt, kreg);
        pg = load_page(blk + 3);
      }
    }

    // softmax of the block: this thread's row, W columns
    const int x = blk * kTPages + (row >> 4);
    const int4 in = info[(blk & 1) * kTPages + (row >> 4)];
    const int j = x < pages ? page_of(x) * 16 + (row & 15) : 0;
    const bool here = x < pages && ((in.x >> (row & 15)) & 1);
    const float c1 = __uint_as_float(static_cast<uint32_t>(in.y));
    const float lv = static_cast<float>(scale_exp(static_cast<uint32_t>(in.z)));
    const float inv = __uint_as_float((254u << 23) - static_cast<uint32_t>(in.z));
    uint32_t keep = here ? 0xffffffffu : 0u;  // bit c: column cg W + c keeps this row
    const bool some = __any_sync(0xffffffffu, here);  // else: nothing in this warp's rows
    const bool all = __all_sync(0xffffffffu, here && j < P && j <= i_first);
    if (!all && here) {
      // bit t of `win`: the warp's t-th token keeps the row
      const int o0 = i_first + ((cg * W) >> LG) - j;  // offset of the first token
      uint32_t win = 0xffffffffu;
      if (j >= P) {
        const int w0 = max(o0, 0) >> 5, sh = max(o0, 0) & 31, last = a.max_window / 32;
        const uint32_t lo = w0 <= last ? msk[w0] : 0u, hi = w0 < last ? msk[w0 + 1] : 0u;
        win = __funnelshift_r(lo, hi, sh);
      }
      if (o0 < 0) win = o0 <= -32 ? 0u : win << -o0;
      if (LG == 0) {
        keep = win;
      } else {
        keep = 0u;
        constexpr uint32_t ones = (1u << (1 << LG)) - 1u;
#pragma unroll
        for (int t = 0; t < (W >> LG); ++t) keep |= ((win >> t) & 1u) ? ones << (t << LG) : 0u;
      }
    }
    // The first block: a column's reference is its score with the block's first row
    // if it keeps that row (a maximum would need a reduction over the rows; a
    // reference too low is found out like any other).
    if (blk == 0) {
      if (wq == 0) {
#pragma unroll
        for (int q = 0; q < kChunks; ++q) {
          uint32_t s[16];
          tmem_load<16>(t_lane + Sh::kS + 16 * q, s);
          tc_wait_ld();
          if (lane == 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              *reinterpret_cast<uint4*>(ref + cg * W + 16 * q + 4 * i) =
                  make_uint4(s[4 * i], s[4 * i + 1], s[4 * i + 2], s[4 * i + 3]);
          }
        }
        __syncwarp();
        const uint32_t keep0 = __shfl_sync(0xffffffffu, keep, 0);
        const float c10 = __shfl_sync(0xffffffffu, c1, 0), lv0 = __shfl_sync(0xffffffffu, lv, 0);
        if (lane < W) {
          const float y = fmaf(ref[cg * W + lane], c10 * up[cg * W + lane], lv0);
          const bool use = ((keep0 >> lane) & 1u) && fabsf(y) < INFINITY;
          ref[cg * W + lane] = use ? y : -INFINITY;
          nref[cg * W + lane] = use ? kTHead - y : INFINITY;
        }
      }
      __syncthreads();
    }
    // weights of the row, stored as the B operand; the row's part of the columns' sums,
    // from copy blk % 2 to the other one
    const float wsum = here ? inv : 0.f;
    const uint32_t l_old = t_lane + Sh::kL + (blk & 1) * kTCols;
    const uint32_t l_new = t_lane + Sh::kL + (~blk & 1) * kTCols;
    const uint32_t p_at = sm + Sh::kP + row * Sh::kPRow;
    auto p_piece = [&](int i) {  // 16-byte piece i of the warp's columns
      const int piece = cg * (W / 8) + i;
      return p_at + ((piece ^ ((row >> 1) & 3)) << 4);
    };
    auto softmax = [&](bool rescale) -> bool {
      const f32x2 c2 = pack2(c1, c1), lv2 = pack2(lv, lv), inv2 = pack2(wsum, wsum);
      uint32_t top = 0u;
#pragma unroll
      for (int q = 0; q < kChunks; ++q) {
        uint32_t s[16], lr[16];
        tmem_load<16>(t_lane + Sh::kS + 16 * q, s);
        if (blk > 0) tmem_load<16>(l_old + 16 * q, lr);
        tc_wait_ld();
        float p[16];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 r = *reinterpret_cast<const float4*>(nref + cg * W + 16 * q + 4 * i);
          const float4 f = *reinterpret_cast<const float4*>(up + cg * W + 16 * q + 4 * i);
          const f32x2 z0 = fma2(pack2(__uint_as_float(s[4 * i]), __uint_as_float(s[4 * i + 1])),
                                mul2(c2, pack2(f.x, f.y)), add2(pack2(r.x, r.y), lv2));
          const f32x2 z1 = fma2(pack2(__uint_as_float(s[4 * i + 2]), __uint_as_float(s[4 * i + 3])),
                                mul2(c2, pack2(f.z, f.w)), add2(pack2(r.z, r.w), lv2));
          unpack2(z0, p[4 * i], p[4 * i + 1]);
          unpack2(z1, p[4 * i + 2], p[4 * i + 3]);
        }
        if (!all) {
#pragma unroll
          for (int c = 0; c < 16; ++c) p[c] = (keep >> (16 * q + c)) & 1u ? p[c] : -INFINITY;
        }
        uint32_t h[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          p[2 * i] = ex2_approx(p[2 * i]);
          p[2 * i + 1] = ex2_approx(p[2 * i + 1]);
          h[i] = f16x2_rn(p[2 * i], p[2 * i + 1]);
          top = hmax2(top, h[i]);
        }
        sts128(p_piece(2 * q), make_uint4(h[0], h[1], h[2], h[3]));
        sts128(p_piece(2 * q + 1), make_uint4(h[4], h[5], h[6], h[7]));
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          f32x2 l = blk > 0 ? pack2(__uint_as_float(lr[2 * i]), __uint_as_float(lr[2 * i + 1]))
                            : pack2(0.f, 0.f);
          if (rescale)
            l = mul2(l, *reinterpret_cast<const f32x2*>(fac + cg * W + 16 * q + 2 * i));
          l = fma2(pack2(p[2 * i], p[2 * i + 1]), inv2, l);
          float u, v;
          unpack2(l, u, v);
          lr[2 * i] = __float_as_uint(u);
          lr[2 * i + 1] = __float_as_uint(v);
        }
        tmem_store16(l_new + 16 * q, lr);
      }
      tc_wait_st();
      // weights of 2^15 and more (0x7800 as fp16): the reference has to move
      return (top & 0xffffu) >= 0x7800u || (top >> 16) >= 0x7800u;
    };
    // a warp none of whose rows is there: no weights, and its sums move on as they are
    auto nothing = [&](bool rescale) {
#pragma unroll
      for (int q = 0; q < kChunks; ++q) {
        uint32_t lr[16];
        if (blk > 0) {
          tmem_load<16>(l_old + 16 * q, lr);
          tc_wait_ld();
#pragma unroll
          for (int c = 0; c < 16; ++c)
            if (rescale)
              lr[c] = __float_as_uint(__uint_as_float(lr[c]) * fac[cg * W + 16 * q + c]);
        } else {
#pragma unroll
          for (int c = 0; c < 16; ++c) lr[c] = 0u;
        }
        tmem_store16(l_new + 16 * q, lr);
        sts128(p_piece(2 * q), make_uint4(0u, 0u, 0u, 0u));
        sts128(p_piece(2 * q + 1), make_uint4(0u, 0u, 0u, 0u));
      }
      tc_wait_st();
    };
    bool over = false;
    if (some) over = softmax(false);
    else nothing(false);
    fence_proxy_async_smem();
    tc_fence_before();
    if (__syncthreads_or(over)) {
      // column maxima over the block, new references, everything so far rescaled
      tc_fence_after();
#pragma unroll
      for (int q = 0; q < kChunks; ++q) {
        uint32_t s[16];
        tmem_load<16>(t_lane + Sh::kS + 16 * q, s);
        tc_wait_ld();
        float y[16];
#pragma unroll
        for (int c = 0; c < 16; ++c)
          y[c] = (keep >> (16 * q + c)) & 1u
                     ? fmaf(__uint_as_float(s[c]), c1 * up[cg * W + 16 * q + c], lv)
                     : -INFINITY;
        const float m = scatter_max(y, lane);
        if ((lane & 1) == 0) cmax[wq * kTCols + cg * W + 16 * q + (lane >> 1)] = m;
      }
      __syncthreads();
      if (tid < kTCols) {
        float m = ref[tid];
        const float was = m;
#pragma unroll
        for (int q = 0; q < 4; ++q) m = fmaxf(m, cmax[q * kTCols + tid]);
        fac[tid] = m == was ? 1.f : ex2_approx(was - m);
        ref[tid] = m;
        nref[tid] = kTHead - m;
      }
      __syncthreads();
      if (blk > 0) {
#pragma unroll
        for (int q = 0; q < kChunks; ++q) {
          uint32_t o[16];
          tmem_load<16>(t_lane + Sh::kO + 16 * q, o);
          tc_wait_ld();
#pragma unroll
          for (int c = 0; c < 16; ++c)
            o[c] = __float_as_uint(__uint_as_float(o[c]) * fac[cg * W + 16 * q + c]);
          tmem_store16(t_lane + Sh::kO + 16 * q, o);
        }
        tc_wait_st();
      }
      if (some) softmax(true);
      else nothing(true);
      fence_proxy_async_smem();
      tc_fence_before();
      __syncthreads();
    }
    ok = *failed == 0;
    if (warp == 0 && ok) {
      tc_fence_after();
      if (elect_one()) {
        issue_o(blk == 0, min(kTPages, pages - blk * kTPages));
        if (blk + 1 < nblocks) issue_s();
      }
      __syncwarp();
    }
  }
  // sums of the columns over all rows
#pragma unroll
  for (int q = 0; q < kChunks; ++q) {
    uint32_t lr[16];
    tmem_load<16>(t_lane + Sh::kL + (nblocks & 1) * kTCols + 16 * q, lr);
    tc_wait_ld();
    float v[16];
#pragma unroll
    for (int c = 0; c < 16; ++c) v[c] = __uint_as_float(lr[c]);
    const float t = reduce_scatter<16>(v, lane);
    if ((lane & 1) == 0) cmax[wq * kTCols + cg * W + 16 * q + (lane >> 1)] = t;
  }
  if (ok) ok = mbar_wait(o_done, (nblocks - 1) & 1);
  if (!ok) *failed = 1;
  __syncthreads();
  ok = *failed == 0;
  if (ok) {
    if (tid < kTCols) {
      const float t = cmax[tid] + cmax[kTCols + tid] + cmax[2 * kTCols + tid] + cmax[3 * kTCols + tid];
      fac[tid] = 1.f / t;
      // columns to be done again should their output hold a NaN: not a place without a query
      // (0 / 0 where it keeps no row), nor one whose own scores are NaN
      const uint32_t out =
          __ballot_sync(0xffffffffu, t0 + (tid >> LG) < t1 && quant_redo_needed(t, ref[tid]));
      const uint32_t sum = __ballot_sync(0xffffffffu, quant_sum_unsure(t, ref[tid]));
      if (tid == 0) {
        quant_redo().out[0] = out;
        quant_redo().sum[0] = sum;
      }
      if (a.lse != nullptr && t0 + (tid >> LG) < t1)
        a.lse[qh_of(tid)] = (ref[tid] - kTHead + log2f(t)) * kLn2;
    }
    __syncthreads();
    tc_fence_after();
    // lane pairs exchange columns: an even lane stores column c, dims row and row + 1,
    // its neighbour column c + 1
    const int odd = lane & 1;
    float probe = 0.f;
#pragma unroll
    for (int q = 0; q < kChunks; ++q) {
      uint32_t o[16];
      tmem_load<16>(t_lane + Sh::kO + 16 * q, o);
      tc_wait_ld();
#pragma unroll
      for (int c = 0; c < 16; c += 2) {
        const float2 r = *reinterpret_cast<const float2*>(fac + cg * W + 16 * q + c);
        const float u = __uint_as_float(o[c]) * r.x, v = __uint_as_float(o[c + 1]) * r.y;
        const float got = __shfl_xor_sync(0xffffffffu, odd ? u : v, 1);
        const float lo = odd ? got : u, hi = odd ? v : got;
        // (column and place worked out again: held in registers until here they spill, 130
        // us instead of 123 on 32 tokens of 64 requests)
        const int col = static_cast<int>(threadIdx.x >> 7) * W + 16 * q + c + odd, t = t0 + (col >> LG);
        if (t < t1) {
          const size_t qh =
              (static_cast<size_t>(b) * a.max_q + t) * a.hq + (hk << LG) + (col & ((1 << LG) - 1));
          *reinterpret_cast<uint32_t*>(a.out + qh * kTD + (row & ~1)) = bf16x2_rn(lo, hi);
          probe += lo + hi;
        }
      }
    }
    // A NaN may come from a row of V that other queries of the CTA keep (weight 0 times
    // NaN), an infinity from a weight past fp16 (scores of 2^20 and more): such a column is done
    // again, from the rows it keeps.
    if (!(fabsf(probe) < INFINITY)) quant_redo().hit = 1;
    tc_fence_before();
  } else {
    // give products in flight a bounded time to finish before the memory goes back
    if (tid == 0) set_error(a.err, DSA_DEV_TIMEOUT);
    mbar_wait(o_done, (nblocks - 1) & 1);
    tc_fence_before();
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    tc_fence_after();
    tmem_dealloc<Sh::kTmem>(tmem);
  }
  if (*reinterpret_cast<volatile int*>(&quant_redo().hit) != 0) quant_redo_tile<kTD, TcTile<LG>>(a);
}

template <int LG>
cudaError_t launch_one(const QuantChunkLaunch& a, cudaStream_t s) {
  auto kern = quant_chunk_tc_kernel<LG>;
  const int smem = TcShape::smem(a.max_window / 32 + 1);
  static KernelSlots cache;
  int per_sm = 0;
  const cudaError_t e =
      cache.get(reinterpret_cast<const void*>(kern), kTThreads, smem, &per_sm);
  if (e != cudaSuccess) return e;
  constexpr int per_cta = kTCols >> LG;
  return launch_pdl(kern, dim3((a.max_q + per_cta - 1) / per_cta, a.hkv, a.batch), dim3(kTThreads),
                    static_cast<size_t>(smem), s, a);
}

}  // namespace

// Which calls this kernel takes: those whose (request, kv head) is one tile, when there are
// enough of them to fill half the GPU or no request passes 2048 rows (a tile is never cut
// along its pages; 8 tiles, cut in quant_chunk.cu / whole here: of 4000 rows 28 / 58 us, of
// 2000 23 / 31, of 1000 21 / 18, of 500 15 / 12, and of 1900 rows of which prompt and window
// leave 60, 16 / 6).  Measured
// against quant_chunk.cu (us, this kernel / that one, batch x kv heads x group, tokens,
// rows): 64x32x1, 32, 300: 80 / 114; 128x8x4, 8, 500: 57 / 82; 128x8x4, 8, 2000: 169 / 235;
// 128x8x4, 4, 1000: 94 / 121.  Against quant_chunk_rows.cu: see there.
bool quant_chunk_tc_fits(const QuantChunkLaunch& a) {
  const int64_t columns = static_cast<int64_t>(a.max_q) << a.group_log2;
  if (columns > 32 || a.split_setting >= 2 || a.batch > 65535 || a.hkv > 65535) return false;
  return a.split_setting == 1 || a.max_pages <= kQuantWholePages ||
         static_cast<int64_t>(a.batch) * a.hkv * 2 >= a.sms;
}

cudaError_t launch_quant_chunk_tc(const QuantChunkLaunch& a, cudaStream_t s) {
  switch (a.group_log2) {
    case 0: return launch_one<0>(a, s);
    case 1: return launch_one<1>(a, s);
    case 2: return launch_one<2>(a, s);
    default: return launch_one<3>(a, s);
  }
}

}  // namespace dsa
