// rows.cuh -- the kept set of one (request, kv head) read straight from its keep
// mask by a warp: the prompt rows, then the window rows by rank.
//
// Lane l holds the bits of window offsets 32l+1 .. 32l+32 that can be kept and the
// inclusive count of them over lanes 0..l; the row of a rank is a binary search over
// the lanes' counts and a rank-select inside the word.  Windows up to 1024 offsets.
#pragma once

#include "common.cuh"

namespace dsa {

// Position (0..31) of the set bit of rank r (0-based, ascending) in w; any
// value in 0..31 when w has no such bit.
__device__ __forceinline__ int select_bit(unsigned w, int r) {
  int pos = 0, c = __popc(w & 0xffffu);
  if (r >= c) { r -= c; w >>= 16; pos += 16; }
  c = __popc(w & 0xffu);
  if (r >= c) { r -= c; w >>= 8; pos += 8; }
  c = __popc(w & 0xfu);
  if (r >= c) { r -= c; w >>= 4; pos += 4; }
  c = __popc(w & 0x3u);
  if (r >= c) { r -= c; w >>= 2; pos += 2; }
  if (r >= static_cast<int>(w & 1u)) pos += 1;
  return pos;
}

struct MaskRows {
  int np, wq, wcnt, wincl;  // prompt rows kept, query row, window rows kept, lane prefix
  unsigned wbits;

  // The number of kept rows, or a negative device error code.  `raw` is lane's mask
  // word; all lanes take part and get the same value.
  __device__ __forceinline__ int init(unsigned raw, int L, int P, int W, int max_pages,
                                      int max_window, int max_kept, int lane) {
    if (L < 1 || L > max_pages * kPage) return -DSA_DEV_BAD_SEQ_LEN;
    if (P < 0) return -DSA_DEV_BAD_PROMPT;
    if (W < 0 || W > max_window) return -DSA_DEV_BAD_WINDOW;
    np = min(P, L);
    wq = L - 1;
    // window rows j = i-o, o = omax..0 (ascending j); none when the query is a prompt row
    const int omax = wq >= np ? min(wq - np, W) : -1;
    const int vb = min(max(omax - 32 * lane, 0), 32);
    wbits = vb == 0 ? 0u : raw & (vb == 32 ? 0xffffffffu : (1u << vb) - 1u);
    wincl = __popc(wbits);
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, wincl, s);
      if (lane >= s) wincl += v;
    }
    wcnt = __shfl_sync(0xffffffffu, wincl, 31);
    const int n = np + (omax >= 0 ? wcnt + 1 : 0);
    return n > max_kept ? -DSA_DEV_BAD_COUNT : n;
  }

  // Row at position p of the ascending window rows (all lanes take part; p outside
  // 0..wcnt gives an unused value).  Position wcnt is the query row.
  __device__ __forceinline__ int window_row(int p) const {
    const int q = wcnt - 1 - p;
    int w = 0;
#pragma unroll
    for (int s = 16; s >= 1; s >>= 1)
      if (__shfl_sync(0xffffffffu, wincl, w + s - 1) <= q) w += s;
    const unsigned word = __shfl_sync(0xffffffffu, wbits, w);
    const int below = __shfl_sync(0xffffffffu, wincl, w) - __popc(word);
    return q < 0 ? wq : wq - (32 * w + select_bit(word, q - below) + 1);
  }
};

}  // namespace dsa
