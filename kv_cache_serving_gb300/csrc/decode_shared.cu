// decode_shared.cu -- the decode kernel over the rows behind a shared prefix: bf16 q and pages,
// dense rows or the kept set of the mask, in the big-batch build (small CTAs, of which some fit
// beside a CTA of the prefix kernel).
#include "decode.cuh"
#include "host.h"

namespace dsa {
namespace {

template <int G>
constexpr int shared_warps() {
  return build_warps<G, true, kBuildBig>();
}

template <int MODE>
cudaError_t launch_mode(const DecodeLaunch& a, cudaStream_t s) {
#define DSA_BODY(DD, GG)                                                                       \
  return launch_decode_one<DD, bf16_t, GG, MODE, true, shared_warps<GG>(),                     \
                           DSA_DECODE_STAGE_BYTES_BIG, DSA_DECODE_STAGES, true>(a, s);
  DSA_FOR_SHAPE(a.head_dim, a.hq / a.hkv, DSA_BODY);
#undef DSA_BODY
  return cudaErrorInvalidValue;
}

template <int MODE>
DecodeShape shape_mode(int head_dim, int group) {
  DecodeShape r{0, 1, 1, DSA_DECODE_WARPS, 0, kBuildBig};
#define DSA_BODY(DD, GG)                                                                       \
  constexpr int kNW = shared_warps<GG>();                                                      \
  using Tl = DecodeTiling<DD, bf16_t, GG, (GG >= 2), kNW, DSA_DECODE_STAGE_BYTES_BIG,          \
                          DSA_DECODE_STAGES>;                                                  \
  auto kern = decode_kernel<DD, bf16_t, GG, MODE, true, kNW, DSA_DECODE_STAGE_BYTES_BIG,       \
                            DSA_DECODE_STAGES, true>;                                          \
  static KernelSlots cache;                                                                    \
  int n = 0;                                                                                   \
  r.warps = kNW;                                                                               \
  r.rows_per_pass = Tl::NW * Tl::T;                                                            \
  r.tile_rows = Tl::T;                                                                         \
  if (cache.get(reinterpret_cast<const void*>(kern), kNW * 32, Tl::kSmem, &n) == cudaSuccess && \
      n > 1)                                                                                   \
    r.ctas_per_sm = n;                                                                         \
  return r;
  DSA_FOR_SHAPE(head_dim, group, DSA_BODY);
#undef DSA_BODY
  return r;
}

}  // namespace

cudaError_t launch_decode_shared(const DecodeLaunch& a, int mode, cudaStream_t s) {
  return mode == kRowsDense ? launch_mode<kRowsDense>(a, s) : launch_mode<kRowsMask>(a, s);
}

DecodeShape decode_shape_shared(int head_dim, int group, int mode) {
  return mode == kRowsDense ? shape_mode<kRowsDense>(head_dim, group)
                            : shape_mode<kRowsMask>(head_dim, group);
}

}  // namespace dsa
