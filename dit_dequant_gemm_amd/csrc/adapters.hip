// The products with per-row adapters for one bit width, DDG_BITS, and (in the
// unit of width 4) the launcher of their pre-pass.  Compiled once per width.
#include <algorithm>

#include "ddg_launch.hpp"

#ifndef DDG_BITS
#error "compile with -DDDG_BITS=<3..7>"
#endif

namespace ddg {

template <>
hipError_t launch_adapter_large<DDG_BITS>(const GemmArgs& a, const AdapterArgs& ad, hipStream_t stream) {
  gemm_large_adapter_kernel<DDG_BITS><<<dim3((unsigned)(a.tiles_m * a.tiles_n)), dim3(512), 0, stream>>>(a, ad);
  return hipGetLastError();
}

template <>
hipError_t launch_adapter_n192<DDG_BITS>(const GemmArgs& a, const AdapterArgs& ad, hipStream_t stream) {
  gemm_n192_adapter_kernel<DDG_BITS><<<dim3((unsigned)(a.tiles_m * a.tiles_n)), dim3(256), 0, stream>>>(a, ad);
  return hipGetLastError();
}

template <>
hipError_t launch_adapter_streamk<DDG_BITS>(const GemmArgs& a, const StreamK& sk, int grid, const AdapterArgs& ad,
                                            hipStream_t stream) {
  gemm_streamk_kernel<DDG_BITS><<<dim3((unsigned)grid), dim3(512), 0, stream>>>(a, sk, ad);
  return hipGetLastError();
}

template <>
hipError_t launch_adapter_small<DDG_BITS>(const GemmArgs& a, int rb, int nc, int nk, const AdapterArgs& ad,
                                          hipStream_t stream) {
  const dim3 grid((unsigned)((a.n + 16 * nc - 1) / (16 * nc)));
#define DDG_SMALL(RB, NC, NK)                                                                         \
  if (rb == RB && nc == NC && nk == NK) {                                                             \
    gemm_small_adapter_kernel<DDG_BITS, RB, NC, NK><<<grid, dim3(64 * NC * NK), 0, stream>>>(a, ad); \
    return hipGetLastError();                                                                         \
  }
  DDG_SMALL(1, 1, 8) DDG_SMALL(1, 2, 4) DDG_SMALL(1, 4, 2)
  DDG_SMALL(2, 1, 4) DDG_SMALL(2, 2, 2)
  DDG_SMALL(4, 1, 4) DDG_SMALL(4, 2, 2)
#undef DDG_SMALL
  return hipErrorInvalidValue;
}

template <>
hipError_t launch_adapter_small_split<DDG_BITS>(const GemmArgs& a, int nc, const SmallSplit& sp,
                                                const AdapterArgs& ad, hipStream_t stream) {
  if (sp.parts < 2 || sp.parts > kSmallMaxParts || nc != 2) return hipErrorInvalidValue;
  const dim3 grid((unsigned)((a.n + 16 * nc - 1) / (16 * nc) * sp.parts));
  gemm_small_split_adapter_kernel<DDG_BITS, 2><<<grid, dim3(128), 0, stream>>>(a, sp, ad);
  return hipGetLastError();
}

template <>
hipError_t launch_adapter_skinny<DDG_BITS>(const GemmArgs& a, int kc, int ncb, const AdapterArgs& ad,
                                           hipStream_t stream) {
  const dim3 grid((unsigned)((a.n + 16 * ncb - 1) / (16 * ncb)));
  if (skinny_static_lds(DDG_BITS, kc, ncb) + skinny_scale_lds(kc) > kLdsLimit) return hipErrorInvalidValue;
#define DDG_SKINNY(KC, NCB)                                                                 \
  if (kc == KC && ncb == NCB) {                                                             \
    gemm_skinny_adapter_kernel<DDG_BITS, KC, NCB><<<grid, dim3(512), 0, stream>>>(a, ad);  \
    return hipGetLastError();                                                               \
  }
  DDG_SKINNY(3, 1) DDG_SKINNY(3, 2) DDG_SKINNY(3, 4)
  DDG_SKINNY(4, 1) DDG_SKINNY(4, 2) DDG_SKINNY(4, 4)
  DDG_SKINNY(5, 1) DDG_SKINNY(5, 2) DDG_SKINNY(5, 4)
#undef DDG_SKINNY
  return hipErrorInvalidValue;
}

#if DDG_BITS == 4
namespace {
constexpr int kFewBlocks = 128;       // row blocks of 16 that leave compute units idle

template <int RBLK, int RR, bool PARTS>
hipError_t launch_down(AdapterDown d, int z, hipStream_t stream) {
  const int blocks = (d.m + 16 * RR - 1) / (16 * RR);
  d.z = z;
  d.rank_parts = ((d.r + 15) / 16 + RBLK - 1) / RBLK;
  // few row blocks: every z = 0 workgroup (the only one with work in a block of
  // one adapter) before the others, so that they spread over the compute units;
  // many: runs of 8 blocks, one per XCD, take all their z before the next run,
  // so that a block's second adapter starts beside its first
  d.run = blocks < kFewBlocks ? 0 : 8;
  const dim3 grid((unsigned)(d.run ? (blocks + 7) / 8 * 8 * z : blocks), (unsigned)d.chunks,
                  (unsigned)(d.run ? d.rank_parts : d.rank_parts * z));
  adapter_down_kernel<RBLK, RR, PARTS><<<grid, dim3(64 * adapter_down_waves(RR, RBLK)), 0, stream>>>(d);
  return hipGetLastError();
}

template <int RBLK>
hipError_t launch_rblk(const AdapterDown& d, int rr, int z, hipStream_t stream) {
  if (rr == 4) return launch_down<RBLK, 4, true>(d, z, stream);
  if (rr == 2) return launch_down<RBLK, 2, true>(d, z, stream);
  return launch_down<RBLK, 1, true>(d, z, stream);
}
}  // namespace

hipError_t launch_adapter_down(const AdapterDown& d, hipStream_t stream) {
  // at most 64 rows: every distinct adapter of a row block and every 16 of
  // the rank in a workgroup of its own
  if (d.m <= kAdapterFewRows) return launch_down<1, 1, false>(d, std::min(d.count, 16), stream);
  // a block's adapters go to different workgroups, two at least (blocks with a
  // request's end inside would otherwise take twice as long as the others),
  // more while all of them are resident at once (two per compute unit; idle ones
  // past that made 4096 rows take 18.5 us instead of 11.4)
  const int blocks = (d.m + 15) / 16;
  const bool few = blocks < kFewBlocks;
  const int wgs = few ? blocks * ((d.r + 15) / 16) : blocks;
  const int z = std::min(d.count, std::max(2, std::min(16, 512 / wgs)));
  // (... and then every 16 of the rank to one of its own)
  if (few) return launch_down<1, 1, true>(d, z, stream);
  // D is read once per workgroup: several row blocks to one while every
  // compute unit gets a workgroup
  const int rr = blocks >= 4 * 256 ? 4 : (blocks >= 2 * 256 ? 2 : 1);
  switch (std::min((d.r + 15) / 16, 4)) {
    case 1: return launch_rblk<1>(d, rr, z, stream);
    case 2: return launch_rblk<2>(d, rr, z, stream);
    case 3: return launch_rblk<3>(d, rr, z, stream);
    default: return launch_rblk<4>(d, rr, z, stream);
  }
}
#endif

}  // namespace ddg
