// The paged Relation Cache's forward of trees of drafted tokens over pages of the tokens'
// own type (relation_paged_fwd_ex): the scan of paged_scan.h with a row of ancestor bits
// per token, or for bf16 batches with many rows and much work (tile_use) the query tiles
// of paged_tile.h. Only the steps that hold new tokens look at the bits.
//
// 48 trees of 2 to 24 tokens over 200 to 9,000 rows of 16 heads of 64 in 4 take 110 us by
// the scan and 89 on tiles (their reads 38); six of 5 to 40 tokens over up to 2,000 fp32 rows
// of 8 heads of 48 in 2 take 19 us and 5 for the join, by the latency of a few steps.
#include "paged_scan.h"
#include "paged_tile.h"

namespace rel {

namespace {

template <typename Tin, int D>
hipError_t launch_typed(const PagedExArgs& a, const HeadParams& hp, hipStream_t s) {
  if constexpr (sizeof(Tin) == 2)
    if (const TileUse use = tile_use(a); use != kToScan)
      return launch_tiles<(D <= 64 ? 64 : 128), D, __bf16, true>(a, hp, use == kToBoth, s);
  return launch_scan<Tin, D, Tin, true>(a, hp, s);
}

}  // namespace

hipError_t launch_paged_tree(const PagedExArgs& a, const HeadParams& hp, bool bf16, hipStream_t s) {
  switch (a.d_h) {
    case 32: return bf16 ? launch_typed<__bf16, 32>(a, hp, s) : launch_typed<float, 32>(a, hp, s);
    case 48: return bf16 ? launch_typed<__bf16, 48>(a, hp, s) : launch_typed<float, 48>(a, hp, s);
    case 64: return bf16 ? launch_typed<__bf16, 64>(a, hp, s) : launch_typed<float, 64>(a, hp, s);
    case 80: return bf16 ? launch_typed<__bf16, 80>(a, hp, s) : launch_typed<float, 80>(a, hp, s);
    case 128: return bf16 ? launch_typed<__bf16, 128>(a, hp, s) : launch_typed<float, 128>(a, hp, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace rel
