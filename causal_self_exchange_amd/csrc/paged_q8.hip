// The paged Relation Cache's forward over 8-bit pages (relation_paged_fwd_ex), without and
// with trees of drafted tokens: the scan of paged_scan.h with e4m3 rows, or for batches
// with many rows and much work (tile_use) the query tiles of paged_tile.h.
//
// The scan is bound by memory: 64 tokens over 1,024 to 4,096 rows of 32 heads of 128 (1.35
// GB) take 248 us, 5.4 TB/s, of 16-bit pages 451; one token over 300 rows of 8 heads of 64
// takes 10 us, the latency of its dependent loads. Six chunks of 100 to 1,500 tokens over up
// to 6,000 rows of 32 heads of 128 in 8 take 680 us by the scan and 295 to 330 on tiles.
#include "paged_scan.h"
#include "paged_tile.h"

namespace rel {

namespace {

template <int D>
hipError_t launch_typed(const PagedExArgs& a, const HeadParams& hp, hipStream_t s) {
  constexpr int kCols = D <= 64 ? 64 : 128;
  if (const TileUse use = tile_use(a); use != kToScan)
    return a.tree ? launch_tiles<kCols, D, e4m3, true>(a, hp, use == kToBoth, s) : launch_tiles<kCols, D, e4m3, false>(a, hp, use == kToBoth, s);
  return a.tree ? launch_scan<__bf16, D, e4m3, true>(a, hp, s) : launch_scan<__bf16, D, e4m3, false>(a, hp, s);
}

}  // namespace

hipError_t launch_paged_q8(const PagedExArgs& a, const HeadParams& hp, hipStream_t s) {
  switch (a.d_h) {
    case 32: return launch_typed<32>(a, hp, s);
    case 48: return launch_typed<48>(a, hp, s);
    case 64: return launch_typed<64>(a, hp, s);
    case 80: return launch_typed<80>(a, hp, s);
    case 128: return launch_typed<128>(a, hp, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace rel
