// The paged Relation Cache's forward over 8-bit pages (relation_paged_fwd_ex): the scan
// of paged_scan.h with e4m3 rows, without and with trees of drafted tokens. Every batch
// goes through the scan, prompts too.
#include "paged_scan.h"
#include "paged_tile.h"

namespace rel {

namespace {

template <int D>
hipError_t launch_typed(const PagedExArgs& a, const HeadParams& hp, hipStream_t s) {
  constexpr int kCols = D <= 64 ? 64 : 128;
  if (tiles_wanted(a))
    return a.tree ? launch_tiles<kCols, D, e4m3, true>(a, hp, s) : launch_tiles<kCols, D, e4m3, false>(a, hp, s);
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
