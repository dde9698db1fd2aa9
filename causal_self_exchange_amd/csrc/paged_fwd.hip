// Relation forward of a packed batch of new tokens against the paged Relation
// Cache (semantics in relation.h; "Ask Self, Ask Others: Relation Is All You
// Need", Eq. (1)-(3) by the scan of Sec. 5.1, Eq. (12)-(14), and the cache of
// Sec. 5.3).
//
// The rows of a request that share a cached head (its new tokens times the
// query heads of the group) are taken in blocks of 16 NB rows. The keys of all
// row blocks are cut into equal ranges, one per work-group (paged_device.h); a
// work-group of four waves scans its segments' keys, each wave its own steps of 32
// (fp32: 16), and keeps (m, l, z) per row; the waves' states meet in LDS. A
// segment with all of its row block's keys finishes the rows itself (Self entry,
// count term, output); otherwise it leaves a partial state, and join_kernel
// finishes the row.
//
// What bounds it: single tokens, the reads of the cache (64 tokens over 1,024 to
// 4,096 rows of 32 heads of 128: 454 us, 5.9 TB/s, every byte read once; 64 over 4000
// rows of 8 heads of 32 to 128: 5.2 to 5.8 TB/s); short calls, the latency of the
// first loads and the meeting (one token over 300 rows: 9.8 us).
//
// Launches: plan (more than kPlanInline requests only), the chunk kernel
// (paged_chunk.hip, where a request can fill its tiles; the rest is left to the
// scan), scan, join (where a row block can have been divided).
#include "paged_scan.h"

namespace rel {

namespace {

template <typename Tin, int D>
hipError_t launch_typed(const PagedArgs& a, const HeadParams& hp, hipStream_t s) {
  return launch_scan<Tin, D, Tin, false>(a, hp, s);
}

}  // namespace

hipError_t launch_paged(const PagedArgs& a, const HeadParams& hp, bool bf16, hipStream_t s) {
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
