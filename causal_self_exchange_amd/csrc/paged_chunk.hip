// Chunks of new tokens of a packed batch against the paged Relation Cache: the
// bf16 MFMA scan of fwd_body.h in its paged form, on query tiles of 256 rows of one
// request: 256 positions of one head, or blocks of 32 positions of several heads
// that share a cached head.
//
// The key tiles of all query tiles are cut into equal ranges (paged_device.h): one
// prompt of 8192, ten ragged ones, or one chunk of 256 rows over 100,000 cached
// ones keep every compute unit busy to the end. The scan's stabiliser is 0 unless
// a segment's evidence overflows it, so joining a divided tile is mostly a sum.
//
// The weights are rounded to bf16 once for the transport, and summed rounded, as in
// the inference forward. Two bf16 terms a weight, as in the scan, took five prompts from
// 951 to 1215 us and 2048 tokens over 30,001 rows from 1160 to 1544.
//
// What bounds it: the weights on VALU next to the MFMA, as in the training forward.
// 2048 tokens of 32 heads of 128 in 8 cached ones over 30,001 rows: 1175 to 1209 us
// with the join, 861 to 886 TFLOP/s (MfmaUtil 41%); five prompts of 500 to 6,000 tokens
// 950 to 1007 us.
#include "fwd_body.h"

namespace rel {

namespace {

using namespace paged;

template <int D, int DR>
__global__ __launch_bounds__(kThreads, 1) void paged_chunk_kernel(PagedArgs a, HeadParams hp) {
  __shared__ PlanLds lds;
  bool chunks = true;
  const Plan plan = load_plan(a, 0, chunks, lds);
  const FwdArgs none{};
  const RopeParams no_rope{};
  fwd_body<D, DR, true, false, true>(none, hp, no_rope, a, plan);
}

template <int D, int DR>
hipError_t launch_typed(const PagedArgs& a, const HeadParams& hp, int groups, hipStream_t s) {
  hipLaunchKernelGGL((paged_chunk_kernel<D, DR>), dim3(groups), dim3(kThreads), 0, s, a, hp);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_paged_chunk(const PagedArgs& a, const HeadParams& hp, int groups, hipStream_t s) {
  switch (a.d_h) {
    case 32: return launch_typed<64, 32>(a, hp, groups, s);
    case 48: return launch_typed<64, 48>(a, hp, groups, s);
    case 64: return launch_typed<64, 64>(a, hp, groups, s);
    case 80: return launch_typed<128, 80>(a, hp, groups, s);
    case 128: return launch_typed<128, 128>(a, hp, groups, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace rel
