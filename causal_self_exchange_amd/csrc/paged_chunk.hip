// Long chunks of a packed batch against the paged Relation Cache: the bf16 MFMA
// scan of fwd_body.h in its paged form, on query tiles of 256 positions of one
// request and one head.
//
// The key tiles of all query tiles form one line of units that is cut into equal
// ranges, one per work-group (paged_device.h): one prompt of 8192, ten ragged
// ones, or one chunk of 256 rows over 100,000 cached ones keep the same share of
// the chip busy. A query tile that a cut divides leaves a partial state in each
// range; chunk_merge_kernel joins them. The scan's stabiliser is 0 unless a
// segment's evidence overflows it, so joining is mostly a sum.
#include "fwd_body.h"

namespace rel {

namespace {

using namespace paged;

template <int D, int DR>
__global__ __launch_bounds__(kThreads, 1) void paged_chunk_kernel(PagedArgs a, HeadParams hp) {
  const FwdArgs none{};
  const RopeParams no_rope{};
  fwd_body<D, DR, true, false, true>(none, hp, no_rope, a);
}

// The query tile that the cut before range k divides, if that is the first cut
// inside it: 16 rows per work-group, 16 lanes per row, and four groups of lanes
// that take every fourth piece and join in LDS in their order.
constexpr int kMergeThreads = 1024;
constexpr int kPieceGroups = 4;

template <int D>
__global__ __launch_bounds__(kMergeThreads) void chunk_merge_kernel(PagedArgs a, HeadParams hp, int groups) {
  __shared__ float s_m[kPieceGroups][16], s_l[kPieceGroups][16];
  __shared__ __attribute__((aligned(16))) float s_z[kPieceGroups][16][D + 4];
  const Ranges rg(a, groups);
  const int k = blockIdx.x + 1;
  const long long cut = k * rg.per;
  if (cut >= rg.units) return;
  Req r;
  const TileOf t(a, cut, &r);
  if (t.start >= cut || cut - rg.per > t.start) return;    // between two tiles, or an earlier cut's tile
  const ChunkWs cw(a.ws, a.S, a.d_h);
  const int tid = threadIdx.x, sl = tid & 15, row = (tid >> 4) & 15, pg = tid >> 8;
  const int ctx = r.total - r.q;
  const int i = 16 * blockIdx.y + row;
  const int pos = (ctx & ~63) + 256 * t.tile + i;
  const bool ok = pos >= ctx && pos < r.total;
  const int pieces = (int)((t.start + t.keys - cut + rg.per - 1) / rg.per) + 1;
  float M = kEmptyMax, L = 0.0f, z[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) z[e] = 0.0f;
  // Piece 0 is the last of range k - 1, the others the first of ranges k, k + 1, ...
  for (int p = pg; p < pieces; p += kPieceGroups) {
    const int slot = p == 0 ? 2 * (k - 1) + 1 : 2 * (k - 1 + p);
    const size_t at = (size_t)slot * 256 + i;
    const float2 ml = cw.ml[at];
    f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f}, y = x;
    if (sl < D / 8) {
      x = reinterpret_cast<const f32x4*>(cw.z + at * D + 8 * sl)[0];
      y = reinterpret_cast<const f32x4*>(cw.z + at * D + 8 * sl)[1];
    }
    const float Mn = fmaxf(M, ml.x);
    const float fo = __builtin_amdgcn_exp2f(M - Mn), fn = __builtin_amdgcn_exp2f(ml.x - Mn);
    M = Mn;
    L = L * fo + ml.y * fn;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      z[e] = z[e] * fo + x[e] * fn;
      z[4 + e] = z[4 + e] * fo + y[e] * fn;
    }
  }
  if (sl == 0) {
    s_m[pg][row] = M;
    s_l[pg][row] = L;
  }
  if (sl < D / 8)
#pragma unroll
    for (int e = 0; e < 8; ++e) s_z[pg][row][8 * sl + e] = z[e];
  __syncthreads();
  if (pg != 0) return;
  M = kEmptyMax;
  L = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) z[e] = 0.0f;
#pragma unroll
  for (int g = 0; g < kPieceGroups; ++g) M = fmaxf(M, s_m[g][row]);
#pragma unroll
  for (int g = 0; g < kPieceGroups; ++g) {
    const float f = __builtin_amdgcn_exp2f(s_m[g][row] - M);
    L = fmaf(f, s_l[g][row], L);
    if (sl < D / 8)
#pragma unroll
      for (int e = 0; e < 8; ++e) z[e] = fmaf(f, s_z[g][row][8 * sl + e], z[e]);
  }
  finish_row<__bf16, D>(a, hp, t.b, r.first + (pos - ctx), t.h, pos, sl, M, L, z, ok);
}

template <int D, int DR>
hipError_t launch_typed(const PagedArgs& a, const HeadParams& hp, int groups, hipStream_t s) {
  hipLaunchKernelGGL((paged_chunk_kernel<D, DR>), dim3(groups), dim3(kThreads), 0, s, a, hp);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || groups == 1) return e;
  hipLaunchKernelGGL((chunk_merge_kernel<DR>), dim3(groups - 1, 16), dim3(kMergeThreads), 0, s, a, hp, groups);
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
