// Device code shared by the kernels of the paged Relation Cache's chunk forward:
// the workspace, the requests' numbers, and the last step of a row.
#pragma once

#include "mfma_tile.h"
#include "rel_internal.h"
#include "rel_device.h"

namespace rel {
namespace paged {

using namespace mfma;
typedef float f32x4 __attribute__((ext_vector_type(4)));

// Workspace of a call.
struct Ws {
  PagedPlan* plan;
  int* units[2];     // [S + 1] each: exclusive sums of row blocks x splits
  int* part;         // [S + 1] partial rows
  int* merge;        // [S + 1] rows to merge
  float2* ml;        // [kPartialRows] stabiliser (log2) and sum
  float* z;          // [kPartialRows][d_h]
  __host__ __device__ Ws(void* ws, int S) {
    char* p = static_cast<char*>(ws);
    const int64_t n = ((int64_t)(S + 1) * 4 + 255) / 256 * 256;
    plan = reinterpret_cast<PagedPlan*>(p);
    p += kPlanHeader;
    units[0] = reinterpret_cast<int*>(p);
    units[1] = reinterpret_cast<int*>(p + n);
    part = reinterpret_cast<int*>(p + 2 * n);
    merge = reinterpret_cast<int*>(p + 3 * n);
    p += kPlanSums * n;
    ml = reinterpret_cast<float2*>(p);
    z = reinterpret_cast<float*>(p + kPartialRows * sizeof(float2));
  }
};

// What the device-side numbers say of request b; rows = 0 for one that is skipped.
struct Req {
  int first, q, total, rows;   // first packed token, new tokens, cached rows, rows per cached head
  __device__ __forceinline__ Req() {}
  __device__ __forceinline__ Req(const PagedArgs& a, int b) {
    first = a.cu[b];
    const int end = a.cu[b + 1];
    total = a.total[b];
    const bool ok = first >= 0 && end > first && end <= a.N && end - first <= a.max_new && total >= end - first &&
                    (long long)total <= ((long long)a.max_pages << a.page_shift);
    q = ok ? end - first : 0;
    rows = q * (a.H / a.H_kv);
  }
};

// A value that is the same in every lane, in a scalar register: buffer
// descriptors are formed from it.
__device__ __forceinline__ int uni(int x) { return __builtin_amdgcn_readfirstlane(x); }

// A split length of kMaxChunk stands for unsplit histories of any length.
constexpr int kMaxChunk = 0x7fffff80;
__device__ __forceinline__ int splits_of(int total, int chunk) {
  return chunk == kMaxChunk ? 1 : (int)(((long long)total + chunk - 1) / chunk);
}

// The last request b with off[b] <= i: 64 entries are compared at a time.
template <typename Int>
__device__ __forceinline__ int find_request(const Int* off, int S, Int i) {
  const int lane = threadIdx.x & 63;
  int lo = 0, n = S;
  while (n > 1) {
    const int stride = (n + 63) >> 6;
    const int k = lane * stride;
    const bool le = k < n && off[lo + k] <= i;
    const int cnt = __popcll(__ballot(le));
    lo += (cnt - 1) * stride;
    n = min(stride, n - (cnt - 1) * stride);
  }
  return __builtin_amdgcn_readfirstlane(lo);
}

// ---- long chunks --------------------------------------------------------------

// Query tiles of a request's chunk: 256 positions each from ctx rounded down to
// a multiple of 64, so that 64-key tiles never straddle a tile's first position
// and a tile's own keys are four key tiles. Tile k needs the key tiles below
// its last position's next: all but the last tile base64 + 4 (k + 1).
struct ChunkTiles {
  int base64, n, last;         // first position / 64, tiles, key tiles of the last tile
  __device__ __forceinline__ ChunkTiles(int ctx, int total) {
    base64 = ctx >> 6;
    n = (int)(((long long)total - 64LL * base64 + 255) >> 8);
    last = (int)(((long long)total + 63) >> 6);
  }
  // Key tiles of the tiles before k.
  __device__ __forceinline__ long long before(int k) const {
    const long long full = (long long)k * base64 + 2LL * k * (k + 1);
    return k < n ? full : (long long)(n - 1) * base64 + 2LL * (n - 1) * n + last;
  }
  __device__ __forceinline__ int keys(int k) const { return k + 1 < n ? base64 + 4 * (k + 1) : last; }
};

// Whether the request's rows go to the long-chunk kernel.
__device__ __forceinline__ bool is_chunk(const Req& r, int chunk_min) { return chunk_min > 0 && r.q >= chunk_min; }

// The long-chunk part of the workspace: exclusive sums of key tiles over the
// requests (all heads; [S] the total) and the partial states, 256 rows each, two
// per work-group.
struct ChunkWs {
  long long* units;
  float2* ml;
  float* z;
  __host__ __device__ ChunkWs(void* ws, int S, int d_h) {
    char* p = static_cast<char*>(ws) + paged_scan_bytes(S, d_h);
    units = reinterpret_cast<long long*>(p);
    p += paged_chunk_sum_bytes(S);
    ml = reinterpret_cast<float2*>(p);
    z = reinterpret_cast<float*>(p + (int64_t)kChunkStates * 256 * sizeof(float2));
  }
};

// A unit is one key tile of one query tile; the units of all query tiles (per
// request, per head, tile by tile) form one line that is cut into equal ranges,
// one per work-group, whatever the requests' lengths. A segment is the part of a
// query tile's key tiles in one range: [tb, te), te = 0 for none. slot: the
// partial state it leaves, or -1 when it holds all of them.
struct Segment {
  int b, h, kvh;
  int first, ctx, total;       // packed token of the chunk's first row, its position, cached rows
  int q0, tb, te, slot;
  // The same, every field in a scalar register.
  __device__ __forceinline__ Segment uniform() const {
    return Segment{uni(b), uni(h), uni(kvh), uni(first), uni(ctx), uni(total), uni(q0), uni(tb), uni(te), uni(slot)};
  }
};

// Equal ranges of at least 8 units.
struct Ranges {
  long long units, per;
  __device__ __forceinline__ Ranges(const PagedArgs& a, int groups) {
    units = ChunkWs(a.ws, a.S, a.d_h).units[a.S];
    per = (units + groups - 1) / groups;
    per = per < 8 ? 8 : per;
  }
};

// The query tile of unit u: its request and head, its index within them, and
// the unit of its first key tile.
struct TileOf {
  int b, h, tile, keys;
  long long start;
  __device__ __forceinline__ TileOf(const PagedArgs& a, long long u, Req* req) {
    const long long* sums = ChunkWs(a.ws, a.S, a.d_h).units;
    b = find_request(sums, a.S, u);
    const Req r(a, b);
    *req = r;
    const ChunkTiles t(r.total - r.q, r.total);
    const long long per_head = t.before(t.n);
    const long long v = u - sums[b];
    h = (int)(v / per_head);
    const long long w = v - h * per_head;
    int lo = 0, hi = t.n - 1;                            // the last tile that starts at or before w
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (t.before(mid) <= w) lo = mid;
      else hi = mid - 1;
    }
    tile = lo;
    keys = t.keys(tile);
    start = sums[b] + h * per_head + t.before(tile);
  }
};

// The segments of one work-group, in order. Work-groups go round the 8 XCDs, and
// each XCD takes a contiguous eighth of the line: neighbouring tiles and heads,
// which read the same keys, share its L2.
struct SegmentSource {
  const PagedArgs& a;
  long long u, end;
  int me;
  __device__ __forceinline__ SegmentSource(const PagedArgs& args, int group, int groups) : a(args) {
    me = groups % 8 == 0 ? (group & 7) * (groups >> 3) + (group >> 3) : group;
    const Ranges r(args, groups);
    u = me * r.per;
    end = u + r.per < r.units ? u + r.per : r.units;
  }
  __device__ __forceinline__ Segment next() {
    Segment s{};
    if (u >= end) return s;
    Req r;
    const TileOf t(a, u, &r);
    s.b = t.b;
    s.h = t.h;
    s.kvh = t.h / (a.H / a.H_kv);
    s.first = r.first;
    s.total = r.total;
    s.ctx = r.total - r.q;
    s.q0 = (s.ctx & ~63) + 256 * t.tile;
    s.tb = (int)(u - t.start);
    const long long stop = t.start + t.keys < end ? t.start + t.keys : end;
    s.te = (int)(stop - t.start);
    s.slot = s.tb == 0 && s.te == t.keys ? -1 : (s.tb > 0 ? 2 * me : 2 * me + 1);
    u = stop;
    return s;
  }
};

// ---- rows ---------------------------------------------------------------------

template <typename Tin>
__device__ __forceinline__ void load8(const Tin* p, float (&x)[8]) {
  if constexpr (sizeof(Tin) == 2) {
    const bf16x8 v = *reinterpret_cast<const bf16x8*>(p);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = (float)v[e];
  } else {
    const f32x4 v = reinterpret_cast<const f32x4*>(p)[0], w = reinterpret_cast<const f32x4*>(p)[1];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[e] = v[e];
      x[4 + e] = w[e];
    }
  }
}

template <typename Tin>
__device__ __forceinline__ void store8(Tin* p, const float (&x)[8]) {
  if constexpr (sizeof(Tin) == 2) {
    *reinterpret_cast<u32x4*>(p) =
        u32x4{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7])};
  } else {
    reinterpret_cast<f32x4*>(p)[0] = f32x4{x[0], x[1], x[2], x[3]};
    reinterpret_cast<f32x4*>(p)[1] = f32x4{x[4], x[5], x[6], x[7]};
  }
}

// Output of one row from its history's state, by 16 lanes of 8 columns each:
// z (sum of weights times V), m (log2 stabiliser) and l (sum of weights); the
// Self evidence and V come from the row's own cached row.
template <typename Tin, int D>
__device__ __forceinline__ void finish_row(const PagedArgs& a, const HeadParams& hp, int b, int t, int h, int pos,
                                           int sl, float m, float l, const float (&z)[8], bool row_ok) {
  const bool live = row_ok && sl < D / 8;
  const int col = live ? 8 * sl : 0;
  const int kvh = h / (a.H / a.H_kv);
  float q[8], k[8], v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) q[e] = k[e] = v[e] = 0.0f;
  if (live) {
    load8(static_cast<const Tin*>(a.P1) + (size_t)t * a.ld1 + (size_t)h * D + col, q);
    const int page = a.table[(size_t)b * a.max_pages + (pos >> a.page_shift)];
    if (page >= 0 && page < a.n_pages) {
      const size_t row =
          ((((size_t)page * a.H_kv + kvh) << a.page_shift) + (pos & ((1 << a.page_shift) - 1))) * D + col;
      load8(static_cast<const Tin*>(a.cP2) + row, k);
      load8(static_cast<const Tin*>(a.cV) + row, v);
    }
  }
  float u = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) u = fmaf(q[e], k[e], u);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) u += __shfl_xor(u, o, 16);
  if (!live) return;
  const float S = sigmoid_f32(u * hp.scale * hp.inv_tau[h]);
  const RowCombine c(S, m * kLn2, l, hp.lambda * logf((float)(pos + 1)));
  float y[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) y[e] = c.w_self * v[e] + c.w_hist * z[e];
  store8(static_cast<Tin*>(a.Y) + ((size_t)t * a.H + h) * D + col, y);
}

}  // namespace paged
}  // namespace rel
