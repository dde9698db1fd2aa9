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

// A value that is the same in every lane, in a scalar register: buffer
// descriptors are formed from it.
__device__ __forceinline__ int uni(int x) { return __builtin_amdgcn_readfirstlane(x); }

// What the device-side numbers say of request b; q = 0 for one that is skipped.
struct Req {
  int first, q, total;         // first packed token, new tokens, cached rows
  __device__ __forceinline__ Req() {}
  __device__ __forceinline__ Req(const PagedArgs& a, int b) {
    first = a.cu[b];
    const int end = a.cu[b + 1];
    total = a.total[b];
    const bool ok = first >= 0 && end > first && end <= a.N && end - first <= a.max_new && total >= end - first &&
                    (long long)total <= ((long long)a.max_pages << a.page_shift);
    q = ok ? end - first : 0;
  }
};

// Query tiles of a long chunk: 256 positions each from ctx rounded down to a
// multiple of 64, so that 64-key tiles never straddle a tile's first position
// and a tile's own keys are four key tiles. Tile k needs the key tiles up to its
// last position: all but the last tile base64 + 4 (k + 1). A last tile with
// fewer than kChunkMin positions would waste more of the long-chunk kernel than
// the scan kernel is slower: its tokens (rest) go there.
struct ChunkTiles {
  int base64, n, last, rest;   // first position / 64, tiles, key tiles of the last one, tokens left to the scan
  __device__ __forceinline__ ChunkTiles(int ctx, int total) {
    base64 = ctx >> 6;
    const long long span = (long long)total - 64LL * base64;
    rest = (int)(span & 255);
    rest = rest < kChunkMin ? rest : 0;
    n = (int)((span - rest + 255) >> 8);
    last = (int)(((long long)total - rest + 63) >> 6);
  }
  // Key tiles of the tiles before k.
  __device__ __forceinline__ long long before(int k) const {
    const long long full = (long long)k * base64 + 2LL * k * (k + 1);
    return k < n ? full : (long long)(n - 1) * base64 + 2LL * (n - 1) * n + last;
  }
  __device__ __forceinline__ int keys(int k) const { return k + 1 < n ? base64 + 4 * (k + 1) : last; }
};

// The part of a request that each kernel takes: its first tokens with
// chunk_min > 0 and at least that many new ones go to the long-chunk kernel, the
// rest to the scan kernel, as requests of their own.
__device__ __forceinline__ Req chunk_part(Req r, int chunk_min) {
  if (chunk_min == 0 || r.q < chunk_min) r.q = 0;
  if (r.q > 0) {
    const int rest = ChunkTiles(r.total - r.q, r.total).rest;
    r.q -= rest;
    r.total -= rest;
  }
  return r;
}
__device__ __forceinline__ Req scan_part(Req r, int chunk_min) {
  if (chunk_min > 0 && r.q >= chunk_min) {
    const int rest = ChunkTiles(r.total - r.q, r.total).rest;
    r.first += r.q - rest;
    r.q = rest;
  }
  return r;
}

// ---- plan ---------------------------------------------------------------------
//
// How the batch's work is cut, from the device-side lengths. Scan kernel: row
// blocks of row_block rows of a request and cached head, times splits of its
// history of `chunk` keys; partial states where a history is split. Long chunks:
// key tiles of all query tiles and heads, in one line. The sums are exclusive,
// over the requests.

constexpr int kMinChunk = 512;            // keys of the shortest split
constexpr int kMaxChunk = 0x7fffff80;     // stands for unsplit histories of any length

// What the host fixes of it.
struct Cut {
  int row_block;          // rows per scan item
  int chunk_min;          // new tokens from which a request is a long chunk; 0: none is
  int scan_groups;        // work-groups of the scan kernel
  int chunk_groups;       // and of the long-chunk kernel
};

struct Plan {
  int chunk, units, merge_rows;
  int* unit_sum;          // row blocks x splits (times H_kv work items)
  int* part_sum;          // partial rows
  int* merge_sum;         // rows to join
  long long* tile_sum;    // key tiles of the long chunks; [S] the total
};

__device__ __forceinline__ int splits_of(int total, int chunk) {
  return chunk == kMaxChunk ? 1 : (int)(((unsigned)total + (unsigned)chunk - 1u) / (unsigned)chunk);
}

// Sums over the first four waves of a work-group, of N values per thread at
// once: inclusive sums in x, totals in total; every thread of the work-group
// calls it, and red is free again when it returns.
template <typename Int, int N>
__device__ __forceinline__ void sum_256(Int (&x)[N], Int (&total)[N], Int (*red)[N]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1)
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const Int y = __shfl_up(x[k], o, 64);
      if (lane >= o) x[k] += y;
    }
  if (lane == 63 && wave < 4)
#pragma unroll
    for (int k = 0; k < N; ++k) red[wave][k] = x[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < N; ++k) {
    Int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      before += w < wave ? red[w][k] : 0;
      all += red[w][k];
    }
    x[k] += before;
    total[k] = all;
  }
  __syncthreads();
}

struct PlanScratch {
  long long wide[4][3];
  int sum[4][3];
};

// Fills p and the arrays it points to, by the work-group's first 256 threads
// (every thread calls). scan / chunks: which sums are wanted.
__device__ __forceinline__ void make_plan(const PagedArgs& a, const Cut& cut, bool scan, bool chunks, PlanScratch& sc,
                                          Plan& p) {
  const int row_block = cut.row_block, chunk_min = cut.chunk_min;
  const int tid = threadIdx.x;
  const int G = a.H / a.H_kv;
  // Up to 256 requests each thread keeps its own.
  Req mine;
  mine.q = 0;
  if (tid < 256 && tid < a.S) mine = Req(a, tid);
  if (scan) {
    // Key visits of the row blocks, the items without splits, and rows times keys:
    // a split length c makes at most visits / c + base items. They should fill the
    // scan's work-groups a whole number of times, with as many again as there are
    // at least: a few items past a round cost a round. The length also keeps the
    // partial rows within the workspace (a split request has at most 2 total /
    // chunk splits).
    long long x[3] = {0, 0, 0}, n[3];
    for (int b = tid; b < a.S && tid < 256; b += 256) {
      const Req r = scan_part(b < 256 ? mine : Req(a, b), chunk_min);
      const long long blocks = (long long)((r.q * G + row_block - 1) / row_block) * a.H_kv;
      x[0] += blocks * r.total;
      x[1] += blocks;
      x[2] += (long long)r.q * a.H * r.total;
    }
    sum_256<long long, 3>(x, n, sc.wide);
    const long long room = (2 * n[1] + cut.scan_groups - 1) / cut.scan_groups * cut.scan_groups - n[1];
    float c1 = room > 0 ? (float)n[0] / (float)room : 0.0f;
    const float c2 = (float)(2 * n[2]) * (1.0f / kPartialRows) * 1.00001f;
    c1 = fmaxf(fmaxf(c1, c2) + 1.0f, (float)kMinChunk);
    p.chunk = c1 < 2.0e9f ? ((int)c1 + 127) & ~127 : kMaxChunk;
  }
  int done[3] = {0, 0, 0};     // units, rows to join, partial rows
  long long tiles = 0;
  for (int b0 = 0; b0 < a.S; b0 += 256) {
    const int b = b0 + tid;
    const bool in = tid < 256 && b < a.S;
    Req r;
    r.q = 0;
    if (in) r = b0 == 0 ? mine : Req(a, b);
    if (scan) {
      const Req s = scan_part(r, chunk_min);
      const int splits = s.q > 0 ? splits_of(s.total, p.chunk) : 0;
      const int rows = splits > 1 ? s.q * a.H : 0;
      const int own[3] = {(s.q * G + row_block - 1) / row_block * splits, rows, rows * splits};
      int x[3] = {own[0], own[1], own[2]}, n[3];
      sum_256<int, 3>(x, n, sc.sum);
      if (in) {
        p.unit_sum[b] = done[0] + x[0] - own[0];
        p.merge_sum[b] = done[1] + x[1] - own[1];
        p.part_sum[b] = done[2] + x[2] - own[2];
      }
#pragma unroll
      for (int k = 0; k < 3; ++k) done[k] += n[k];
    }
    if (chunks) {
      const Req s = chunk_part(r, chunk_min);
      long long own = 0;
      if (s.q > 0) {
        const ChunkTiles t(s.total - s.q, s.total);
        own = t.before(t.n) * a.H;
      }
      long long x[3] = {own, 0, 0}, n[3];
      sum_256<long long, 3>(x, n, sc.wide);
      if (in) p.tile_sum[b] = tiles + x[0] - own;
      tiles += n[0];
    }
  }
  p.units = done[0];
  p.merge_rows = done[1];
  if (chunks && tid == 0) p.tile_sum[a.S] = tiles;
}

// The plan in the workspace: written by plan_kernel for more than kPlanInline
// requests, else by the scan kernel's first work-group for the join.
struct WsPlan {
  int* head;              // chunk, units, merge_rows
  Plan p;
  __device__ __forceinline__ void put_head(const Plan& q) {
    head[0] = q.chunk;
    head[1] = q.units;
    head[2] = q.merge_rows;
  }
  __device__ __forceinline__ Plan get() {
    p.chunk = uni(head[0]);
    p.units = uni(head[1]);
    p.merge_rows = uni(head[2]);
    return p;
  }
  __device__ __forceinline__ WsPlan(const PagedArgs& a) {
    char* w = static_cast<char*>(a.ws);
    head = reinterpret_cast<int*>(w);
    w += kPlanHeader;
    const int64_t n = paged_sum_bytes(a.S, 4);
    p.unit_sum = reinterpret_cast<int*>(w);
    p.part_sum = reinterpret_cast<int*>(w + n);
    p.merge_sum = reinterpret_cast<int*>(w + 2 * n);
    p.tile_sum = reinterpret_cast<long long*>(w + 3 * n);
  }
};

// A kernel's plan: formed in LDS by each work-group for up to kPlanInline
// requests (a launch of its own and the wait for it take 5 us), else read from
// the workspace.
struct PlanLds {
  PlanScratch sc;
  int unit_sum[kPlanInline + 1], part_sum[kPlanInline + 1], merge_sum[kPlanInline + 1];
  long long tile_sum[kPlanInline + 1];
};
__device__ __forceinline__ Plan load_plan(const PagedArgs& a, const Cut& cut, bool scan, bool chunks, PlanLds& lds) {
  if (a.S > kPlanInline) {
    WsPlan w(a);
    return w.get();
  }
  Plan p{};
  p.unit_sum = lds.unit_sum;
  p.part_sum = lds.part_sum;
  p.merge_sum = lds.merge_sum;
  p.tile_sum = lds.tile_sum;
  make_plan(a, cut, scan, chunks, lds.sc, p);
  __syncthreads();
  p.chunk = uni(p.chunk);
  p.units = uni(p.units);
  p.merge_rows = uni(p.merge_rows);
  return p;
}

// Partial states in the workspace: of the scan's split histories, and of the
// long chunks' divided tiles.
struct States {
  float2* ml;
  float* z;
  __device__ __forceinline__ static States scan(const PagedArgs& a) {
    char* w = static_cast<char*>(a.ws) + paged_plan_bytes(a.S);
    return {reinterpret_cast<float2*>(w), reinterpret_cast<float*>(w + kPartialRows * sizeof(float2))};
  }
  __device__ __forceinline__ static States chunk(const PagedArgs& a) {
    char* w = static_cast<char*>(a.ws) + paged_plan_bytes(a.S) + paged_scan_bytes(a.d_h) + kCutBytes;
    return {reinterpret_cast<float2*>(w), reinterpret_cast<float*>(w + (int64_t)kChunkStates * 256 * sizeof(float2))};
  }
};

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

// A unit is one key tile of one query tile; the units of all query tiles (per
// request, per head, tile by tile) form one line that is cut into equal ranges
// of at least 8, one per work-group, whatever the requests' lengths. A segment
// is the part of a query tile's key tiles in one range: [tb, te), te = 0 for
// none. slot: the partial state it leaves, or -1 when it holds all of them.
struct Segment {
  int b, h, kvh;
  int first, ctx, total;       // packed token of the chunk's first row, its position, cached rows
  int q0, tb, te, slot;
  // The same, every field in a scalar register.
  __device__ __forceinline__ Segment uniform() const {
    return Segment{uni(b), uni(h), uni(kvh), uni(first), uni(ctx), uni(total), uni(q0), uni(tb), uni(te), uni(slot)};
  }
};

// The query tile that the end of a work-group's range divides, for the join:
// pieces = 0 when there is none. Piece 0 is the last segment of range k, the
// others the first segments of the ranges after it.
struct CutTile {
  int pieces, b, h, first, ctx, total, q0, pad;
};
static_assert(sizeof(CutTile) == 32 && kChunkGroups * sizeof(CutTile) == kCutBytes, "workspace layout");

__device__ __forceinline__ long long range_length(long long units, int groups) {
  const long long per = (units + groups - 1) / groups;
  return per < 8 ? 8 : per;
}

// The query tile of unit u: its request and head, its index within them, and
// the unit of its first key tile.
struct TileOf {
  int b, h, tile, keys;
  long long start;
  Req r;
  __device__ __forceinline__ TileOf(const PagedArgs& a, const Plan& p, long long u) {
    b = find_request(p.tile_sum, a.S, u);
    r = chunk_part(Req(a, b), kChunkMin);
    const ChunkTiles t(r.total - r.q, r.total);
    const long long per_head = t.before(t.n);
    const long long v = u - p.tile_sum[b];
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
    start = p.tile_sum[b] + h * per_head + t.before(tile);
  }
};

// The segments of one work-group, in order. Work-groups go round the 8 XCDs, and
// each XCD takes a contiguous eighth of the line: neighbouring tiles and heads,
// which read the same keys, share its L2.
struct SegmentSource {
  const PagedArgs& a;
  const Plan& p;
  long long u, end, per;
  int me;
  __device__ __forceinline__ SegmentSource(const PagedArgs& args, const Plan& plan, int group, int groups)
      : a(args), p(plan) {
    me = groups % 8 == 0 ? (group & 7) * (groups >> 3) + (group >> 3) : group;
    const long long units = p.tile_sum[a.S];
    per = range_length(units, groups);
    u = me * per;
    end = u + per < units ? u + per : units;
    if (threadIdx.x == 0) cuts()[me].pieces = 0;
  }
  __device__ __forceinline__ CutTile* cuts() const {
    return reinterpret_cast<CutTile*>(static_cast<char*>(a.ws) + paged_plan_bytes(a.S) + paged_scan_bytes(a.d_h));
  }
  __device__ __forceinline__ Segment next() {
    Segment s{};
    if (u >= end) return s;
    const TileOf t(a, p, u);
    s.b = t.b;
    s.h = t.h;
    s.kvh = t.h / (a.H / a.H_kv);
    s.first = t.r.first;
    s.total = t.r.total;
    s.ctx = t.r.total - t.r.q;
    s.q0 = (s.ctx & ~63) + 256 * t.tile;
    s.tb = (int)(u - t.start);
    const long long stop = t.start + t.keys < end ? t.start + t.keys : end;
    s.te = (int)(stop - t.start);
    s.slot = s.tb == 0 && s.te == t.keys ? -1 : (s.tb > 0 ? 2 * me : 2 * me + 1);
    if (s.slot == 2 * me + 1 && threadIdx.x == 0)
      cuts()[me] = CutTile{1 + (int)((t.start + t.keys - end + per - 1) / per), s.b, s.h, s.first, s.ctx, s.total, s.q0, 0};
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

// A partial state at row `at` of st joined to (M, L, z), 16 lanes of 8 columns.
template <int D>
__device__ __forceinline__ void join_state(const States& st, int64_t at, int sl, float& M, float& L, float (&z)[8]) {
  const float2 ml = st.ml[at];
  f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f}, y = x;
  if (sl < D / 8) {
    x = reinterpret_cast<const f32x4*>(st.z + at * D + 8 * sl)[0];
    y = reinterpret_cast<const f32x4*>(st.z + at * D + 8 * sl)[1];
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

}  // namespace paged
}  // namespace rel
