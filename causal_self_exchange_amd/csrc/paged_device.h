// Device code shared by the kernels of the paged Relation Cache's chunk forward:
// the workspace, the requests' numbers, and the last step of a row.
#pragma once

#include <type_traits>

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
__device__ __forceinline__ long long uni(long long x) {
  return (long long)((unsigned long long)(unsigned)uni((int)(x >> 32)) << 32 | (unsigned)uni((int)x));
}

// The arguments of the kernels for pages of type Tc and tokens of type Tin.
template <typename Tin, typename Tc, bool kTree>
using ScanArgs = typename std::conditional<kTree || !std::is_same<Tin, Tc>::value, PagedExArgs, PagedArgs>::type;

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

// The cut of the work (below; kScanUnit, kExtra and whole row blocks in rel_internal.h):
//   kChunkExtra kExtra of the chunks: five prompts of 500 to 6,000 tokens 1000 us at
//               2, 981 at 4, 1004 at 10.
//   kSnap       the least units that a cut leaves; in fp32, where a unit takes longer,
//               1: four chunks of 16 tokens over 1000 rows 24.5 us at 2, 21.9 at 1.
//   kWhole      in its place, where row blocks stay whole.
//   kMinRange   units of the scan's shortest range (single tokens lose 1 us at 1); in
//               fp32 1: six chunks of up to 97 tokens of 8 heads of 48 34 us at 4, 27 at 1.
//               The chunks need none: kChunkWork units of the scan are more than 1,000
//               of theirs (a query tile takes the place of 8 row blocks at most), 4 and
//               more to a work-group.
constexpr int kChunkExtra = 4;
constexpr int kSnap = 2;
constexpr int kSnapF32 = 1;
constexpr int kWhole = 1 << 30;
constexpr int kMinRange = 4;
constexpr int kMinRangeF32 = 1;

// The least work on query tiles, in units of the scan (32 rows by 128 keys, kExtra
// more a row block): a batch with less leaves it to the scan, whose fixed costs are
// lower. 32 heads of 128 in 8, scan (by selection, without a chunk kernel's launch) and
// tiles: a prompt of 300 tokens (1,800 units) 19 and 33 us, 16 chunks of 32 tokens over
// 1000 rows (5,600) 35 and 58, 64 of 32 over 100 (8,200) 55 and 44, a prompt of 1024
// (10,200) 52 and 49, 8 chunks of 127 over 2000 (19,500) 88 and 96, 32 of 32 over 4000
// (34,800) 174 and 130. The work alone does not part the two: it leaves out into how many
// parts the tiles are cut (the 8 chunks: 192 tiles to 256 work-groups), and between 8,000
// and 30,000 either may be up to a quarter faster than the one that runs.
constexpr int kChunkWork = 8000;

// Query tiles of a request's new tokens (chunk kernel): 256 rows, 32 for each of 8 waves.
//   Full tiles: 256 positions of one head, from ctx rounded down to a multiple of
//   64 (64-key tiles then never straddle a tile's first position, and its own keys
//   are four key tiles). Full tile k needs base64 + 4 (k + 1) key tiles.
//   Shared tiles: the positions left, from a multiple of 32, are `blocks` blocks of
//   32; the blocks of all query heads of a cached head, one head after the other,
//   fill the 8 waves of `tiles` tiles, so that a short chunk, or the end of a long
//   one, leaves few waves idle. Where the tiles would hold fewer than kChunkRows
//   rows each, two row blocks of the scan kernel, which read the keys together, are
//   faster: the tokens left (rest) go there. 32 chunks over 4000 rows, 8 cached
//   heads: 64 rows 113 us by the scan, 128 on tiles; 80 rows 200 and 126.
struct ChunkTiles {
  int base64, full;            // first position / 64, full tiles
  int start, blocks, tiles, keys;   // shared tiles: first position, blocks of a head, per cached head, key tiles each
  int rest;                    // tokens left to the scan
  __device__ __forceinline__ ChunkTiles(int ctx, int total, int G) {
    base64 = ctx >> 6;
    full = (int)(((long long)total - 64LL * base64) >> 8);
    start = full > 0 ? 64 * base64 + 256 * full : ctx & ~31;
    const int tokens = total - max(start, ctx);
    blocks = (total - start + 31) >> 5;
    tiles = (G * blocks + 7) >> 3;
    keys = (int)(((long long)total + 63) >> 6);
    rest = tokens * G < tiles * kChunkRows ? tokens : 0;
    if (rest > 0) tiles = 0;
  }
  // Key tiles and set-ups of the full tiles before k.
  __device__ __forceinline__ long long before(int k) const {
    return (long long)k * (base64 + kChunkExtra) + 2LL * k * (k + 1);
  }
  __device__ __forceinline__ long long units(int H, int H_kv) const {
    return before(full) * H + (long long)tiles * H_kv * (keys + kChunkExtra);
  }
};

// The scan's part of a request: all of its new tokens, or those that the chunk
// kernel leaves (chunks), as a request of their own.
__device__ __forceinline__ Req scan_part(Req r, bool chunks, int G) {
  if (chunks && r.q > 0) {
    const int rest = ChunkTiles(r.total - r.q, r.total, G).rest;
    r.first += r.q - rest;
    r.q = rest;
  }
  return r;
}

// ---- work ---------------------------------------------------------------------
//
// Both kernels cut their work the same way, from the device-side lengths. A unit
// is 128 keys of one row block (scan: row_block rows of a request and cached head)
// or one 64-key tile of one query tile (chunks). The units of all row blocks or
// tiles form one line, request by request, which is cut into equal ranges, one per
// work-group: one request or many, ragged or not. Every row block of a request counts
// the units of its last one, so in a prompt that the scan takes, where a row block ends
// at its own position, the ranges of early row blocks have less to do than those of late
// ones, up to half the work being no keys. Units of a row block's own took fp32 prompts
// of 2,000 tokens from 85 to 78 us, but 3 chunks of 600 over 100 rows from 70 to 94, as
// a segment costs more than two units there. A row
// block or tile counts kExtra (kChunkExtra) units more than its keys: what a segment
// costs beside them (set-up, the waves' states meeting, the output: 3 to 5 us;
// without it the work-group with the most short histories came last, 64 us
// against a median of 43 on drafted tokens of 48 requests). A cut less than kSnap
// units from either end of the keys moves there. A row block or tile that a cut
// divides leaves a partial state in each range it lies in, at most two per range,
// and the join kernel finishes it.

struct Plan {
  long long* unit_sum;    // exclusive sums over the requests; [S] the total
  long long* tile_sum;
  Req* part;              // the requests' parts that the sums count (null: not kept)
};

// The scan's part of a request.
struct ScanRows {
  int rows, blocks, units;     // rows per cached head, row blocks, units of each
  __device__ __forceinline__ ScanRows(const PagedArgs& a, const Req& r, int row_block) {
    rows = r.q * (a.H / a.H_kv);
    blocks = (rows + row_block - 1) / row_block;
    units = paged_scan_units(r.total);
  }
};

struct PlanScratch { long long red[4][2]; };

// What a request's rows on query tiles would be in the scan (units as ScanRows counts
// them: of a prompt about twice its keys).
__device__ __forceinline__ long long tile_work(const PagedArgs& a, const Req& r) {
  if (r.q == 0) return 0;
  Req t = r;
  t.q -= ChunkTiles(r.total - r.q, r.total, a.H / a.H_kv).rest;
  const ScanRows n(a, t, 32);
  return (long long)n.blocks * a.H_kv * (n.units + kExtra);
}

// Fills the sums whose arrays p has, by the work-group's first 256 threads; every
// thread calls. row_block: rows per scan item; chunks: whether the chunk kernel
// is launched. Returns whether there is work for it.
__device__ __forceinline__ bool make_plan(const PagedArgs& a, int row_block, bool chunks, PlanScratch& sc, const Plan& p) {
  const int G = a.H / a.H_kv;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  if (chunks) {
    long long work = 0;
    for (int b = tid; b < a.S && tid < 256; b += 256) work += tile_work(a, Req(a, b));
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) work += __shfl_xor(work, o, 64);
    if (lane == 0 && wave < 4) sc.red[wave][0] = work;
    __syncthreads();
    chunks = sc.red[0][0] + sc.red[1][0] + sc.red[2][0] + sc.red[3][0] >= kChunkWork;
    __syncthreads();
  }
  long long done[2] = {0, 0};
  for (int b0 = 0; b0 < a.S; b0 += 256) {
    const int b = b0 + tid;
    const bool in = tid < 256 && b < a.S;
    long long own[2] = {0, 0};
    Req part;
    if (in) {
      const Req r(a, b);
      const Req s = scan_part(r, chunks, G);
      part = p.unit_sum ? s : r;
      if (p.unit_sum && s.q > 0) {
        const ScanRows n(a, s, row_block);
        own[0] = (long long)n.blocks * a.H_kv * (n.units + kExtra);
      }
      if (p.tile_sum && chunks && r.q > 0) own[1] = ChunkTiles(r.total - r.q, r.total, G).units(a.H, a.H_kv);
    }
    long long x[2] = {own[0], own[1]};
#pragma unroll
    for (int o = 1; o < 64; o <<= 1)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const long long y = __shfl_up(x[k], o, 64);
        if (lane >= o) x[k] += y;
      }
    if (lane == 63 && wave < 4) {
      sc.red[wave][0] = x[0];
      sc.red[wave][1] = x[1];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      long long all = 0;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        x[k] += w < wave ? sc.red[w][k] : 0;
        all += sc.red[w][k];
      }
      x[k] += done[k] - own[k];
      done[k] += all;
    }
    if (in && p.unit_sum) p.unit_sum[b] = x[0];
    if (in && p.tile_sum) p.tile_sum[b] = x[1];
    if (in && p.part) p.part[b] = part;
    __syncthreads();
  }
  if (tid == 0) {
    if (p.unit_sum) p.unit_sum[a.S] = done[0];
    if (p.tile_sum) p.tile_sum[a.S] = done[1];
  }
  return chunks;
}

// The sums that plan_kernel left in the workspace (more than kPlanInline requests).
__device__ __forceinline__ Plan ws_plan(const PagedArgs& a) {
  char* w = static_cast<char*>(a.ws);
  return Plan{reinterpret_cast<long long*>(w), reinterpret_cast<long long*>(w + paged_sum_bytes(a.S)), nullptr};
}

// A kernel's sums: formed in LDS by each work-group for up to kPlanInline
// requests (a launch of its own and the wait for it take 5 us), else read from
// the workspace. chunks: in, whether the chunk kernel is launched; out, whether there
// is work for it.
struct PlanLds {
  PlanScratch sc;
  long long sum[kPlanInline + 1];
  Req part[kPlanInline];
};
__device__ __forceinline__ Plan load_plan(const PagedArgs& a, int row_block, bool& chunks, PlanLds& lds) {
  if (a.S > kPlanInline) {
    const Plan w = ws_plan(a);
    chunks = chunks && w.tile_sum[a.S] > 0;
    return w;
  }
  const Plan p = row_block > 0 ? Plan{lds.sum, nullptr, lds.part} : Plan{nullptr, lds.sum, lds.part};
  chunks = make_plan(a, row_block, chunks, lds.sc, p);
  __syncthreads();
  return p;
}

// The last request b with off[b] <= u: 64 entries are compared at a time.
__device__ __forceinline__ int find_request(const long long* off, int S, long long u) {
  const int lane = threadIdx.x & 63;
  int lo = 0, n = S;
  while (n > 1) {
    const int stride = (n + 63) >> 6;
    const int k = lane * stride;
    const bool le = k < n && off[lo + k] <= u;
    const int cnt = __popcll(__ballot(le));
    lo += (cnt - 1) * stride;
    n = min(stride, n - (cnt - 1) * stride);
  }
  return uni(lo);
}

// v / n; the 64-bit division takes longer than the rest of a segment's numbers.
__device__ __forceinline__ int divide(long long v, long long n) {
  return (v | n) >> 32 == 0 ? (int)((unsigned)v / (unsigned)n) : (int)(v / n);
}

// The row block or tile that the end of a work-group's range divides, for the
// join: pieces = 0 when there is none. Piece 0 is the last segment of the range
// `owner`, piece p the first segment of the p-th range after it.
struct CutRecord {
  int pieces, owner, b, head, first, ctx, total, row0, rows;
  int blocks, slot0;      // of a query tile
  int pad;
};
static_assert(sizeof(CutRecord) == kCutBytes, "workspace layout");

// Records and partial states of the scan or of the chunks.
struct States {
  CutRecord* cuts;
  float2* ml;
  float* z;
  __device__ __forceinline__ static States scan(const PagedArgs& a) {
    return at(static_cast<char*>(a.ws) + paged_scan_offset(a.S), kScanGroups, kScanStateRows);
  }
  __device__ __forceinline__ static States chunk(const PagedArgs& a) {
    return at(static_cast<char*>(a.ws) + paged_chunk_offset(a.S, a.d_h), kChunkGroups, kChunkStateRows);
  }
  __device__ __forceinline__ static States at(char* w, int groups, int rows) {
    char* m = w + groups * kCutBytes;
    return {reinterpret_cast<CutRecord*>(w), reinterpret_cast<float2*>(m),
            reinterpret_cast<float*>(m + (int64_t)rows * sizeof(float2))};
  }
};

// A work-group's range of the line. Work-groups go round the 8 XCDs, and each
// XCD takes a contiguous eighth of the line: neighbouring row blocks, tiles and
// heads, which read the same keys, share its L2. The end of an item that the range
// before began comes last (late): then the work-groups start at the first keys and
// go through them side by side (2048 tokens over 30,001 rows 1284 us in the line's
// order, 1223 so).
struct Range {
  long long u, end, per, units;
  long long late = 0, late_end = 0;
  int me, extra, snap;
  __device__ __forceinline__ Range(long long all, int least, int set_up, int shortest, int group, int groups)
      : units(all), extra(set_up), snap(shortest) {
    me = groups % 8 == 0 ? (group & 7) * (groups >> 3) + (group >> 3) : group;
    per = (units + groups - 1) / groups;
    per = uni(per < least ? least : per);
    u = uni(me * per);
    end = uni(u + per < units ? u + per : units);
  }
  // The first cut moves to its place: u is in the item [start, start + extra + n).
  __device__ __forceinline__ void settle(long long start, int n) {
    const long long k = u - start - extra, stop = start + extra + n;
    if (k < snap) {
      u = uni(start);
    } else if (n - k < snap) {
      u = uni(stop);
    } else if (stop < end) {
      late = u;
      late_end = stop;
      u = uni(stop);
    }
  }
  // Whether there is an item left, or the part kept for last.
  __device__ __forceinline__ bool more() {
    if (u >= end && late < late_end) {
      u = uni(late);
      end = uni(late_end);
      late = late_end;
    }
    return u < end;
  }
  // The part of an item of n units at `start` that begins at u: units [k0, k1) of
  // its keys, in the partial state `slot` (-1: all of them); where the range's end
  // divides it, pieces and owner as in CutRecord. false: the item belongs to the
  // next range.
  __device__ __forceinline__ bool take(long long start, int n, int& k0, int& k1, int& slot, int& pieces, int& owner) {
    const long long stop = start + extra + n;
    const bool inside = u > start;
    k0 = inside ? (int)(u - start - extra) : 0;
    k1 = n;
    pieces = 0;
    u = uni(stop);
    if (end < stop) {
      const long long k = end - start - extra;
      if (k < snap) return false;
      if (n - k >= snap) {
        k1 = (int)k;
        // The range of the first cut that stays in the item; the cuts after it, and one.
        owner = inside ? (int)((start + extra + snap + per - 1) / per) - 1 : me;
        pieces = 2 + (int)((stop - snap - (owner + 1) * per) / per);
      }
    }
    slot = inside ? 2 * me : (pieces ? 2 * me + 1 : -1);
    return true;
  }
};

// A range's part of one row block: keys [k0, k1) (any = 0 for none).
struct ScanSegment {
  int b, kvh, first, ctx, total, row0, rows, k0, k1, slot, any;
};

struct ScanSource {
  const PagedArgs& a;
  const Plan& p;
  Range rg;
  int row_block;
  bool chunks;
  CutRecord* cuts;
  struct Block {
    int b, kvh, row0, rows, units;
    long long start;
    Req r;
  };
  __device__ __forceinline__ ScanSource(const PagedArgs& args, const Plan& plan, int rows, bool with_chunks, int least, int snap)
      : a(args), p(plan), rg(plan.unit_sum[args.S], least, kExtra, snap, blockIdx.x, gridDim.x), row_block(rows),
        chunks(with_chunks), cuts(States::scan(args).cuts) {
    if (threadIdx.x == 0) cuts[rg.me].pieces = 0;
    if (rg.u < rg.end) {
      const Block k = block_of(rg.u);
      rg.settle(k.start, k.units);
    }
  }
  __device__ __forceinline__ Block block_of(long long u) const {
    Block k;
    k.b = find_request(p.unit_sum, a.S, u);
    k.r = p.part ? p.part[k.b] : scan_part(Req(a, k.b), chunks, a.H / a.H_kv);
    const ScanRows n(a, k.r, row_block);
    k.units = n.units;
    const long long v = u - p.unit_sum[k.b];
    const int item = divide(v, n.units + kExtra);
    k.start = p.unit_sum[k.b] + (long long)item * (n.units + kExtra);
    // Stripes of as many heads as a range has items, row block by row block: the
    // row blocks of a head lie in neighbouring ranges, which read its keys at the
    // same time, and not one after the other in the same (64 requests of 8 tokens of
    // 64 heads in 8 over 4096 rows: 212 us, head by head 374).
    const int most = min(a.H_kv, max(1, divide(rg.per, n.units + kExtra)));
    const int first = item / (most * n.blocks) * most;   // the stripe's first head
    const int width = min(most, a.H_kv - first);
    const int rest = item - first * n.blocks, rb = rest / width;
    k.kvh = first + rest - rb * width;
    k.row0 = rb * row_block;
    k.rows = min(row_block, n.rows - k.row0);
    return k;
  }
  __device__ __forceinline__ ScanSegment next() {
    ScanSegment s{};
    Block k;
    int u0, u1, pieces, owner;
    do {
      if (!rg.more()) return s;
      k = block_of(rg.u);
    } while (!rg.take(k.start, k.units, u0, u1, s.slot, pieces, owner));
    s.any = 1;
    s.b = k.b;
    s.kvh = k.kvh;
    s.row0 = k.row0;
    s.rows = k.rows;
    s.first = k.r.first;
    s.ctx = k.r.total - k.r.q;
    s.total = k.r.total;
    // Keys below the block's last row's position.
    const int last = s.ctx + (s.row0 + s.rows - 1) / (a.H / a.H_kv);
    s.k0 = u0 * kScanUnit;
    s.k1 = (int)min((long long)last, (long long)u1 * kScanUnit);
    if (pieces > 0 && threadIdx.x == 0)
      cuts[rg.me] = CutRecord{pieces, owner, s.b, s.kvh, s.first, s.ctx, s.total, s.row0, s.rows, 0, 0, 0};
    return s;
  }
};

// A range's part of one query tile: key tiles [tb, te), te = 0 for none. Rows
// 32 w .. 32 w + 31 of the tile are block (slot0 + w) % blocks of positions from q0
// of the group's head h + (slot0 + w) / blocks (none past the group).
struct Segment {
  int b, h, kvh;
  int first, ctx, total;       // packed token of the chunk's first row, its position, cached rows
  int q0, blocks, slot0;
  int tb, te, slot;
  // The same, every field in a scalar register.
  __device__ __forceinline__ Segment uniform() const {
    return Segment{uni(b),  uni(h),      uni(kvh),   uni(first), uni(ctx), uni(total),
                   uni(q0), uni(blocks), uni(slot0), uni(tb),    uni(te),  uni(slot)};
  }
};

struct ChunkSource {
  const PagedArgs& a;
  const Plan& p;
  Range rg;
  CutRecord* cuts;
  __device__ __forceinline__ ChunkSource(const PagedArgs& args, const Plan& plan)
      : a(args), p(plan), rg(plan.tile_sum[args.S], 1, kChunkExtra, kSnap, blockIdx.x, gridDim.x),
        cuts(States::chunk(args).cuts) {
    if (threadIdx.x == 0) cuts[rg.me].pieces = 0;
    if (rg.u < rg.end) {
      Segment s;
      int keys;
      const long long start = tile_of(rg.u, s, keys);
      rg.settle(start, keys);
    }
  }
  // The query tile of unit u in s, its key tiles, and the unit it starts at.
  __device__ __forceinline__ long long tile_of(long long u, Segment& s, int& keys) const {
    const int G = a.H / a.H_kv;
    s.b = find_request(p.tile_sum, a.S, u);
    const Req r = p.part ? p.part[s.b] : Req(a, s.b);
    s.first = r.first;
    s.total = r.total;
    s.ctx = r.total - r.q;
    const ChunkTiles t(s.ctx, s.total, G);
    const long long v = u - p.tile_sum[s.b], per_head = t.before(t.full), all_full = per_head * a.H;
    if (v < all_full) {
      s.h = divide(v, per_head);
      const long long w = v - s.h * per_head;
      int lo = 0, hi = t.full - 1;                       // the last tile that starts at or before w
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (t.before(mid) <= w) lo = mid;
        else hi = mid - 1;
      }
      s.kvh = s.h / G;
      s.q0 = 64 * t.base64 + 256 * lo;
      s.blocks = 8;
      s.slot0 = 0;
      keys = t.base64 + 4 * (lo + 1);
      return u - (w - t.before(lo));
    }
    const int item = divide(v - all_full, t.keys + kChunkExtra);   // cached head, tile
    s.kvh = item / t.tiles;
    s.h = s.kvh * G;
    s.q0 = t.start;
    s.blocks = t.blocks;
    s.slot0 = 8 * (item - s.kvh * t.tiles);
    keys = t.keys;
    return p.tile_sum[s.b] + all_full + (long long)item * (t.keys + kChunkExtra);
  }
  __device__ __forceinline__ Segment next() {
    Segment s{};
    while (rg.more()) {
      int keys, pieces, owner;
      const long long start = tile_of(rg.u, s, keys);
      if (rg.take(start, keys, s.tb, s.te, s.slot, pieces, owner)) {
        if (pieces > 0 && threadIdx.x == 0)
          cuts[rg.me] = CutRecord{pieces, owner, s.b, s.h, s.first, s.ctx, s.total, s.q0, 256, s.blocks, s.slot0, 0};
        return s;
      }
    }
    s.te = 0;
    return s;
  }
};

// ---- 8-bit rows -----------------------------------------------------------------

// The value of a scale byte: 2^(e - 127). 255, which is none, reads as 2^127, so that a
// masked row's weight of 0 stays 0 whatever its page holds; 0 reads as 0.
__device__ __forceinline__ float scale_of(unsigned e) { return __uint_as_float(min(e, 254u) << 23); }

// Eight e4m3 values times a power of two, as bf16: exact where the product is a normal
// bf16 number.
__device__ __forceinline__ u32x4 e4m3_to_bf16(u32x2 x, float scale) {
  return u32x4{__builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x[0], scale, false)),
               __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x[0], scale, true)),
               __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x[1], scale, false)),
               __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x[1], scale, true))};
}

// Lane i of a group of 16 receives byte i % 8 of the 8-byte rows that the group's lanes
// i / 8 + 2 k address, k = 0 .. 7.
__device__ __forceinline__ u32x2 lds_tr8_read(const char* p) {
  typedef int i32x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr8_b64_v2i32((__attribute__((address_space(3))) i32x2*)(p)));
}

// ---- trees ----------------------------------------------------------------------

// Which of the new tokens o .. o + 3 of its request the packed token t sees, in bits 0 to
// 3: its ancestors, and all rows that were cached before (o < 0). Bits at and past its own
// place are the caller's to mask.
__device__ __forceinline__ unsigned tree_bits(const PagedExArgs& a, int t, int o) {
  const uint32_t* const row = a.tree + (size_t)t * a.words;
  const int w = o >> 5;
  const unsigned lo = w < 0 ? ~0u : (w < a.words ? row[w] : 0u);
  const unsigned hi = w + 1 < 0 ? ~0u : (w + 1 < a.words ? row[w + 1] : 0u);
  return (unsigned)(((unsigned long long)hi << 32 | lo) >> (o & 31)) & 15u;
}

// How many new tokens the packed token t, the tq'th of its request, sees; below, the same
// by 16 lanes.
__device__ __forceinline__ int ancestors_of(const PagedExArgs& a, int t, int tq) {
  int n = 0;
  for (int w = 0; 32 * w < tq; ++w) {
    const uint32_t x = a.tree[(size_t)t * a.words + w];
    const int left = tq - 32 * w;
    n += __popc(left < 32 ? x & ((1u << left) - 1) : x);
  }
  return n;
}
__device__ __forceinline__ int ancestors(const PagedExArgs& a, int t, int tq, int sl) {
  int n = 0;
  for (int w = sl; 32 * w < tq; w += 16) {
    const uint32_t x = a.tree[(size_t)t * a.words + w];
    const int left = tq - 32 * w;
    n += __popc(left < 32 ? x & ((1u << left) - 1) : x);
  }
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) n += __shfl_xor(n, o, 16);
  return n;
}

// ---- rows ---------------------------------------------------------------------

// Eight elements as they lie in memory.
template <typename Tin>
struct Raw8 {
  static constexpr int kWords = sizeof(Tin) / 2;
  u32x4 w[kWords];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = u32x4{0u, 0u, 0u, 0u};
  }
  __device__ __forceinline__ void load(const Tin* p) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = reinterpret_cast<const u32x4*>(p)[i];
  }
  __device__ __forceinline__ float operator[](int e) const {
    if constexpr (sizeof(Tin) == 2) return (float)__builtin_bit_cast(bf16x8, w[0])[e];
    else return __builtin_bit_cast(f32x4, w[e >> 2])[e & 3];
  }
};

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

// A row's own P1, P2 and V (zeros where it has none), by 16 lanes of 8 columns
// each: loaded ahead of finish_row, behind whose table lookup they would wait. 8-bit rows
// become bf16 here, exactly.
template <typename Tin, int D, typename Tc>
struct OwnRow {
  Raw8<Tin> q, k, v;
  __device__ __forceinline__ void load(const ScanArgs<Tin, Tc, false>& a, int b, int t, int h, int pos, int sl, bool row_ok) {
    q.zero();
    k.zero();
    v.zero();
    if (!row_ok || sl >= D / 8) return;
    const int page = a.table[(size_t)b * a.max_pages + (pos >> a.page_shift)];
    q.load(static_cast<const Tin*>(a.P1) + (size_t)t * a.ld1 + (size_t)h * D + 8 * sl);
    if (page >= 0 && page < a.n_pages) {
      const int kvh = h / (a.H / a.H_kv), off = pos & ((1 << a.page_shift) - 1);
      const size_t head = (size_t)page * a.H_kv + kvh, row = ((head << a.page_shift) + off) * D + 8 * sl;
      if constexpr (sizeof(Tc) == 1) {
        const uint8_t* const sc = a.scale + (head << (a.page_shift + 1)) + off;
        k.w[0] = e4m3_to_bf16(*reinterpret_cast<const u32x2*>(static_cast<const uint8_t*>(a.cP2) + row), scale_of(sc[0]));
        v.w[0] = e4m3_to_bf16(*reinterpret_cast<const u32x2*>(static_cast<const uint8_t*>(a.cV) + row),
                              scale_of(sc[1 << a.page_shift]));
      } else {
        k.load(static_cast<const Tin*>(a.cP2) + row);
        v.load(static_cast<const Tin*>(a.cV) + row);
      }
    }
  }
};

// Output of one row from its history's state, by 16 lanes of 8 columns each:
// z (sum of weights times V), m (log2 stabiliser) and l (sum of weights); the
// Self evidence and V come from the row's own cached row.
// seen: the rows before its own that it sees.
template <typename Tin, int D, typename Tc>
__device__ __forceinline__ void finish_row(const PagedArgs& a, const HeadParams& hp, const OwnRow<Tin, D, Tc>& own, int t,
                                           int h, int seen, int sl, float m, float l, const float (&z)[8], bool row_ok) {
  float u = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) u = fmaf(own.q[e], own.k[e], u);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) u += __shfl_xor(u, o, 16);
  if (!row_ok || sl >= D / 8) return;
  const float S = sigmoid_f32(u * hp.scale * hp.inv_tau[h]);
  const RowCombine c(S, m * kLn2, l, hp.lambda * logf((float)(seen + 1)));
  float y[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) y[e] = c.w_self * own.v[e] + c.w_hist * z[e];
  store8(static_cast<Tin*>(a.Y) + ((size_t)t * a.H + h) * D + 8 * sl, y);
}

// The state (m, l, zp) joined to (M, L, z).
__device__ __forceinline__ void merge(float& M, float& L, float (&z)[8], float m, float l, const float (&zp)[8]) {
  const float Mn = fmaxf(M, m);
  const float f = __builtin_amdgcn_exp2f(M - Mn), fp = __builtin_amdgcn_exp2f(m - Mn);
  M = Mn;
  L = L * f + l * fp;
#pragma unroll
  for (int e = 0; e < 8; ++e) z[e] = z[e] * f + zp[e] * fp;
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
  float zp[8];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    zp[e] = x[e];
    zp[4 + e] = y[e];
  }
  merge(M, L, z, ml.x, ml.y, zp);
}

}  // namespace paged
}  // namespace rel
