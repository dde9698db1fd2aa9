// Query tiles for the paged Relation Cache's rows over 8-bit pages and of trees
// (relation_paged_fwd_ex): where a request has many rows to a cached head, the keys are
// brought into LDS once for 256 of them. tile_use below says which requests come here.
//
// A work-group of eight waves takes 256 rows (whole tokens of a request, times the query
// heads of a cached head), 32 to a wave, and goes through its keys in tiles of 64, which
// pass through LDS as bf16 in the layouts of QTile: two buffers, one barrier a tile (of four
// waves, two to a compute unit, for up to 128 rows of heads of up to 64). A tile of 16-bit
// rows is loaded into registers while the one before is computed, an 8-bit tile straight
// into a ring in LDS, four tiles ahead, and becomes bf16 on its way from there, its values
// times their scale, exactly. The products are the 32x32x16 ones of the forward: a lane
// holds one query row's scores and weights, and no state of a row is divided between waves.
//
// The weights are rounded to bf16 once for the transport, and summed rounded, as in the
// forward. Two bf16 terms a weight, as in the scan, took six chunks of 100 to 1,500 tokens of
// 32 heads in 8 of 128 from 317 to 408 us, 48 trees of 2 to 24 tokens of 16 in 4 of 64 from 84
// to 99, 16 of 20 to 64 over up to 30,000 rows of 32 in 8 of 128 from 324 to 398. The results
// are off by 0.0021 to 0.0022 of their norm, with two terms by 0.0017, the rounding of Y.
//
// Bound by the loop's issue: a wave's tile is 36 products (1,090 cycles of the matrix unit),
// 96 transcendentals and about 290 other instructions; a compute unit's takes 4,450 cycles
// where the products alone would take 2,180 (with one wave to a SIMD 3,240, of 1,090). Those
// six chunks, over up to 6,000 8-bit rows, take 295 to 330 us, 0.65 to 0.73 PFLOP/s; two of
// 4,000 of 32 heads in 4, whose segments are longer, 550 us, 0.82 (a large bf16 product by the
// library 1.32). A segment costs about eight tiles beside its keys (kTileExtra).
//
// The keys of all row blocks are cut into equal ranges as in the scan (paged_device.h);
// here a row block counts its own keys, so early blocks of a prompt take less of a range
// than late ones.
#pragma once

#include "paged_scan.h"

namespace rel {

namespace {

using namespace paged;

constexpr int kTileExtra = 8;             // units (64 keys of a row block) that a segment costs beside its keys
constexpr int kTileSnap = 2;
constexpr int kTileMin = 4;               // units of the shortest range

// Row blocks of a request: `tokens` of its new ones each.
// A tile of up to 128 rows, one wave to a SIMD, takes 3,240 cycles, of more 4,450: 12 to 16.
struct RowBlocks {
  int tokens, blocks, ctx, weight;
  __device__ __forceinline__ RowBlocks(const PagedArgs& a, const Req& r, int rows) {
    tokens = rows / (a.H / a.H_kv);
    blocks = (r.q + tokens - 1) / tokens;
    ctx = r.total - r.q;
    weight = rows == 256 && (long long)r.q * (a.H / a.H_kv) <= 128 ? 12 : 16;
  }
  // Units of the row blocks before k of one cached head: each has ctx and the tokens up to
  // its own last one, in 64ths times the weight, rounded over the sum, and one for what that
  // leaves.
  __device__ __forceinline__ long long before(int k) const {
    return (long long)k * (kTileExtra + 1) + ((((long long)k * ctx + (long long)tokens * k * (k + 1) / 2) * weight) >> 10);
  }
  __device__ __forceinline__ int size(int k) const { return (int)(before(k + 1) - before(k)); }
};

struct TilePlanLds {
  long long red[8];
  long long sum[kPlanInline + 1];
  Req part[kPlanInline];
};

// Exclusive sums of the requests' units in sum[0 .. S], by a whole work-group of W waves.
// Requests of up to `few` new tokens are the scan's.
template <int W>
__device__ __forceinline__ void tile_plan(const PagedArgs& a, int rows, int few, long long* sum, Req* part, long long* red) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  long long done = 0;
  for (int b0 = 0; b0 < a.S; b0 += 64 * W) {
    const int b = b0 + tid;
    long long own = 0;
    if (b < a.S) {
      const Req r(a, b);
      if (part) part[b] = r;
      if (r.q > few) {
        const RowBlocks n(a, r, rows);
        own = n.before(n.blocks) * a.H_kv;
      }
    }
    long long x = own;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const long long y = __shfl_up(x, o, 64);
      if (lane >= o) x += y;
    }
    if (lane == 63) red[wave] = x;
    __syncthreads();
    long long all = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      x += w < wave ? red[w] : 0;
      all += red[w];
    }
    if (b < a.S) sum[b] = done + x - own;
    done += all;
    __syncthreads();
  }
  if (tid == 0) sum[a.S] = done;
}

// The tiles' sums, and in the second work-group the scan's.
__global__ __launch_bounds__(256) void tile_plan_kernel(PagedArgs a, int rows, int few) {
  __shared__ long long red[4];
  __shared__ PlanScratch sc;
  const Plan p = ws_plan(a);
  if (blockIdx.x == 0) {
    tile_plan<4>(a, rows, few, p.tile_sum, nullptr, red);
  } else {
    a.max_new = min(few, a.max_new);
    make_plan(a, 32, false, sc, Plan{p.unit_sum, nullptr, nullptr});
  }
}

// States of divided row blocks: the second half of the scan's records (it has two row blocks
// to an item here), room for two of every work-group's in the chunks' part of the workspace
// (which is there: paged_chunks_possible).
constexpr int tile_groups(int rows) { return kChunkStateRows / (2 * rows); }
static_assert(tile_groups(128) <= kScanGroups / 2, "a record for each");
__device__ __forceinline__ States tile_states(const PagedArgs& a) {
  States s = States::chunk(a);
  s.cuts = States::scan(a).cuts + kScanGroups / 2;
  return s;
}

struct TileSource {
  const PagedArgs& a;
  const long long* sum;
  const Req* part;
  Range rg;
  int rows;
  CutRecord* cuts;
  struct Block {
    int b, kvh, rb, units;
    long long start;
    Req r;
  };
  __device__ __forceinline__ TileSource(const PagedArgs& args, int block_rows, const long long* s, const Req* p)
      : a(args), sum(s), part(p), rg(s[args.S], kTileMin, kTileExtra, kTileSnap, blockIdx.x, gridDim.x), rows(block_rows),
        cuts(tile_states(args).cuts) {
    if (threadIdx.x == 0) cuts[rg.me].pieces = 0;
    if (rg.u < rg.end) {
      const Block k = block_of(rg.u);
      rg.settle(k.start, k.units);
    }
  }
  // Stripes of as many heads as a range has items, row block by row block (ScanSource).
  __device__ __forceinline__ Block block_of(long long u) const {
    Block k;
    k.b = find_request(sum, a.S, u);
    k.r = part ? part[k.b] : Req(a, k.b);
    const RowBlocks n(a, k.r, rows);
    const long long head = n.before(n.blocks);
    long long v = u - sum[k.b];
    const int most = min(a.H_kv, max(1, divide(rg.per * n.blocks, head)));
    const int first = divide(v, head * most) * most;      // the stripe's first head
    const int width = min(most, a.H_kv - first);
    v -= head * first;
    int lo = 0, hi = n.blocks - 1;                        // the last row block that starts at or before v
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (width * n.before(mid) <= v) lo = mid;
      else hi = mid - 1;
    }
    const int size = n.size(lo);
    v -= width * n.before(lo);
    const int x = divide(v, size);
    k.kvh = first + x;
    k.rb = lo;
    k.units = size - kTileExtra;
    k.start = u - (v - (long long)x * size);
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
    const RowBlocks n(a, k.r, rows);
    const int G = a.H / a.H_kv;
    const int tokens = min(n.tokens, k.r.q - k.rb * n.tokens);
    s.any = 1;
    s.b = k.b;
    s.kvh = k.kvh;
    s.row0 = k.rb * n.tokens * G;
    s.rows = tokens * G;
    s.first = k.r.first;
    s.ctx = n.ctx;
    s.total = k.r.total;
    // Keys below the block's last row's position, by whole tiles. Units cover them, and up to
    // two more.
    const int last = n.ctx + k.rb * n.tokens + tokens - 1;
    auto key_of = [&](int u) __attribute__((always_inline)) -> long long {
      return 64 * ((n.weight == 16 ? u : ((long long)u * 16 + 11) / 12));
    };
    s.k0 = (int)min((long long)((last + 63) & ~63), key_of(u0));
    s.k1 = u1 == k.units ? last : (int)min((long long)last, key_of(u1));
    if (pieces > 0 && threadIdx.x == 0)
      cuts[rg.me] = CutRecord{pieces, owner, s.b, s.kvh, s.first, s.ctx, s.total, s.row0, s.rows, 0, 0, 0};
    return s;
  }
};

// A tile of 64 rows in LDS, blocks of 8 rows by 8 chunks of 16 bytes: P2's block has its
// chunks 144 bytes apart, rows of a chunk next to each other; V's is the transposed layout
// of mfma_tile.h. Operand reads are a lane base and an immediate, without bank conflicts.
// So are the stores of a row's pieces, by lanes that hold neighbouring ones (an 8-bit piece
// is two chunks, so a store has every other chunk of a row; the second eight chunks are
// 128 bytes further on, in the other half of the banks).
template <int D>
struct QTile {
  using L = TileLayout<D>;
  static constexpr int kKBlock = 1152, kChunk = 144, kPad = 128;
  static constexpr int kHalves = D / 64;
  static constexpr int kKHalf = 8 * kKBlock + kPad, kVHalf = 8 * L::kVBlock + kPad;
  static constexpr int kVOff = kHalves * kKHalf;
  static constexpr int kBuf = kVOff + kHalves * kVHalf;
  static constexpr int k_imm(int kb, int ds) { return kKHalf * (ds / 4) + 4 * kKBlock * kb + 2 * kChunk * (ds % 4); }
  // Rows 8 half .. of the transport operand (kb, ks, db).
  static constexpr int v_imm(int kb, int ks, int db, int half) { return kVHalf * (db >> 1) + L::kVBlock * (4 * kb + 2 * ks + half); }
  __device__ static int k_base(int lq, int hf) { return kKBlock * (lq >> 3) + 16 * (lq & 7) + kChunk * hf; }
  __device__ static int k_at(int row, int cc) { return kKHalf * (cc >> 3) + kKBlock * (row >> 3) + 16 * (row & 7) + kChunk * (cc & 7); }
  __device__ static int v_at(int row, int cc) {
    const int rr = row & 7;
    return kVOff + kVHalf * (cc >> 3) + L::kVBlock * (row >> 3) + 16 * (8 * rr + ((cc & 7) ^ (4 * ((rr >> 1) & 1))));
  }
  __device__ static bf16x8 v_operand(const VBase& vb, int kb, int ks, int db) {
    const char* const p = (db & 1) ? vb.odd : vb.even;
    bf16x8 v;
    v.lo = lds_tr_read(p + v_imm(kb, ks, db, 0));
    v.hi = lds_tr_read(p + v_imm(kb, ks, db, 1));
    return v;
  }
};

// A work-group barrier for LDS data alone: the next tiles' loads are not waited for.
__device__ __forceinline__ void tile_barrier() {
  asm volatile("" ::: "memory");
  wait_vm_lgkm<63, 0>();
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// The wait states between the last products and the first read of their results.
__device__ __forceinline__ void settle(f32x16 (&o)[2], f32x4& l) {
  asm volatile("s_nop 15\n\ts_nop 3" : "+v"(o[0]), "+v"(o[1]), "+v"(l) : : "memory");
}
__device__ __forceinline__ void settle(f32x16 (&o)[4], f32x4& l) {
  asm volatile("s_nop 15\n\ts_nop 3" : "+v"(o[0]), "+v"(o[1]), "+v"(o[2]), "+v"(o[3]), "+v"(l) : : "memory");
}

// What a block step does with the weights.
enum : int { kNoWeights = 0, kAllSeen = 1, kMasked = 2 };

// D: the layout's columns (64, 128), DR those of a row in memory; W: waves.
template <int D, int DR, int W, typename Tc, bool kTree>
__global__ __launch_bounds__(64 * W, 2) void tile_kernel(ScanArgs<__bf16, Tc, kTree> a, HeadParams hp, int few) {
  constexpr int kTileWaves = W, kTileRowsQ = 32 * W;
  using L = TileLayout<D>;
  using Q = QTile<D>;
  constexpr bool k8 = sizeof(Tc) == 1;
  constexpr int kEs = (int)sizeof(Tc);
  constexpr int kPiece = 16 / kEs;                        // elements of a 16-byte piece of a row
  constexpr int kPieces = D / kPiece;                     // of a row in the layout
  constexpr int kWaveRows = 64 / kPieces;                 // rows of a wave's piece, within one page
  // Where four waves hold a tile of P2, the others take V's.
  constexpr bool kSplit = kWaveRows * kTileWaves > 64;
  static_assert(!kSplit || k8, "16-bit rows have two pieces a lane");
  constexpr int kMovers = kSplit ? kTileWaves / 2 : kTileWaves;
  constexpr int kStepRows = kMovers * kWaveRows;          // rows between a thread's pieces
  constexpr int kUnits = 64 / kStepRows;                  // pieces of a tile (of P2, of V) per thread
  constexpr int kYStride = 2 * D + 16;                    // bytes of a row of Y on its way out
  // 8-bit tiles wait in LDS, each lane's pieces where it alone reads them: kAhead tiles of
  // a wave's P2 and V pieces and of their scales.
  constexpr int kAhead = k8 ? 4 : 0;
  constexpr int kParts = kSplit ? 1 : 2;
  constexpr int kRaw = kParts * 1024 + 256;
  constexpr int kTileLoads = kParts + 1;                  // direct loads of a wave and tile
  constexpr int kRing = 2 * Q::kBuf;
  constexpr int kScan = kRing + kTileWaves * kAhead * kRaw;
  constexpr int kBytes = kScan > kTileRowsQ * kYStride ? kScan : kTileRowsQ * kYStride;
  constexpr int kNS = 2 * L::kDs;                         // MFMA steps of a block
  constexpr float kFinite = 0x1p100f;
  constexpr float kPartFinite = 0x1p127f / tile_groups(kTileRowsQ);   // a row block has at most one part to a range
  __shared__ __attribute__((aligned(16))) char smem[kBytes];
  __shared__ int s_bad[kTileWaves];
  __shared__ TilePlanLds lds;

  const long long* sum = ws_plan(a).tile_sum;
  if (a.S <= kPlanInline) {
    tile_plan<W>(a, kTileRowsQ, few, lds.sum, lds.part, lds.red);
    __syncthreads();
    sum = lds.sum;
  }
  const States states = tile_states(a);
  const int G = a.H / a.H_kv;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lq = lane & 31, hf = lane >> 5;
  const float k2 = hp.scale * kLog2e;
  const int pmask = (1 << a.page_shift) - 1;

  // A operand of the row-sum product (16x16x32, the weights as B operand): with ones where
  // lane bits 2 and 4 agree, lane l's results are the sum of its own row l % 32.
  bf16x8 sel;
  {
    const __bf16 v = (((lane >> 2) ^ (lane >> 4)) & 1) ? (__bf16)0.0f : (__bf16)1.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) sel[e] = v;
  }

  // This thread's pieces of a tile: rows prow + kStepRows i, piece pc.
  const int wrow = lane / kPieces, pc = lane % kPieces;
  const int mover = wave % kMovers;
  const int prow = kWaveRows * mover + wrow;
  const int src = pc * kPiece < DR ? wrow * DR * kEs + 16 * pc : kOutOfRange;
  struct Pieces { u32x4 x[kUnits]; };

  // Token of a row block that its row x belongs to, x / G (0.5 / G from an integer, far more
  // than the product is off for x, G <= 256).
  const float per_head = 1.0f / (float)G;
  auto token = [&](int x) __attribute__((always_inline)) -> int { return (int)(((float)x + 0.5f) * per_head); };

  const int koff = Q::k_base(lq, hf), te = L::tr_base(lane, false), to = L::tr_base(lane, true);
  TileSource source(a, kTileRowsQ, sum, a.S <= kPlanInline ? lds.part : nullptr);
  ScanSegment cur = source.next();
  while (cur.any) {
    const int b = uni(cur.b), kvh = uni(cur.kvh), first = uni(cur.first), ctx = uni(cur.ctx), total = uni(cur.total);
    const int row0 = uni(cur.row0), rows = uni(cur.rows), slot = uni(cur.slot), k0 = uni(cur.k0), k1 = uni(cur.k1);
    const int t0 = k0 >> 6, J = max(((k1 + 63) >> 6) - t0, 0);   // key tiles t0 .. t0 + J - 1, counted from 0 below
    bool tree = false;
    if constexpr (kTree) tree = total - ctx <= 32 * a.words;

    // Page of the wave's rows of each piece: lane x holds the entry of tile win0 + x, -1 for
    // tiles past the segment and for pages outside the cache. P2 is loaded a tile ahead of V.
    int win[kUnits], win0 = 0;
    auto load_window = [&](int t) __attribute__((always_inline)) {
      win0 = max(t - 32, 0);
#pragma unroll
      for (int i = 0; i < kUnits; ++i) {
        const int key = 64 * (t0 + win0 + lane) + kStepRows * i + kWaveRows * mover;
        win[i] = win0 + lane < J && key < total ? a.table[(size_t)b * a.max_pages + (key >> a.page_shift)] : -1;
      }
      // Waited for here, and not at the first use of each iteration.
#pragma unroll
      for (int i = 0; i < kUnits; ++i) {
        win[i] = win[i] < a.n_pages ? win[i] : -1;
        asm volatile("" : "+v"(win[i]));
      }
    };
    load_window(0);
    // Rows at and past the request's end, tiles past the segment and pages outside the
    // cache are zeros.
    struct Rows { size_t head; int off, left; };          // cached head's page, row in it, rows
    auto rows_of = [&](int t, int i) __attribute__((always_inline)) -> Rows {
      const int key = 64 * (t0 + t) + kStepRows * i + kWaveRows * mover;
      const int page = __builtin_amdgcn_readlane(win[i], (t - win0) & 63);
      const bool in = page >= 0;
      return Rows{(size_t)(in ? page : 0) * a.H_kv + kvh, key & pmask, in ? min(total - key, kWaveRows) : 0};
    };
    auto base_of = [&](int part, const Rows& r) __attribute__((always_inline)) -> const char* {
      return static_cast<const char*>(part ? a.cV : a.cP2) + ((r.head << a.page_shift) + r.off) * (DR * kEs);
    };
    auto put = [&](int part, int t, int row, int cc, const u32x4& x) __attribute__((always_inline)) {
      *reinterpret_cast<u32x4*>(smem + (t & 1) * Q::kBuf + (part ? Q::v_at(row, cc) : Q::k_at(row, cc))) = x;
    };
    // 16-bit pages: a tile's pieces in registers.
    auto load = [&](int part, int t, Pieces& p) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < kUnits; ++i) {
        const Rows r = rows_of(t, i);
        p.x[i] = __builtin_amdgcn_raw_buffer_load_b128(rsrc(base_of(part, r), r.left * DR * kEs), src, 0, 0);
      }
    };
    auto store = [&](int part, int t, const Pieces& p) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < kUnits; ++i) put(part, t, prow + kStepRows * i, pc, p.x[i]);
    };
    // 8-bit pages: direct loads of tile t into its place in LDS (its window is there), and
    // from there as bf16. No branches: they would part a block step's products from its
    // weights.
    char* const raw = smem + kRing + wave * (kAhead * kRaw);
    const int second = kSplit ? wave >= kMovers : 0;      // the part that a wave with one moves
    auto fetch = [&](int t) __attribute__((always_inline)) {
      const Rows r = rows_of(t, 0);
      char* const at = raw + (t & 3) * kRaw;
      auto words = [&](const void* base, int bytes) __attribute__((always_inline)) -> u32x4 {
        u32x4 w = rsrc_words(base, bytes);
#pragma unroll
        for (int x = 0; x < 3; ++x) w[x] = (unsigned)uni((int)w[x]);
        return w;
      };
#pragma unroll
      for (int i = 0; i < kParts; ++i) dma16(words(base_of(kSplit ? second : i, r), r.left * DR), at + 1024 * i, src);
      // Scales: dwords of four rows, of P2 by the first lanes, of V (its rows lie a page's
      // rows further on) by the next; one of the two where the wave moves one.
      constexpr int kDw = kWaveRows / 4;
      const int ps = 1 << a.page_shift;
      const u32x4 sc = words(a.scale + (r.head << (a.page_shift + 1)) + r.off, r.left > 0 ? 2 * ps - r.off : 0);
      dma4(sc, at + 1024 * kParts, lane < kDw ? 4 * lane + second * ps : (!kSplit && lane < 2 * kDw ? ps + 4 * (lane - kDw) : kOutOfRange));
    };
    // Where this lane's piece of an even tile goes, of P2 or of V; odd tiles kBuf further on.
    const int kput = Q::k_at(prow, 2 * pc), vput = Q::v_at(prow, 2 * pc);
    const int vput1 = Q::v_at(prow, 2 * pc + 1) - vput;
    struct Wide { u32x4 x; int e; };
    auto peek = [&](int part, int t) __attribute__((always_inline)) -> Wide {
      const char* const at = raw + (t & 3) * kRaw;
      return Wide{*reinterpret_cast<const u32x4*>(at + (kSplit ? 0 : 1024 * part) + 16 * lane),
                  reinterpret_cast<const uint8_t*>(at + 1024 * kParts)[(kSplit ? 0 : kWaveRows * part) + wrow]};
    };
    auto widen = [&](int part, int t, const Wide& w) __attribute__((always_inline)) {
      const float f = scale_of((unsigned)w.e);
      char* const to = smem + (t & 1) * Q::kBuf + (part ? vput : kput);
      *reinterpret_cast<u32x4*>(to) = e4m3_to_bf16(u32x2{w.x[0], w.x[1]}, f);
      *reinterpret_cast<u32x4*>(to + (part ? vput1 : Q::kChunk)) = e4m3_to_bf16(u32x2{w.x[2], w.x[3]}, f);
    };
    // Tile tk of P2 and tv of V, by the waves that move them.
    auto widen_both = [&](int tk, int tv) __attribute__((always_inline)) {
      if constexpr (kSplit) {
        widen(second, second ? tv : tk, peek(0, second ? tv : tk));
      } else {
        widen(0, tk, peek(0, tk));
        widen(1, tv, peek(1, tv));
      }
    };

    if constexpr (k8) {
      if (J > 0) {
#pragma unroll
        for (int t = 0; t < kAhead; ++t) fetch(t);
      }
    }

    // The wave's rows as B operands: row 32 wave + lq, columns 16 ds + 8 hf.
    const bool active = 32 * wave < rows;                 // waves without rows only move tiles
    const int mine = 32 * wave + lq;
    const bool ok = mine < rows;
    const int tok0 = row0 / G;
    const int tq = tok0 + (ok ? token(mine) : 0);
    const int pos = ok ? ctx + tq : 0;                    // no key is below 0
    const int tok = first + tq;
    bf16x8 q[L::kDs];
    {
      const int h = kvh * G + (ok ? mine - token(mine) * G : 0);
      const __bf16* const p = static_cast<const __bf16*>(a.P1) + (size_t)tok * a.ld1 + (size_t)h * DR + 8 * hf;
#pragma unroll
      for (int ds = 0; ds < L::kDs; ++ds) {
        u32x4 x = {0u, 0u, 0u, 0u};
        if (ok && 16 * ds < DR) x = *reinterpret_cast<const u32x4*>(p + 16 * ds);
        q[ds] = __builtin_bit_cast(bf16x8, x);
      }
    }
    const ScanSegment nxt = source.next();                // while the first tiles are on their way
    // Blocks of 32 keys, counted from the segment's first, that all of the wave's rows see.
    const int seen_all = (tree ? ctx : ctx + tok0 + uni(token(32 * wave))) / 32 - 2 * t0;
    // Which of the lane's 16 keys of block x its row sees.
    auto sees = [&](int x) -> unsigned {
      unsigned v = 0;
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int key = 64 * t0 + 32 * x + 8 * g + 4 * hf;
        unsigned s = (1u << min(max(pos - key, 0), 4)) - 1;
        if constexpr (kTree)
          if (tree) s &= tree_bits(a, tok, key - ctx);
        v |= s << (4 * g);
      }
      return v;
    };

    f32x16 o[L::kDb];
    f32x4 l16 = {0.0f, 0.0f, 0.0f, 0.0f};
    float m2 = 0.0f, l = 0.0f;
#pragma unroll
    for (int db = 0; db < L::kDb; ++db) o[db] = f32x16{};

    // ---- the scan: one block step forms the evidence of one block (E), the weights of the
    // block before (W) and the transport of the one before that (T), the products one by one
    // beside parts of the weights; the offset is 0 (see below).
    auto kslot = [&](int t) -> const char* { return smem + (t & 1) * Q::kBuf + koff; };
    auto vslot = [&](int t) -> VBase {
      const char* const v = smem + (t & 1) * Q::kBuf + Q::kVOff;
      return VBase{v + te, v + to};
    };
    bf16x8 ring[4];                                       // step i reads ring[i % 4]
    auto operand = [&](int i, const char* kt, int kbE, const VBase& vt, int kbT) __attribute__((always_inline)) -> bf16x8 {
      if ((i & 1) == 0) return *reinterpret_cast<const bf16x8*>(kt + Q::k_imm(kbE, i >> 1));
      return Q::v_operand(vt, kbT, (i >> 1) / L::kDb, (i >> 1) % L::kDb);
    };
    auto step = [&](auto doE, auto doW, auto doT, f32x16& sE, const f32x16& sW, u32x4 (&pW)[2], const u32x4 (&pT)[2],
                    const char* kt, int kbE, const VBase& vt, int kbT, int blockW, auto beside) __attribute__((always_inline)) {
      constexpr bool E = decltype(doE)::value, T = decltype(doT)::value;
      constexpr int kW = decltype(doW)::value;
      float xv[16], tv[16];
      unsigned vis = 0;
      if constexpr (kW == kMasked) vis = sees(blockW);
      // Weight of score n in four parts, x log2 e and 2^-x, 1 / (1 + 2^-x), 2^(x / (1 + 2^-x))
      // and the rounding, each in a later step than the transcendental that it needs: right
      // behind it, every such pair cost a wait instruction (469 instructions a tile, now 424;
      // 16 trees of 20 to 64 tokens over 2,000 to 30,000 rows of 64 heads of 64 in 8: 401 and
      // 391 us, 32 of 128 in 8 356 and 342).
      constexpr int kLast = kNS - 4;                      // step of the last first part
      auto part = [&](int i) __attribute__((always_inline)) {
#pragma unroll
        for (int n = 0; n < 16; ++n) {
          const int at = n * (kLast + 1) / 16;
          if (i == at + 3) {
            float w = tv[n];
            if constexpr (kW == kMasked) w = __uint_as_float(__float_as_uint(w) & (unsigned)__builtin_amdgcn_sbfe((int)vis, n, 1));
            if (n & 1) pW[n >> 3][(n & 7) >> 1] = pack_bf16(tv[n - 1], w);
            else tv[n] = w;
          }
          if (i == at + 2) tv[n] = __builtin_amdgcn_exp2f(xv[n] * tv[n]);
          if (i == at + 1) tv[n] = __builtin_amdgcn_rcpf(1.0f + tv[n]);
          if (i == at) {
            xv[n] = sW[n] * k2;
            tv[n] = __builtin_amdgcn_exp2f(-xv[n]);
          }
        }
      };
      // Two operands at a time, the second one's first: its wait is the first one's.
      auto reads = [&](int i) __attribute__((always_inline)) {
        if (i >= kNS) return;
        if (T) ring[(i + 1) & 3] = operand(i + 1, kt, kbE, vt, kbT);
        if (E) ring[i & 3] = operand(i, kt, kbE, vt, kbT);
      };
      reads(0);
#pragma unroll
      for (int i = 0; i < kNS; ++i) {
        if ((i & 1) == 0) reads(i + 2);
        if ((i & 1) == 0) {
          if constexpr (E) {
            const int ds = i >> 1;
            if (ds == 0) {
              const f32x16 zero = {};
              sE = __builtin_amdgcn_mfma_f32_32x32x16_bf16(ring[i & 3], q[0], zero, 0, 0, 0);
            } else {
              sE = __builtin_amdgcn_mfma_f32_32x32x16_bf16(ring[i & 3], q[ds], sE, 0, 0, 0);
            }
          }
        } else if constexpr (T) {
          const int k = i >> 1, ks = k / L::kDb, db = k % L::kDb;
          const bf16x8 w = __builtin_bit_cast(bf16x8, pT[ks]);
          o[db] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(ring[i & 3], w, o[db], 0, 0, 0);
          if (db == L::kDb - 1) l16 = __builtin_amdgcn_mfma_f32_16x16x32_bf16(sel, w, l16, 0, 0, 0);
        }
        beside(i);
        if constexpr (kW != kNoWeights) part(i);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    using On = std::true_type;
    using Off = std::false_type;
    using None = std::integral_constant<int, kNoWeights>;
    using All = std::integral_constant<int, kAllSeen>;
    using Some = std::integral_constant<int, kMasked>;

    auto nothing = [](int) __attribute__((always_inline)) {};
    Pieces rk, rv;
    Wide wk, wv;
    f32x16 sA = {}, sB = {};
    u32x4 pA[2] = {}, pB[2] = {};
    if (J > 0) {
      if constexpr (k8) {
        wait_vm_lgkm<2 * kTileLoads, 15>();
        asm volatile("" ::: "memory");
        widen_both(0, 0);
        if (!kSplit || !second) widen(0, 1, peek(0, 1));
      } else {
        Pieces k1st, v1st, k2nd;
        load(0, 0, k1st);
        load(1, 0, v1st);
        load(0, 1, k2nd);
        load(0, 2, rk);
        load(1, 1, rv);
        store(0, 0, k1st);
        store(1, 0, v1st);
        store(0, 1, k2nd);
      }
      tile_barrier();
      if (active) {
        const char* const kt = kslot(0);
        const VBase none = vslot(0);
        step(On{}, None{}, Off{}, sA, sB, pB, pA, kt, 0, none, 0, 0, nothing);
        if (seen_all > 0) step(On{}, All{}, Off{}, sB, sA, pB, pA, kt, 1, none, 0, 0, nothing);
        else step(On{}, Some{}, Off{}, sB, sA, pB, pA, kt, 1, none, 0, 0, nothing);
      }
      tile_barrier();
    }
    // P1's loads have landed on every path: where one leaves that open, the compiler waits for
    // all of a loop's own loads at the first product of each iteration.
#pragma unroll
    for (int ds = 0; ds < L::kDs; ++ds) asm volatile("" : "+v"(q[ds]));
    // Tile j's blocks are transported in iteration j, whose evidence is of tile j + 1. Its
    // stores go where tile j of P2 and tile j - 1 of V were, last read in iteration j - 1.
    // One loop for the iterations whose weights all rows see, one for the others, and the
    // last one by itself: as branches in one loop they cost 100 registers.
    // What iteration j moves, in the kNS parts of its first block step.
    auto move = [&](int j, int i) __attribute__((always_inline)) {
      if constexpr (k8) {
        static_assert(kNS >= 8, "parts of a step");
        if (i == 0) {
          // Tile j + 2 has landed (vector memory operations complete in order; tile j + 3's
          // may be on their way).
          asm volatile("" ::: "memory");
          wait_vm_lgkm<kTileLoads, 15>();
          asm volatile("" ::: "memory");
          if constexpr (kSplit) {
            wk = peek(0, second ? j + 1 : j + 2);
          } else {
            wk = peek(0, j + 2);
            wv = peek(1, j + 1);
          }
        }
        if (i == kNS / 4) {
          if constexpr (kSplit) widen(second, second ? j + 1 : j + 2, wk);
          else widen(0, j + 2, wk);
        }
        if (i == kNS / 2 && !kSplit) widen(1, j + 1, wv);
        if (i == 3 * kNS / 4) {
          asm volatile("" ::: "memory");
          fetch(j + 4);                                   // where tile j was
          asm volatile("" ::: "memory");
        }
      } else {
        if (i == 0) store(0, j + 2, rk);
        if (i == kNS / 4) store(1, j + 1, rv);
        if (i == kNS / 2) load(0, j + 3, rk);
        if (i == 3 * kNS / 4) load(1, j + 2, rv);
      }
    };
    auto window = [&](int j) __attribute__((always_inline)) {
      if (j + 4 >= win0 + 64) load_window(j + 4);
    };
    if (active) {
      const int steady = min((seen_all - 1) >> 1, J - 1);   // 2 j + 2 < seen_all
      int j = 0;
#pragma nounroll
      for (; j < steady; ++j) {
        window(j);
        const char* const kt = kslot(j + 1);
        const VBase vt = vslot(j);
        step(On{}, All{}, On{}, sA, sB, pA, pB, kt, 0, vt, 0, 0, [&](int i) __attribute__((always_inline)) { move(j, i); });
        step(On{}, All{}, On{}, sB, sA, pB, pA, kt, 1, vt, 1, 0, nothing);
        tile_barrier();
      }
#pragma nounroll
      for (; j < J - 1; ++j) {
        window(j);
        const char* const kt = kslot(j + 1);
        const VBase vt = vslot(j);
        step(On{}, Some{}, On{}, sA, sB, pA, pB, kt, 0, vt, 0, 2 * j + 1, [&](int i) __attribute__((always_inline)) { move(j, i); });
        step(On{}, Some{}, On{}, sB, sA, pB, pA, kt, 1, vt, 1, 2 * j + 2, nothing);
        tile_barrier();
      }
      if (J > 0) {
        const VBase vt = vslot(j);
        step(Off{}, Some{}, On{}, sA, sB, pA, pB, nullptr, 0, vt, 0, 2 * j + 1, nothing);
        step(Off{}, None{}, On{}, sB, sA, pB, pA, nullptr, 1, vt, 1, 0, nothing);
        tile_barrier();
      }
    } else {
#pragma nounroll
      for (int j = 0; j < J; ++j) {
        window(j);
#pragma unroll
        for (int i = 0; i < kNS; ++i) move(j, i);
        tile_barrier();
      }
    }
    // The compiler has left out wait states between a product and what reads it behind a
    // branch; the results go through the wait, so that no read of them moves before it. And
    // the last direct loads.
    settle(o, l16);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    l = l16[0];

    // The offset 0 is exact where nothing overflows: SiLU >= -0.2785, so no weight is small.
    // Row sums up to 2^100 and, in parts, results of which all together reach 2^127 (2^119 of
    // eight waves, 2^118 of four) pass; else the segment is scanned again with a stabiliser
    // that follows the scores. The maximum keeps a NaN (products of both signs past the range
    // leave nothing else), which is below no limit.
    float omax = 0.0f;
#pragma unroll
    for (int db = 0; db < L::kDb; ++db)
#pragma unroll
      for (int r = 0; r < 16; ++r) omax = __builtin_elementwise_maximum(omax, fabsf(o[db][r]));
    const bool fine = l <= kFinite && omax < (slot >= 0 ? kPartFinite : INFINITY);
    const bool bad = __any(ok && !fine);
    if (lane == 0) s_bad[wave] = bad ? 1 : 0;
    __syncthreads();
    int redo = 0;
#pragma unroll
    for (int w = 0; w < kTileWaves; ++w) redo |= s_bad[w];
    redo = __builtin_amdgcn_readfirstlane(redo);
    __syncthreads();
    if (redo) {
#pragma unroll
      for (int db = 0; db < L::kDb; ++db) o[db] = f32x16{};
      l = 0.0f;
#pragma nounroll
      for (int t = 0; t < J; ++t) {
        if (t < win0 || t >= win0 + 64) load_window(t);
        if constexpr (k8) {
          fetch(t);
          wait_vm_lgkm<0, 15>();
          asm volatile("" ::: "memory");
          widen_both(t, t);
        } else {
          load(0, t, rk);
          load(1, t, rv);
          store(0, t, rk);
          store(1, t, rv);
        }
        __syncthreads();
#pragma nounroll
        for (int kb = 0; kb < 2; ++kb) {
          f32x16 s = {};
#pragma unroll
          for (int ds = 0; ds < L::kDs; ++ds) {
            const bf16x8 x = *reinterpret_cast<const bf16x8*>(kslot(t) + (kb ? Q::k_imm(1, 0) : 0) + Q::k_imm(0, ds));
            s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x, q[ds], s, 0, 0, 0);
          }
          const unsigned vis = sees(2 * t + kb);
          float mx = -INFINITY;
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const float x = s[r] * k2;
            s[r] = vis >> r & 1u ? x * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-x)) : -INFINITY;
            mx = fmaxf(mx, s[r]);
          }
          const float top = fmaxf(m2, lane_pair_max(mx)), f = __builtin_amdgcn_exp2f(m2 - top);
          m2 = top;
          l *= f;
#pragma unroll
          for (int db = 0; db < L::kDb; ++db)
#pragma unroll
            for (int r = 0; r < 16; ++r) o[db][r] *= f;
          u32x4 w[2];
#pragma unroll
          for (int r = 0; r < 16; r += 2) {
            const float x = __builtin_amdgcn_exp2f(s[r] - m2), y = __builtin_amdgcn_exp2f(s[r + 1] - m2);
            l += x + y;
            w[r >> 3][(r >> 1) & 3] = pack_bf16(x, y);
          }
          const VBase vt = vslot(t);
          const VBase vb{vt.even + 4 * L::kVBlock * kb, vt.odd + 4 * L::kVBlock * kb};
#pragma unroll
          for (int ks = 0; ks < 2; ++ks)
#pragma unroll
            for (int db = 0; db < L::kDb; ++db)
              o[db] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(Q::v_operand(vb, 0, ks, db), __builtin_bit_cast(bf16x8, w[ks]),
                                                              o[db], 0, 0, 0);
        }
        __syncthreads();
      }
      settle(o, l16);
      l = lane_pair_sum(l);
    }

    if (slot < 0) {
      // Self evidence of the lane's row from its own cached row, the columns that the lane
      // holds of P1; then its V, in the columns that it holds of the result. Y passes through
      // LDS (the wave's own part), so that each store writes whole rows.
      const int page = ok ? a.table[(size_t)b * a.max_pages + (pos >> a.page_shift)] : -1;
      const bool has = page >= 0 && page < a.n_pages;
      const size_t head = (size_t)(has ? page : 0) * a.H_kv + kvh;
      const size_t at = ((head << a.page_shift) + (pos & pmask)) * DR;
      const char* const kp = static_cast<const char*>(a.cP2) + (at + 8 * hf) * kEs;
      const char* const vp = static_cast<const char*>(a.cV) + (at + 4 * hf) * kEs;
      typedef unsigned words8 __attribute__((ext_vector_type(2 * kEs)));
      typedef unsigned words4 __attribute__((ext_vector_type(kEs)));
      words8 ko[DR / 16];
      words4 vo[DR / 8];
      float ks = 1.0f, vs = 1.0f;
#pragma unroll
      for (int ds = 0; ds < DR / 16; ++ds) ko[ds] = has ? *reinterpret_cast<const words8*>(kp + 16 * ds * kEs) : words8{};
#pragma unroll
      for (int c = 0; c < DR / 8; ++c) vo[c] = has ? *reinterpret_cast<const words4*>(vp + 8 * c * kEs) : words4{};
      if constexpr (k8) {
        const uint8_t* const sc = a.scale + (head << (a.page_shift + 1)) + (pos & pmask);
        ks = has ? scale_of(sc[0]) : 0.0f;
        vs = has ? scale_of(sc[1 << a.page_shift]) : 0.0f;
      }
      int seen = tq;
      if constexpr (kTree)
        if (tree) seen = ancestors_of(a, tok, tq);
      float u = 0.0f;
#pragma unroll
      for (int ds = 0; ds < DR / 16; ++ds) {
        bf16x8 x;
        if constexpr (k8) x = __builtin_bit_cast(bf16x8, e4m3_to_bf16(u32x2{ko[ds][0], ko[ds][1]}, ks));
        else x = __builtin_bit_cast(bf16x8, ko[ds]);
#pragma unroll
        for (int e = 0; e < 8; ++e) u = fmaf((float)q[ds][e], (float)x[e], u);
      }
      u = lane_pair_sum(u);
      const int h = kvh * G + (ok ? mine - token(mine) * G : 0);
      const float S = sigmoid_f32(u * hp.scale * hp.inv_tau[h]);
      const RowCombine c(S, m2 * kLn2, l, hp.lambda * logf((float)(ctx + seen + 1)));
      char* const y = smem + wave * (32 * kYStride);
#pragma unroll
      for (int db = 0; db < L::kDb; ++db)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          if (32 * db + 8 * g >= DR) continue;            // the layout's other columns
          bf16x4 v, out;
          if constexpr (k8) {
            const u32x4 w = e4m3_to_bf16(u32x2{vo[4 * db + g][0], 0u}, vs);
            v = __builtin_bit_cast(bf16x4, u32x2{w[0], w[1]});
          } else {
            v = __builtin_bit_cast(bf16x4, vo[4 * db + g]);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) out[e] = (__bf16)(c.w_self * (float)v[e] + c.w_hist * o[db][4 * g + e]);
          *reinterpret_cast<bf16x4*>(y + lq * kYStride + 2 * (32 * db + 8 * g + 4 * hf)) = out;
        }
      tile_barrier();
      constexpr int kC = D / 8, kStoreRows = 64 / kC;     // 16-byte chunks of a row, rows of a store
      const int ch = lane % kC;
#pragma unroll
      for (int i = 0; i < 32 / kStoreRows; ++i) {
        const int r = i * kStoreRows + lane / kC, row = 32 * wave + r;
        if (row >= rows || ch >= DR / 8) continue;
        const int x = token(row);
        *reinterpret_cast<u32x4*>(static_cast<__bf16*>(a.Y) +
                                  ((size_t)(first + tok0 + x) * a.H + kvh * G + row - x * G) * DR + 8 * ch) =
            *reinterpret_cast<const u32x4*>(y + r * kYStride + 16 * ch);
      }
    } else if (ok) {
      const int64_t at = (int64_t)slot * kTileRowsQ + mine;
      if (hf == 0) states.ml[at] = make_float2(m2, l);
      float* const zp = states.z + at * DR + 4 * hf;
#pragma unroll
      for (int db = 0; db < L::kDb; ++db)
#pragma unroll
        for (int g = 0; g < 4; ++g)
          if (32 * db + 8 * g < DR)
            *reinterpret_cast<f32x4*>(zp + 32 * db + 8 * g) =
                f32x4{o[db][4 * g], o[db][4 * g + 1], o[db][4 * g + 2], o[db][4 * g + 3]};
    }
    tile_barrier();                        // read before the next segment's keys
    cur = nxt;
  }
}

// Joins of the row blocks that ranges divide: of the tiles' ranges rows / 16 work-groups to
// each, then of the scan's two.
template <int DR, typename Tc, bool kTree>
__global__ __launch_bounds__(kThreads) void tile_join_kernel(ScanArgs<__bf16, Tc, kTree> a, HeadParams hp, int rows, int groups) {
  const int scan = (int)blockIdx.x - groups * (rows / 16), i = scan < 0 ? (int)blockIdx.x : scan, shares = scan < 0 ? rows / 16 : 2;
  join_rows<__bf16, DR, Tc, kTree>(a, hp, scan < 0 ? tile_states(a) : States::scan(a), i / shares, i % shares, shares,
                                   scan < 0 ? rows : 32, false);
}

// Where a batch's requests go, by what the host knows: kToScan, kToTiles (but for those of one
// new token), or kToBoth (those of up to kTileRowsLeast rows to a cached head to the scan).
//   Single tokens are the scan's in any batch, so that their weights have two terms whatever
//   the other requests are. Where there are none the scan's launch adds 2 to 4 us to a call:
//   48 trees of 2 to 24 tokens, as below, 87 us without it and 89 with it, 65 of 60 over none
//   35 and 38.5, 64 of 1 to 30 of 32 heads of 64 in 8, some of them single, 117 and 130.
//   Two row blocks of the scan, 64 rows, are faster than a tile: 32 requests of 64 rows over
//   4,000 8-bit rows of 8 heads of 128 120 us by the scan, 153 on tiles; of 96 rows 172 and
//   159, of 256 387 and 230.
//   The tiles' fixed costs have to be worth their while, by the rows of all heads times the
//   most keys that a request can have, and 500 for what a row block costs beside them, scan
//   and tiles: a prompt of 500 tokens of 8 heads (4 million) 19 and 29 us, a chunk of 64
//   tokens of 32 heads over 4,000 rows (9) 35 and 37, 8 of 100 over none (16) 31 and 28, 16 of
//   64 over 1,000 (49) 68 and 63, 65 trees of 60 over none (78) 84 and 35. The host knows the
//   tables' width, not the lengths: short requests in wide tables lose up to 10 us.
//   Where the requests have like numbers of tokens (kTileLike: the average is a quarter of the
//   most), tiles for all are fastest, scan, both and tiles: 48 trees of 2 to 24 tokens of 16
//   heads of 64 in 4 110, 98 and 89 us.
//   Where few have many, tiles of few rows are slow, and those few alone are worth launches
//   of their own from some 500 rows on. 62 tokens over 1,024 to 4,096 rows beside two chunks
//   of 512, 32 heads of 128: 387, 357 and 707 us, in 8 cached heads 190, 177 and 216; 60
//   beside four of 60, 16 heads in 4: 65, 88 and 98. (The tiles' figures of ragged batches are
//   of single tokens on tiles.)
// And the workspace has to have the chunks' part.
constexpr int kTileRowsLeast = 64;
constexpr int kTileRowsBeside = 512;
constexpr int64_t kTileWork = 12000000;
constexpr int kTileKeys = 500;
constexpr int kTileLike = 4;
enum TileUse { kToScan, kToTiles, kToBoth };
inline TileUse tile_use(const PagedArgs& a) {
  const int G = a.H / a.H_kv;
  const int64_t most = a.max_new < a.N ? a.max_new : a.N, keys = ((int64_t)a.max_pages << a.page_shift) + kTileKeys;
  if (!a.tiles || G > 128 || most < 2 || most * G <= kTileRowsLeast || !paged_chunks_possible(most, G) || (int64_t)a.N * a.H * keys < kTileWork)
    return kToScan;
  if (kTileLike * (int64_t)a.N >= a.S * most) return kToTiles;
  return most * G >= kTileRowsBeside ? kToBoth : kToScan;
}

template <int D, int DR, int W, typename Tc, bool kTree>
hipError_t launch_tiles_of(const ScanArgs<__bf16, Tc, kTree>& a, const HeadParams& hp, int few, hipStream_t s) {
  int cu = 0;
  hipError_t e = device_cu_count(&cu);
  if (e != hipSuccess) return e;
  const int groups = cu * 8 / W < tile_groups(32 * W) ? cu * 8 / W : tile_groups(32 * W);
  // The scan takes requests of up to `few` tokens, one at least.
  ScanArgs<__bf16, Tc, kTree> small = a;
  small.max_new = few < a.max_new ? few : a.max_new;
  int scan_groups = cu * Geom<Tc, DR, 2>::kPerCu;
  scan_groups = scan_groups < kScanGroups / 2 ? scan_groups : kScanGroups / 2;
  if (a.S > kPlanInline) {
    hipLaunchKernelGGL(tile_plan_kernel, dim3(2), dim3(256), 0, s, (const PagedArgs&)a, 32 * W, few);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((tile_kernel<D, DR, W, Tc, kTree>), dim3(groups), dim3(64 * W), 0, s, a, hp, few);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((scan_kernel<__bf16, DR, 2, Tc, kTree>), dim3(scan_groups), dim3(kThreads), 0, s, small, hp, 0, 0);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((tile_join_kernel<DR, Tc, kTree>), dim3(groups * 2 * W + scan_groups * 2), dim3(kThreads), 0, s, a, hp, 32 * W,
                     groups);
  return hipGetLastError();
}

template <int D, int DR, typename Tc, bool kTree>
hipError_t launch_tiles(const ScanArgs<__bf16, Tc, kTree>& a, const HeadParams& hp, bool both, hipStream_t s) {
  // Up to 128 rows to a cached head: work-groups of four waves, two to a compute unit, where
  // the LDS holds both.
  const int G = a.H / a.H_kv, few = both && kTileRowsLeast > G ? kTileRowsLeast / G : 1;
  if constexpr (D == 64) {
    const int64_t most = a.max_new < a.N ? a.max_new : a.N;
    if (most * G <= 128) return launch_tiles_of<D, DR, 4, Tc, kTree>(a, hp, few, s);
  }
  return launch_tiles_of<D, DR, 8, Tc, kTree>(a, hp, few, s);
}

}  // namespace

}  // namespace rel
