// The scan and the join of the paged Relation Cache's forward (paged_fwd.hip has what
// they compute and their figures): kernels for pages in fp32, bf16 and 8 bits, with and
// without trees of drafted tokens.
#pragma once

#include "paged_device.h"

namespace rel {

namespace {

using namespace paged;

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
// log2 slack before the stabiliser moves, as in decode.hip: n keys' weights times V then
// stay below n 2^8 max |V|. 2^32 overflowed for V from 2^96 on, where the outputs are
// finite (decode_batch and decode_long 455 and 219 us at either).
constexpr float kLazy = 8.0f;
constexpr float kHeadroom = 0x1p8f;

// A work-group barrier for LDS data alone: outstanding vector memory operations
// (the next segment's loads) are not waited for.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("" ::: "memory");
  wait_vm_lgkm<63, 0>();
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

__global__ __launch_bounds__(kThreads) void plan_kernel(PagedArgs a, int row_block, int chunks) {
  __shared__ PlanScratch sc;
  Plan p = ws_plan(a);
  if (!chunks) p.tile_sum = nullptr;
  make_plan(a, row_block, chunks != 0, sc, p);
}

// ---- scan ---------------------------------------------------------------------
//
// v_mfma_f32_16x16x32_bf16 and v_mfma_f32_16x16x4_f32 (lane l, i = l % 16, j =
// l / 16): A row i, B column i, the contraction index in the elements and j; C
// register r holds row 4 j + r of column i. With keys as A rows and query rows
// as B columns a lane holds 4 keys' scores of one query row, and its own
// weights are the B operand of the transport O^T[d][row] += V^T[d][key]
// W[key][row], whose contraction runs over the keys in that same order (bf16:
// two 16-key blocks to a step; fp32: one, contraction over d in the order
// {16 t + 4 j + e}).
//
// Both operands of the keys pass through a wave-private LDS slot, filled by
// direct loads of 1 KB of consecutive memory each. The order matters more than
// the traffic: reading the rows straight into the A layout (16 rows x 64 bytes
// per instruction), or V in blocks of 8 rows x 128 bytes, the same bytes took
// eight times as long from the L2 (196 rows over 32,000 keys: 94 us of loads
// against 12). The 16-byte chunks of a row are stored in an order that depends
// on the row, so that the operand reads spread over the banks. A wave holds its
// step's operands in registers, and the slot is refilled while it computes.
//
// 8-bit pages (Tc = e4m3): as the 16-bit ones, with the operands formed in registers:
// v_cvt_scalef32_pk_bf16_fp8 gives two bf16 values, exact, times a power of two, which
// for a P2 row is its scale; V's scales multiply the weights instead (a lane's V operand
// has eight keys), over 2^8, which the values take: a weight may be 2^8 (kLazy) and a scale
// 2^127. An A operand of P2 is 8 consecutive bytes a lane, two to a 16-byte
// read where the row has whole groups of four chunks; V^T comes from ds_read_b64_tr_b8:
// lane i of a group of 16 receives byte i % 8 of the 8-byte rows that lanes i / 8 + 2 k
// address, k = 0 .. 7, so one read has all eight keys of the lane's column. The 32
// scales of a step are loaded into the slot behind its rows, 16 of P2 and 16 of V for
// each 16-key block.
template <typename Tc, int D, int NB>
struct Geom {
  static constexpr bool k8 = sizeof(Tc) == 1;
  static constexpr bool kBf = sizeof(Tc) <= 2;               // operands in bf16
  static constexpr int kEs = (int)sizeof(Tc);
  static constexpr int kHalves = kBf ? 2 : 1;                // 16-key blocks per step
  static constexpr int kStep = 16 * kHalves;                 // keys of a wave's step
  static constexpr int kCh = D * kEs / 16;                   // 16-byte chunks per row
  static constexpr int kDma = (kCh + 3) / 4;                 // 1 KB loads per 16 rows
  static constexpr int kHalf = kDma * 1024;
  static constexpr int kRows = 2 * kHalves * kHalf;          // P2, then V
  static constexpr int kSlot = kRows + (k8 ? kHalves * 256 : 0);   // 8 bits: then the scales
  static constexpr int kStepLoads = 2 * kHalves * kDma + (k8 ? kHalves : 0);   // direct loads of a step
  static constexpr bool kWide = k8 && D % 64 == 0;           // 8 bits: P2 read 16 bytes at a time
  static constexpr int kKs = k8 ? (D / 8 + 3) / 4 : (kCh + 3) / 4;   // A operands per row block
  // Group of 8 columns that lanes of group j have in A operand ks (past the row: none).
  __device__ static int cols(int ks, int j) { return kWide ? 2 * (j + 4 * (ks >> 1)) + (ks & 1) : 4 * ks + j; }
  static constexpr int kDb = D / 16;                         // 16-row blocks of O^T
  static constexpr int kZStride = D + 4;
  static constexpr int kZBytes = 16 * kZStride * 4;          // 16 rows where the waves' states meet
  // Work-groups per compute unit and slots per wave: together about 128 KB of loads in
  // flight on a compute unit. The registers admit them but in two fp32 kernels: d = 128
  // with two row blocks keeps 43 in scratch, most of them addresses of operand reads that
  // each step loads again (8 chunks of 64 tokens over 2000 rows of 8 heads in 2: 81 us, 53
  // TFLOP/s; d = 64, without any, 42 us and 51), d = 64 with one row block 4, outside its
  // key loop. 8-bit rows are half as long: one row block has three work-groups of one slot
  // above d = 64, four below (64 tokens over 1,024 to 4,096 rows of 32 heads: d = 80 185 us,
  // with two of two slots 211, d = 128 256 at either; d = 64 150 us, d = 32 100, with three
  // of two slots 157 and 124).
  static constexpr int kPerCu = NB == 1 && D <= 64 ? 4 : (k8 && NB == 1 ? 3 : 2);
  static constexpr int kSlots = NB == 2 && kSlot <= (k8 ? 9000 : 8192) ? 2 : 1;
  static constexpr int kRing = kWaves * kSlots * kSlot;
  // Chunk c of row q lies at position c ^ swz(q). Rows of 160 and 96 bytes spread
  // over the banks by themselves; wider fp32 rows of 320 and 192 bytes leave
  // four-way conflicts in the V reads.
  __device__ static int swz(int q) {
    if (kBf) return kCh == 16 ? 2 * (q & 7) : (kCh == 8 ? 2 * ((q >> 1) & 3) : (kCh == 4 ? 2 * ((q >> 2) & 1) : 0));
    return kCh >= 32 || kCh == 16 ? q & 15 : (kCh == 8 ? (q >> 1) & 7 : q & 3);
  }
};

// Tc: the pages' type, Tin that of the tokens; kTree: whether the call has trees.
template <typename Tin, int D, int NB, typename Tc, bool kTree>
__global__ __launch_bounds__(kThreads, (Geom<Tc, D, NB>::kPerCu)) void scan_kernel(ScanArgs<Tin, Tc, kTree> a, HeadParams hp,
                                                                                  int with_chunks, int whole) {
  using C = Geom<Tc, D, NB>;
  constexpr bool kBf = C::kBf;
  constexpr int kRb = 16 * NB;
  constexpr int kEs = C::kEs;
  constexpr int kStep = C::kStep;
  __shared__ __attribute__((aligned(16))) char smem[C::kRing + C::kZBytes];
  __shared__ float s_m[kWaves][16], s_l[kWaves][16];
  __shared__ PlanLds lds;

  bool chunks = with_chunks != 0;
  const Plan plan = load_plan(a, kRb, chunks, lds);
  const States states = States::scan(a);
  const int G = a.H / a.H_kv;
  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lane = tid & 63;
  const int li = lane & 15, lj = lane >> 4;
  const float k2 = hp.scale * kLog2e;
  const int pmask = (1 << a.page_shift) - 1;
  char* const ring = smem + wave * C::kSlots * C::kSlot;

  // Source of this lane's 16 bytes in load u of a 16-row block: LDS position
  // 64 u + lane is row / chunk position of the block.
  int src[C::kDma];
#pragma unroll
  for (int u = 0; u < C::kDma; ++u) {
    const int p = 64 * u + lane, q = p / C::kCh, c = p - q * C::kCh;
    src[u] = q < 16 ? q * D * kEs + 16 * (c ^ C::swz(q)) : kOutOfRange;
  }

  // A segment's numbers, in scalar registers. This wave's steps are first + 4 n.
  struct Run {
    int b, kvh, first_tok, ctx, total, row0, rows, slot, first, nsteps;
    bool any;
  };
  ScanSource source(a, plan, kRb, chunks, kBf ? kMinRange : kMinRangeF32,
                    whole ? kWhole : (kBf ? kSnap : kSnapF32));
  auto next_run = [&]() __attribute__((always_inline)) -> Run {
    const ScanSegment sg = source.next();
    const int k0 = uni(sg.k0), k1 = uni(sg.k1);
    const int mine = k1 - k0 - kStep * wave;        // keys from this wave's first step on
    return Run{uni(sg.b), uni(sg.kvh), uni(sg.first), uni(sg.ctx), uni(sg.total), uni(sg.row0), uni(sg.rows), uni(sg.slot),
               k0 / kStep + wave, mine > 0 ? (mine + kWaves * kStep - 1) / (kWaves * kStep) : 0, uni(sg.any) != 0};
  };
  // Lane x holds the table entry of 16-key block x of this wave's steps, for 64
  // blocks from step n0 on (checked when it is used).
  constexpr int kWin = 64 / C::kHalves;             // steps per window
  auto load_pages = [&](const Run& r, int n0) __attribute__((always_inline)) -> int {
    const int n = n0 + lane / C::kHalves;
    const int key = (r.first + kWaves * n) * kStep + 16 * (lane % C::kHalves);
    int pg = -1;
    if (n < r.nsteps && key < r.total) pg = a.table[(size_t)r.b * a.max_pages + (key >> a.page_shift)];
    return pg;
  };
  // Direct loads of step n of a run into a slot. Rows at and past the request's
  // end and rows of a page outside the cache are zeros.
  auto fetch = [&](const Run& r, int pages, int n, int g) __attribute__((always_inline)) {
    char* const slot = ring + (g % C::kSlots) * C::kSlot;
#pragma unroll
    for (int hb = 0; hb < C::kHalves; ++hb) {
      const int key = (r.first + kWaves * n) * kStep + 16 * hb;
      const int pg = __builtin_amdgcn_readlane(pages, C::kHalves * (n % kWin) + hb);
      const bool in = pg >= 0 && pg < a.n_pages;
      const int left = min(16, r.total - key);
      const int bytes = in && left > 0 ? left * D * kEs : 0;
      const size_t row = (((size_t)(in ? pg : 0) * a.H_kv + r.kvh) << a.page_shift) + (key & pmask);
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        u32x4 rw = rsrc_words(static_cast<const char*>(w ? a.cV : a.cP2) + row * D * kEs, bytes);
#pragma unroll
        for (int x = 0; x < 3; ++x) rw[x] = (unsigned)uni((int)rw[x]);
#pragma unroll
        for (int u = 0; u < C::kDma; ++u) dma16(rw, slot + (w * C::kHalves + hb) * C::kHalf + 1024 * u, src[u]);
      }
      if constexpr (C::k8) {
        // The block's scales: of P2 by lanes 0 to 3, of V, a page's rows further on, by lanes 4 to 7.
        const int ps = 1 << a.page_shift, off = key & pmask;
        const size_t at = (((size_t)(in ? pg : 0) * a.H_kv + r.kvh) << (a.page_shift + 1)) + off;
        u32x4 rw = rsrc_words(a.scale + at, bytes > 0 ? 2 * ps - off : 0);
#pragma unroll
        for (int x = 0; x < 3; ++x) rw[x] = (unsigned)uni((int)rw[x]);
        dma4(rw, slot + C::kRows + 256 * hb, lane < 4 ? 4 * lane : (lane < 8 ? ps + 4 * (lane - 4) : kOutOfRange));
      }
    }
  };

  // The segments of the range. The next one's numbers are formed while the first
  // loads of the current one are in flight, and its own first loads are issued
  // before the current one's states meet: base counts this wave's steps of the
  // segments before, got the steps whose loads are issued.
  Run cur = next_run();
  if (!cur.any) return;
  int pages = load_pages(cur, 0);
  int base = 0, got = 0;
  for (; got < C::kSlots && got < cur.nsteps; ++got) fetch(cur, pages, got, got);
  while (true) {
    const Run nxt = next_run();
    int npages = load_pages(nxt, 0);
    const int b = cur.b, kvh = cur.kvh, ctx = cur.ctx, row0 = cur.row0, rows = cur.rows;
    // Steps below it are seen whole by all rows; the new tokens of a tree are not.
    bool tree = false;
    if constexpr (kTree) tree = cur.total - ctx <= 32 * a.words;
    const int pos_lo = tree ? ctx : ctx + row0 / G;

    // The query rows as B operands, and their positions (0 for rows past the end:
    // no key is below it).
    u32x4 qf[NB][C::kKs];
    int pos[NB], tok[NB];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int row = row0 + 16 * nb + li;
      const bool ok = 16 * nb + li < rows;
      const int tq = ok ? row / G : 0;
      const int h = kvh * G + (ok ? row - tq * G : 0);
      pos[nb] = ok ? ctx + tq : 0;
      tok[nb] = cur.first_tok + tq;
      const char* p = static_cast<const char*>(a.P1) + ((size_t)(cur.first_tok + tq) * a.ld1 + (size_t)h * D) * sizeof(Tin);
#pragma unroll
      for (int ks = 0; ks < C::kKs; ++ks) {
        const int c = C::cols(ks, lj);
        qf[nb][ks] = ok && c < D * (int)sizeof(Tin) / 16 ? *reinterpret_cast<const u32x4*>(p + 16 * c) : u32x4{0u, 0u, 0u, 0u};
      }
    }

    f32x4 acc[NB][C::kDb];
    float m2[NB], l[NB];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      m2[nb] = l[nb] = 0.0f;
#pragma unroll
      for (int db = 0; db < C::kDb; ++db) acc[nb][db] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }

    u32x4 kf[C::kHalves][C::k8 ? 1 : C::kKs];       // P2 rows as A operands
    bf16x8 vb[kBf && !C::k8 ? C::kDb : 1];          // V^T as A operands
    float vs[kBf ? 1 : 4][C::kDb];
    // 8 bits: the bytes of both, the scale of the lane's P2 row and those of its keys' V.
    u32x2 kf8[C::kHalves][C::k8 ? C::kKs : 1], vb8[C::k8 ? C::kDb : 1];
    float ksc[C::kHalves], vsc[C::kHalves][4];
    auto read_operands = [&](int g) __attribute__((always_inline)) {
      const char* const slot = ring + (g % C::kSlots) * C::kSlot;
      if constexpr (C::k8) {
#pragma unroll
        for (int hb = 0; hb < C::kHalves; ++hb) {
          const char* const row = slot + hb * C::kHalf + li * D;
#pragma unroll
          for (int ks = 0; ks < C::kKs; ks += C::kWide ? 2 : 1) {
            if constexpr (C::kWide) {
              const u32x4 x = *reinterpret_cast<const u32x4*>(row + 16 * ((4 * (ks >> 1) + lj) ^ C::swz(li)));
              kf8[hb][ks] = u32x2{x[0], x[1]};
              kf8[hb][ks + 1 < C::kKs ? ks + 1 : ks] = u32x2{x[2], x[3]};
            } else {
              const int c = C::cols(ks, lj);
              const bool in = 4 * ks + 3 < D / 8 || c < D / 8;
              const u32x2 x = *reinterpret_cast<const u32x2*>(row + 16 * (((in ? c : 0) >> 1) ^ C::swz(li)) + 8 * (c & 1));
              kf8[hb][ks] = in ? x : u32x2{0u, 0u};
            }
          }
          const unsigned char* const sc = reinterpret_cast<const unsigned char*>(slot + C::kRows + 256 * hb);
          ksc[hb] = scale_of(sc[li]);
          const unsigned x = *reinterpret_cast<const unsigned*>(sc + 16 + 4 * lj);
#pragma unroll
          for (int rr = 0; rr < 4; ++rr) vsc[hb][rr] = scale_of(x >> (8 * rr) & 255u) * (1.0f / kHeadroom);
        }
        const int k = li >> 1, q = 4 * lj + (k & 3);
        const char* const v = slot + (C::kHalves + (k >> 2)) * C::kHalf + q * D + 8 * (li & 1);
#pragma unroll
        for (int db = 0; db < C::kDb; ++db) vb8[db] = lds_tr8_read(v + 16 * (db ^ C::swz(q)));
        return;
      }
#pragma unroll
      for (int hb = 0; hb < C::kHalves; ++hb)
#pragma unroll
        for (int ks = 0; ks < C::kKs; ++ks) {
          const int c = 4 * ks + lj;
          const bool in = 4 * ks + 3 < C::kCh || c < C::kCh;
          const u32x4 x = *reinterpret_cast<const u32x4*>(slot + hb * C::kHalf + 16 * (li * C::kCh + ((in ? c : 0) ^ C::swz(li))));
          kf[hb][ks] = in ? x : u32x4{0u, 0u, 0u, 0u};
        }
      const char* v = slot + C::kHalves * C::kHalf;
      if constexpr (kBf) {
        // Transposing reads: lane m of group j addresses row 4 j + m / 4 of a
        // 16-row block at columns 16 db + 4 (m % 4).
        const int q = 4 * lj + (li >> 2), h = (li & 3) >> 1;
#pragma unroll
        for (int db = 0; db < C::kDb; ++db) {
          const char* p = v + 16 * (q * C::kCh + ((2 * db + h) ^ C::swz(q))) + 8 * (li & 1);
          const bf16x4 x = lds_tr_read(p), y = lds_tr_read(p + C::kHalf);
          vb[db] = bf16x8{x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
        }
      } else {
#pragma unroll
        for (int rr = 0; rr < 4; ++rr)
#pragma unroll
          for (int db = 0; db < C::kDb; ++db) {
            const int q = 4 * lj + rr, c = 4 * db + (li >> 2);
            vs[rr][db] = *reinterpret_cast<const float*>(v + 16 * (q * C::kCh + (c ^ C::swz(q))) + 4 * (li & 3));
          }
      }
    };

    // Scores, weights and transport of step n. Row blocks past the item's rows
    // run along: with a branch around their MFMAs the compiler (ROCm 7.2) left
    // out the wait states between an MFMA and the read of its result behind the
    // branch, and results were wrong.
    auto compute = [&](int n) __attribute__((always_inline)) {
      const int key0 = (cur.first + kWaves * n) * kStep;
      const bool full = key0 + kStep <= pos_lo;
      float w[NB][C::kHalves][4];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        float e2[C::kHalves][4];
#pragma unroll
        for (int hb = 0; hb < C::kHalves; ++hb) {
          f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int ks = 0; ks < C::kKs; ++ks) {
            if constexpr (kBf) {
              u32x4 x;
              if constexpr (C::k8) x = e4m3_to_bf16(kf8[hb][ks], ksc[hb]);
              else x = kf[hb][ks];
              s = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x), __builtin_bit_cast(bf16x8, qf[nb][ks]),
                                                          s, 0, 0, 0);
            } else {
              const f32x4 x = __builtin_bit_cast(f32x4, kf[hb][ks]), y = __builtin_bit_cast(f32x4, qf[nb][ks]);
#pragma unroll
              for (int e = 0; e < 4; ++e) s = __builtin_amdgcn_mfma_f32_16x16x4f32(x[e], y[e], s, 0, 0, 0);
            }
          }
#pragma unroll
          for (int rr = 0; rr < 4; ++rr) {
            // SiLU(u) log2 e = a / (1 + 2^-a), a = u log2 e.
            const float av = s[rr] * k2;
            e2[hb][rr] = av * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-av));
          }
        }
        if (!full) {
#pragma unroll
          for (int hb = 0; hb < C::kHalves; ++hb) {
            const int key = key0 + 16 * hb + 4 * lj;
            unsigned sees = 15u;
            if constexpr (kTree)
              if (tree) sees = tree_bits(a, tok[nb], key - ctx);
#pragma unroll
            for (int rr = 0; rr < 4; ++rr)
              e2[hb][rr] = key + rr < pos[nb] && (!kTree || (sees >> rr & 1u)) ? e2[hb][rr] : -INFINITY;
          }
        }
        // The stabiliser starts at 0 (SiLU >= -0.2785, so no weight is small) and
        // moves only when a score passes it by 2^kLazy.
        float mx = -INFINITY;
#pragma unroll
        for (int hb = 0; hb < C::kHalves; ++hb)
          mx = fmaxf(mx, fmaxf(fmaxf(e2[hb][0], e2[hb][1]), fmaxf(e2[hb][2], e2[hb][3])));
        if (__any(mx > m2[nb] + kLazy)) {
          mx = fmaxf(mx, __shfl_xor(mx, 16));
          mx = fmaxf(mx, __shfl_xor(mx, 32));
          const float mn = fmaxf(mx, m2[nb]);
          const float f = __builtin_amdgcn_exp2f(m2[nb] - mn);
          m2[nb] = mn;
          l[nb] *= f;
#pragma unroll
          for (int db = 0; db < C::kDb; ++db)
#pragma unroll
            for (int rr = 0; rr < 4; ++rr) acc[nb][db][rr] *= f;
        }
#pragma unroll
        for (int hb = 0; hb < C::kHalves; ++hb) {
#pragma unroll
          for (int rr = 0; rr < 4; ++rr) w[nb][hb][rr] = __builtin_amdgcn_exp2f(e2[hb][rr] - m2[nb]);
          l[nb] += (w[nb][hb][0] + w[nb][hb][1]) + (w[nb][hb][2] + w[nb][hb][3]);
        }
      }
      if constexpr (kBf) {
        auto v_of = [&](int db) __attribute__((always_inline)) -> bf16x8 {
          if constexpr (C::k8) return __builtin_bit_cast(bf16x8, e4m3_to_bf16(vb8[db], kHeadroom));
          else return vb[db];
        };
        // The transport's operand: each weight as two bf16 terms, itself rounded and what that
        // leaves (an fp32 difference, exact), so at most 2^-16 of a weight is lost, where one
        // term loses 2^-8 and single tokens would be less exact than relation_decode's. One
        // and two terms: single tokens (decode_batch of 64 over 1,024 to 4,096 rows of 32
        // heads) 455 and 455 us, 32 requests of 8 tokens of 64 heads in 8 of 128 over 4,096
        // rows 112 and 116, 64 of 6 tokens of 32 heads in 4 of 64 over 4000 70 and 75.
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          u32x4 hi, lo;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float x = w[nb][k >> 1][2 * (k & 1)], y = w[nb][k >> 1][2 * (k & 1) + 1];
            if constexpr (C::k8) {
              x *= vsc[k >> 1][2 * (k & 1)];
              y *= vsc[k >> 1][2 * (k & 1) + 1];
            }
            hi[k] = pack_bf16(x, y);
            lo[k] = pack_bf16(x - __builtin_bit_cast(float, hi[k] << 16), y - __builtin_bit_cast(float, hi[k] & 0xffff0000u));
          }
#pragma unroll
          for (int db = 0; db < C::kDb; ++db)
            acc[nb][db] =
                __builtin_amdgcn_mfma_f32_16x16x32_bf16(v_of(db), __builtin_bit_cast(bf16x8, hi), acc[nb][db], 0, 0, 0);
#pragma unroll
          for (int db = 0; db < C::kDb; ++db)
            acc[nb][db] =
                __builtin_amdgcn_mfma_f32_16x16x32_bf16(v_of(db), __builtin_bit_cast(bf16x8, lo), acc[nb][db], 0, 0, 0);
        }
      } else {
#pragma unroll
        for (int rr = 0; rr < 4; ++rr)
#pragma unroll
          for (int db = 0; db < C::kDb; ++db)
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
              acc[nb][db] = __builtin_amdgcn_mfma_f32_16x16x4f32(vs[rr][db], w[nb][0][rr], acc[nb][db], 0, 0, 0);
      }
    };

    for (int n = 0; n < cur.nsteps; ++n) {
      // The step's loads have landed (vector memory operations complete in order:
      // all but the next step's, where they are in flight already); then its
      // operands are in registers and the slot is free.
      asm volatile("" ::: "memory");
      if (C::kSlots == 2 && got > base + n + 1) wait_vm_lgkm<C::kStepLoads, 15>();
      else wait_vm_lgkm<0, 15>();
      asm volatile("" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
      read_operands(base + n);
      asm volatile("" ::: "memory");
      wait_vm_lgkm<63, 0>();
      asm volatile("" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
      const int k = got - base;                     // the next step to load: this run's, or the next one's
      if (k < cur.nsteps) {
        if (k % kWin == 0) pages = load_pages(cur, k);
        fetch(cur, pages, k, got);
        ++got;
      } else if (k - cur.nsteps < nxt.nsteps) {
        fetch(nxt, npages, k - cur.nsteps, got);
        ++got;
      }
      __builtin_amdgcn_sched_barrier(0);
      compute(n);
    }
    base += cur.nsteps;
    for (; got - base < C::kSlots && got - base < nxt.nsteps; ++got) fetch(nxt, npages, got - base, got);

    // The waves' states meet in LDS, 16 rows at a time: each wave adds its share to
    // a quarter of the columns per phase, so the four add side by side and every
    // column has its own fixed order; then 16 lanes per row.
    float* const zrow = reinterpret_cast<float*>(smem + C::kRing);
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      if (16 * nb >= rows) continue;
      float ls = l[nb];
      ls += __shfl_xor(ls, 16);
      ls += __shfl_xor(ls, 32);
      if (lj == 0) {
        s_m[wave][li] = m2[nb];
        s_l[wave][li] = ls;
      }
      lds_barrier();
      float M = s_m[0][li];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) M = fmaxf(M, s_m[w][li]);
      const float f = __builtin_amdgcn_exp2f(m2[nb] - M);
      const int rr = tid >> 4, sl = tid & 15;
      const int row = row0 + 16 * nb + rr;
      const bool ok = 16 * nb + rr < rows;
      const int tq = ok ? row / G : 0;
      const int h = kvh * G + (ok ? row - tq * G : 0);
      // The row's own entries, while the states meet (fp32: behind it, where the
      // registers that it takes are free).
      OwnRow<Tin, D, Tc> own;
      if (kBf && cur.slot < 0) own.load(a, b, cur.first_tok + tq, h, ctx + tq, sl, ok);
      f32x4 share[C::kDb];
#pragma unroll
      for (int db = 0; db < C::kDb; ++db)
#pragma unroll
        for (int rr = 0; rr < 4; ++rr) share[db][rr] = acc[nb][db][rr] * f;
#pragma unroll
      for (int ph = 0; ph < kWaves; ++ph) {
#pragma unroll
        for (int db = 0; db < C::kDb; ++db) {
          if (((wave + ph) & 3) != (db & 3)) continue;
          f32x4* z = reinterpret_cast<f32x4*>(zrow + li * C::kZStride + 16 * db + 4 * lj);
          *z = ph == 0 ? share[db] : *z + share[db];
        }
        lds_barrier();
      }
      float L = 0.0f, zs[8];
      M = s_m[0][rr];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) M = fmaxf(M, s_m[w][rr]);
#pragma unroll
      for (int w = 0; w < kWaves; ++w) L = fmaf(__builtin_amdgcn_exp2f(s_m[w][rr] - M), s_l[w][rr], L);
      {
        const float* zw = zrow + rr * C::kZStride + 8 * (sl < D / 8 ? sl : 0);
        const f32x4 x = reinterpret_cast<const f32x4*>(zw)[0], y = reinterpret_cast<const f32x4*>(zw)[1];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          zs[e] = x[e];
          zs[4 + e] = y[e];
        }
      }
      lds_barrier();                                // read before the next rows' states
      if (cur.slot < 0) {
        if (!kBf) own.load(a, b, cur.first_tok + tq, h, ctx + tq, sl, ok);
        int seen = tq;
        if constexpr (kTree)
          if (tree) seen = ancestors(a, cur.first_tok + tq, tq, sl);
        finish_row(a, hp, own, cur.first_tok + tq, h, ctx + seen, sl, M, L, zs, ok);
      } else if (ok) {
        const int64_t p = (int64_t)cur.slot * kRb + 16 * nb + rr;
        if (sl == 0) states.ml[p] = make_float2(M, L);
        if (sl < D / 8) {
          reinterpret_cast<f32x4*>(states.z + p * D + 8 * sl)[0] = f32x4{zs[0], zs[1], zs[2], zs[3]};
          reinterpret_cast<f32x4*>(states.z + p * D + 8 * sl)[1] = f32x4{zs[4], zs[5], zs[6], zs[7]};
        }
      }
    }
    if (!nxt.any) break;
    cur = nxt;
    pages = npages;
  }
}

// ---- join ---------------------------------------------------------------------

// Rows of the row block or query tile that the end of range k divides, by the
// share'th of its `shares` work-groups. A block in n pieces has n - 1 ranges that it
// ends, so shares * (n - 1) work-groups: as they suffice, each takes one row (every
// 16th piece to a group of 16 lanes), 4 (a wave each, every 4th piece) or 16. One
// token of 16 heads over 131,072 rows of one cached head leaves 256 pieces of 16
// rows: 66 us with one work-group for all of them, 33 us so.
template <typename Tin, int D, typename Tc, bool kTree>
__device__ __forceinline__ void join_rows(const ScanArgs<Tin, Tc, kTree>& a, const HeadParams& hp, const States& st, int k, int share,
                                          int shares, int state_rows, bool tile) {
  __shared__ float s_state[kWaves - 1][16][10];
  const CutRecord c = st.cuts[k];
  if (c.pieces == 0) return;
  const int groups = shares * (c.pieces - 1);
  const int per = c.rows <= groups ? 1 : (c.rows <= 4 * groups ? 4 : 16);
  const int first_row = per * (shares * (k - c.owner) + share);
  if (first_row >= c.rows) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, sl = lane & 15;
  const int i = first_row + (per == 1 ? 0 : (per == 4 ? wave : (int)threadIdx.x >> 4));
  const int from = per == 1 ? (int)threadIdx.x >> 4 : (per == 4 ? lane >> 4 : 0), by = 16 / per;
  // A tile's rows are blocks of 32 positions of the group's heads (Segment); a row
  // block's are tokens times the heads of a group.
  const int G = a.H / a.H_kv;
  const int block = tile ? c.slot0 + (i >> 5) : 0;
  const int x = tile ? block / c.blocks : 0;
  const int tq = tile ? c.row0 + 32 * (block - x * c.blocks) + (i & 31) - c.ctx : (c.row0 + i) / G;
  const int h = tile ? c.head + x : c.head * G + (c.row0 + i) - tq * G;
  const bool ok = i < c.rows && tq >= 0 && c.ctx + tq < c.total && x < G;
  OwnRow<Tin, D, Tc> own;
  own.load(a, c.b, c.first + tq, h, c.ctx + tq, sl, ok && from == 0);
  float M = kEmptyMax, L = 0.0f, z[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) z[e] = 0.0f;
  if (i < c.rows) {
#pragma unroll 4
    for (int p = from; p < c.pieces; p += by)
      join_state<D>(st, (int64_t)(p == 0 ? 2 * c.owner + 1 : 2 * (c.owner + p)) * state_rows + i, sl, M, L, z);
  }
  if (per < 16) {
#pragma unroll
    for (int o = 16; o < 64; o <<= 1) {
      float zo[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) zo[e] = __shfl_xor(z[e], o);
      merge(M, L, z, __shfl_xor(M, o), __shfl_xor(L, o), zo);
    }
  }
  if (per == 1) {
    if (wave > 0 && lane < 16) {
      float* s = s_state[wave - 1][sl];
      s[0] = M;
      s[1] = L;
#pragma unroll
      for (int e = 0; e < 8; ++e) s[2 + e] = z[e];
    }
    __syncthreads();
    if (wave > 0) return;
#pragma unroll
    for (int w = 0; w < kWaves - 1; ++w) {
      const float* s = s_state[w][sl];
      float zo[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) zo[e] = s[2 + e];
      merge(M, L, z, s[0], s[1], zo);
    }
  }
  int seen = tq;
  if constexpr (kTree)
    if (c.total - c.ctx <= 32 * a.words) seen = ancestors(a, c.first + tq, ok ? tq : 0, sl);
  finish_row(a, hp, own, c.first + tq, h, c.ctx + seen, sl, M, L, z, ok && from == 0);
}

// The first scan_groups * row_block / 16 work-groups join the scan's row blocks,
// the others, 16 per range, the query tiles.
template <typename Tin, int D, typename Tc, bool kTree>
__global__ __launch_bounds__(kThreads) void join_kernel(ScanArgs<Tin, Tc, kTree> a, HeadParams hp, int scan_groups, int row_block) {
  const int blocks = row_block / 16;
  int i = (int)blockIdx.x;
  if (i < scan_groups * blocks) {
    join_rows<Tin, D, Tc, kTree>(a, hp, States::scan(a), i / blocks, i % blocks, blocks, row_block, false);
  } else if constexpr (sizeof(Tc) == 2 && !kTree) {
    i -= scan_groups * blocks;
    join_rows<Tin, D, Tc, kTree>(a, hp, States::chunk(a), i / 16, i % 16, 16, 256, true);
  }
}

template <typename Tin, int D, int NB, typename Tc, bool kTree>
hipError_t launch_rows(const ScanArgs<Tin, Tc, kTree>& a, const HeadParams& hp, hipStream_t s) {
  using C = Geom<Tc, D, NB>;
  int cu = 0;
  hipError_t e = device_cu_count(&cu);
  if (e != hipSuccess) return e;
  // The chunk kernel: bf16 unless the scan is selected, where a request can fill a query
  // tile (the workspace counts on no more tokens than the batch has), with a token stride
  // whose 256 rows a 31-bit byte offset reaches, and where the lengths can add up to its
  // least work (its launch without any takes 5 us).
  const int table_rows = a.max_pages << a.page_shift;
  const int64_t most = ((int64_t)a.N * a.H / 32 + (int64_t)a.S * a.H_kv + 1) * (paged_scan_units(table_rows) + kExtra);
  const bool chunks = sizeof(Tc) == 2 && !kTree && a.tiles && paged_chunks_possible(a.max_new < a.N ? a.max_new : a.N, a.H / a.H_kv) &&
                      a.ld1 < (1 << 22) && most >= kChunkWork;
  const int chunk_groups = chunks ? (cu < kChunkGroups ? cu : kChunkGroups) : 0;
  int scan_groups = cu * C::kPerCu;
  scan_groups = scan_groups * NB < kScanGroups ? scan_groups : kScanGroups / NB;
  if (a.S > kPlanInline) {
    hipLaunchKernelGGL(plan_kernel, dim3(1), dim3(kThreads), 0, s, a, 16 * NB, (int)chunks);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (chunks) {
    e = launch_paged_chunk(a, hp, chunk_groups, s);
    if (e != hipSuccess) return e;
  }
  // Few short row blocks stay whole, one per work-group at most, and need no join.
  const bool whole = !chunks && paged_whole(table_rows, (int64_t)a.N * a.H / (16 * NB) + (int64_t)a.S * a.H_kv,
                                            scan_groups, C::kBf);
  hipLaunchKernelGGL((scan_kernel<Tin, D, NB, Tc, kTree>), dim3(scan_groups), dim3(kThreads), 0, s, a, hp, (int)chunks, (int)whole);
  e = hipGetLastError();
  if (e != hipSuccess || whole) return e;
  hipLaunchKernelGGL((join_kernel<Tin, D, Tc, kTree>), dim3(scan_groups * NB + 16 * chunk_groups), dim3(kThreads), 0, s, a, hp,
                     scan_groups, 16 * NB);
  return hipGetLastError();
}

// The rows of a cached head decide on one or two row blocks of 16 in an item.
template <typename Tin, int D, typename Tc, bool kTree>
hipError_t launch_scan(const ScanArgs<Tin, Tc, kTree>& a, const HeadParams& hp, hipStream_t s) {
  const long long rows = (long long)a.max_new * (a.H / a.H_kv);
  return rows <= 16 ? launch_rows<Tin, D, 1, Tc, kTree>(a, hp, s) : launch_rows<Tin, D, 2, Tc, kTree>(a, hp, s);
}

}  // namespace

}  // namespace rel
