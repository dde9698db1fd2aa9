// Relation forward of a packed batch of new tokens against the paged Relation
// Cache (semantics in relation.h; "Ask Self, Ask Others: Relation Is All You
// Need", Eq. (1)-(3) by the scan of Sec. 5.1, Eq. (12)-(14), and the cache of
// Sec. 5.3).
//
// The rows of a request that share a cached head (its new tokens times the
// query heads of the group) are taken in blocks of 16 NB rows. A work item is
// (request, split of its history, cached head, row block); a work-group of four
// waves scans the item's keys, each wave its own 32 keys at a time, and keeps
// (m, l, z) per row; the waves' states meet in LDS. Where a history is split,
// the item leaves a partial state and merge_kernel joins them; otherwise the
// item finishes the row itself (Self entry, count term, output).
//
// Three launches: plan (one work-group: the split length and prefix sums of the
// work over the requests, from the device-side lengths), scan (persistent), and
// merge.
#include "paged_device.h"

namespace rel {

namespace {

using namespace paged;

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kStep = 32;                 // keys of a wave's step
constexpr float kLazy = 32.0f;            // log2 slack before the stabiliser moves

__global__ __launch_bounds__(kThreads) void plan_kernel(PagedArgs a, Cut cut) {
  __shared__ PlanScratch sc;
  WsPlan w(a);
  make_plan(a, cut, true, cut.chunk_min > 0, sc, w.p);
  if (threadIdx.x == 0) {
    w.head[0] = w.p.chunk;
    w.head[1] = w.p.units;
    w.head[2] = w.p.merge_rows;
  }
}

// ---- scan ---------------------------------------------------------------------
//
// v_mfma_f32_16x16x32_bf16 and v_mfma_f32_16x16x4_f32 (lane l, i = l % 16, j =
// l / 16): A row i, B column i, the contraction index in the elements and j; C
// register r holds row 4 j + r of column i. With keys as A rows and query rows
// as B columns a lane holds 4 keys' scores of one query row, and its own
// weights are the B operand of the transport O^T[d][row] += V^T[d][key]
// W[key][row], whose contraction runs over the keys in that same order.
//   bf16: two 16-key blocks make one transport step; V^T comes from a
//     wave-private LDS tile (direct loads, transposing reads).
//   fp32: contraction over d in the order {16 t + 4 j + e}, so each lane loads 16
//     bytes of a P2 row; output rows in the order {d / 16 i + e}, so each lane
//     loads d_h / 16 consecutive floats of a V row as the A operands of all
//     output blocks.
template <typename Tin, int D>
struct Geom {
  static constexpr bool kBf = sizeof(Tin) == 2;
  static constexpr int kKs = kBf ? (D + 31) / 32 : D / 16;   // 16-byte loads per lane and 16-key block
  static constexpr int kDb = D / 16;                         // 16-row blocks of O^T
  static constexpr int kCb = (D + 63) / 64;                  // 64-column blocks of a V tile
  static constexpr int kVTile = 4 * kCb * 1024;              // 32 rows: blocks of 8 rows x 8 chunks, 1 KB each
  static constexpr int kRing = kBf ? kWaves * 2 * kVTile : 0;
  static constexpr int kZStride = D + 4;
  static constexpr int kZBytes = kWaves * 16 * kZStride * 4;
  static constexpr int kLds = kRing > kZBytes ? kRing : kZBytes;
};

// Work-groups per compute unit: as many as the LDS ring and the registers of
// the row blocks admit.
template <typename Tin, int D, int NB>
constexpr int kPerCu = sizeof(Tin) == 4 && D == 128 && NB == 2 ? 1 : (D <= 64 && NB == 1 ? 4 : 2);

template <typename Tin, int D, int NB>
__global__ __launch_bounds__(kThreads, (kPerCu<Tin, D, NB>)) void scan_kernel(PagedArgs a, HeadParams hp, Cut cut) {
  using C = Geom<Tin, D>;
  constexpr bool kBf = C::kBf;
  constexpr int kRb = 16 * NB;
  constexpr int kEs = (int)sizeof(Tin);
  __shared__ __attribute__((aligned(16))) char smem[C::kLds];
  __shared__ float s_m[kWaves][16], s_l[kWaves][16];
  __shared__ PlanLds lds;

  const int chunk_min = cut.chunk_min;
  const Plan plan = load_plan(a, cut, true, false, lds);
  const int n_items = plan.units * a.H_kv;
  const int chunk = plan.chunk;
  const States states = States::scan(a);
  const int G = a.H / a.H_kv;
  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lane = tid & 63;
  const int li = lane & 15, lj = lane >> 4;
  const float k2 = hp.scale * kLog2e;
  const int pmask = (1 << a.page_shift) - 1;
  const int per = (n_items + 7) >> 3;

  // Work-groups go round the 8 XCDs: each takes a contiguous eighth of the items,
  // so the row blocks of one (request, split, cached head), which lie together,
  // read its keys through one L2.
  for (int it = blockIdx.x; it < 8 * per; it += gridDim.x) {
    const int item = (it & 7) * per + (it >> 3);
    if (item >= n_items) continue;
    const int b = find_request(plan.unit_sum, a.S, item / a.H_kv);
    Req r = scan_part(Req(a, b), chunk_min);
    r.first = uni(r.first);
    r.q = uni(r.q);
    r.total = uni(r.total);
    const int all_rows = r.q * G;
    const int nrb = (all_rows + kRb - 1) / kRb;
    const int nsplit = splits_of(r.total, chunk);
    const int local = item - uni(plan.unit_sum[b]) * a.H_kv;   // 0 .. nrb * nsplit * H_kv - 1
    const int rb = local % nrb;
    const int kvh = (local / nrb) % a.H_kv;
    const int split = local / nrb / a.H_kv;
    const int ctx = r.total - r.q;
    const int row0 = rb * kRb;
    const int rows = min(kRb, all_rows - row0);
    const int pos_lo = ctx + row0 / G, pos_hi = ctx + (row0 + rows - 1) / G;
    const int k0 = split * chunk;
    if (split > 0 && k0 >= pos_hi) continue;        // no keys; the merge does not read this state
    const int k1 = (int)min((long long)k0 + chunk, (long long)pos_hi);

    // The query rows as B operands, and their positions (0 for rows past the end:
    // no key is below it).
    u32x4 qf[NB][C::kKs];
    int pos[NB];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int row = row0 + 16 * nb + li;
      const bool ok = 16 * nb + li < rows;
      const int tq = ok ? row / G : 0;
      const int h = kvh * G + (ok ? row - tq * G : 0);
      pos[nb] = ok ? ctx + tq : 0;
      const Tin* p = static_cast<const Tin*>(a.P1) + (size_t)(r.first + tq) * a.ld1 + (size_t)h * D;
#pragma unroll
      for (int ks = 0; ks < C::kKs; ++ks) {
        const int col = kBf ? 32 * ks + 8 * lj : 16 * ks + 4 * lj;
        qf[nb][ks] = ok && col < D ? *reinterpret_cast<const u32x4*>(p + col) : u32x4{0u, 0u, 0u, 0u};
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

    // This wave's steps: first + 4 n. Lane x holds the page of half x % 2 of step
    // n0 + x / 2, for 32 steps at a time.
    const int first = k0 / kStep + wave;
    const int nsteps = k1 > k0 + kStep * wave ? ((k1 - k0 + kStep - 1) / kStep - wave + kWaves - 1) / kWaves : 0;
    int pages = -1;
    auto load_pages = [&](int n0) {
      const int key = (first + kWaves * (n0 + (lane >> 1))) * kStep + 16 * (lane & 1);
      pages = -1;
      if (n0 + (lane >> 1) < nsteps && key < r.total) {
        const int pg = a.table[(size_t)b * a.max_pages + (key >> a.page_shift)];
        pages = pg >= 0 && pg < a.n_pages ? pg : -1;
      }
    };
    // Byte address of the first row of 16-key half hb of step n in a cache, and
    // the bytes of its rows that exist (0: page outside the cache).
    auto half_at = [&](const void* cache, int n, int hb, int* bytes) -> const char* {
      const int key = (first + kWaves * n) * kStep + 16 * hb;
      const int pg = __builtin_amdgcn_readlane(pages, 2 * (n & 31) + hb);
      const int left = min(16, r.total - key);
      *bytes = pg >= 0 && left > 0 ? left * D * kEs : 0;
      const size_t row = (((size_t)(pg >= 0 ? pg : 0) * a.H_kv + kvh) << a.page_shift) + (key & pmask);
      return static_cast<const char*>(cache) + row * D * kEs;
    };

    constexpr int kBuf = kBf ? 2 : 1;
    u32x4 kf[kBuf][2][C::kKs];                      // P2 rows of this step (bf16: and the next)
    float vf[2][4][C::kDb];                         // fp32: V rows of the step
    char* const ring = smem + wave * 2 * C::kVTile;
    auto fetch = [&](int n, int buf) __attribute__((always_inline)) {
      if ((n & 31) == 0) load_pages(n);
#pragma unroll
      for (int hb = 0; hb < 2; ++hb) {
        int bytes;
        const char* p = half_at(a.cP2, n, hb, &bytes);
        const auto rs = rsrc(p, bytes);
#pragma unroll
        for (int ks = 0; ks < C::kKs; ++ks) {
          const int col = kBf ? 32 * ks + 8 * lj : 16 * ks + 4 * lj;
          const int o = col < D ? (li * D + col) * kEs : kOutOfRange;
          kf[buf][hb][ks] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, o, 0, 0));
        }
        const char* v = half_at(a.cV, n, hb, &bytes);
        if constexpr (kBf) {
#pragma unroll
          for (int rg = 0; rg < 2; ++rg) {
            u32x4 rw = rsrc_words(v + 8 * rg * D * kEs, bytes - 8 * rg * D * kEs);
#pragma unroll
            for (int w = 0; w < 3; ++w) rw[w] = (unsigned)uni((int)rw[w]);
#pragma unroll
            for (int cb = 0; cb < C::kCb; ++cb) {
              const int ch = 8 * cb + (lane >> 3);
              dma16(rw, ring + (n & 1) * C::kVTile + (2 * hb + rg + 4 * cb) * 1024,
                    ch < D / 8 ? (lane & 7) * D * 2 + 16 * ch : kOutOfRange);
            }
          }
        }
      }
    };
    // fp32: the V rows of 16-key half hb, key 4 j + rr, columns d / 16 i ..
    auto fetch_v = [&](int n) __attribute__((always_inline)) {
      if constexpr (!kBf) {
#pragma unroll
        for (int hb = 0; hb < 2; ++hb) {
          int bytes;
          const char* v = half_at(a.cV, n, hb, &bytes);
          const auto rs = rsrc(v, bytes);
#pragma unroll
          for (int rr = 0; rr < 4; ++rr) {
            const int o = ((4 * lj + rr) * D + C::kDb * li) * 4;
#pragma unroll
            for (int e = 0; e < C::kDb; e += 4) {
              if constexpr (C::kDb >= 4) {
                if (e + 4 <= C::kDb) {
                  const f32x4 x = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, o + 4 * e, 0, 0));
#pragma unroll
                  for (int w = 0; w < 4; ++w) vf[hb][rr][e + w] = x[w];
                  continue;
                }
              }
#pragma unroll
              for (int w = e; w < C::kDb; ++w)
                vf[hb][rr][w] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rs, o + 4 * w, 0, 0));
            }
          }
        }
      }
    };

    // Scores, weights and transport of step n from P2 buffer buf. Row blocks past
    // the item's rows run along: with a branch around their MFMAs the compiler
    // (ROCm 7.2) left out the wait states between an MFMA and the read of its
    // result behind the branch, and results were wrong.
    auto compute = [&](int n, int buf) __attribute__((always_inline)) {
      const int key0 = (first + kWaves * n) * kStep;
      const bool full = key0 + kStep <= pos_lo;
      u32x4 wf[NB];
      float w32[kBf ? 1 : NB][2][4];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        float e2[2][4];
#pragma unroll
        for (int hb = 0; hb < 2; ++hb) {
          f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int ks = 0; ks < C::kKs; ++ks) {
            if constexpr (kBf) {
              s = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, kf[buf][hb][ks]),
                                                          __builtin_bit_cast(bf16x8, qf[nb][ks]), s, 0, 0, 0);
            } else {
              const f32x4 x = __builtin_bit_cast(f32x4, kf[buf][hb][ks]), y = __builtin_bit_cast(f32x4, qf[nb][ks]);
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
          for (int hb = 0; hb < 2; ++hb)
#pragma unroll
            for (int rr = 0; rr < 4; ++rr)
              e2[hb][rr] = key0 + 16 * hb + 4 * lj + rr < pos[nb] ? e2[hb][rr] : -INFINITY;
        }
        // The stabiliser starts at 0 (SiLU >= -0.2785, so no weight is small) and
        // moves only when a score passes it by 2^32.
        float mx = fmaxf(fmaxf(fmaxf(e2[0][0], e2[0][1]), fmaxf(e2[0][2], e2[0][3])),
                         fmaxf(fmaxf(e2[1][0], e2[1][1]), fmaxf(e2[1][2], e2[1][3])));
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
        float w[2][4];
#pragma unroll
        for (int hb = 0; hb < 2; ++hb) {
#pragma unroll
          for (int rr = 0; rr < 4; ++rr) w[hb][rr] = __builtin_amdgcn_exp2f(e2[hb][rr] - m2[nb]);
          l[nb] += (w[hb][0] + w[hb][1]) + (w[hb][2] + w[hb][3]);
        }
        if constexpr (kBf) {
          // The transport's operand: weights rounded to bf16, like the other bf16 forwards.
          wf[nb] = u32x4{pack_bf16(w[0][0], w[0][1]), pack_bf16(w[0][2], w[0][3]), pack_bf16(w[1][0], w[1][1]),
                         pack_bf16(w[1][2], w[1][3])};
        } else {
#pragma unroll
          for (int hb = 0; hb < 2; ++hb)
#pragma unroll
            for (int rr = 0; rr < 4; ++rr) w32[nb][hb][rr] = w[hb][rr];
        }
      }
      if constexpr (kBf) {
        // Transposing reads: lane m of group j addresses row 4 j + m / 4 of a
        // 16-row block at columns 16 db + 4 (m % 4).
        const int q = 4 * lj + (li >> 2), c = (li & 3) >> 1;
        const char* tb = ring + (n & 1) * C::kVTile + 1024 * (q >> 3) + 16 * ((q & 7) + 8 * c) + 8 * (li & 1);
#pragma unroll
        for (int db = 0; db < C::kDb; ++db) {
          const char* p = tb + 4096 * (db / 4) + 256 * (db % 4);
          const bf16x4 x = lds_tr_read(p), y = lds_tr_read(p + 2048);
          const bf16x8 vt = {x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
            acc[nb][db] =
                __builtin_amdgcn_mfma_f32_16x16x32_bf16(vt, __builtin_bit_cast(bf16x8, wf[nb]), acc[nb][db], 0, 0, 0);
        }
      } else {
#pragma unroll
        for (int hb = 0; hb < 2; ++hb)
#pragma unroll
          for (int rr = 0; rr < 4; ++rr)
#pragma unroll
            for (int db = 0; db < C::kDb; ++db)
#pragma unroll
              for (int nb = 0; nb < NB; ++nb)
                acc[nb][db] = __builtin_amdgcn_mfma_f32_16x16x4f32(vf[hb][rr][db], w32[nb][hb][rr], acc[nb][db], 0, 0, 0);
      }
    };

    if constexpr (kBf) {
      // One step ahead: the next step's loads are issued once this step's have
      // landed and the LDS reads of the step before are done.
      if (nsteps > 0) fetch(0, 0);
      for (int n = 0; n < nsteps; n += 2) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          if (n + u < nsteps) {
            asm volatile("" ::: "memory");
            wait_vm_lgkm<0, 0>();
            asm volatile("" ::: "memory");
            __builtin_amdgcn_sched_barrier(0);
            if (n + u + 1 < nsteps) fetch(n + u + 1, u ^ 1);
            __builtin_amdgcn_sched_barrier(0);
            compute(n + u, u);
          }
        }
      }
    } else {
      for (int n = 0; n < nsteps; ++n) {
        fetch(n, 0);
        fetch_v(n);
        compute(n, 0);
      }
    }

    // The waves' states meet in LDS, 16 rows at a time; then 16 lanes per row.
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      if (16 * nb >= rows) continue;
      float ls = l[nb];
      ls += __shfl_xor(ls, 16);
      ls += __shfl_xor(ls, 32);
      __syncthreads();                              // ring or the previous rows' states are no longer read
      if (lj == 0) {
        s_m[wave][li] = m2[nb];
        s_l[wave][li] = ls;
      }
      float* z = reinterpret_cast<float*>(smem) + (wave * 16 + li) * C::kZStride;
#pragma unroll
      for (int db = 0; db < C::kDb; ++db) {
        if constexpr (kBf) {
          *reinterpret_cast<f32x4*>(z + 16 * db + 4 * lj) = acc[nb][db];
        } else {
#pragma unroll
          for (int rr = 0; rr < 4; ++rr) z[C::kDb * (4 * lj + rr) + db] = acc[nb][db][rr];
        }
      }
      __syncthreads();
      const int rr = tid >> 4, sl = tid & 15;
      const int row = row0 + 16 * nb + rr;
      const bool ok = 16 * nb + rr < rows;
      float M = s_m[0][rr], L = 0.0f, zs[8];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) M = fmaxf(M, s_m[w][rr]);
#pragma unroll
      for (int e = 0; e < 8; ++e) zs[e] = 0.0f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const float f = __builtin_amdgcn_exp2f(s_m[w][rr] - M);
        L = fmaf(f, s_l[w][rr], L);
        if (sl < D / 8) {
          const float* zw = reinterpret_cast<const float*>(smem) + (w * 16 + rr) * C::kZStride + 8 * sl;
          const f32x4 x = reinterpret_cast<const f32x4*>(zw)[0], y = reinterpret_cast<const f32x4*>(zw)[1];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            zs[e] = fmaf(f, x[e], zs[e]);
            zs[4 + e] = fmaf(f, y[e], zs[4 + e]);
          }
        }
      }
      const int tq = ok ? row / G : 0;
      const int h = kvh * G + (ok ? row - tq * G : 0);
      if (nsplit == 1) {
        finish_row<Tin, D>(a, hp, b, r.first + tq, h, ctx + tq, sl, M, L, zs, ok);
      } else if (ok) {
        const int64_t p = (int64_t)plan.part_sum[b] + (int64_t)split * all_rows * a.H_kv + (int64_t)kvh * all_rows + row;
        if (sl == 0) states.ml[p] = make_float2(M, L);
        if (sl < D / 8) {
          reinterpret_cast<f32x4*>(states.z + p * D + 8 * sl)[0] = f32x4{zs[0], zs[1], zs[2], zs[3]};
          reinterpret_cast<f32x4*>(states.z + p * D + 8 * sl)[1] = f32x4{zs[4], zs[5], zs[6], zs[7]};
        }
      }
    }
    __syncthreads();                                // the states are read before the next item's loads land
  }
}

// ---- join ---------------------------------------------------------------------

// Rows of split histories, a wave each: four groups of 16 lanes join every
// fourth split, then the groups join.
template <typename Tin, int D>
__device__ __forceinline__ void join_rows(const PagedArgs& a, const HeadParams& hp, const Plan& plan, int chunk_min,
                                          int wave, int waves) {
  const States st = States::scan(a);
  const int G = a.H / a.H_kv;
  const int lane = threadIdx.x & 63, g = lane >> 4, sl = lane & 15;
  for (int i = wave; i < plan.merge_rows; i += waves) {
    const int b = find_request(plan.merge_sum, a.S, i);
    const Req r = scan_part(Req(a, b), chunk_min);
    const int all_rows = r.q * G;
    const int id = i - plan.merge_sum[b];           // kvh * all_rows + row
    const int kvh = id / all_rows, row = id - kvh * all_rows;
    const int tq = row / G, h = kvh * G + row - tq * G;
    const int pos = r.total - r.q + tq;
    const int ns = (int)(((long long)pos + plan.chunk - 1) / plan.chunk);   // splits with keys of this row
    float M = kEmptyMax, L = 0.0f, z[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) z[e] = 0.0f;
#pragma unroll 4
    for (int s = g; s < ns; s += 4)
      join_state<D>(st, (int64_t)plan.part_sum[b] + (int64_t)s * all_rows * a.H_kv + id, sl, M, L, z);
#pragma unroll
    for (int o = 16; o < 64; o <<= 1) {
      const float Mo = __shfl_xor(M, o), Mn = fmaxf(M, Mo);
      const float f = __builtin_amdgcn_exp2f(M - Mn), fo = __builtin_amdgcn_exp2f(Mo - Mn);
      L = L * f + __shfl_xor(L, o) * fo;
#pragma unroll
      for (int e = 0; e < 8; ++e) z[e] = z[e] * f + __shfl_xor(z[e], o) * fo;
      M = Mn;
    }
    finish_row<Tin, D>(a, hp, b, r.first + tq, h, pos, sl, M, L, z, g == 0);
  }
}

// 16 rows of the query tile that the end of range k of the long chunks divides,
// 16 lanes per row.
template <typename Tin, int D>
__device__ __forceinline__ void join_tile(const PagedArgs& a, const HeadParams& hp, int k, int rows16) {
  const CutTile t = reinterpret_cast<const CutTile*>(static_cast<const char*>(a.ws) + paged_plan_bytes(a.S) +
                                                     paged_scan_bytes(a.d_h))[k];
  if (t.pieces == 0) return;
  const States st = States::chunk(a);
  const int sl = threadIdx.x & 15, i = 16 * rows16 + (threadIdx.x >> 4);
  const int pos = t.q0 + i;
  const bool ok = pos >= t.ctx && pos < t.total;
  float M = kEmptyMax, L = 0.0f, z[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) z[e] = 0.0f;
#pragma unroll 4
  for (int p = 0; p < t.pieces; ++p)
    join_state<D>(st, (int64_t)(p == 0 ? 2 * k + 1 : 2 * (k + p)) * 256 + i, sl, M, L, z);
  finish_row<Tin, D>(a, hp, t.b, ok ? t.first + (pos - t.ctx) : 0, t.h, ok ? pos : 0, sl, M, L, z, ok);
}

// The first row_groups work-groups join the scan's split histories, the others
// 16 rows each of the long chunks' divided tiles.
template <typename Tin, int D>
__global__ __launch_bounds__(kThreads) void join_kernel(PagedArgs a, HeadParams hp, Cut cut, int row_groups) {
  __shared__ PlanLds lds;
  if ((int)blockIdx.x < row_groups) {
    const Plan plan = load_plan(a, cut, true, false, lds);
    join_rows<Tin, D>(a, hp, plan, cut.chunk_min, blockIdx.x * kWaves + (threadIdx.x >> 6), row_groups * kWaves);
  } else if constexpr (sizeof(Tin) == 2) {
    const int i = (int)blockIdx.x - row_groups;
    join_tile<Tin, D>(a, hp, i / 16, i % 16);
  }
}

template <typename Tin, int D, int NB>
hipError_t launch_rows(const PagedArgs& a, const HeadParams& hp, hipStream_t s) {
  int cu = 0;
  hipError_t e = device_cu_count(&cu);
  if (e != hipSuccess) return e;
  // Long chunks: bf16, with a token stride whose 256 rows a 31-bit byte offset
  // reaches.
  const bool chunks = sizeof(Tin) == 2 && a.max_new >= kChunkMin && a.N >= kChunkMin && a.ld1 < (1 << 22);
  const Cut cut{16 * NB, chunks ? kChunkMin : 0, cu * kPerCu<Tin, D, NB>, chunks ? (cu < kChunkGroups ? cu : kChunkGroups) : 0};
  if (a.S > kPlanInline) {
    hipLaunchKernelGGL(plan_kernel, dim3(1), dim3(kThreads), 0, s, a, cut);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (chunks) {
    e = launch_paged_chunk(a, hp, cut.chunk_groups, s);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((scan_kernel<Tin, D, NB>), dim3(cut.scan_groups), dim3(kThreads), 0, s, a, hp, cut);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  // The last range has no end inside a tile.
  const int row_groups = 4 * cu, tile_groups = chunks ? 16 * (cut.chunk_groups - 1) : 0;
  hipLaunchKernelGGL((join_kernel<Tin, D>), dim3(row_groups + tile_groups), dim3(kThreads), 0, s, a, hp, cut, row_groups);
  return hipGetLastError();
}

template <typename Tin, int D>
hipError_t launch_typed(const PagedArgs& a, const HeadParams& hp, hipStream_t s) {
  const long long rows = (long long)a.max_new * (a.H / a.H_kv);
  return rows <= 16 ? launch_rows<Tin, D, 1>(a, hp, s) : launch_rows<Tin, D, 2>(a, hp, s);
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
