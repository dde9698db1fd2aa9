// The cut of each request back to the new tokens that it keeps: their cached rows move to
// the front of the new ones, the request's length follows, and the pages that then hold
// nothing return to the free list (semantics in relation.h).
//
// One work-group per request and cached head moves the rows, P2's and V's; one more forms
// the lengths and the list (as page_map does: a prefix sum, then a page per thread). Both
// check the kept tokens for themselves, so that neither waits for the other. A round of
// rows is loaded into registers before any of it is stored: a kept row's new place may be
// another's old one, but never one that a later round reads, as places only grow.
// Bound by latency, of a table entry, a row, a barrier and a store, and of the list's sums
// and searches: 48 requests that keep up to 6 of 2 to 24 tokens of 4 heads 4.1 us, 512 that
// keep up to 16 of 20 to 64 in 8-bit pages of 8 heads 15.7 (the rows alone 12.2, the list
// alone 14.6; with four kept tokens' searches side by side the list took longer, 15.8).
#include "page_list.h"
#include "rel_internal.h"

namespace rel {

namespace {

constexpr int kThreads = 256;
constexpr int kAtOnce = 4;                // 16-byte pieces, or pages, that a thread moves together

// What the device-side numbers say of request b; ok = false for one that is left alone.
struct Kept {
  int first, q, ctx, n;
  bool ok;
  __device__ __forceinline__ Kept(const PagedKeepArgs& a, int b) {
    first = q = ctx = n = 0;
    ok = false;
    if (b >= a.S) return;
    first = a.cu[b];
    const int end = a.cu[b + 1], total = a.total[b];
    ok = first >= 0 && end >= first && end <= a.N && total >= end - first &&
         (long long)total <= ((long long)a.max_pages << a.page_shift);
    if (!ok) return;
    q = end - first;
    ctx = total - q;
    n = a.n_keep[b];
    if (n < 0 || n > q) n = 0;
  }
};

// Whether kept token k of a request follows the one before it.
__device__ __forceinline__ bool follows(const PagedKeepArgs& a, const Kept& r, int k) {
  const int x = a.keep[r.first + k];
  return x < r.q && x > (k > 0 ? a.keep[r.first + k - 1] : -1);
}

// The wave's loads are in registers (a barrier alone orders LDS).
__device__ __forceinline__ void loaded() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

__device__ void move_rows(const PagedKeepArgs& a, int b, int h) {
  const Kept r(a, b);
  if (!r.ok || r.n == 0) return;          // uniform for the work-group
  const int tid = threadIdx.x;
  bool fine = true;
  for (int k = tid; k < r.n; k += kThreads) fine = fine && follows(a, r, k);
  if (!__syncthreads_and(fine)) return;
  const int pmask = (1 << a.page_shift) - 1;
  // The row of a position in the pages, -1 where its page is none.
  auto row_of = [&](int pos) -> long long {
    const int page = a.table[(size_t)b * a.max_pages + (pos >> a.page_shift)];
    return page >= 0 && page < a.n_pages ? ((((long long)page * a.H_kv + h) << a.page_shift) + (pos & pmask)) : -1;
  };
  const int pieces = a.row_bytes / 16;    // of a row
  const long long units = (long long)r.n * 2 * pieces;
  for (long long u0 = tid; u0 - tid < units; u0 += kAtOnce * kThreads) {
    uint4 x[kAtOnce];
    char* to[kAtOnce];
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      const long long u = u0 + j * kThreads;
      to[j] = nullptr;
      if (u >= units) continue;
      const int k = (int)(u / (2 * pieces)), c = (int)(u - (long long)k * 2 * pieces);
      const int from = a.keep[r.first + k];
      if (from == k) continue;
      char* const cache = static_cast<char*>(c >= pieces ? a.cV : a.cP2);
      const size_t at = (size_t)16 * (c >= pieces ? c - pieces : c);
      const long long src = row_of(r.ctx + from), dst = row_of(r.ctx + k);
      if (dst < 0) continue;
      to[j] = cache + (size_t)dst * a.row_bytes + at;
      x[j] = src < 0 ? make_uint4(0, 0, 0, 0) : *reinterpret_cast<const uint4*>(cache + (size_t)src * a.row_bytes + at);
    }
    loaded();
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j)
      if (to[j]) *reinterpret_cast<uint4*>(to[j]) = x[j];
  }
  if (!a.scale) return;
  // A page's scales of a head: its P2 rows', then its V rows'.
  auto scale_at = [&](long long row, int part) -> uint8_t* {
    return a.scale + (((row >> a.page_shift) * 2 + part) << a.page_shift) + (row & pmask);
  };
  for (long long u0 = tid; u0 - tid < 2LL * r.n; u0 += kThreads) {
    uint8_t x = 0;
    uint8_t* to = nullptr;
    if (u0 < 2LL * r.n) {
      const int k = (int)(u0 >> 1), part = (int)u0 & 1, from = a.keep[r.first + k];
      if (from != k) {
        const long long src = row_of(r.ctx + from), dst = row_of(r.ctx + k);
        if (dst >= 0) {
          to = scale_at(dst, part);
          x = src < 0 ? 0 : *scale_at(src, part);
        }
      }
    }
    loaded();
    __syncthreads();
    if (to) *to = x;
  }
}

__device__ void cut_lists(const PagedKeepArgs& a) {
  __shared__ long long red[kThreads / 64];
  __shared__ long long s_sum[kThreads], s_first[kThreads];   // any offsets, overlapping ones too
  __shared__ int s_end[kThreads], s_from[kThreads], s_q[kThreads], s_bad[kThreads];
  const int tid = threadIdx.x;
  int have = a.n_free[0];
  have = have < 0 ? 0 : (have > a.F ? a.F : have);
  long long back = 0, all;
  for (int b0 = 0; b0 < a.S; b0 += kThreads) {
    const int b = b0 + tid;
    Kept r(a, b);
    // The kept tokens of these requests, one per thread.
    long long sum = block_sum<kThreads>(r.n, red, &all);
    s_sum[tid] = sum;
    s_first[tid] = r.first - (sum - r.n);
    s_q[tid] = r.q;
    s_bad[tid] = 0;
    __syncthreads();
    for (long long i = tid; i < all; i += kThreads) {
      const int x = first_past_of<kThreads>(s_sum, i);
      const long long t = s_first[x] + i;
      const int at = a.keep[t], before = i > (x > 0 ? s_sum[x - 1] : 0) ? a.keep[t - 1] : -1;
      if (!(at < s_q[x] && at > before)) s_bad[x] = 1;
    }
    __syncthreads();
    if (s_bad[tid]) r.n = 0;
    if (r.ok) a.lens[b] = r.ctx + r.n;
    const int kept = pages_of(r.ctx + r.n, a.page_shift);
    const int held = r.ok ? pages_of(r.ctx + r.q, a.page_shift) - kept : 0;
    sum = block_sum<kThreads>(held, red, &all);
    // The sums saturate at F: what is past it is dropped.
    const long long room = a.F - have - back;
    const int n = (int)(all < room ? all : (room > 0 ? room : 0));
    s_end[tid] = (int)(sum < n ? sum : n);
    s_from[tid] = kept - (int)(sum - held < n ? sum - held : n);
    __syncthreads();
    for (int k0 = tid; k0 < n; k0 += kAtOnce * kThreads) {
      int page[kAtOnce];
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        const int k = min(k0 + j * kThreads, n - 1), x = first_past_of<kThreads>(s_end, k);
        page[j] = a.table[(size_t)(b0 + x) * a.max_pages + (s_from[x] + k)];
      }
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j)
        if (k0 + j * kThreads < n) a.free_pages[have + back + k0 + j * kThreads] = page[j];
    }
    back += all;
    __syncthreads();
  }
  if (tid == 0) a.n_free_out[0] = have + back > a.F ? a.F : (int)(have + back);
}

__global__ __launch_bounds__(kThreads) void paged_keep_kernel(PagedKeepArgs a, int first, int last) {
  const int x = blockIdx.x;
  if (last && x == 0) cut_lists(a);
  else move_rows(a, first + (x - last) / a.H_kv, (x - last) % a.H_kv);
}

}  // namespace

hipError_t launch_paged_keep(const PagedKeepArgs& a, hipStream_t s) {
  // A launch has fewer than 2^32 threads.
  const int most = (1 << 23) / a.H_kv;
  for (int first = 0; first < a.S; first += most) {
    const int n = a.S - first < most ? a.S - first : most, list = first == 0;
    hipLaunchKernelGGL(paged_keep_kernel, dim3((unsigned)(n * a.H_kv + list)), dim3(kThreads), 0, s, a, first, list);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace rel
