// Block tables, slots and positions of a packed batch of the paged Relation
// Cache, from the request lengths (integers only; semantics in relation.h).
//
// page_map: one work-group walks the requests 1024 at a time, twice. The first
//   walk numbers the pages that finished requests return (a prefix sum) and
//   pushes them on the free list; the second sums the new tokens (the packed
//   offsets) and the pages needed, and moves each request's pages from the top
//   of the list to its table row. One work-group, because both sums run through
//   all requests and the second needs the whole first one.
// page_slots: one thread per packed token finds its request by bisection in
//   the offsets and its page in the table.
// The call moves a few KB: it is bound by the latency of its dependent steps.
#include "rel_internal.h"
#include "rel_device.h"

namespace rel {

namespace {

constexpr int kMapThreads = 1024;
constexpr int kMapWaves = kMapThreads / 64;
constexpr int kSlotThreads = 256;

// Inclusive sum over the work-group and the work-group's total.
__device__ __forceinline__ long long block_sum(long long v, long long* red, long long* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  long long x = v;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const long long y = __shfl_up(x, o, 64);
    if (lane >= o) x += y;
  }
  __syncthreads();                     // the previous use of red is over
  if (lane == 63) red[wave] = x;
  __syncthreads();
  long long before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kMapWaves; ++w) {
    const long long r = red[w];
    before += w < wave ? r : 0;
    all += r;
  }
  *total = all;
  return before + x;
}

__device__ __forceinline__ int pages_of(int rows, int shift) {
  return (int)(((long long)rows + (1 << shift) - 1) >> shift);
}

struct Request {
  int len, q;        // cached tokens, new tokens (0 for a finished request)
  bool gone, fits;   // finished with a valid length; sizes within the table row
  __device__ __forceinline__ Request(const PageMapArgs& a, int b) {
    len = 0;
    q = 0;
    gone = fits = false;
    if (b < a.S) {
      const int n = a.n_new[b];
      len = a.len[b];
      q = n > 0 ? n : 0;
      const bool in_row = len >= 0 && (long long)len + q <= ((long long)a.max_pages << a.page_shift);
      gone = n == -1 && in_row;
      fits = n >= 0 && in_row;
    }
  }
};

// Slot and position of packed token t of request b, whose cached rows are len.
__device__ __forceinline__ void write_slot(const PageMapArgs& a, int t, int b, int first, bool live) {
  int slot = -1, pos = -1;
  if (live) {
    pos = a.len[b] + (t - first);
    const int page = a.table[(size_t)b * a.max_pages + (pos >> a.page_shift)];
    if (page >= 0 && page < a.n_pages) slot = (page << a.page_shift) + (pos & ((1 << a.page_shift) - 1));
  }
  a.slot[t] = slot;
  a.pos[t] = pos;
}

__device__ __forceinline__ void token_slot(const PageMapArgs& a, int t) {
  // The request with cu[b] <= t < cu[b + 1]: the first b whose end is past t.
  int lo = 0, hi = a.S;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (a.cu[mid + 1] > t) hi = mid;
    else lo = mid + 1;
  }
  const bool in = lo < a.S;
  const int b = in ? lo : 0;
  write_slot(a, t, b, a.cu[b], in && a.total[b] >= 0);
}

__global__ __launch_bounds__(kMapThreads) void page_map_kernel(PageMapArgs a, int with_slots) {
  __shared__ long long red[kMapWaves];
  const int tid = threadIdx.x;
  long long all;

  // Returned pages.
  int have = a.n_free[0];
  have = have < 0 ? 0 : (have > a.F ? a.F : have);
  long long back = 0;
  for (int b0 = 0; b0 < a.S; b0 += kMapThreads) {
    const int b = b0 + tid;
    const Request r(a, b);
    const int held = r.gone ? pages_of(r.len, a.page_shift) : 0;
    const long long at = have + back + block_sum(held, red, &all) - held;
    for (int k = 0; k < held && at + k < a.F; ++k) a.free_pages[at + k] = a.table[(size_t)b * a.max_pages + k];
    back += all;
  }
  const int top = (int)(have + back > a.F ? (long long)a.F : have + back);
  __syncthreads();                     // the list is whole before pages are taken from it

  // Offsets, totals and pages for the new tokens.
  long long tokens = 0, needed = 0, taken = 0;
  for (int b0 = 0; b0 < a.S; b0 += kMapThreads) {
    const int b = b0 + tid;
    const Request r(a, b);
    const long long end = tokens + block_sum(r.q, red, &all);
    tokens += all;
    const int held = pages_of(r.len, a.page_shift);
    bool ok = r.fits && end <= a.N;
    const int need = ok ? pages_of(r.len + r.q, a.page_shift) - held : 0;
    const long long upto = needed + block_sum(need, red, &all);
    needed += all;
    ok = ok && (need == 0 || upto <= top);
    if (b < a.S) {
      constexpr long long kMost = 0x7fffffff;
      a.cu[b + 1] = (int)(end < kMost ? end : kMost);
      a.total[b] = ok ? r.len + r.q : (r.gone ? 0 : -1);
    }
    if (ok) {
      int* row = a.table + (size_t)b * a.max_pages + held;
      const int* from = a.free_pages + (top - 1 - (upto - need));
      for (int k = 0; k < need; ++k) row[k] = from[-k];
    }
    block_sum(ok ? need : 0, red, &all);
    taken += all;
  }
  if (tid == 0) {
    a.cu[0] = 0;
    a.n_free_out[0] = top - (int)taken;
  }
  if (!with_slots) return;
  __threadfence_block();
  __syncthreads();                     // offsets, totals and table are written
  for (int t = tid; t < a.N; t += kMapThreads) token_slot(a, t);
}

__global__ __launch_bounds__(kSlotThreads) void page_slots_kernel(PageMapArgs a) {
  const int t = blockIdx.x * kSlotThreads + threadIdx.x;
  if (t < a.N) token_slot(a, t);
}

}  // namespace

hipError_t launch_page_map(const PageMapArgs& a, hipStream_t s) {
  const int with_slots = a.N <= kMapThreads;
  hipLaunchKernelGGL(page_map_kernel, dim3(1), dim3(kMapThreads), 0, s, a, with_slots);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || with_slots) return e;
  const unsigned blocks = (unsigned)(((long long)a.N + kSlotThreads - 1) / kSlotThreads);
  hipLaunchKernelGGL(page_slots_kernel, dim3(blocks), dim3(kSlotThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace rel
