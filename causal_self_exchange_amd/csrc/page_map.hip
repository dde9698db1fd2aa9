// Block tables, slots and positions of a packed batch of the paged Relation
// Cache, from the request lengths (integers only; semantics in relation.h).
//
// page_map: one work-group takes the requests 1024 at a time, twice. The first
//   walk numbers the pages that finished requests return (a prefix sum) and
//   pushes them on the free list; the second sums the new tokens (the packed
//   offsets) and the pages needed, and moves pages from the top of the list to
//   the table rows. One work-group, because both sums run through all requests
//   and the second needs the whole first one. Pages are moved one per thread,
//   whichever request they belong to (found by bisection in the sums, in LDS): a
//   request of 2000 tokens returns 125 pages, which one thread would move in 25 us.
//   A thread has four in flight: 1024 prompts, which move 10,000 pages, 19.0 us one
//   by one, 14.7 so. Up to 256 requests and 512 tokens take 4 waves instead of 16,
//   whose barriers and sums are shorter: 256 requests of one token 8.3 us by 16
//   waves, 5.3 by 4.
// page_slots: one thread per packed token finds its request by bisection in
//   the offsets and its page in the table (60,000 tokens 4 us). Up to kSlotsInline
//   tokens page_map does it itself.
// The call moves a few KB: it is bound by the latency of its dependent steps.
#include "rel_internal.h"
#include "rel_device.h"

namespace rel {

namespace {

constexpr int kMapThreads = 1024;
constexpr int kMapFew = 256;              // threads for as many requests
constexpr int kAtOnce = 4;                // pages that a thread moves together
constexpr int kSlotThreads = 256;
constexpr int kSlotsInline = 4096;
constexpr int kSlotsLds = 4096;           // requests whose offsets page_slots keeps in LDS

// Inclusive sum over a work-group of T threads, and its total.
template <int T>
__device__ __forceinline__ long long block_sum(long long x, long long* red, long long* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const long long y = __shfl_up(x, o, 64);
    if (lane >= o) x += y;
  }
  if (lane == 63) red[wave] = x;
  __syncthreads();
  long long before = 0, all = 0;
#pragma unroll 4
  for (int w = 0; w < T / 64; ++w) {
    const long long r = red[w];
    before += w < wave ? r : 0;
    all += r;
  }
  __syncthreads();
  *total = all;
  return before + x;
}

// The first k of n with end[k] > i (n when there is none).
template <typename Int>
__device__ __forceinline__ int first_past(const Int* end, int n, Int i) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (end[mid] > i) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

// The same for n = T, where there is one, in a fixed number of steps: several
// searches run side by side.
template <int T>
__device__ __forceinline__ int first_past_of(const int* end, int i) {
  int at = 0;
#pragma unroll
  for (int step = T / 2; step > 0; step >>= 1) at += end[at + step - 1] <= i ? step : 0;
  return at;
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

// Slot and position of packed token t, the (t - first)th new one of request b,
// which is granted its pages (live) and holds len tokens already.
__device__ __forceinline__ void write_slot(const PageMapArgs& a, int t, int b, int first, int len, bool live) {
  int slot = -1, pos = -1;
  if (live) {
    pos = len + (t - first);
    const int page = a.table[(size_t)b * a.max_pages + (pos >> a.page_shift)];
    if (page >= 0 && page < a.n_pages) slot = (page << a.page_shift) + (pos & ((1 << a.page_shift) - 1));
  }
  a.slot[t] = slot;
  a.pos[t] = pos;
}

template <int T>
__global__ __launch_bounds__(T) void page_map_kernel(PageMapArgs a, int with_slots) {
  __shared__ long long red[T / 64];
  __shared__ int s_end[T], s_held[T], s_to[T], s_ok[T], s_taken;
  const int tid = threadIdx.x;
  const Request own(a, tid);
  long long all;
  if (tid == 0) s_taken = 0;

  // Returned pages. The sums saturate at F: what is past it is dropped.
  int have = a.n_free[0];
  have = have < 0 ? 0 : (have > a.F ? a.F : have);
  long long back = 0;
  for (int b0 = 0; b0 < a.S; b0 += T) {
    const Request r = b0 == 0 ? own : Request(a, b0 + tid);
    const int held = r.gone ? pages_of(r.len, a.page_shift) : 0;
    const long long sum = block_sum<T>(held, red, &all);
    const long long room = a.F - have - back;             // entries left above the list
    const int n = (int)(all < room ? all : (room > 0 ? room : 0));
    s_end[tid] = (int)(sum < n ? sum : n);
    s_held[tid] = (int)(sum - held < n ? sum - held : n);
    __syncthreads();
    for (int k0 = tid; k0 < n; k0 += kAtOnce * T) {
      int page[kAtOnce];
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        const int k = min(k0 + j * T, n - 1), x = first_past_of<T>(s_end, k);
        page[j] = a.table[(size_t)(b0 + x) * a.max_pages + (k - s_held[x])];
      }
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j)
        if (k0 + j * T < n) a.free_pages[have + back + k0 + j * T] = page[j];
    }
    back += all;
    __syncthreads();                   // s_end is read; the last time, the list is whole too
  }
  const int top = (int)(have + back > a.F ? (long long)a.F : have + back);

  // Offsets, totals and pages for the new tokens.
  long long tokens = 0, needed = 0;
  constexpr long long kMost = 0x7fffffff;
  for (int b0 = 0; b0 < a.S; b0 += T) {
    const int b = b0 + tid;
    const Request r = b0 == 0 ? own : Request(a, b);
    const long long end = tokens + block_sum<T>(r.q, red, &all);
    tokens += all;
    const int held = pages_of(r.len, a.page_shift);
    bool ok = r.fits && end <= a.N;
    const int need = ok ? pages_of(r.len + r.q, a.page_shift) - held : 0;
    const long long upto = needed + block_sum<T>(need, red, &all);
    ok = ok && (need == 0 || upto <= top);
    if (b < a.S) {
      a.cu[b + 1] = (int)(end < kMost ? end : kMost);
      a.total[b] = ok ? r.len + r.q : (r.gone ? 0 : -1);
    }
    // The requests that find their pages come first: the list closes at the first
    // that does not, and taken is the last one's sum.
    const bool takes = ok && need > 0;
    if (takes) atomicMax(&s_taken, (int)upto);
    s_end[tid] = (int)(upto < kMost ? upto : kMost);      // pages up to and with this request
    s_to[tid] = held;
    s_held[tid] = need;
    __syncthreads();
    const int taken = s_taken, before = (int)(needed < top ? needed : top);
    for (int k0 = before + tid; k0 < taken; k0 += kAtOnce * T) {
      int page[kAtOnce];
      size_t to[kAtOnce];
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        const int k = min(k0 + j * T, taken - 1), x = first_past_of<T>(s_end, k);
        page[j] = a.free_pages[top - 1 - k];
        to[j] = (size_t)(b0 + x) * a.max_pages + s_to[x] + (k - (s_end[x] - s_held[x]));
      }
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j)
        if (k0 + j * T < taken) a.table[to[j]] = page[j];
    }
    needed += all;
    __syncthreads();                   // the lists are read, the pages are in the table
    if (with_slots && a.S <= T) {
      s_end[tid] = b < a.S ? (int)(end < kMost ? end : kMost) : (int)kMost;
      s_to[tid] = r.len;
      s_held[tid] = (int)(end - r.q < kMost ? end - r.q : kMost);
      s_ok[tid] = ok;
    }
  }
  if (tid == 0) {
    a.cu[0] = 0;
    a.n_free_out[0] = top - s_taken;
  }
  if (!with_slots) return;
  __syncthreads();
  for (int t = tid; t < a.N; t += T) {
    const int x = first_past(s_end, a.S, t);
    const bool in = x < a.S;
    write_slot(a, t, in ? x : 0, s_held[in ? x : 0], s_to[in ? x : 0], in && s_ok[x]);
  }
}

__global__ __launch_bounds__(kSlotThreads) void page_slots_kernel(PageMapArgs a) {
  __shared__ int s_end[kSlotsLds];
  const bool lds = a.S <= kSlotsLds;
  if (lds) {
    for (int b = threadIdx.x; b < a.S; b += kSlotThreads) s_end[b] = a.cu[b + 1];
    __syncthreads();
  }
  const int t = blockIdx.x * kSlotThreads + threadIdx.x;
  if (t >= a.N) return;
  const int x = lds ? first_past<int>(s_end, a.S, t) : first_past<int>(a.cu + 1, a.S, t);
  const bool in = x < a.S;
  const int b = in ? x : 0;
  write_slot(a, t, b, a.cu[b], a.len[b], in && a.total[b] >= 0);
}

}  // namespace

hipError_t launch_page_map(const PageMapArgs& a, hipStream_t s) {
  const int with_slots = a.N <= kSlotsInline && a.S <= kMapThreads;
  if (a.S <= kMapFew && a.N <= 2 * kMapFew) {
    hipLaunchKernelGGL(page_map_kernel<kMapFew>, dim3(1), dim3(kMapFew), 0, s, a, with_slots);
  } else {
    hipLaunchKernelGGL(page_map_kernel<kMapThreads>, dim3(1), dim3(kMapThreads), 0, s, a, with_slots);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || with_slots) return e;
  const unsigned blocks = (unsigned)(((long long)a.N + kSlotThreads - 1) / kSlotThreads);
  hipLaunchKernelGGL(page_slots_kernel, dim3(blocks), dim3(kSlotThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace rel
