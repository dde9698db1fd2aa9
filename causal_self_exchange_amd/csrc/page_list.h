// Sums and searches over a batch's requests, shared by the kernels that take pages from
// the paged Relation Cache's free list and give them back.
#pragma once

#include <hip/hip_runtime.h>

namespace rel {

namespace {

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
template <int T, typename Int>
__device__ __forceinline__ int first_past_of(const Int* end, Int i) {
  int at = 0;
#pragma unroll
  for (int step = T / 2; step > 0; step >>= 1) at += end[at + step - 1] <= i ? step : 0;
  return at;
}

__device__ __forceinline__ int pages_of(int rows, int shift) {
  return (int)(((long long)rows + (1 << shift) - 1) >> shift);
}

}  // namespace

}  // namespace rel
