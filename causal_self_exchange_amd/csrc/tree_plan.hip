// Ancestor bits and positions of the tokens of drafted trees, from their parents
// (integers only; semantics in relation.h).
//
// One work-group per request, and one for the rows behind the last: the parents go to
// LDS, and each thread walks from its token to the root for one word of the token's bits.
// A walk is as long as the token is deep, so the call is bound by the latency of a few
// dependent steps.
#include "rel_internal.h"

namespace rel {

namespace {

constexpr int kThreads = 256;

__global__ __launch_bounds__(kThreads) void tree_plan_kernel(TreePlanArgs a) {
  __shared__ int s_up[32 * REL_MAX_TREE_WORDS];
  const int b = blockIdx.x, tid = threadIdx.x;
  if (b == a.S) {
    for (int64_t t = (int64_t)max(a.cu[a.S], 0) + tid; t < a.N; t += kThreads) a.pos[t] = -1;
    return;
  }
  const int first = a.cu[b], end = a.cu[b + 1], total = a.total[b];
  if (first < 0 || end <= first || end > a.N) return;
  const int q = end - first;
  if (total < q || q > 32 * a.words) {
    for (int k = tid; k < q; k += kThreads) a.pos[first + k] = total < q ? -1 : total - q + k;
    return;
  }
  for (int k = tid; k < q; k += kThreads) {
    const int p = a.parent[first + k];
    s_up[k] = p >= 0 && p < k ? p : -1;
  }
  __syncthreads();
  for (int i = tid; i < q * a.words; i += kThreads) {
    const int k = i / a.words, w = i - k * a.words;
    unsigned bits = 0;
    int depth = 0;
    for (int up = s_up[k]; up >= 0; up = s_up[up]) {       // s_up[k] < k, so the walk ends
      bits |= up >> 5 == w ? 1u << (up & 31) : 0u;
      ++depth;
    }
    a.tree[(size_t)(first + k) * a.words + w] = bits;
    if (w == 0) a.pos[first + k] = total - q + depth;
  }
}

}  // namespace

hipError_t launch_tree_plan(const TreePlanArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(tree_plan_kernel, dim3(a.S + 1), dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace rel
