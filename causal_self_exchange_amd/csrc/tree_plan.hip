// Ancestor bits and positions of the tokens of drafted trees, from their parents
// (integers only; semantics in relation.h).
//
// One work-group per request, and one for the rows behind the last. The parents go to LDS;
// each token walks up to the first ancestor outside its own 32 tokens (a parent comes
// before its child, so a walk never returns to them), and the words of its bits are formed
// by going from one such ancestor to the next: at most 31 steps and then one for each 32
// tokens, where a walk from each token to the root was as many as the token is deep for
// each of its words (8 requests of 1024 tokens in a line, 32 words: 3.8 ms, now 0.2). Bound by the
// latency of these steps: 256 requests of up to 60 tokens 3.5 us.
#include "rel_internal.h"

namespace rel {

namespace {

constexpr int kThreads = 256;

__global__ __launch_bounds__(kThreads) void tree_plan_kernel(TreePlanArgs a) {
  __shared__ int s_up[32 * REL_MAX_TREE_WORDS];     // a token's parent
  __shared__ int s_out[32 * REL_MAX_TREE_WORDS];    // its nearest ancestor outside its 32 tokens
  __shared__ unsigned s_own[32 * REL_MAX_TREE_WORDS];   // those among them
  const int b = blockIdx.x, tid = threadIdx.x;
  if (b == a.S) {
    // Behind the last request; where that one ends past N, behind the last that does not.
    int from = max(a.cu[a.S], 0);
    if (from > a.N) {
      from = 0;
      for (int k = tid; k < a.S; k += kThreads) from = max(from, a.cu[k] <= a.N ? a.cu[k] : 0);
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) from = max(from, __shfl_xor(from, o, 64));
      if ((tid & 63) == 0) s_up[tid >> 6] = from;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kThreads / 64; ++w) from = max(from, s_up[w]);
    }
    for (int64_t t = (int64_t)from + tid; t < a.N; t += kThreads) a.pos[t] = -1;
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
  for (int k = tid; k < q; k += kThreads) {
    unsigned bits = 0;
    int up = s_up[k];
    for (; up >= (k & ~31); up = s_up[up]) bits |= 1u << (up & 31);   // s_up[k] < k, so the walk ends
    s_own[k] = bits;
    s_out[k] = up;
  }
  __syncthreads();
  for (int i = tid; i < q * a.words; i += kThreads) {
    const int k = i / a.words, w = i - k * a.words;
    unsigned bits = 0;
    int depth = 0;
    for (int x = k; x >= 32 * w;) {
      const unsigned own = s_own[x];
      const int out = s_out[x];
      bits |= x >> 5 == w ? own : 0u;
      bits |= out >= 0 && out >> 5 == w ? 1u << (out & 31) : 0u;
      depth += __popc(own) + (out >= 0);
      x = out;
    }
    a.tree[(size_t)(first + k) * a.words + w] = bits;
    if (w == 0) a.pos[first + k] = total - q + depth;      // the walk to the root
  }
}

}  // namespace

hipError_t launch_tree_plan(const TreePlanArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(tree_plan_kernel, dim3(a.S + 1), dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace rel
