// Relation forward of a packed batch of new tokens against the paged Relation
// Cache (semantics in relation.h).
//
// One work-group per (packed token, query head): its rows of lanes scan the
// token's history with a running maximum each, the states meet in LDS, and the
// Self entry and the count term enter once (RowCombine).
#include "rel_internal.h"
#include "rel_device.h"

namespace rel {

namespace {

constexpr int kThreads = 256;

// The request of packed token t: cu[b] <= t < cu[b + 1], the first such b.
__device__ __forceinline__ int request_of(const PagedArgs& a, int t) {
  int lo = 0, hi = a.S;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (a.cu[mid + 1] > t) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

template <typename Tin, int D>
__global__ __launch_bounds__(kThreads) void paged_scan_kernel(PagedArgs a, HeadParams hp) {
  constexpr int VEC = 16 / (int)sizeof(Tin);
  constexpr int LIVE = D / VEC;
  constexpr int LPR = LIVE <= 4 ? 4 : (LIVE <= 8 ? 8 : (LIVE <= 16 ? 16 : 32));
  constexpr int GROUPS = kThreads / LPR;
  __shared__ float s_m[GROUPS], s_l[GROUPS], s_z[GROUPS][D + 1], s_u;
  const int t = blockIdx.x, h = blockIdx.y;
  const int b = request_of(a, t);
  if (b >= a.S) return;
  const int c0 = a.cu[b], q = a.cu[b + 1] - c0, total = a.total[b];
  if (c0 < 0 || c0 > t || a.cu[b + 1] > a.N || q > a.max_new || total < q ||
      total > ((long long)a.max_pages << a.page_shift))
    return;
  const int p = total - q + (t - c0);
  const int kvh = h / (a.H / a.H_kv);
  const int tid = threadIdx.x, g = tid / LPR, sl = tid % LPR;
  const bool live = sl < LIVE;
  const int so = live ? sl * VEC : 0;
  const Tin* p1 = static_cast<const Tin*>(a.P1) + (size_t)t * a.ld1 + (size_t)h * D + so;
  auto row = [&](const void* cache, int j, float (&x)[VEC]) {
    const int page = a.table[(size_t)b * a.max_pages + (j >> a.page_shift)];
    const bool in = live && page >= 0 && page < a.n_pages;
    const Tin* r = static_cast<const Tin*>(cache) +
                   (((((size_t)(in ? page : 0) * a.H_kv + kvh) << a.page_shift) + (j & ((1 << a.page_shift) - 1))) * D + so);
#pragma unroll
    for (int e = 0; e < VEC; ++e) x[e] = in ? to_f32(r[e]) : 0.0f;
  };
  float qv[VEC], z[VEC], x[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    qv[e] = live ? to_f32(p1[e]) : 0.0f;
    z[e] = 0.0f;
  }
  float m = kEmptyMax, l = 0.0f;
  for (int j = g; j <= p; j += GROUPS) {
    row(a.cP2, j, x);
    float u = 0.0f;
#pragma unroll
    for (int e = 0; e < VEC; ++e) u = fmaf(qv[e], x[e], u);
#pragma unroll
    for (int off = LPR / 2; off > 0; off >>= 1) u += __shfl_xor(u, off);
    u *= hp.scale;
    if (j == p) {
      if (sl == 0) s_u = u;
      break;
    }
    const float E = silu_f32(u), mn = fmaxf(m, E);
    const float w = expf(E - mn), k = expf(m - mn);
    m = mn;
    l = l * k + w;
    row(a.cV, j, x);
#pragma unroll
    for (int e = 0; e < VEC; ++e) z[e] = z[e] * k + w * x[e];
  }
  if (sl == 0) {
    s_m[g] = m;
    s_l[g] = l;
  }
  if (live)
#pragma unroll
    for (int e = 0; e < VEC; ++e) s_z[g][so + e] = z[e];
  __syncthreads();
  float M = kEmptyMax, ls = 0.0f;
  for (int k = 0; k < GROUPS; ++k) M = fmaxf(M, s_m[k]);
  for (int k = 0; k < GROUPS; ++k) ls += s_l[k] * expf(s_m[k] - M);
  const RowCombine cmb(sigmoid_f32(s_u * hp.inv_tau[h]), M, ls, hp.lambda * logf((float)(p + 1)));
  if (g == 0 && live) {
    row(a.cV, p, x);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      float zs = 0.0f;
      for (int k = 0; k < GROUPS; ++k) zs += s_z[k][so + e] * expf(s_m[k] - M);
      static_cast<Tin*>(a.Y)[((size_t)t * a.H + h) * D + so + e] = from_f32<Tin>(cmb.w_self * x[e] + cmb.w_hist * zs);
    }
  }
}

template <typename Tin, int D>
hipError_t launch_typed(const PagedArgs& a, const HeadParams& hp, hipStream_t s) {
  hipLaunchKernelGGL((paged_scan_kernel<Tin, D>), dim3((unsigned)a.N, a.H), dim3(kThreads), 0, s, a, hp);
  return hipGetLastError();
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
