// Append of a packed batch of new tokens to the paged Relation Cache: rotary
// encoding of P1 and P2 and Givens mixing of the information heads as in
// prestep.hip, with P2 and the mixed information stored to the tokens' slots
// (semantics in relation.h).
//
// One work-group per token: its first d_h / 2 threads form the token's sines
// and cosines once, in LDS, for all heads; then each thread takes units of 16
// elements: a group of 8 rotary pairs of one head of P1 or P2, or 16 channels
// of an information head (of both heads of a Givens pair).
//
// Bound by memory: 16,384 tokens of 32 + 8 heads of 128 in bf16 take 75 us, 5.4 TB/s
// read and written (204 and 201 MB by the counters, each byte once; on inputs rotated
// through 3 GB, so that none are left in the last-level cache); 64 tokens of 32 + 32 heads
// 4.9 us.
#include "rel_internal.h"
#include "rel_device.h"

namespace rel {

namespace {

constexpr int kThreads = 256;

template <typename Tin>
__device__ __forceinline__ void load8(const Tin* p, float (&x)[8]) {
  if constexpr (sizeof(Tin) == 2) {
    typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
    const bf16x8 v = *reinterpret_cast<const bf16x8*>(p);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = (float)v[e];
  } else {
    const float4 a = reinterpret_cast<const float4*>(p)[0];
    const float4 b = reinterpret_cast<const float4*>(p)[1];
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
}

template <typename Tin>
__device__ __forceinline__ void store8(Tin* p, const float (&x)[8]) {
  if constexpr (sizeof(Tin) == 2) {
    typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
    bf16x8 v;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = (__bf16)x[e];
    *reinterpret_cast<bf16x8*>(p) = v;
  } else {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
  }
}

template <typename Tin, int D>
__global__ __launch_bounds__(kThreads) void paged_append_kernel(PagedAppendArgs a, PrestepParams pp, int first) {
  constexpr int kGroups = D / 16;
  __shared__ float s_cos[D / 2], s_sin[D / 2];
  const int t = first + (int)blockIdx.x;
  const int slot = a.slot[t];
  if (slot < 0 || (slot >> a.page_shift) >= a.n_pages) return;   // uniform for the work-group
  const int tid = threadIdx.x;
  if (a.rope != 0 && tid < D / 2) {
    float sn, cs;
    sincos_of((double)a.pos[t] * pp.inv_freq[tid], &sn, &cs);
    s_cos[tid] = cs;
    s_sin[tid] = sn;
  }
  __syncthreads();
  const int page = slot >> a.page_shift, off = slot & ((1 << a.page_shift) - 1);
  // Row of head h in the pages.
  auto cache_row = [&](void* cache, int h) -> Tin* {
    return static_cast<Tin*>(cache) + (((((size_t)page * a.H_kv + h) << a.page_shift) + off) * D);
  };
  const int coord = (a.H + a.H_kv) * kGroups;
  const int info = (a.mix ? a.H_kv / 2 : a.H_kv) * kGroups;
  for (int u = tid; u < coord + info; u += kThreads) {
    const int g = u % kGroups;
    if (u < coord) {
      const int hh = u / kGroups;
      const Tin* src;
      Tin* dst;
      if (hh < a.H) {
        src = static_cast<const Tin*>(a.P1) + (size_t)t * a.ld1 + (size_t)hh * D;
        dst = static_cast<Tin*>(a.P1o) + ((size_t)t * a.H + hh) * D;
      } else {
        src = static_cast<const Tin*>(a.P2) + (size_t)t * a.ld2 + (size_t)(hh - a.H) * D;
        dst = cache_row(a.cP2, hh - a.H);
      }
      const int oa = a.rope == 2 ? 8 * g : 16 * g;
      const int ob = a.rope == 2 ? D / 2 + 8 * g : 16 * g + 8;
      float x[8], y[8];
      load8(src + oa, x);
      load8(src + ob, y);
      if (a.rope == 1) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float c0 = s_cos[8 * g + e], n0 = s_sin[8 * g + e], c1 = s_cos[8 * g + 4 + e], n1 = s_sin[8 * g + 4 + e];
          const float p = x[2 * e], q = x[2 * e + 1], r = y[2 * e], w = y[2 * e + 1];
          x[2 * e] = fmaf(p, c0, -q * n0);
          x[2 * e + 1] = fmaf(p, n0, q * c0);
          y[2 * e] = fmaf(r, c1, -w * n1);
          y[2 * e + 1] = fmaf(r, n1, w * c1);
        }
      } else if (a.rope == 2) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float c0 = s_cos[8 * g + e], n0 = s_sin[8 * g + e], p = x[e], q = y[e];
          x[e] = fmaf(p, c0, -q * n0);
          y[e] = fmaf(p, n0, q * c0);
        }
      }
      store8(dst + oa, x);
      store8(dst + ob, y);
    } else {
      const int k = (u - coord) / kGroups;
      const Tin* src = static_cast<const Tin*>(a.I) + (size_t)t * a.ldi + 16 * g;
      float x[2][8];
      if (a.mix) {
        const int ha = a.pairing == 0 ? 2 * k : 2 * k + 1, hb = (ha + 1) % a.H_kv;
        const float c = pp.cos_theta[k], s = pp.sin_theta[k];
        float y[2][8];
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          load8(src + (size_t)ha * D + 8 * w, x[w]);
          load8(src + (size_t)hb * D + 8 * w, y[w]);
        }
#pragma unroll
        for (int w = 0; w < 2; ++w) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float p = x[w][e], q = y[w][e];
            x[w][e] = fmaf(c, p, -s * q);
            y[w][e] = fmaf(s, p, c * q);
          }
          store8(cache_row(a.cV, ha) + 16 * g + 8 * w, x[w]);
          store8(cache_row(a.cV, hb) + 16 * g + 8 * w, y[w]);
        }
      } else {
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          load8(src + (size_t)k * D + 8 * w, x[w]);
          store8(cache_row(a.cV, k) + 16 * g + 8 * w, x[w]);
        }
      }
    }
  }
}

template <typename Tin, int D>
hipError_t launch_typed(const PagedAppendArgs& a, const PrestepParams& pp, hipStream_t s) {
  // A launch has fewer than 2^32 threads.
  constexpr int kMost = 1 << 23;
  for (int64_t first = 0; first < a.N; first += kMost) {
    const unsigned n = (unsigned)(a.N - first < kMost ? a.N - first : kMost);
    hipLaunchKernelGGL((paged_append_kernel<Tin, D>), dim3(n), dim3(kThreads), 0, s, a, pp, (int)first);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_paged_append(const PagedAppendArgs& a, const PrestepParams& pp, bool bf16, hipStream_t s) {
  switch (a.d_h) {
    case 32: return bf16 ? launch_typed<__bf16, 32>(a, pp, s) : launch_typed<float, 32>(a, pp, s);
    case 48: return bf16 ? launch_typed<__bf16, 48>(a, pp, s) : launch_typed<float, 48>(a, pp, s);
    case 64: return bf16 ? launch_typed<__bf16, 64>(a, pp, s) : launch_typed<float, 64>(a, pp, s);
    case 80: return bf16 ? launch_typed<__bf16, 80>(a, pp, s) : launch_typed<float, 80>(a, pp, s);
    case 128: return bf16 ? launch_typed<__bf16, 128>(a, pp, s) : launch_typed<float, 128>(a, pp, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace rel
