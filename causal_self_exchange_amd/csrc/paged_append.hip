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

// The 8 rotary pairs of a group, by their cosines and sines: x and y are the group's 16
// elements in order (interleaved pairs) or its 8 of either half (half split).
__device__ __forceinline__ void turn(int rope, const float* cs, const float* sn, float (&x)[8], float (&y)[8]) {
  if (rope == 1) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float c0 = cs[e], n0 = sn[e], c1 = cs[4 + e], n1 = sn[4 + e];
      const float p = x[2 * e], q = x[2 * e + 1], r = y[2 * e], w = y[2 * e + 1];
      x[2 * e] = fmaf(p, c0, -q * n0);
      x[2 * e + 1] = fmaf(p, n0, q * c0);
      y[2 * e] = fmaf(r, c1, -w * n1);
      y[2 * e + 1] = fmaf(r, n1, w * c1);
    }
  } else if (rope == 2) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float c0 = cs[e], n0 = sn[e], p = x[e], q = y[e];
      x[e] = fmaf(p, c0, -q * n0);
      y[e] = fmaf(p, n0, q * c0);
    }
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
      turn(a.rope, s_cos + 8 * g, s_sin + 8 * g, x, y);
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

// ---- 8-bit pages ------------------------------------------------------------------
//
// A row x of P2 or of the information state is stored as e4m3 values q and one exponent
// k, x = q 2^k: k is the least with max |x| <= 448 2^k. A power of two loses nothing
// against a finer scale, as e4m3 rounds relative to each value (2^-4 of it, down to 2^-6
// 2^k, below which steps are 2^-9 2^k); it costs a byte, and no multiplication where the
// forward turns the values back into bf16. Lanes of a power of two share a row (16
// elements each), so that its maximum is a few exchanges between lanes.
//
// The row is rounded once, from the fp32 of its rotation or mixing, as above but for the
// cosines and sines, which are fp64 ones in two parts (the mixing's from fp64 angles). A value
// of 2^-6 2^k and more that is near the middle between two steps then (one in 60,000) is formed
// again in fp64, so that the nearest is stored. All rotations and mixings in fp64 took 16,384
// tokens of 32 + 8 heads of 128 from 75 to 105 us.
//
// Bound by memory: those tokens read 201 MB and write 168 MB in 83 to 85 us, 4.4 TB/s (a copy
// of 4 GB 4.7; without the values formed again 77 us); 64 tokens of 32 + 32 heads take 7.5 us.
constexpr int kLowScale = -100, kHighScale = 119;
constexpr float kMostE4m3 = 448.0f;

// k from a row's maximum (of its finite elements); 2^-k is a normal fp32 number.
__device__ __forceinline__ int scale_exponent(float most) {
  const unsigned b = __float_as_uint(most);
  const int k = (int)(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);   // 448 = 1.75 2^8
  return min(max(k, kLowScale), kHighScale);
}

// sin and cos of an angle by their Taylor series after the reduction by pi / 2: to x^17 on
// [-pi/4, pi/4], where the next term is below 2^-58.
__device__ __forceinline__ void sincos_f64(double ang, double* s, double* c) {
  const double k = rint(ang * 0.63661977236758134);           // 2 / pi
  const double r = fma(-k, 6.123233995736766e-17, fma(-k, 1.5707963267948966, ang));
  const int q = (int)(long long)k & 3;
  const double z = r * r;
  double sr = 1.0 / 355687428096000.0, cr = -1.0 / 6402373705728000.0;
  sr = fma(z, sr, -1.0 / 1307674368000.0);
  sr = fma(z, sr, 1.0 / 6227020800.0);
  sr = fma(z, sr, -1.0 / 39916800.0);
  sr = fma(z, sr, 1.0 / 362880.0);
  sr = fma(z, sr, -1.0 / 5040.0);
  sr = fma(z, sr, 1.0 / 120.0);
  sr = fma(z, sr, -1.0 / 6.0);
  sr = fma(r * z, sr, r);
  cr = fma(z, cr, 1.0 / 20922789888000.0);
  cr = fma(z, cr, -1.0 / 87178291200.0);
  cr = fma(z, cr, 1.0 / 479001600.0);
  cr = fma(z, cr, -1.0 / 3628800.0);
  cr = fma(z, cr, 1.0 / 40320.0);
  cr = fma(z, cr, -1.0 / 720.0);
  cr = fma(z, cr, 1.0 / 24.0);
  cr = fma(z, cr, -0.5);
  cr = fma(z, cr, 1.0);
  const double sv = (q & 1) ? cr : sr, cv = (q & 1) ? sr : cr;
  *s = (q & 2) ? -sv : sv;
  *c = ((q + 1) & 2) ? -cv : cv;
}

__device__ __forceinline__ float finite_max(const float (&x)[8], const float (&y)[8]) {
  float m = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float p = fabsf(x[e]), q = fabsf(y[e]);
    m = fmaxf(m, fmaxf(p <= 3.4028234e38f ? p : 0.0f, q <= 3.4028234e38f ? q : 0.0f));
  }
  return m;
}

// Eight elements as e4m3, to nearest even; what is past the largest scale saturates,
// NaN and infinities become NaN.
__device__ __forceinline__ uint2 quantise8(const float (&x)[8], float inv) {
  float y[8];
#pragma unroll
  for (int e = 0; e < 8; ++e)
    y[e] = fabsf(x[e]) <= 3.4028234e38f ? __builtin_amdgcn_fmed3f(x[e] * inv, -kMostE4m3, kMostE4m3) : x[e];
  int lo = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], lo, true);
  int hi = __builtin_amdgcn_cvt_pk_fp8_f32(y[4], y[5], 0, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(y[6], y[7], hi, true);
  return make_uint2((unsigned)lo, (unsigned)hi);
}

// Whether x is within 8 steps of fp32 of the middle between two e4m3 values (of 2^-6 and
// more over the row's scale, where these have four bits, whatever the scale).
__device__ __forceinline__ bool near_tie(float x) { return (__float_as_uint(x) & 0xfffffu) - 0x7fff8u <= 16u; }

// x in fp32, but not in the middle unless it is there.
__device__ __forceinline__ float beside_tie(double x) {
  const float f = (float)x;
  unsigned b = __float_as_uint(f);
  if ((b & 0xfffffu) == 0x80000u && (double)f != x) b += fabs(x) > fabs((double)f) ? 1u : -1u;
  return __uint_as_float(b);
}

// Values that are looked at together: with 8 the registers cost two work-groups (of the
// mixing: 96 us).
constexpr int kTogether = 4;

// A number in two parts: 16 bits, whose products with bf16 numbers are exact in fp32, and
// what they leave, to 2^-39.
__device__ __forceinline__ float2 split(double x) {
  const float hi = __uint_as_float(__float_as_uint((float)x) & 0xffffff00u);
  return make_float2(hi, (float)(x - hi));
}

// kTogether pairs u(e), v(e) of a row that is quantised turned by factors(e), a split cosine
// and sine: each sum of exact products is rounded once, and again with what the rests give, so
// that its error is a few steps of the result also where a pair nearly cancels.
struct Factors { float2 c, n; };
template <typename U, typename V, typename F>
__device__ __forceinline__ void turn_together(U u, V v, F factors) {
  float p[kTogether], q[kTogether];
  bool near = false;
#pragma unroll
  for (int e = 0; e < kTogether; ++e) {
    const auto [c, n] = factors(e);
    p[e] = u(e);
    q[e] = v(e);
    u(e) = fmaf(c.x, p[e], -n.x * q[e]) + fmaf(c.y, p[e], -n.y * q[e]);
    v(e) = fmaf(n.x, p[e], c.x * q[e]) + fmaf(n.y, p[e], c.y * q[e]);
    near |= near_tie(u(e));
    near |= near_tie(v(e));
  }
  if (near) {
#pragma unroll
    for (int e = 0; e < kTogether; ++e) {
      const auto [c, n] = factors(e);
      const double cd = (double)c.x + c.y, nd = (double)n.x + n.y;
      u(e) = beside_tie(cd * p[e] - nd * q[e]);
      v(e) = beside_tie(nd * p[e] + cd * q[e]);
    }
  }
}

// turn for a row that is quantised.
template <int kRope>
__device__ __forceinline__ void turn_q8(const float2* cs, const float2* sn, float (&x)[8], float (&y)[8]) {
#pragma unroll
  for (int e0 = 0; e0 < 8; e0 += kTogether) {
    turn_together(
        [&](int e) __attribute__((always_inline)) -> float& {
          const int k = e0 + e;
          return kRope == 2 ? x[k] : (k < 4 ? x[2 * k] : y[2 * k - 8]);
        },
        [&](int e) __attribute__((always_inline)) -> float& {
          const int k = e0 + e;
          return kRope == 2 ? y[k] : (k < 4 ? x[2 * k + 1] : y[2 * k - 7]);
        },
        [&](int e) __attribute__((always_inline)) { return Factors{cs[e0 + e], sn[e0 + e]}; });
  }
}

// One work-group per token, as above: the rows that are quantised first, then P1.
template <int D>
__global__ __launch_bounds__(kThreads) void paged_append_q8_kernel(PagedAppendArgs a, uint8_t* scale, AppendQ8Params qp, int first) {
  const PrestepParams& pp = qp.pre;
  constexpr int kGroups = D / 16;
  constexpr int kLanes = kGroups <= 2 ? 2 : (kGroups <= 4 ? 4 : 8);   // of a row
  __shared__ float s_cos[D / 2], s_sin[D / 2];
  __shared__ float2 s_cos2[D / 2], s_sin2[D / 2];         // P2's, split
  const int t = first + (int)blockIdx.x;
  const int slot = a.slot[t];
  if (slot < 0 || (slot >> a.page_shift) >= a.n_pages) return;   // uniform for the work-group
  const int tid = threadIdx.x;
  if (a.rope != 0 && tid < D / 2) {
    const double ang = (double)a.pos[t] * pp.inv_freq[tid];
    float sn, cs;
    sincos_of(ang, &sn, &cs);
    s_cos[tid] = cs;
    s_sin[tid] = sn;
    double sn2, cs2;
    sincos_f64(ang, &sn2, &cs2);
    s_cos2[tid] = split(cs2);
    s_sin2[tid] = split(sn2);
  }
  __syncthreads();
  const int page = slot >> a.page_shift, off = slot & ((1 << a.page_shift) - 1);
  // Quantises the row of head h that the lanes hold 16 elements of each, 8 of them at
  // column oa and 8 at ob (nothing where the lane has none).
  auto store_row = [&](int part, int h, int g, int oa, int ob, const float (&x)[8], const float (&y)[8]) {
    float most = g < kGroups ? finite_max(x, y) : 0.0f;
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) most = fmaxf(most, __shfl_xor(most, o, 64));
    if (g >= kGroups) return;
    const int k = scale_exponent(most);
    const float inv = __uint_as_float((unsigned)(127 - k) << 23);
    const size_t head = (size_t)page * a.H_kv + h;
    uint8_t* const row = static_cast<uint8_t*>(part ? a.cV : a.cP2) + ((head << a.page_shift) + off) * D;
    const uint2 p = quantise8(x, inv), q = quantise8(y, inv);
    if (ob == oa + 8) {
      *reinterpret_cast<uint4*>(row + oa) = make_uint4(p.x, p.y, q.x, q.y);
    } else {
      *reinterpret_cast<uint2*>(row + oa) = p;
      *reinterpret_cast<uint2*>(row + ob) = q;
    }
    if (g == 0) scale[(((head << 1) + part) << a.page_shift) + off] = (uint8_t)(k + 127);
  };
  const int keys = a.H_kv * kLanes;
  const int info = (a.mix ? a.H_kv / 2 : a.H_kv) * kLanes;
  const int all = keys + info + a.H * kGroups;
  for (int u = tid; u < all; u += kThreads) {
    float x[2][8], y[2][8];
    if (u < keys) {
      const int h = u / kLanes, g = u % kLanes;
      const int oa = a.rope == 2 ? 8 * g : 16 * g, ob = a.rope == 2 ? D / 2 + 8 * g : 16 * g + 8;
      if (g < kGroups) {
        const __bf16* src = static_cast<const __bf16*>(a.P2) + (size_t)t * a.ld2 + (size_t)h * D;
        load8(src + oa, x[0]);
        load8(src + ob, x[1]);
        if (a.rope == 1) turn_q8<1>(s_cos2 + 8 * g, s_sin2 + 8 * g, x[0], x[1]);
        else if (a.rope == 2) turn_q8<2>(s_cos2 + 8 * g, s_sin2 + 8 * g, x[0], x[1]);
      }
      store_row(0, h, g, oa, ob, x[0], x[1]);
    } else if (u < keys + info) {
      const int k = (u - keys) / kLanes, g = (u - keys) % kLanes;
      const __bf16* src = static_cast<const __bf16*>(a.I) + (size_t)t * a.ldi + 16 * g;
      if (a.mix) {
        const int ha = a.pairing == 0 ? 2 * k : 2 * k + 1, hb = (ha + 1) % a.H_kv;
        if (g < kGroups) {
          const Factors by{{pp.cos_theta[k], qp.cos_rest[k]}, {pp.sin_theta[k], qp.sin_rest[k]}};
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            load8(src + (size_t)ha * D + 8 * w, x[w]);
            load8(src + (size_t)hb * D + 8 * w, y[w]);
          }
#pragma unroll
          for (int e0 = 0; e0 < 16; e0 += kTogether) {
            turn_together([&](int e) __attribute__((always_inline)) -> float& { return x[(e0 + e) >> 3][(e0 + e) & 7]; },
                          [&](int e) __attribute__((always_inline)) -> float& { return y[(e0 + e) >> 3][(e0 + e) & 7]; },
                          [&](int) __attribute__((always_inline)) { return by; });
          }
        }
        store_row(1, ha, g, 16 * g, 16 * g + 8, x[0], x[1]);
        store_row(1, hb, g, 16 * g, 16 * g + 8, y[0], y[1]);
      } else {
        if (g < kGroups) {
          load8(src + (size_t)k * D, x[0]);
          load8(src + (size_t)k * D + 8, x[1]);
        }
        store_row(1, k, g, 16 * g, 16 * g + 8, x[0], x[1]);
      }
    } else {
      const int v = u - keys - info, h = v / kGroups, g = v % kGroups;
      const int oa = a.rope == 2 ? 8 * g : 16 * g, ob = a.rope == 2 ? D / 2 + 8 * g : 16 * g + 8;
      const __bf16* src = static_cast<const __bf16*>(a.P1) + (size_t)t * a.ld1 + (size_t)h * D;
      __bf16* dst = static_cast<__bf16*>(a.P1o) + ((size_t)t * a.H + h) * D;
      load8(src + oa, x[0]);
      load8(src + ob, x[1]);
      turn(a.rope, s_cos + 8 * g, s_sin + 8 * g, x[0], x[1]);
      store8(dst + oa, x[0]);
      store8(dst + ob, x[1]);
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

template <int D>
hipError_t launch_q8(const PagedAppendArgs& a, uint8_t* scale, const AppendQ8Params& qp, hipStream_t s) {
  constexpr int kMost = 1 << 23;
  for (int64_t first = 0; first < a.N; first += kMost) {
    const unsigned n = (unsigned)(a.N - first < kMost ? a.N - first : kMost);
    hipLaunchKernelGGL(paged_append_q8_kernel<D>, dim3(n), dim3(kThreads), 0, s, a, scale, qp, (int)first);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_paged_append_q8(const PagedAppendArgs& a, uint8_t* scale, const AppendQ8Params& qp, hipStream_t s) {
  switch (a.d_h) {
    case 32: return launch_q8<32>(a, scale, qp, s);
    case 48: return launch_q8<48>(a, scale, qp, s);
    case 64: return launch_q8<64>(a, scale, qp, s);
    case 80: return launch_q8<80>(a, scale, qp, s);
    case 128: return launch_q8<128>(a, scale, qp, s);
    default: return hipErrorInvalidValue;
  }
}

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
