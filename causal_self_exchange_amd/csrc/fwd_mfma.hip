// bf16 MFMA FlashRelation forward for gfx950: the kernels and launchers of the
// scan in fwd_body.h.
#include <atomic>

#include "fwd_body.h"

namespace rel {

namespace {

template <int D, int DR, bool kLse>
__global__ __launch_bounds__(kThreads, 1) void fwd_mfma_kernel(FwdArgs a, HeadParams hp) {
  const RopeParams none{};
  fwd_body<D, DR, kLse, false>(a, hp, none);
}

template <int D, int DR, bool kLse>
__global__ __launch_bounds__(kThreads, 1) void fwd_mfma_rope_kernel(FwdArgs a, HeadParams hp, RopeParams rp) {
  fwd_body<D, DR, kLse, true>(a, hp, rp);
}

template <int D, int DR>
hipError_t launch_typed(const FwdArgs& a, const HeadParams& hp, hipStream_t s, const RopeParams* rp) {
  const int nq = (a.T + kBM - 1) / kBM;
  const long long nwork = (long long)((nq + 1) / 2) * a.B * a.H;
  if (nwork > 0x7fffffffLL) return hipErrorInvalidValue;
  // One persistent work-group per compute unit (the LDS rings admit one).
  int n_cu = 0;
  const hipError_t e = device_cu_count(&n_cu);
  if (e != hipSuccess) return e;
  const long long grid = nwork < n_cu ? nwork : n_cu;
  if (rp != nullptr) {
    if (a.lse != nullptr) {
      hipLaunchKernelGGL((fwd_mfma_rope_kernel<D, DR, true>), dim3((unsigned)grid), dim3(kThreads), 0, s, a, hp, *rp);
    } else {
      hipLaunchKernelGGL((fwd_mfma_rope_kernel<D, DR, false>), dim3((unsigned)grid), dim3(kThreads), 0, s, a, hp, *rp);
    }
  } else if (a.lse != nullptr) {
    hipLaunchKernelGGL((fwd_mfma_kernel<D, DR, true>), dim3((unsigned)grid), dim3(kThreads), 0, s, a, hp);
  } else {
    hipLaunchKernelGGL((fwd_mfma_kernel<D, DR, false>), dim3((unsigned)grid), dim3(kThreads), 0, s, a, hp);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t device_cu_count(int* n_cu) {
  // Cached per device; concurrent first calls store the same value.
  static std::atomic<int> cus[64];
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  if (dev < 0 || dev >= 64) return hipErrorInvalidDevice;
  int n = cus[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    e = hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev);
    if (e != hipSuccess) return e;
    n = n > 0 ? n : 1;
    cus[dev].store(n, std::memory_order_relaxed);
  }
  *n_cu = n;
  return hipSuccess;
}

bool fwd_mfma_supported(int d_h, int T) {
  // Buffer descriptors address one head with 31-bit byte offsets, including
  // the rows past T of the last query tile.
  return (d_h == 32 || d_h == 48 || d_h == 64 || d_h == 80 || d_h == 128) && ((long long)T + kBM) * d_h * 2 < 0x7fffffffLL;
}

bool fwd_mfma_rope_fusable(int d_h, int rope) {
  return (d_h == 32 || d_h == 48 || d_h == 64 || d_h == 80 || d_h == 128) && (rope == 1 || (rope == 2 && d_h % 32 == 0));
}

hipError_t launch_fwd_mfma_bf16(const FwdArgs& a, const HeadParams& hp, hipStream_t s, const RopeParams* rp) {
  if (rp != nullptr && !fwd_mfma_rope_fusable(a.d_h, rp->rope)) return hipErrorInvalidValue;
  switch (a.d_h) {
    case 32: return launch_typed<64, 32>(a, hp, s, rp);
    case 48: return launch_typed<64, 48>(a, hp, s, rp);
    case 64: return launch_typed<64, 64>(a, hp, s, rp);
    case 80: return launch_typed<128, 80>(a, hp, s, rp);
    case 128: return launch_typed<128, 128>(a, hp, s, rp);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace rel
