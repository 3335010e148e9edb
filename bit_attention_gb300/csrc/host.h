// host.h -- host-side argument checks shared by the C entry points of the
// rotation and of the paged cache.  Internal to the library.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/sage_fp4.h"
#include "kernels.h"

namespace sagefp4 {

inline bool is_aligned(const void* p, uintptr_t a) { return p && (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// The current device is an sm_103 one (the kernels are compiled for sm_103a
// only); its number of SMs in *sms.
inline int check_device_103(int* sms) {
  // 0 unknown, -1 not supported, else the number of SMs: one word, so that a
  // thread sees all of what another found out, or nothing
  static std::atomic<int> cache[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return SAGE_FP4_ECUDA;
  if (dev < 0 || dev >= 64) return SAGE_FP4_EUNSUPPORTED;
  int n = cache[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    int major = 0, minor = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return SAGE_FP4_ECUDA;
    if (major != 10 || minor != 3) n = -1;
    cache[dev].store(n, std::memory_order_relaxed);
  }
  if (n < 0) return SAGE_FP4_EUNSUPPORTED;
  *sms = n;
  return SAGE_FP4_OK;
}

// A stride triple for the kernels: >= 0, multiples of 8 elements (16-byte
// rows), the largest offset within 2^62 elements.
inline bool take_strides(const sage_fp4_strides& in, int64_t B, int64_t H, int64_t N, int64_t D, Strides* out) {
  const int64_t st[3] = {in.b, in.h, in.n}, dims[3] = {B, H, N};
  int64_t last = D;
  for (int i = 0; i < 3; ++i) {
    if (st[i] < 0 || st[i] % 8 != 0) return false;
    int64_t span = 0;
    if (dims[i] > 0 &&
        (__builtin_mul_overflow(st[i], dims[i] - 1, &span) || __builtin_add_overflow(last, span, &last)))
      return false;
  }
  if (last > (int64_t(1) << 62)) return false;
  *out = Strides{st[0], st[1], st[2]};
  return true;
}

// Read and reset a status word after the stream's work, on that stream alone:
// the default stream may be busy with something else, and a reset there could
// come after a later call's error.
inline int read_status(int32_t* status, void* stream) {
  if (!is_aligned(status, 4)) return SAGE_FP4_EINVAL;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int32_t h = 0;
  if (cudaMemcpyAsync(&h, status, sizeof(h), cudaMemcpyDeviceToHost, st) != cudaSuccess ||
      cudaStreamSynchronize(st) != cudaSuccess)
    return SAGE_FP4_ECUDA;
  if (h != 0 && (cudaMemsetAsync(status, 0, sizeof(h), st) != cudaSuccess || cudaStreamSynchronize(st) != cudaSuccess))
    return SAGE_FP4_ECUDA;
  return h;
}

inline int launched(cudaError_t e) { return e == cudaSuccess ? SAGE_FP4_OK : SAGE_FP4_ECUDA; }

}  // namespace sagefp4
