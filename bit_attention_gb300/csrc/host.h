// host.h -- host-side argument checks shared by the C entry points of the
// rotation and of the paged cache.  Internal to the library.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/sage_fp4.h"
#include "kernels.h"

namespace sagefp4 {

inline bool is_aligned(const void* p, uintptr_t a) { return p && (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// The current device is an sm_103 one (the kernels are compiled for sm_103a
// only); its number of SMs in *sms.
inline int check_device_103(int* sms) {
  struct Seen {
    int state, sms;  // state: 0 unknown, 1 supported, 2 not
  };
  static Seen cache[64];  // racing threads write the same values
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return SAGE_FP4_ECUDA;
  if (dev < 0 || dev >= 64) return SAGE_FP4_EUNSUPPORTED;
  if (!cache[dev].state) {
    int major = 0, minor = 0, n = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return SAGE_FP4_ECUDA;
    cache[dev].sms = n;
    cache[dev].state = (major == 10 && minor == 3) ? 1 : 2;
  }
  *sms = cache[dev].sms;
  return cache[dev].state == 1 ? SAGE_FP4_OK : SAGE_FP4_EUNSUPPORTED;
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
