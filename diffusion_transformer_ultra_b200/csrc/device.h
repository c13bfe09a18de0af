// The device a call runs on, and the driver's tensor map encoder (api.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <initializer_list>
#include <mutex>

namespace ug {

// Whether an output begins where one of the other operands does (null: not there).  Overlap that begins
// elsewhere is the caller's to avoid: strided tensors may lie between one another's rows.
inline bool begins_at(const void* out, std::initializer_list<const void*> others) {
  for (const void* p : others)
    if (out && out == p) return true;
  return false;
}

// What a kernel needs once on each device before its first launch there (a static of the code that
// launches it): `set` runs until it succeeds, and no two threads run it at once.
class OncePerDevice {
  static constexpr int kMost = 64;
  std::mutex mu_;
  bool done_[kMost] = {};

 public:
  template <typename F>
  cudaError_t operator()(F set) {
    int dev = -1;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMost) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu_);
    if (done_[dev]) return cudaSuccess;
    e = set();
    done_[dev] = e == cudaSuccess;
    return e;
  }
};

// The current device, or ULTRAGEN_ERR_NO_DEVICE when it is not an sm_100 one.
int current_device(int* dev);

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
// cuTensorMapEncodeTiled, or null when the driver has none.
EncodeTiledFn encode_fn();

}  // namespace ug
