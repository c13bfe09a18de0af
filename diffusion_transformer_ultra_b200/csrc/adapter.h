// Projection with adapters: what its entry points and small kernels (adapter.cu) and its matrix
// product (adapter_gemm.cu) share.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace ug {

constexpr int kTileRows = 256;         // rows of a tile of the product (two CTAs of 128)

struct AdapterArgs {
  const void* x;
  const void* w;
  const void* a;
  const void* b;
  const void* bias;
  const float* scales;
  const int32_t* ids;
  void* y;
  int64_t x_row, y_row;
  int M, N, K, R, adapters;
  int Rp;                              // R rounded up to 16
  void* t;                             // [M][2 Rp]: s A x as two 16-bit numbers, high parts then low
                                       // (fp32 [M][R] for the general kernel)
  int32_t* lists;                      // per tile: count, then the adapters its rows use
  int b16;                             // rows of b can be read 16 bytes at a time
  int y16;                             // rows of y can be written 16 bytes at a time
  unsigned long long timeout_ns;
};
constexpr int kListInts = 1 + kTileRows;

// y of `a` on the tensor cores, after the kernel that makes t and the lists (adapter.cu); launched
// so that it may begin before that kernel ends.
cudaError_t launch_adapter_gemm(const AdapterArgs& a, int dtype, cudaStream_t s);
cudaError_t adapter_status(int* code, cudaStream_t s);

}  // namespace ug
