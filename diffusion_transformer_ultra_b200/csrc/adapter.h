// Projection with adapters: what its entry points and small kernels (adapter.cu) and its matrix
// product (adapter_gemm.cu) share.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

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
  void* t;                             // [M][2 Rp]: s A x as two 16-bit numbers, high parts then low (see kLowScale)
                                       // (fp32 [M][R] for the general kernel)
  int32_t* lists;                      // per tile: count, then the adapters its rows use
  int b16;                             // rows of b can be read 16 bytes at a time
  int y16;                             // rows of y can be written 16 bytes at a time
  unsigned long long timeout_ns;
};
constexpr int kListInts = 1 + kTileRows;

// What the low parts of t are multiplied by.  t = high + low / kLowScale: in fp16 a low part as it is would
// end at the type's smallest step, 2^-24, and t below 2^-9 would keep less than 16 bits, none below 2^-25;
// times 2^11 it has high's size, and the products take it against 2^-11 B.  The term t B is then off by
// 2^-22 |t B| + 2^-36 |B| + min(2^-26 |t|, 2^-12 |t B|), the last because 2^-11 B may be below the smallest
// step in its turn.  bf16 has fp32's exponents: 2^-16 |t B|.
template <typename T>
constexpr float kLowScale = std::is_same<T, __half>::value ? 2048.0f : 1.0f;

// y of `a` on the tensor cores, after the kernel that makes t and the lists (adapter.cu); launched
// so that it may begin before that kernel ends.
cudaError_t launch_adapter_gemm(const AdapterArgs& a, int dtype, cudaStream_t s);
cudaError_t adapter_status(int* code, cudaStream_t s);

}  // namespace ug
