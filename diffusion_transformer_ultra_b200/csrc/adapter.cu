// Projection shared by all rows, with the low-rank adapter of each row beside it:
//   y_m = W x_m + bias + s_a B_a (A_a x_m),   a = ids[m] (no adapter outside [0, adapters))
// Two kernels: t_m = s_a A_a x_m (fp32, [rows, rank]), then the projection with the adapters'
// second factor in its epilogue.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "device.h"
#include "elem.cuh"
#include "kernels.h"
#include "nvtx_range.h"
#include "ultragen.h"

namespace ug {
namespace {

struct AdapterArgs {
  const void* x;
  const void* w;
  const void* a;
  const void* b;
  const void* bias;
  const float* scales;
  const int32_t* ids;
  void* y;
  float* t;
  int64_t x_row, y_row;
  int M, N, K, R, adapters;
};

template <typename T>
__global__ void __launch_bounds__(128) adapter_shrink_kernel(const AdapterArgs p) {
  const int m = blockIdx.x, id = p.ids[m], lane = threadIdx.x & 31;
  const bool on = id >= 0 && id < p.adapters;
  const T* x = static_cast<const T*>(p.x) + m * p.x_row;
  const float scale = !on ? 0.f : p.scales ? p.scales[id] : 1.f;
  for (int r = threadIdx.x >> 5; r < p.R; r += 4) {
    float s = 0.f;
    if (on) {
      const T* a = static_cast<const T*>(p.a) + ((int64_t)id * p.R + r) * p.K;
      for (int k = lane; k < p.K; k += 32) s += to_f32(x[k]) * to_f32(a[k]);
    }
    s = warp_sum(s) * scale;
    if (lane == 0) p.t[(int64_t)m * p.R + r] = on ? s : 0.f;
  }
}

template <typename T>
__global__ void __launch_bounds__(256) adapter_general_kernel(const AdapterArgs p) {
  constexpr int TM = 64, TN = 64, TK = 16;
  __shared__ float xs[TK][TM + 4], ws[TK][TN + 4];
  const int m0 = blockIdx.x * TM, n0 = blockIdx.y * TN;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const T* x = static_cast<const T*>(p.x);
  const T* w = static_cast<const T*>(p.w);
  float acc[4][4] = {};
  for (int k0 = 0; k0 < p.K; k0 += TK) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int k = threadIdx.x & 15, r = (threadIdx.x >> 4) + i * 16;
      const bool kin = k0 + k < p.K;
      xs[k][r] = kin && m0 + r < p.M ? to_f32(x[(int64_t)(m0 + r) * p.x_row + k0 + k]) : 0.f;
      ws[k][r] = kin && n0 + r < p.N ? to_f32(w[(int64_t)(n0 + r) * p.K + k0 + k]) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < TK; ++k) {
      float xv[4], wv[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        xv[i] = xs[k][ty + 16 * i];
        wv[i] = ws[k][tx + 16 * i];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] += xv[i] * wv[j];
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int m = m0 + ty + 16 * i;
    if (m >= p.M) continue;
    const int id = p.ids[m];
    const bool on = id >= 0 && id < p.adapters;
    const float* t = p.t + (int64_t)m * p.R;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = n0 + tx + 16 * j;
      if (n >= p.N) continue;
      float v = acc[i][j];
      if (on) {
        const T* b = static_cast<const T*>(p.b) + ((int64_t)id * p.N + n) * p.R;
        for (int r = 0; r < p.R; ++r) v += t[r] * to_f32(b[r]);
      }
      if (p.bias) v += to_f32(static_cast<const T*>(p.bias)[n]);
      static_cast<T*>(p.y)[(int64_t)m * p.y_row + n] = from_f32<T>(v);
    }
  }
}

int check(const ultragen_adapter_t* c) {
  if (!c || c->rows < 0 || c->k < 1 || c->n < 1 || c->rank < 1 || c->adapters < 1) return ULTRAGEN_ERR_INVALID_ARG;
  if (c->dtype != ULTRAGEN_BF16 && c->dtype != ULTRAGEN_F16 && c->dtype != ULTRAGEN_F32) return ULTRAGEN_ERR_INVALID_ARG;
  if (c->rank > 128 || c->n > 65535 * 64) return ULTRAGEN_ERR_UNSUPPORTED;
  return ULTRAGEN_OK;
}

template <typename T>
cudaError_t launch(const AdapterArgs& a, cudaStream_t s) {
  adapter_shrink_kernel<T><<<a.M, 128, 0, s>>>(a);
  adapter_general_kernel<T><<<dim3((a.M + 63) / 64, (a.N + 63) / 64), 256, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace
}  // namespace ug

using namespace ug;

extern "C" {

int ultragen_adapter_project_workspace(const ultragen_adapter_t* c, size_t* bytes) {
  int st = check(c);
  if (st != ULTRAGEN_OK) return st;
  if (!bytes) return ULTRAGEN_ERR_INVALID_ARG;
  *bytes = (size_t)c->rows * c->rank * sizeof(float);
  return ULTRAGEN_OK;
}

int ultragen_adapter_project(const ultragen_adapter_t* c, const void* x, const void* w, const void* bias,
                             const void* a, const void* b, const float* scales, const int32_t* ids, void* y,
                             void* workspace, size_t workspace_bytes, ultragen_stream_t stream) {
  ug::NvtxRange nvtx_range("ultragen_adapter_project");
  int st = check(c);
  if (st != ULTRAGEN_OK) return st;
  if (c->rows == 0) return ULTRAGEN_OK;
  size_t need = 0;
  ultragen_adapter_project_workspace(c, &need);
  if (!x || !w || !a || !b || !ids || !y || !workspace || workspace_bytes < need) return ULTRAGEN_ERR_INVALID_ARG;
  int dev;
  if ((st = current_device(&dev)) != ULTRAGEN_OK) return st;
  AdapterArgs p = {x, w, a, b, bias, scales, ids, y, static_cast<float*>(workspace), c->x_row, c->y_row,
                   c->rows, c->n, c->k, c->rank, c->adapters};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = c->dtype == ULTRAGEN_BF16  ? launch<__nv_bfloat16>(p, s)
                  : c->dtype == ULTRAGEN_F16 ? launch<__half>(p, s)
                                             : launch<float>(p, s);
  return e == cudaSuccess ? ULTRAGEN_OK : ULTRAGEN_ERR_CUDA;
}

}  // extern "C"
