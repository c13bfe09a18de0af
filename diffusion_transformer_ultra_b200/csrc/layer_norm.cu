// Layer norm over the last dimension, forward and backward, with one weight for every row or
// one per sample (the modulation of a diffusion transformer).
//
//   mu = sum(x) / C,  r = (sum((x - mu)^2) / C + eps)^-1/2,  xh = (x - mu) r
//   y  = xh w' + b,   w' = w, or 1 + w (plus_one), or 1 without a weight
//   g  = dy w',       dx = r (g - sum(g) / C - xh sum(g xh) / C)
//   dw = sum over rows of dy xh,   db = sum over rows of dy
//
// Both passes are bound by HBM: x is read and y written once (x, dy read and dx written once).
// A row lives in the registers of its block, kElems elements per thread, so that the variance
// takes a second pass over registers (no cancellation of sum(x^2) against mu^2) and nothing is
// read twice.  All sums are fp32.  A row of up to 512 elements belongs to one warp and a block
// holds several rows; a longer one to a block of just enough warps, so that few lanes idle at
// any width.
//
// The weight's gradient: a block of the backward pass walks a run of rows of one sample (of the
// whole batch with a shared weight), keeps its columns' sums in registers, and writes them once
// to the caller's workspace; a second kernel adds the runs in a fixed order.  No atomics: the
// same inputs give the same bits.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "device.h"
#include "elem.cuh"
#include "kernels.h"
#include "nvtx_range.h"
#include "ultragen.h"

namespace ug {
namespace {

constexpr int kElems = 16;                 // elements of a row per thread
constexpr int kMaxCols = 16384;            // 1,024 threads of kElems elements
constexpr int kWarpCols = 32 * kElems;     // rows up to this belong to one warp
constexpr int kWarpRows = 8;               // rows per block then

struct NormArgs {
  const void* x;
  const void* dy;
  const void* w;
  const void* b;
  void* y;                 // y, or dx
  float* mean;
  float* rstd;
  float* part;             // [runs][2][C] sums of the backward pass (null: not wanted)
  int64_t x_row, x_batch, y_row, y_batch, dy_row, dy_batch;
  int64_t total;           // rows of all samples
  int rows, C;             // rows per sample
  int64_t w_batch;         // C with a weight per sample, else 0
  int runs_per_group;      // runs of a sample (of everything with a shared weight)
  int64_t group_rows;      // rows of a sample (of everything with a shared weight)
  float plus, inv_c, eps;
};

// Sum of x over the threads of a row: one warp, or the whole block (two barriers; `red` holds a
// float per warp and may be reused at once by the next call because of the second).
template <bool WARP>
__device__ __forceinline__ float row_sum(float x, float* red) {
  x = warp_sum(x);
  if (WARP) return x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  if (lane == 0) red[warp] = x;
  __syncthreads();
  x = warp_sum(lane < nw ? red[lane] : 0.f);
  __syncthreads();
  return x;
}

// Two sums with one pair of barriers.
template <bool WARP>
__device__ __forceinline__ float2 row_sum2(float a, float b, float2* red) {
  a = warp_sum(a);
  b = warp_sum(b);
  if (WARP) return make_float2(a, b);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  if (lane == 0) red[warp] = make_float2(a, b);
  __syncthreads();
  const float2 v = lane < nw ? red[lane] : make_float2(0.f, 0.f);
  a = warp_sum(v.x);
  b = warp_sum(v.y);
  __syncthreads();
  return make_float2(a, b);
}

template <typename T, typename W, int VEC, bool WARP, int MAXT>
__global__ void __launch_bounds__(MAXT) norm_fwd_kernel(const NormArgs p) {
  constexpr int NV = kElems / VEC;
  __shared__ float red[32];
  const int tpr = WARP ? 32 : blockDim.x;                       // threads of a row
  const int t = WARP ? (threadIdx.x & 31) : threadIdx.x;
  const int64_t row = WARP ? (int64_t)blockIdx.x * kWarpRows + (threadIdx.x >> 5) : (int64_t)blockIdx.x;
  if (WARP && row >= p.total) return;
  const int64_t s = row / p.rows, i = row - s * p.rows;
  const T* x = static_cast<const T*>(p.x) + s * p.x_batch + i * p.x_row;
  float v[NV][VEC];
  float sum = 0.f;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = (t + k * tpr) * VEC;
    if (c < p.C) {
      load_f32<T, VEC>(x + c, v[k]);
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[k][e] = 0.f;
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) sum += v[k][e];
  }
  const float mean = row_sum<WARP>(sum, red) * p.inv_c;
  float sq = 0.f;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = (t + k * tpr) * VEC;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      v[k][e] -= mean;
      if (c < p.C) sq += v[k][e] * v[k][e];
    }
  }
  const float rstd = 1.0f / sqrtf(row_sum<WARP>(sq, red) * p.inv_c + p.eps);
  T* y = static_cast<T*>(p.y) + s * p.y_batch + i * p.y_row;
  const W* w = p.w ? static_cast<const W*>(p.w) + s * p.w_batch : nullptr;
  const W* b = p.b ? static_cast<const W*>(p.b) + s * p.w_batch : nullptr;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = (t + k * tpr) * VEC;
    if (c >= p.C) continue;
    float wv[VEC], bv[VEC];
    if (w) load_f32<W, VEC>(w + c, wv);
    if (b) load_f32<W, VEC>(b + c, bv);
#pragma unroll
    for (int e = 0; e < VEC; ++e)
      v[k][e] = v[k][e] * rstd * (w ? wv[e] + p.plus : 1.0f) + (b ? bv[e] : 0.0f);
    store_f32<T, VEC>(y + c, v[k]);
  }
  if (t == 0) {
    if (p.mean) p.mean[row] = mean;
    if (p.rstd) p.rstd[row] = rstd;
  }
}

// One block walks the rows [r0, r1) of run blockIdx.x; with WARP its warps take them in turn.
template <typename T, typename W, int VEC, bool WARP, int MAXT>
__global__ void __launch_bounds__(MAXT) norm_bwd_kernel(const NormArgs p) {
  constexpr int NV = kElems / VEC;
  __shared__ float2 red[32];
  const int tpr = WARP ? 32 : blockDim.x;
  const int t = WARP ? (threadIdx.x & 31) : threadIdx.x;
  const int warp = WARP ? threadIdx.x >> 5 : 0, step = WARP ? kWarpRows : 1;
  const int64_t group = blockIdx.x / p.runs_per_group;
  const int64_t run = blockIdx.x - group * p.runs_per_group;
  const int64_t r0 = group * p.group_rows + p.group_rows * run / p.runs_per_group;
  const int64_t r1 = group * p.group_rows + p.group_rows * (run + 1) / p.runs_per_group;
  float dw[NV][VEC], db[NV][VEC];
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int e = 0; e < VEC; ++e) dw[k][e] = db[k][e] = 0.f;
  for (int64_t row = r0 + warp; row < r1; row += step) {
    const int64_t s = row / p.rows, i = row - s * p.rows;
    const T* x = static_cast<const T*>(p.x) + s * p.x_batch + i * p.x_row;
    const T* dy = static_cast<const T*>(p.dy) + s * p.dy_batch + i * p.dy_row;
    const W* w = p.w ? static_cast<const W*>(p.w) + s * p.w_batch : nullptr;
    const float mean = p.mean[row], rstd = p.rstd[row];
    float xh[NV][VEC], g[NV][VEC];
    float a = 0.f, b = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = (t + k * tpr) * VEC;
      if (c < p.C) {
        load_f32<T, VEC>(x + c, xh[k]);
        load_f32<T, VEC>(dy + c, g[k]);
        float wv[VEC];
        if (w) load_f32<W, VEC>(w + c, wv);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          xh[k][e] = (xh[k][e] - mean) * rstd;
          dw[k][e] += g[k][e] * xh[k][e];
          db[k][e] += g[k][e];
          if (w) g[k][e] *= wv[e] + p.plus;
          a += g[k][e];
          b += g[k][e] * xh[k][e];
        }
      }
    }
    const float2 ab = row_sum2<WARP>(a, b, red);
    T* dx = static_cast<T*>(p.y) + s * p.y_batch + i * p.y_row;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = (t + k * tpr) * VEC;
      if (c >= p.C) continue;
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        g[k][e] = rstd * (g[k][e] - ab.x * p.inv_c - xh[k][e] * (ab.y * p.inv_c));
      store_f32<T, VEC>(dx + c, g[k]);
    }
  }
  if (!p.part) return;
  float* out = p.part + (int64_t)blockIdx.x * 2 * p.C;
  if constexpr (WARP) {
    // the block's warps hold sums of the same columns: add them in warp order
    __shared__ float acc[2][kWarpCols];
    for (int q = 0; q < kWarpRows; ++q) {
      if (warp == q) {
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            const int c = (t + k * 32) * VEC + e;
            acc[0][c] = dw[k][e] + (q ? acc[0][c] : 0.f);
            acc[1][c] = db[k][e] + (q ? acc[1][c] : 0.f);
          }
      }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < p.C; c += blockDim.x) {
      out[c] = acc[0][c];
      out[p.C + c] = acc[1][c];
    }
  } else {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = (t + k * tpr) * VEC;
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        if (c + e < p.C) {
          out[c + e] = dw[k][e];
          out[p.C + c + e] = db[k][e];
        }
    }
  }
}

// Adds the runs of a group: block (32 columns, 8 lanes of runs), grid (columns / 32, groups, 2).
template <typename O>
__global__ void __launch_bounds__(256) norm_reduce_kernel(const float* part, int C, int runs, O* dw, O* db) {
  O* out = blockIdx.z ? db : dw;
  if (!out) return;
  __shared__ float acc[8][33];
  const int c = blockIdx.x * 32 + threadIdx.x;
  const int64_t g = blockIdx.y;
  float s = 0.f;
  if (c < C)
    for (int r = threadIdx.y; r < runs; r += 8) s += part[((g * runs + r) * 2 + blockIdx.z) * C + c];
  acc[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y == 0 && c < C) {
#pragma unroll
    for (int q = 1; q < 8; ++q) s += acc[q][threadIdx.x];
    out[g * C + c] = from_f32<O>(s);
  }
}

// Threads of a row's block: one warp up to kWarpCols columns, else just enough warps.
int row_threads(int C) { return std::max(32, (C + kWarpCols - 1) / kWarpCols * 32); }

// Runs of a group in the backward pass: about 512 threads per multiprocessor (its accumulators
// take about 128 registers), no more runs than rows.
int runs_of(int64_t group_rows, int64_t groups, int C, int sms) {
  const int block = C <= kWarpCols ? 32 * kWarpRows : row_threads(C);
  const int64_t want = std::max<int64_t>(1, (int64_t)sms * std::max(1, 512 / block) / groups);
  const int64_t most = C <= kWarpCols ? (group_rows + kWarpRows - 1) / kWarpRows : group_rows;
  return (int)std::max<int64_t>(1, std::min(want, most));
}

template <typename T, typename W, int VEC>
cudaError_t launch_vec(bool bwd, const NormArgs& a, int blocks, cudaStream_t st) {
  const int tpr = row_threads(a.C);
  if (a.C <= kWarpCols) {
    if (bwd) norm_bwd_kernel<T, W, VEC, true, 256><<<blocks, 32 * kWarpRows, 0, st>>>(a);
    else norm_fwd_kernel<T, W, VEC, true, 256><<<blocks, 32 * kWarpRows, 0, st>>>(a);
  } else if (tpr <= 512) {
    if (bwd) norm_bwd_kernel<T, W, VEC, false, 512><<<blocks, tpr, 0, st>>>(a);
    else norm_fwd_kernel<T, W, VEC, false, 512><<<blocks, tpr, 0, st>>>(a);
  } else {
    if (bwd) norm_bwd_kernel<T, W, VEC, false, 1024><<<blocks, tpr, 0, st>>>(a);
    else norm_fwd_kernel<T, W, VEC, false, 1024><<<blocks, tpr, 0, st>>>(a);
  }
  return cudaGetLastError();
}

template <typename T, typename W>
cudaError_t launch_norm(bool bwd, bool vec, const NormArgs& a, int blocks, cudaStream_t st) {
  return vec ? launch_vec<T, W, (int)(16 / sizeof(T))>(bwd, a, blocks, st)
             : launch_vec<T, W, 1>(bwd, a, blocks, st);
}

cudaError_t dispatch(bool bwd, int dtype, int wdtype, bool vec, const NormArgs& a, int blocks, cudaStream_t st) {
  const bool wf = wdtype == ULTRAGEN_F32;
  if (dtype == ULTRAGEN_BF16)
    return wf ? launch_norm<__nv_bfloat16, float>(bwd, vec, a, blocks, st)
              : launch_norm<__nv_bfloat16, __nv_bfloat16>(bwd, vec, a, blocks, st);
  if (dtype == ULTRAGEN_F16)
    return wf ? launch_norm<__half, float>(bwd, vec, a, blocks, st)
              : launch_norm<__half, __half>(bwd, vec, a, blocks, st);
  return launch_norm<float, float>(bwd, vec, a, blocks, st);
}

int elem_size(int dtype) { return dtype == ULTRAGEN_F32 ? 4 : 2; }
bool known(int dtype) { return dtype == ULTRAGEN_BF16 || dtype == ULTRAGEN_F16 || dtype == ULTRAGEN_F32; }

int check(const ultragen_norm_t* n) {
  if (!n || n->batch < 0 || n->rows < 0 || n->cols < 1) return ULTRAGEN_ERR_INVALID_ARG;
  if (!known(n->dtype) || (n->wdtype != n->dtype && n->wdtype != ULTRAGEN_F32)) return ULTRAGEN_ERR_INVALID_ARG;
  if (!(n->eps >= 0.f) || !std::isfinite(n->eps)) return ULTRAGEN_ERR_INVALID_ARG;
  if (n->cols > kMaxCols || (int64_t)n->batch * n->rows > 0x7fffffffLL) return ULTRAGEN_ERR_UNSUPPORTED;
  if (n->per_sample && n->batch > 65535) return ULTRAGEN_ERR_UNSUPPORTED;
  return ULTRAGEN_OK;
}

// Whether a row operand can be read 16 bytes at a time.
bool rows16(const void* p, int64_t row, int64_t batch, int vec, int dtype) {
  return p == nullptr || (((uintptr_t)p & 15u) == 0 && row * elem_size(dtype) % 16 == 0 &&
                          batch * elem_size(dtype) % 16 == 0 && vec > 1);
}

NormArgs args_of(const ultragen_norm_t* n) {
  NormArgs a = {};
  a.total = (int64_t)n->batch * n->rows;
  a.rows = n->rows;
  a.C = n->cols;
  a.w_batch = n->per_sample ? n->cols : 0;
  a.plus = n->plus_one ? 1.0f : 0.0f;
  a.inv_c = 1.0f / (float)n->cols;
  a.eps = n->eps;
  a.x_row = n->x_row;
  a.x_batch = n->x_batch;
  a.y_row = n->y_row;
  a.y_batch = n->y_batch;
  a.dy_row = n->dy_row;
  a.dy_batch = n->dy_batch;
  a.group_rows = n->per_sample ? n->rows : a.total;
  return a;
}

// 16-byte vectors need every row, and every sample's weight, to start on a 16-byte boundary (a
// weight wider than the rows then does too, its vectors being a multiple of theirs).
bool vectorised(const ultragen_norm_t* n, const void* x, const void* dy, const void* y, const void* w,
                const void* b) {
  const int vec = 16 / elem_size(n->dtype);
  const int64_t wb = n->per_sample ? n->cols : 0;
  return n->cols % vec == 0 && rows16(x, n->x_row, n->x_batch, vec, n->dtype) &&
         rows16(dy, n->dy_row, n->dy_batch, vec, n->dtype) && rows16(y, n->y_row, n->y_batch, vec, n->dtype) &&
         rows16(w, wb, wb, vec, n->wdtype) && rows16(b, wb, wb, vec, n->wdtype);
}

int status_of(cudaError_t e) { return e == cudaSuccess ? ULTRAGEN_OK : ULTRAGEN_ERR_CUDA; }

}  // namespace
}  // namespace ug

using namespace ug;

extern "C" {

int ultragen_layer_norm(const ultragen_norm_t* n, const void* x, const void* weight, const void* bias, void* y,
                        float* mean, float* rstd, ultragen_stream_t stream) {
  ug::NvtxRange nvtx_range("ultragen_layer_norm");
  int st = check(n);
  if (st != ULTRAGEN_OK) return st;
  if (n->batch == 0 || n->rows == 0) return ULTRAGEN_OK;
  if (!x || !y) return ULTRAGEN_ERR_INVALID_ARG;
  int dev;
  if ((st = current_device(&dev)) != ULTRAGEN_OK) return st;
  NormArgs a = args_of(n);
  a.x = x;
  a.w = weight;
  a.b = bias;
  a.y = y;
  a.mean = mean;
  a.rstd = rstd;
  const int blocks = (int)(n->cols <= kWarpCols ? (a.total + kWarpRows - 1) / kWarpRows : a.total);
  return status_of(dispatch(false, n->dtype, n->wdtype, vectorised(n, x, nullptr, y, weight, bias), a, blocks,
                            reinterpret_cast<cudaStream_t>(stream)));
}

int ultragen_layer_norm_backward_workspace(const ultragen_norm_t* n, size_t* bytes) {
  int st = check(n);
  if (st != ULTRAGEN_OK) return st;
  if (!bytes) return ULTRAGEN_ERR_INVALID_ARG;
  const NormArgs a = args_of(n);
  const int64_t groups = n->per_sample ? n->batch : 1;
  *bytes = a.total == 0 ? 0 : (size_t)groups * runs_of(a.group_rows, groups, n->cols, sm_count()) * 2 * n->cols * sizeof(float);
  return ULTRAGEN_OK;
}

int ultragen_layer_norm_backward(const ultragen_norm_t* n, const void* dy, const void* x, const void* weight,
                                 const float* mean, const float* rstd, void* dx, void* dweight, void* dbias,
                                 int grad_dtype, void* workspace, size_t workspace_bytes,
                                 ultragen_stream_t stream) {
  ug::NvtxRange nvtx_range("ultragen_layer_norm_backward");
  int st = check(n);
  if (st != ULTRAGEN_OK) return st;
  if (!known(grad_dtype)) return ULTRAGEN_ERR_INVALID_ARG;
  NormArgs a = args_of(n);
  const int64_t groups = n->per_sample ? n->batch : 1;
  int dev;
  if (a.total == 0) {                         // no rows: the sums over them are zero
    if ((st = current_device(&dev)) != ULTRAGEN_OK) return st;
    for (void* g : {dweight, dbias})
      if (g && cudaMemsetAsync(g, 0, (size_t)groups * n->cols * elem_size(grad_dtype),
                               reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
        return ULTRAGEN_ERR_CUDA;
    return ULTRAGEN_OK;
  }
  if (!dy || !x || !mean || !rstd || !dx) return ULTRAGEN_ERR_INVALID_ARG;
  if ((st = current_device(&dev)) != ULTRAGEN_OK) return st;
  a.runs_per_group = runs_of(a.group_rows, groups, n->cols, sm_count());
  if (dweight || dbias) {
    const size_t need = (size_t)groups * a.runs_per_group * 2 * n->cols * sizeof(float);
    if (!workspace || workspace_bytes < need || ((uintptr_t)workspace & 15u)) return ULTRAGEN_ERR_INVALID_ARG;
    a.part = static_cast<float*>(workspace);
  }
  a.x = x;
  a.dy = dy;
  a.w = weight;
  a.y = dx;
  a.mean = const_cast<float*>(mean);
  a.rstd = const_cast<float*>(rstd);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  st = status_of(dispatch(true, n->dtype, n->wdtype, vectorised(n, x, dy, dx, weight, nullptr), a,
                          (int)(groups * a.runs_per_group), s));
  if (st != ULTRAGEN_OK || !a.part) return st;
  const dim3 grid((n->cols + 31) / 32, (unsigned)groups, 2), block(32, 8);
  if (grad_dtype == ULTRAGEN_F32)
    norm_reduce_kernel<float><<<grid, block, 0, s>>>(a.part, n->cols, a.runs_per_group, (float*)dweight, (float*)dbias);
  else if (grad_dtype == ULTRAGEN_BF16)
    norm_reduce_kernel<__nv_bfloat16><<<grid, block, 0, s>>>(a.part, n->cols, a.runs_per_group,
                                                             (__nv_bfloat16*)dweight, (__nv_bfloat16*)dbias);
  else
    norm_reduce_kernel<__half><<<grid, block, 0, s>>>(a.part, n->cols, a.runs_per_group, (__half*)dweight, (__half*)dbias);
  return status_of(cudaGetLastError());
}

}  // extern "C"
