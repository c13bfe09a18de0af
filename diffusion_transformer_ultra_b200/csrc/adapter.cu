// Projection shared by all rows, with the low-rank adapter of each row beside it:
//   y_m = W x_m + bias + s_a B_a (A_a x_m),   a = ids[m] (no adapter outside [0, adapters))
// Two kernels: t_m = s_a A_a x_m, then the projection with the adapters' second factor in it:
//   16-bit types, 16-byte aligned rows   few rows: adapter_few_kernel (bound by W's bytes)
//                                        else the tensor-core product of adapter_gemm.cu
//   fp32, or rows that 16-byte accesses cannot read   adapter_general_kernel
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "adapter.h"
#include "cross.cuh"
#include "device.h"
#include "elem.cuh"
#include "kernels.h"
#include "nvtx_range.h"
#include "ptx.cuh"
#include "ultragen.h"

namespace ug {
namespace {

template <typename T>
__global__ void __launch_bounds__(128) adapter_general_shrink_kernel(const AdapterArgs p) {
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
    if (lane == 0) static_cast<float*>(p.t)[(int64_t)m * p.R + r] = on ? s : 0.f;
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
    const float* t = static_cast<const float*>(p.t) + (int64_t)m * p.R;
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

// ------------------------------------------------------------------ 16-bit types
// D += A B of 16 x 8 x 16 (fp32 sums); lane (g, t) = (lane / 4, lane % 4) holds rows g, g + 8 of A
// and column g of B.
template <typename T>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  if constexpr (std::is_same<T, __half>::value)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Products of two 16-byte pieces of A's rows g, g + 8 and one of B's column g, each holding 8
// consecutive k of lane t: a sum over k may take them in any order, so the pieces are used as they
// were loaded, two k-halves at a time.
template <typename T>
__device__ __forceinline__ void mma_pieces(float (&c)[4], const uint4& a, const uint4& a8, const uint4& b) {
  mma16816<T>(c, a.x, a8.x, a.y, a8.y, b.x, b.y);
  mma16816<T>(c, a.z, a8.z, a.w, a8.w, b.z, b.w);
}

__device__ __forceinline__ uint4 piece(const void* row, int64_t k, bool on) {
  return on ? __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(row) + k)) : make_uint4(0, 0, 0, 0);
}

constexpr int kShrinkRows = 32;        // rows of a block of the shrink kernel

// t = s A x of 32 rows: their distinct adapters' rows of A, 8 to a tile, NT tiles a pass over K.  The block's 8 warps take every eighth 32-element piece of K, so that few rows still bring
// enough loads into flight; their sums meet in shared memory, in warp order.  Bound by x's bytes.
template <typename T, int NT>
__device__ __forceinline__ void shrink_pass(const AdapterArgs& p, const int* ids, int tile0, int ntiles, float* red) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int m0 = blockIdx.x * kShrinkRows, per = (p.R + 7) >> 3;
  const T* x[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int m = m0 + g + 8 * i;
    x[i] = m < p.M ? static_cast<const T*>(p.x) + m * p.x_row : nullptr;
  }
  const T* a[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int q = tile0 + i, r = q % per * 8 + g;
    a[i] = i < ntiles && r < p.R ? static_cast<const T*>(p.a) + ((int64_t)ids[q / per] * p.R + r) * p.K : nullptr;
  }
  float c[2][NT][4] = {};
#pragma unroll(NT <= 2 ? 4 : 2)
  for (int k0 = warp * 32; k0 < p.K; k0 += 256) {
    const int k = k0 + t * 8;
    uint4 xv[4], av[NT];
#pragma unroll
    for (int i = 0; i < 4; ++i) xv[i] = piece(x[i], k, x[i] && k < p.K);
#pragma unroll
    for (int i = 0; i < NT; ++i) av[i] = piece(a[i], k, a[i] && k < p.K);
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      mma_pieces<T>(c[0][i], xv[0], xv[1], av[i]);
      mma_pieces<T>(c[1][i], xv[2], xv[3], av[i]);
    }
  }
  // red[warp][row][NT * 8]
  float* mine = red + warp * (kShrinkRows * NT * 8);
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      *reinterpret_cast<float2*>(mine + (h * 16 + g) * (NT * 8) + i * 8 + 2 * t) = make_float2(c[h][i][0], c[h][i][1]);
      *reinterpret_cast<float2*>(mine + (h * 16 + g + 8) * (NT * 8) + i * 8 + 2 * t) = make_float2(c[h][i][2], c[h][i][3]);
    }
}

// Blocks behind the last row block make the lists of adapters of the product's 256-row tiles.
template <typename T, int NT>
__global__ void __launch_bounds__(256, NT <= 4 ? 2 : 1) adapter_shrink_kernel(const AdapterArgs p) {
  extern __shared__ float red[];
  __shared__ int sid[kTileRows];
  __shared__ int first[8];
  grid_dep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nrow = (p.M + kShrinkRows - 1) / kShrinkRows;
  if (blockIdx.x >= nrow) {
    if (blockIdx.y) return;
    const int tile = blockIdx.x - nrow, m = tile * kTileRows + threadIdx.x;
    const int id = m < p.M ? p.ids[m] : -1;
    sid[threadIdx.x] = id;
    __syncthreads();
    bool mine = id >= 0 && id < p.adapters;                  // the first row of its adapter
    for (int j = 0; j < threadIdx.x && mine; ++j) mine = sid[j] != id;
    const uint32_t b = __ballot_sync(0xffffffffu, mine);
    if (lane == 0) first[warp] = __popc(b);
    __syncthreads();
    int at = __popc(b & ((1u << lane) - 1u)), total = 0;
    for (int w = 0; w < 8; ++w) {
      at += w < warp ? first[w] : 0;
      total += first[w];
    }
    int32_t* list = p.lists + (int64_t)tile * kListInts;
    if (mine) list[1 + at] = id;
    if (threadIdx.x == 0) list[0] = total;
    return;
  }
  const int m0 = blockIdx.x * kShrinkRows, row = m0 + lane;
  const int id = row < p.M ? p.ids[row] : -1;
  const bool on = id >= 0 && id < p.adapters;
  const uint32_t same = __match_any_sync(0xffffffffu, on ? id : -1);
  const uint32_t lead = __ballot_sync(0xffffffffu, on && __ffs(same) - 1 == lane);
  const int nd = __popc(lead);                               // distinct adapters
  if (nd == 0) return;
  const int at = __popc(lead & ((1u << (__ffs(same) - 1)) - 1u));
  if (warp == 0) {
    sid[32 + lane] = on ? at : -1;
    if (on && __ffs(same) - 1 == lane) sid[at] = id;
  }
  __syncthreads();
  const int per = (p.R + 7) >> 3, tiles = nd * per;
  for (int t0 = blockIdx.y * NT; t0 < tiles; t0 += gridDim.y * NT) {
    const int nt = min(NT, tiles - t0);
    shrink_pass<T, NT>(p, sid, t0, nt, red);
    __syncthreads();
    // rows x columns of this pass; a row takes the columns of its own adapter
    for (int e = threadIdx.x; e < kShrinkRows * nt * 8; e += 256) {
      const int r = e / (nt * 8), c = e - r * nt * 8, q = t0 + (c >> 3), j = q % per * 8 + (c & 7);
      if (sid[32 + r] != q / per) continue;
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < 8; ++w) s += red[(w * kShrinkRows + r) * (NT * 8) + c];
      const int a = sid[q / per];
      s = j < p.R ? s * (p.scales ? p.scales[a] : 1.f) : 0.f;
      T* t = static_cast<T*>(p.t) + (int64_t)(m0 + r) * 2 * p.Rp + j;
      const T hi = from_f32<T>(s);
      t[0] = hi;
      t[p.Rp] = from_f32<T>(fabsf(to_f32(hi)) < INFINITY ? (s - to_f32(hi)) * kLowScale<T> : 0.f);
      if (per * 8 < p.Rp && q % per == per - 1) {            // the columns up to Rp
        t[8] = from_f32<T>(0.f);
        t[p.Rp + 8] = from_f32<T>(0.f);
      }
    }
    __syncthreads();
  }
}

// Few rows: bound by reading W once.  A block takes 16 RT rows of W; its 8 warps take every eighth
// 32-element piece of K of them and of the rows of x, 8 to a tile, straight from global memory in
// the layout of the products.  The adapters' second factor comes last, when the kernel before is
// done: until then this one runs beside it.
template <typename T, int NT, int RT>
__global__ void __launch_bounds__(256) adapter_few_kernel(const AdapterArgs p) {
  extern __shared__ float red[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int n0 = blockIdx.x * 16 * RT;
  const T* w[2 * RT];
#pragma unroll
  for (int i = 0; i < 2 * RT; ++i) {
    const int n = n0 + g + 8 * i;
    w[i] = n < p.N ? static_cast<const T*>(p.w) + (int64_t)n * p.K : nullptr;
  }
  const T* x[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int m = g + 8 * i;
    x[i] = m < p.M ? static_cast<const T*>(p.x) + m * p.x_row : nullptr;
  }
  float c[RT][NT][4] = {};
#pragma unroll 4
  for (int k0 = warp * 32; k0 < p.K; k0 += 256) {
    const int k = k0 + t * 8;
    uint4 wv[2 * RT], xv[NT];
#pragma unroll
    for (int i = 0; i < 2 * RT; ++i) wv[i] = piece(w[i], k, w[i] && k < p.K);
#pragma unroll
    for (int i = 0; i < NT; ++i) xv[i] = piece(x[i], k, x[i] && k < p.K);
#pragma unroll
    for (int h = 0; h < RT; ++h)
#pragma unroll
      for (int i = 0; i < NT; ++i) mma_pieces<T>(c[h][i], wv[2 * h], wv[2 * h + 1], xv[i]);
  }
  // red[warp][row of x][16 RT rows of W]
  constexpr int W = 16 * RT;
#pragma unroll
  for (int h = 0; h < RT; ++h)
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) red[(warp * (NT * 8) + i * 8 + 2 * t + (e & 1)) * W + h * 16 + g + 8 * (e >> 1)] = c[h][i][e];
  __syncthreads();
  grid_dep_wait();                                           // t
  for (int e = threadIdx.x; e < NT * 8 * W; e += 256) {
    const int m = e / W, n = n0 + e % W;
    if (m >= p.M || n >= p.N) continue;
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) s += red[(k * (NT * 8) + m) * W + e % W];
    const int id = __ldg(p.ids + m);
    if (id >= 0 && id < p.adapters) {
      const T* b = static_cast<const T*>(p.b) + ((int64_t)id * p.N + n) * p.R;
      const T* tt = static_cast<const T*>(p.t) + (int64_t)m * 2 * p.Rp;
      if (p.b16) {
        for (int r = 0; r < p.R; r += 8) {
          float bv[8], hi[8], lo[8];
          load_f32<T, 8>(b + r, bv);
          load_f32<T, 8>(tt + r, hi);
          load_f32<T, 8>(tt + p.Rp + r, lo);
#pragma unroll
          for (int q = 0; q < 8; ++q) s += (hi[q] + lo[q] * (1.0f / kLowScale<T>)) * bv[q];
        }
      } else {
        for (int r = 0; r < p.R; ++r) s += (to_f32(tt[r]) + to_f32(tt[p.Rp + r]) * (1.0f / kLowScale<T>)) * to_f32(b[r]);
      }
    }
    if (p.bias) s += to_f32(static_cast<const T*>(p.bias)[n]);
    static_cast<T*>(p.y)[m * p.y_row + n] = from_f32<T>(s);
  }
}

template <typename K>
cudaError_t launch_after(K kernel, int blocks, int smem, const AdapterArgs& a, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <typename T, int NT, int RT>
cudaError_t launch_few(const AdapterArgs& a, cudaStream_t s) {
  return launch_after(adapter_few_kernel<T, NT, RT>, (a.N + 16 * RT - 1) / (16 * RT), 8 * NT * 8 * 16 * RT * 4, a, s);
}

// Up to here the rows of x are few enough to pass by every 16 rows of W (2,048 -> 6,144: 33 rows take 27 us,
// 64 take 33.7; as tensor-core tiles of 256 rows 34 and 33.9).
constexpr int kFewRows = 64;

template <typename T, int NT>
cudaError_t launch_shrink(const AdapterArgs& a, int blocks, int lists, int gy, cudaStream_t s) {
  constexpr int kBytes = 8 * kShrinkRows * NT * 8 * 4;
  if (kBytes > 48 * 1024) {
    static OncePerDevice limit;
    const cudaError_t e = limit([] {
      return cudaFuncSetAttribute(adapter_shrink_kernel<T, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
    });
    if (e != cudaSuccess) return e;
  }
  adapter_shrink_kernel<T, NT><<<dim3(blocks + lists, gy), 256, kBytes, s>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch16(const AdapterArgs& a, int dtype, cudaStream_t s) {
  const int per = (a.R + 7) / 8, most = std::min(a.adapters, std::min(a.M, kShrinkRows)) * per;   // column tiles of a block
  const int blocks = (a.M + kShrinkRows - 1) / kShrinkRows;
  const bool few = a.M <= kFewRows;
  const int lists = few ? 0 : (a.M + kTileRows - 1) / kTileRows;
  // Two tiles to a block while that leaves multiprocessors idle (8 rows with 8 adapters of rank 16: 17 us
  // with 8 tiles to a block), else one pass over x for all of them, if its registers allow: 4 tiles leave
  // room for two blocks per multiprocessor (70,144 rows, one adapter of rank 32 in a block: 105 us; 193 us
  // with 8).
  const cudaError_t e = most <= 2 || (int64_t)blocks * ((most + 1) / 2) <= sm_count() ? launch_shrink<T, 2>(a, blocks, lists, (most + 1) / 2, s)
                        : a.R <= 32 ? launch_shrink<T, 4>(a, blocks, lists, 1, s) : launch_shrink<T, 8>(a, blocks, lists, 1, s);
  if (e != cudaSuccess) return e;
  if (!few) return launch_adapter_gemm(a, dtype, s);
  return a.M <= 8 ? launch_few<T, 1, 1>(a, s) : a.M <= 16 ? launch_few<T, 2, 1>(a, s) : a.M <= 32 ? launch_few<T, 4, 1>(a, s) : launch_few<T, 8, 1>(a, s);
}

constexpr int kMostRows = 0x7fffffff - (kTileRows - 1), kMostColumns = 0x7fffffff - 511;

int check(const ultragen_adapter_t* c) {
  if (!c || c->rows < 0 || c->k < 1 || c->n < 1 || c->rank < 1 || c->adapters < 1) return ULTRAGEN_ERR_INVALID_ARG;
  if (c->dtype != ULTRAGEN_BF16 && c->dtype != ULTRAGEN_F16 && c->dtype != ULTRAGEN_F32) return ULTRAGEN_ERR_INVALID_ARG;
  if (c->rank > 128 || c->n > 65535 * 64) return ULTRAGEN_ERR_UNSUPPORTED;
  // rows and columns of k are counted in int, up to a tile of rows, or the 8 warps' next pieces of k, behind the last
  if (c->rows > kMostRows || c->k > kMostColumns) return ULTRAGEN_ERR_UNSUPPORTED;
  return ULTRAGEN_OK;
}

template <typename T>
cudaError_t launch_general(const AdapterArgs& a, cudaStream_t s) {
  adapter_general_shrink_kernel<T><<<a.M, 128, 0, s>>>(a);
  adapter_general_kernel<T><<<dim3((a.M + 63) / 64, (a.N + 63) / 64), 256, 0, s>>>(a);
  return cudaGetLastError();
}

// Bytes of t and of the lists, for whichever kernels the call takes.
size_t t_bytes(const ultragen_adapter_t* c) {
  return ((size_t)c->rows * std::max((c->rank + 15) / 16 * 16, c->rank) * sizeof(float) + 15) & ~size_t(15);
}
size_t list_bytes(const ultragen_adapter_t* c) {
  return ((size_t)c->rows + kTileRows - 1) / kTileRows * kListInts * sizeof(int32_t);
}

bool aligned(const void* p) { return ((uintptr_t)p & 15u) == 0; }

}  // namespace
}  // namespace ug

using namespace ug;

extern "C" {

int ultragen_adapter_project_workspace(const ultragen_adapter_t* c, size_t* bytes) {
  int st = check(c);
  if (st != ULTRAGEN_OK) return st;
  if (!bytes) return ULTRAGEN_ERR_INVALID_ARG;
  *bytes = t_bytes(c) + list_bytes(c);
  return ULTRAGEN_OK;
}

int ultragen_adapter_project(const ultragen_adapter_t* c, const void* x, const void* w, const void* bias,
                             const void* a, const void* b, const float* scales, const int32_t* ids, void* y,
                             void* workspace, size_t workspace_bytes, ultragen_stream_t stream) {
  ug::NvtxRange nvtx_range("ultragen_adapter_project");
  int st = check(c);
  if (st != ULTRAGEN_OK) return st;
  if (c->rows == 0) return ULTRAGEN_OK;
  if (!x || !w || !a || !b || !ids || !y || !workspace || !aligned(workspace) ||
      workspace_bytes < t_bytes(c) + list_bytes(c))
    return ULTRAGEN_ERR_INVALID_ARG;
  if (begins_at(y, {x, w, bias, a, b, scales, ids, workspace})) return ULTRAGEN_ERR_INVALID_ARG;   // (x is read for every column tile of y)
  int dev;
  if ((st = current_device(&dev)) != ULTRAGEN_OK) return st;
  AdapterArgs p = {};
  p.x = x;
  p.w = w;
  p.a = a;
  p.b = b;
  p.bias = bias;
  p.scales = scales;
  p.ids = ids;
  p.y = y;
  p.x_row = c->x_row;
  p.y_row = c->y_row;
  p.M = c->rows;
  p.N = c->n;
  p.K = c->k;
  p.R = c->rank;
  p.adapters = c->adapters;
  p.Rp = (c->rank + 15) / 16 * 16;
  p.t = workspace;
  p.lists = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(workspace) + t_bytes(c));
  p.b16 = c->rank % 8 == 0 && aligned(b);
  p.y16 = c->n % 8 == 0 && c->y_row % 8 == 0 && aligned(y);
  p.timeout_ns = 2000ull * 1000 * 1000;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool fast = c->dtype != ULTRAGEN_F32 && c->k % 8 == 0 && c->x_row % 8 == 0 && aligned(x) && aligned(w) && aligned(a);
  cudaError_t e;
  if (fast) e = c->dtype == ULTRAGEN_BF16 ? launch16<__nv_bfloat16>(p, c->dtype, s) : launch16<__half>(p, c->dtype, s);
  else e = c->dtype == ULTRAGEN_BF16 ? launch_general<__nv_bfloat16>(p, s)
         : c->dtype == ULTRAGEN_F16 ? launch_general<__half>(p, s) : launch_general<float>(p, s);
  return e == cudaSuccess ? ULTRAGEN_OK : ULTRAGEN_ERR_CUDA;
}

}  // extern "C"
