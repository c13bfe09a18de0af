// Device helpers of the cross attention kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "cross.h"
#include "elem.cuh"
#include "ptx.cuh"

namespace ug {

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }

template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (std::is_same<T, __half>::value) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  } else {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
}

// Instruction descriptor of kind::f16 with fp32 accumulation for either 16-bit type: bits 7 and
// 10 select bf16 for A and B.  b_mn = 1: B is MN-major.
template <typename T>
__host__ __device__ constexpr uint32_t idesc_half(int M, int N, int b_mn) {
  return std::is_same<T, __half>::value ? idesc_bf16(M, N, b_mn) & ~((1u << 7) | (1u << 10)) : idesc_bf16(M, N, b_mn);
}

// Generic-proxy writes to shared memory become visible to the tensor core and to TMA.
__device__ __forceinline__ void fence_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

__device__ __forceinline__ int cross_len(const CrossParams& p, int b) {
  return p.lens ? cross_clamp_len(__ldg(p.lens + b), p.ns) : p.ns;
}

// Query of a row of a packed query tile (r < 128), relative to the tile's first.
__device__ __forceinline__ int row_tok(const CrossParams& p, int r) { return (r * p.group_inv) >> 16; }

// Visibility of the 128 keys of tile j of sample b: bit c % 32 of word c / 32.
__device__ __forceinline__ uint4 cross_words(const CrossParams& p, int b, int j, int len) {
  if (p.words) return __ldg(reinterpret_cast<const uint4*>(p.words) + (int64_t)b * p.word_tiles + j);
  const int n = len - j * 128;            // visible keys of the tile, from its first
  auto word = [n](int w) { const int k = n - 32 * w; return k >= 32 ? ~0u : (k <= 0 ? 0u : (1u << k) - 1u); };
  return make_uint4(word(0), word(1), word(2), word(3));
}

__device__ __forceinline__ uint32_t word_of(const uint4& w, int i) {
  return i == 0 ? w.x : (i == 1 ? w.y : (i == 2 ? w.z : w.w));
}
__device__ __forceinline__ bool all_visible(const uint4& w) { return (w.x & w.y & w.z & w.w) == ~0u; }

// Key tiles [k0, k1) of split s of a sample with `len` visible keys.  (At most 2^24 tiles and 64
// splits: 32 bits hold the products.)
__device__ __forceinline__ void split_range(int len, int s, int nsplit, int& k0, int& k1) {
  const uint32_t n = (len + 127) >> 7;
  if (nsplit == 1) {
    k0 = 0;
    k1 = n;
  } else {
    k0 = n * s / (uint32_t)nsplit;
    k1 = n * (s + 1) / (uint32_t)nsplit;
  }
}

// Rows of a warp's accumulator (lane = row), scaled and rounded, to 16-bit global memory.  A lane's
// row is one piece, but 32 lanes' 16-byte stores to 32 rows go one by one: the 64-column chunks pass
// through 4 KB of the warp's shared memory and leave as whole 128-byte pieces, 8 lanes each.
// `row` is the lane's row, null for one that is not stored.
template <typename T, int COLS>
__device__ __forceinline__ void store_rows(uint32_t tmem, uint8_t* stage, T* row, float f) {
  const int lane = threadIdx.x & 31, c = lane & 7;
#pragma unroll 1
  for (int ch = 0; ch < COLS / 64; ++ch) {
    uint32_t o[64];
    __syncwarp();
    tmem_ld64_sync(tmem + ch * 64, o);
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      uint4 v;
      v.x = pack2<T>(__uint_as_float(o[8 * q + 0]) * f, __uint_as_float(o[8 * q + 1]) * f);
      v.y = pack2<T>(__uint_as_float(o[8 * q + 2]) * f, __uint_as_float(o[8 * q + 3]) * f);
      v.z = pack2<T>(__uint_as_float(o[8 * q + 4]) * f, __uint_as_float(o[8 * q + 5]) * f);
      v.w = pack2<T>(__uint_as_float(o[8 * q + 6]) * f, __uint_as_float(o[8 * q + 7]) * f);
      *reinterpret_cast<uint4*>(stage + lane * 128 + ((q ^ (lane & 7)) * 16)) = v;
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = i * 4 + (lane >> 3);
      const uint4 v = *reinterpret_cast<const uint4*>(stage + r * 128 + ((c ^ (r & 7)) * 16));
      T* dst = reinterpret_cast<T*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(row), r));
      if (dst) *reinterpret_cast<uint4*>(dst + ch * 64 + c * 8) = v;
    }
  }
}

// Zeroes the rows of hidden keys of a [rows x D] tile in shared memory (rows of 128 bytes in
// D / 64 boxes box_bytes apart; a row's 128 bytes stay one piece under the 128-byte swizzle).
// One warp; `first` is the tile row of key 0 of `bits`' word range.
template <int D>
__device__ __forceinline__ void scrub_rows(uint32_t tile, uint32_t box_bytes, const uint4& w, int row0, int rows) {
  const int lane = threadIdx.x & 31;
  for (int r = lane; r < rows; r += 32) {
    const int c = row0 + r;
    if ((word_of(w, c >> 5) >> (c & 31)) & 1u) continue;
#pragma unroll
    for (int bx = 0; bx < D / 64; ++bx)
#pragma unroll
      for (int q = 0; q < 8; ++q)
        asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(tile + bx * box_bytes + r * 128 + q * 16), "r"(0)
                     : "memory");
  }
}

}  // namespace ug
