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

constexpr int BOX_BYTES = 128 * 64 * 2;                // one box of 128 rows x 64 elements
constexpr uint64_t kDrainNs = 50ull * 1000 * 1000;    // bounded drain on the abort path

// Bounded waits of a role on the CTA's barriers.
struct Waiter {
  uint32_t bar;                        // first barrier
  uint32_t abort_word;
  int code;
  uint32_t limit_ns;
  __device__ __forceinline__ bool operator()(int b, uint32_t parity) const {
    return mbar_wait_short(bar + 8 * b, parity, abort_word, code, limit_ns);
  }
  // all lanes of the warp
  __device__ __forceinline__ bool warp(int b, uint32_t parity) const {
    return __all_sync(0xffffffffu, (*this)(b, parity));
  }
  __device__ __forceinline__ void drain(int b, uint32_t parity, int* error) const {
    mbar_wait(bar + 8 * b, parity, nullptr, error, DEV_TIMEOUT_DRAIN, kDrainNs);
  }
};

// After a wait that ran out: the copies in flight land well within this time, and none may land after
// this CTA exits.
__device__ __noinline__ inline void settle() {
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t looks = 0; !wait_over(globaltimer_ns(), t0, kDrainNs, looks); ++looks) __nanosleep(1000);
}

__device__ __forceinline__ void warp_arrive(uint32_t bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// One [128 x D] tile: D / 64 boxes of 64 elements.
template <int D>
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap* m, int row, int hk, int b, uint32_t bar) {
#pragma unroll
  for (int bx = 0; bx < D / 64; ++bx) tma_load_5d_elect(dst + bx * BOX_BYTES, m, bx * 64, 0, row, hk, b, bar);
}

// D[128 x 128] = A B^T over K = D, both tiles K-major.
template <typename T, int D>
__device__ __forceinline__ void mma_scores(uint32_t d, uint32_t a, uint32_t b) {
  mma_ss_tile_elect<D>(d, desc_lo(a, 16), desc_lo(b, 16), desc_hi_sw128(1024), idesc_half<T>(128, 128, 0));
}

// D[128 x D] (+)= A B: A a packed 16-bit operand in TMEM, B a [128 x D] tile read MN-major.
template <typename T, int D>
__device__ __forceinline__ void mma_accum(uint32_t d, uint32_t a, uint32_t b, bool first) {
  mma_ts_tile_elect(d, a, desc_lo(b, BOX_BYTES), desc_hi_sw128(1024), idesc_half<T>(128, D, 1), first ? 0u : 1u);
}

// W columns of a row of an accumulator per lane, scaled and rounded, to 16-bit global memory.  Stores
// by row would go to 32 rows each; N = W / 8 lanes exchange their 16-byte pieces first (a transpose of
// N x N pieces in log2(N) rounds), so that N lanes write one row's 2 W bytes together.  `row` is the
// lane's destination, null for a row that is not stored.
template <typename T, int W>
__device__ __forceinline__ void store_piece(uint32_t tmem, T* row, float f) {
  constexpr int N = W / 8;
  const int lane = threadIdx.x & 31, c = lane & (N - 1);
  uint4 v[N];
  {
    uint32_t o[W];
    __syncwarp();
    if constexpr (W == 64) tmem_ld64_sync(tmem, o);
    else tmem_ld32_sync(tmem, o);
#pragma unroll
    for (int q = 0; q < N; ++q) {
      v[q].x = pack2<T>(__uint_as_float(o[8 * q + 0]) * f, __uint_as_float(o[8 * q + 1]) * f);
      v[q].y = pack2<T>(__uint_as_float(o[8 * q + 2]) * f, __uint_as_float(o[8 * q + 3]) * f);
      v[q].z = pack2<T>(__uint_as_float(o[8 * q + 4]) * f, __uint_as_float(o[8 * q + 5]) * f);
      v[q].w = pack2<T>(__uint_as_float(o[8 * q + 6]) * f, __uint_as_float(o[8 * q + 7]) * f);
    }
  }
#pragma unroll
  for (int b = 1; b < N; b *= 2) {
    const bool up = lane & b;
#pragma unroll
    for (int q = 0; q < N; ++q) {
      if (q & b) continue;
      uint4 &lo = v[q], &hi = v[q | b];
      uint4 t = up ? lo : hi;
      t.x = __shfl_xor_sync(0xffffffffu, t.x, b);
      t.y = __shfl_xor_sync(0xffffffffu, t.y, b);
      t.z = __shfl_xor_sync(0xffffffffu, t.z, b);
      t.w = __shfl_xor_sync(0xffffffffu, t.w, b);
      if (up) lo = t;
      else hi = t;
    }
  }
  // v[q] is now piece c of the row of lane (lane - c + q)
#pragma unroll
  for (int q = 0; q < N; ++q) {
    T* dst = reinterpret_cast<T*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(row), lane - c + q));
    if (dst) *reinterpret_cast<uint4*>(dst + c * 8) = v[q];
  }
}

}  // namespace ug
