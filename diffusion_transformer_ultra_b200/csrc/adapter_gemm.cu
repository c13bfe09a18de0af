// Projection with adapters on the tensor cores (tcgen05, CTA pairs): y = x W^T + T B'^T + 1 bias^T.
//
// A tile is 256 rows of x by BN rows of W, computed by two CTAs with cta_group::2: each holds 128
// rows of x and half of W's rows, so that a stage brings (128 + BN / 2) x 64 elements per SM for
// 128 x BN x 64 products.  (Alone, a CTA would bring 128 + BN rows for them, half as much again,
// and the loads from L2, not the products, would set the pace.)
// The adapters are more columns of the same sum, in granules of 16: for each adapter a that rows
// of the tile use, t_m = s_a A_a x_m (from a kernel before, as two 16-bit numbers, so that its
// rounding does not show in y: see kLowScale) in the rows that use it and zero in the others, against
// B_a (the low parts against B_a / kLowScale); and one granule whose first column is 1 against the bias.
//
// Roles per CTA (10 warps): 0-3 epilogue (TMEM -> 16 bits -> shared memory -> rows of y), 4 TMA
// producer, 5 MMA issuer (first CTA of the pair), 6-9 extension: writes the granules.
// TMEM: two accumulators of BN columns, so that a tile's epilogue runs beside the next products.
// With the kernel that makes t, of which the second case hides little: 9,728 x 1,536 -> 4,608, 105 us,
// 1.31 PF/s, in a burst of calls; 70,144 x 2,048 -> 2,048 with rank 32, 529 us, of which t takes 103 to 126.
// In a loop of seconds 124 and 606 us: the power limit holds the clock at 1,552 and 1,395 of 1,965 MHz.  (A
// library product reaches 1.63 PF/s in a burst, 1.39 over seconds.)
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <mutex>
#include <type_traits>

#include "adapter.h"
#include "cross.cuh"
#include "device.h"
#include "kernels.h"
#include "ptx.cuh"
#include "ultragen.h"

namespace ug {
namespace {

__device__ int g_error;                // first wait that ran out since the last status read

constexpr int kThreads = 320;
constexpr int kWarpProducer = 4, kWarpMma = 5, kWarpExt = 6;

template <int BN>
struct Cfg {
  static constexpr int A_BYTES = 128 * 128, B_BYTES = BN / 2 * 128;       // 64 16-bit columns
  static constexpr int STAGE = A_BYTES + B_BYTES;
  static constexpr int NS = BN == 256 ? 4 : (BN == 128 ? 6 : 7);          // stages of x and W
  static constexpr int NE = 2;                                            // stages of granules
  static constexpr int OUT_OFF = (NS + NE) * STAGE;                       // 4 warps x 32 rows x 128 bytes
  static constexpr int BAR_OFF = OUT_OFF + 4 * 4096;
  static constexpr int B_F = 0, B_E = B_F + NS, B_XF = B_E + NS, B_XE = B_XF + NE, B_TF = B_XE + NE, B_TE = B_TF + 2,
                       B_DRAIN = B_TE + 2, NBAR = B_DRAIN + 1;
  static constexpr int FLAG_OFF = BAR_OFF + NBAR * 8;                     // 8 ints: see the extension role
  static constexpr int MISC_OFF = FLAG_OFF + 32;
  static constexpr int SMEM = MISC_OFF + 16;
  static_assert(SMEM <= 227 * 1024, "shared memory per CTA exceeds 227 KB");
  static __device__ __forceinline__ uint32_t arrivals(int i) {
    return (i >= B_XF && i < B_XE) || i == B_TE || i == B_TE + 1 ? 8 : 1;   // four warps of each CTA
  }
};

struct Wait {
  uint32_t bar;
  volatile int* abort_flag;
  int code;
  uint64_t timeout_ns;
  __device__ __forceinline__ bool operator()(int b, uint32_t parity) const {
    return mbar_wait(bar + 8 * b, parity, abort_flag, &g_error, code, timeout_ns);
  }
  __device__ __forceinline__ bool warp(int b, uint32_t parity) const {
    return __all_sync(0xffffffffu, (*this)(b, parity));
  }
};

struct GemmMaps {
  CUtensorMap x, w;
};

struct Tiles {
  int nt, total;                       // tiles along N, in all
  __device__ __forceinline__ Tiles(const AdapterArgs& p, int BN) {
    nt = (p.N + BN - 1) / BN;
    total = (p.M + kTileRows - 1) / kTileRows * nt;
  }
};

// Granules of row tile mt: two sets of Rp / 16 per adapter of the list, and the bias.
__device__ __forceinline__ int granules(const AdapterArgs& p, int mt) {
  return __ldcg(p.lists + (int64_t)mt * kListInts) * (p.Rp >> 3) + (p.bias ? 1 : 0);
}

template <typename T>
__device__ __forceinline__ bool finite16(uint32_t v) {            // both 16-bit numbers of v
  constexpr uint32_t e = std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;
  return (v & e) != e && ((v >> 16) & e) != e;
}

template <int BN>
__device__ void producer_role(const GemmMaps& m, const AdapterArgs& p, uint32_t sbase, uint32_t rank, const Wait& wait) {
  using C = Cfg<BN>;
  const Tiles tl(p, BN);
  const int nk = (p.K + 63) >> 6;
  uint32_t st = 0;
  for (int t = blockIdx.x >> 1; t < tl.total; t += gridDim.x >> 1) {
    const int mt = t / tl.nt, row = mt * kTileRows + (int)rank * 128, col = (t - mt * tl.nt) * BN + (int)rank * (BN / 2);
    for (int k = 0; k < nk; ++k, ++st) {
      const uint32_t s = st % C::NS;
      if (!wait(C::B_E + s, ((st / C::NS) & 1) ^ 1)) {
        settle();                      // both CTAs stay until the copies in flight have landed
        return;
      }
      const uint32_t full = wait.bar + 8 * (C::B_F + s);
      if (rank == 0) mbar_expect_tx(full, 2 * C::STAGE);
      const uint32_t dst = sbase + s * C::STAGE, to = map_cta(full, 0);
      tma_load_2d_pair(dst, &m.x, k * 64, row, to);
      tma_load_2d_pair(dst + C::A_BYTES, &m.w, k * 64, col, to);
    }
  }
}

// Products of `n` granules (16 columns each) of a stage.
template <typename T, int BN>
__device__ __forceinline__ void mma_stage(uint32_t d, uint32_t stage, int n, bool first) {
  constexpr uint32_t id = idesc_half<T>(256, BN, 0);
  const uint32_t a = desc_lo(stage, 16), b = desc_lo(stage + Cfg<BN>::A_BYTES, 16);
#pragma unroll
  for (int kk = 0; kk < 4; ++kk)
    if (kk < n) mma_ss_pair(d, a + kk * 2, b + kk * 2, desc_hi_sw128(1024), id, first && kk == 0 ? 0u : 1u);
}

template <typename T, int BN>
__device__ void mma_role(const AdapterArgs& p, uint32_t sbase, uint32_t tbase, const Wait& wait) {
  using C = Cfg<BN>;
  const Tiles tl(p, BN);
  const int nk = (p.K + 63) >> 6;
  uint32_t st = 0, xs = 0, n = 0;
  bool ok = true;
  grid_dep_wait();                     // the lists
  for (int t = blockIdx.x >> 1; ok && t < tl.total; t += gridDim.x >> 1, ++n) {
    const int ng = granules(p, t / tl.nt);
    const uint32_t d = tbase + (n & 1) * BN;
    if (!(ok = wait(C::B_TE + (n & 1), ((n >> 1) & 1) ^ 1))) break;
    tc_fence_after();
    for (int k = 0; k < nk; ++k, ++st) {
      const uint32_t s = st % C::NS;
      if (!(ok = wait(C::B_F + s, (st / C::NS) & 1))) break;
      tc_fence_after();
      mma_stage<T, BN>(d, sbase + s * C::STAGE, min(4, (p.K - k * 64 + 15) >> 4), k == 0);
      mma_commit_pair(wait.bar + 8 * (C::B_E + s));
    }
    for (int g = 0; ok && g < ng; g += 4, ++xs) {
      const uint32_t s = xs % C::NE;
      if (!(ok = wait(C::B_XF + s, (xs / C::NE) & 1))) break;
      tc_fence_after();
      mma_stage<T, BN>(d, sbase + (C::NS + s) * C::STAGE, min(4, ng - g), false);
      mma_commit_pair(wait.bar + 8 * (C::B_XE + s));
    }
    if (ok) mma_commit_pair(wait.bar + 8 * (C::B_TF + (n & 1)));
  }
  if (!ok) {
    mma_commit_pair(wait.bar + 8 * C::B_DRAIN);
    mbar_wait(wait.bar + 8 * C::B_DRAIN, 0, nullptr, &g_error, DEV_TIMEOUT_DRAIN, kDrainNs);
  }
}

// Thread i writes row i of T and row i of B' of each granule, 32 bytes each.  A row of B with an
// infinity or NaN is written as zeros, since it would reach the rows of other adapters as 0 * inf,
// and the tile is flagged (in both CTAs, by its number among the tiles with granules, in one of 8
// places: this role is at most 5 of those ahead of the epilogue): the epilogue then adds such
// terms for the rows that use them.
template <typename T, int BN>
__device__ void extension_role(const AdapterArgs& p, uint8_t* smem, uint32_t sbase, uint32_t rank, const Wait& wait) {
  using C = Cfg<BN>;
  const Tiles tl(p, BN);
  const int i = threadIdx.x - 32 * kWarpExt;
  const int half = p.Rp >> 4;                    // granules of one set
  uint32_t xs = 0, n = 0;
  grid_dep_wait();                               // t and the lists
  for (int t = blockIdx.x >> 1; t < tl.total; t += gridDim.x >> 1) {
    const int mt = t / tl.nt, row = mt * kTileRows + (int)rank * 128 + i;
    const int col = (t - mt * tl.nt) * BN + (int)rank * (BN / 2) + i;
    const int ng = granules(p, mt);
    if (ng == 0) continue;
    ++n;
    const int32_t* list = p.lists + (int64_t)mt * kListInts + 1;
    const int id = row < p.M ? __ldg(p.ids + row) : -1;
    bool bad = false;
    for (int g0 = 0; g0 < ng; g0 += 4, ++xs) {
      const uint32_t s = xs % C::NE;
      if (!wait.warp(C::B_XE + s, ((xs / C::NE) & 1) ^ 1)) return;
      uint8_t* a_dst = smem + (C::NS + s) * C::STAGE + i * 128;
      uint8_t* b_dst = a_dst + C::A_BYTES;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int g = g0 + k;
        if (g >= ng) break;
        uint32_t av[8] = {}, bv[8] = {};
        if (p.bias && g == ng - 1) {
          const T one = from_f32<T>(1.0f);
          av[0] = *reinterpret_cast<const uint16_t*>(&one);
          if (i < BN / 2 && col < p.N) bv[0] = __ldg(static_cast<const uint16_t*>(p.bias) + col);
        } else {
          const int e = g / (2 * half), sub = g - e * 2 * half, r0 = (sub < half ? sub : sub - half) * 16;
          const int ad = __ldcg(list + e);
          if (id == ad) {
            const uint4* src = reinterpret_cast<const uint4*>(static_cast<const T*>(p.t) + (int64_t)row * 2 * p.Rp + sub * 16);
            const uint4 u = __ldcg(src), v = __ldcg(src + 1);
            av[0] = u.x; av[1] = u.y; av[2] = u.z; av[3] = u.w;
            av[4] = v.x; av[5] = v.y; av[6] = v.z; av[7] = v.w;
          }
          if (i < BN / 2 && col < p.N) {
            const uint16_t* src = static_cast<const uint16_t*>(p.b) + ((int64_t)ad * p.N + col) * p.R;
            bool fin = true;
            if (p.b16) {                         // R is a multiple of 8
              const uint4 u = __ldg(reinterpret_cast<const uint4*>(src + r0));
              uint4 v = make_uint4(0, 0, 0, 0);
              if (r0 + 8 < p.R) v = __ldg(reinterpret_cast<const uint4*>(src + r0 + 8));
              bv[0] = u.x; bv[1] = u.y; bv[2] = u.z; bv[3] = u.w;
              bv[4] = v.x; bv[5] = v.y; bv[6] = v.z; bv[7] = v.w;
            } else {
#pragma unroll
              for (int r = 0; r < 16; ++r)
                if (r0 + r < p.R) bv[r >> 1] |= (uint32_t)__ldg(src + r0 + r) << (16 * (r & 1));
            }
#pragma unroll
            for (int r = 0; r < 8; ++r) fin = fin && finite16<T>(bv[r]);
            if (!fin) {
              bad = true;
#pragma unroll
              for (int r = 0; r < 8; ++r) bv[r] = 0u;
            }
            if constexpr (kLowScale<T> != 1.0f)
              if (sub >= half) {
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                  __half2 h = *reinterpret_cast<__half2*>(&bv[r]);
                  h = __hmul2(h, __float2half2_rn(1.0f / kLowScale<T>));
                  bv[r] = *reinterpret_cast<uint32_t*>(&h);
                }
              }
          }
        }
        const int c0 = ((2 * k) ^ (i & 7)) * 16, c1 = ((2 * k + 1) ^ (i & 7)) * 16;    // 128-byte swizzle
        *reinterpret_cast<uint4*>(a_dst + c0) = make_uint4(av[0], av[1], av[2], av[3]);
        *reinterpret_cast<uint4*>(a_dst + c1) = make_uint4(av[4], av[5], av[6], av[7]);
        if (i < BN / 2) {
          *reinterpret_cast<uint4*>(b_dst + c0) = make_uint4(bv[0], bv[1], bv[2], bv[3]);
          *reinterpret_cast<uint4*>(b_dst + c1) = make_uint4(bv[4], bv[5], bv[6], bv[7]);
        }
      }
      if (bad) {
        const uint32_t f = sbase + C::FLAG_OFF + (n & 7) * 4;
        st_cluster_s32(map_cta(f, 0), (int)n);
        st_cluster_s32(map_cta(f, 1), (int)n);
      }
      fence_async_smem();
      __syncwarp();
      if ((threadIdx.x & 31) == 0) mbar_arrive_cluster(map_cta(wait.bar + 8 * (C::B_XF + s), 0));
    }
  }
}

// The terms of a column that the products left out: sums over the granules of its row `b` of B
// that hold an infinity or NaN (0 when there is none).
template <typename T>
__device__ __noinline__ float odd_terms(const T* b, const T* t, int R, int Rp) {
  float v = 0.f;
  for (int r0 = 0; r0 < R; r0 += 16) {
    bool fin = true;
    float s = 0.f;
    for (int r = r0; r < min(R, r0 + 16); ++r) {
      const float x = to_f32(b[r]);
      fin = fin && fabsf(x) < INFINITY;
      s += (to_f32(t[r]) + to_f32(t[Rp + r]) * (1.0f / kLowScale<T>)) * x;
    }
    if (!fin) v += s;
  }
  return v;
}

template <typename T, int BN>
__device__ void epilogue_role(const AdapterArgs& p, uint8_t* smem, uint32_t tbase, uint32_t rank, const Wait& wait) {
  using C = Cfg<BN>;
  const Tiles tl(p, BN);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* out = smem + C::OUT_OFF + warp * 4096;
  volatile int* flags = reinterpret_cast<volatile int*>(smem + C::FLAG_OFF);
  uint32_t n = 0, ext = 0;
  grid_dep_wait();                     // the lists
  for (int t = blockIdx.x >> 1; t < tl.total; t += gridDim.x >> 1, ++n) {
    const int mt = t / tl.nt, row0 = mt * kTileRows + (int)rank * 128 + warp * 32, col0 = (t - mt * tl.nt) * BN;
    const bool has = granules(p, mt) > 0;
    if (has) ++ext;
    if (!wait.warp(C::B_TF + (n & 1), (n >> 1) & 1)) return;
    tc_fence_after();
    const bool odd = has && flags[ext & 7] == (int)ext;
    const uint32_t acc = tbase + (n & 1) * BN + ((uint32_t)warp * 32u << 16);
#pragma unroll 1
    for (int ch = 0; ch < BN / 64; ++ch) {
      const int col = col0 + ch * 64;
      uint32_t v[64];
      tmem_ld64_sync(acc + ch * 64, v);
      if (ch == BN / 64 - 1) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(map_cta(wait.bar + 8 * (C::B_TE + (n & 1)), 0));
      }
      __syncwarp();
      if (col >= p.N) continue;
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        uint4 u;
        u.x = pack2<T>(__uint_as_float(v[8 * c]), __uint_as_float(v[8 * c + 1]));
        u.y = pack2<T>(__uint_as_float(v[8 * c + 2]), __uint_as_float(v[8 * c + 3]));
        u.z = pack2<T>(__uint_as_float(v[8 * c + 4]), __uint_as_float(v[8 * c + 5]));
        u.w = pack2<T>(__uint_as_float(v[8 * c + 6]), __uint_as_float(v[8 * c + 7]));
        *reinterpret_cast<uint4*>(out + lane * 128 + ((c ^ (lane & 7)) * 16)) = u;
      }
      if (odd && row0 + lane < p.M) {
        const int id = __ldg(p.ids + row0 + lane);
        const T* b = static_cast<const T*>(p.b) + ((int64_t)id * p.N + col) * p.R;
        const T* tr = static_cast<const T*>(p.t) + (int64_t)(row0 + lane) * 2 * p.Rp;
        for (int c = 0; c < 64 && id >= 0 && id < p.adapters && col + c < p.N; ++c) {
          T* e = reinterpret_cast<T*>(out + lane * 128 + (((c >> 3) ^ (lane & 7)) * 16) + (c & 7) * 2);
          *e = from_f32<T>(to_f32(*e) + odd_terms<T>(b + (int64_t)c * p.R, tr, p.R, p.Rp));
        }
      }
      __syncwarp();
      if (p.y16) {
        const int c = lane & 7;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = i * 4 + (lane >> 3);
          const uint4 u = *reinterpret_cast<const uint4*>(out + r * 128 + ((c ^ (r & 7)) * 16));
          if (row0 + r < p.M && col + c * 8 < p.N)
            *reinterpret_cast<uint4*>(static_cast<T*>(p.y) + (int64_t)(row0 + r) * p.y_row + col + c * 8) = u;
        }
      } else {
        const int rows = min(32, p.M - row0);
        for (int r = 0; r < rows; ++r) {
          const uint32_t u = *reinterpret_cast<const uint32_t*>(out + r * 128 + (((lane >> 2) ^ (r & 7)) * 16) + (lane & 3) * 4);
          uint16_t* y = static_cast<uint16_t*>(p.y) + (int64_t)(row0 + r) * p.y_row + col + 2 * lane;
          if (col + 2 * lane < p.N) y[0] = (uint16_t)u;
          if (col + 2 * lane + 1 < p.N) y[1] = (uint16_t)(u >> 16);
        }
      }
      __syncwarp();
    }
  }
}

template <typename T, int BN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    adapter_gemm_kernel(const __grid_constant__ GemmMaps m, const AdapterArgs p) {
  using C = Cfg<BN>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem), bar = sbase + C::BAR_OFF, rank = cluster_rank();
  if (sbase & 1023) {                  // the swizzle needs it; the declaration asks for it
    if (threadIdx.x == 0) atomicExch(&g_error, (int)DEV_TIMEOUT_PRODUCER);
    return;
  }
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + C::MISC_OFF);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NBAR; ++i) mbar_init(bar + 8 * i, C::arrivals(i));
    for (int i = 0; i < 8; ++i) reinterpret_cast<int*>(smem + C::FLAG_OFF)[i] = 0;
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kWarpMma) {
    tmem_alloc_pair(smem_u32(misc), 2 * BN);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tbase = misc[0];
  Wait wait{bar, abort_flag, DEV_TIMEOUT_SOFTMAX, p.timeout_ns};
  if (warp == kWarpProducer) {
    wait.code = DEV_TIMEOUT_PRODUCER;
    if (lane == 0) producer_role<BN>(m, p, sbase, rank, wait);
  } else if (warp == kWarpMma) {
    wait.code = DEV_TIMEOUT_MMA;
    if (lane == 0 && rank == 0) mma_role<T, BN>(p, sbase, tbase, wait);
  } else if (warp >= kWarpExt) {
    extension_role<T, BN>(p, smem, sbase, rank, wait);
  } else {
    epilogue_role<T, BN>(p, smem, tbase, rank, wait);
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();                      // neither CTA leaves while the other reads its memory
  tc_fence_after();
  if (warp == kWarpMma) {
    __syncwarp();
    tmem_dealloc_pair(tbase, 2 * BN);
  }
}

// [rows, K] of 16-bit elements with [64 x box] boxes and the 128-byte swizzle.
int make_map(CUtensorMap* m, const void* base, int64_t stride, int dtype, int rows, int K, int box) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return 1;
  const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)stride * 2};
  const cuuint32_t bx[2] = {64, (cuuint32_t)box}, es[2] = {1, 1};
  return fn(m, dtype == ULTRAGEN_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
            const_cast<void*>(base), dims, strides, bx, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS;
}

template <typename T, int BN>
cudaError_t launch(const AdapterArgs& a, int dtype, cudaStream_t s) {
  constexpr int kMaxDev = 64;
  static std::mutex mu;
  static bool attr_set[kMaxDev] = {};
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDev) return cudaErrorInvalidDevice;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!attr_set[dev]) {
      e = cudaFuncSetAttribute(adapter_gemm_kernel<T, BN>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<BN>::SMEM);
      if (e != cudaSuccess) return e;
      attr_set[dev] = true;
    }
  }
  GemmMaps m;
  if (make_map(&m.x, a.x, a.x_row, dtype, a.M, a.K, 128) || make_map(&m.w, a.w, a.K, dtype, a.N, a.K, BN / 2))
    return cudaErrorInvalidValue;
  const int tiles = (a.M + kTileRows - 1) / kTileRows * ((a.N + BN - 1) / BN);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * std::min(tiles, std::max(1, sm_count() / 2)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Cfg<BN>::SMEM;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, adapter_gemm_kernel<T, BN>, m, a);
}

template <typename T>
cudaError_t launch_bn(const AdapterArgs& a, int dtype, cudaStream_t s) {
  // The tile's width: rounds of tiles over the CTA pairs, each of its width's products and about
  // 32 columns' time per k-step on top.
  const int64_t pairs = std::max(1, sm_count() / 2), mt = (a.M + kTileRows - 1) / kTileRows;
  int best = 256;
  int64_t cost = 0;
  for (int bn : {256, 128, 64}) {
    const int64_t c = (mt * ((a.N + bn - 1) / bn) + pairs - 1) / pairs * (bn + 32);
    if (bn == 256 || c < cost) {
      cost = c;
      best = bn;
    }
  }
  return best == 256 ? launch<T, 256>(a, dtype, s) : best == 128 ? launch<T, 128>(a, dtype, s) : launch<T, 64>(a, dtype, s);
}

}  // namespace

cudaError_t launch_adapter_gemm(const AdapterArgs& a, int dtype, cudaStream_t s) {
  return dtype == ULTRAGEN_BF16 ? launch_bn<__nv_bfloat16>(a, dtype, s) : launch_bn<__half>(a, dtype, s);
}

cudaError_t adapter_status(int* code, cudaStream_t s) { return read_clear_error(&g_error, code, s); }

}  // namespace ug
