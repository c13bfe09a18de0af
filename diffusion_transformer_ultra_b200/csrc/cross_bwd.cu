// Cross attention backward for sm_100a (tcgen05 + TMEM + TMA), two kernels:
//   dQ:     per 128-row query tile, over its key tiles:  S = Q K^T, dP = dO V^T,
//           dS = P (dP - delta), dQ += dS K.  Also makes delta for the second kernel.
//   dK/dV:  per 128-key tile, over query tiles:  S^T = K Q^T, dP^T = V dO^T,
//           dV += P^T dO, dK += dS^T Q.
// P = exp2(scale log2(e) S - lse log2(e)) from the forward pass's lse, so no running maximum.
// The split in two costs S and dP twice (seven products per pair of tiles instead of five) and
// saves the sum of dQ over key tiles through memory: with the 512 keys of a prompt that would be
// four fp32 copies of dQ, eight times the bytes of all the operands.
// P and dS pass through TMEM as 16-bit A operands (the tensor core's type); sums, P's exponent
// and dS before its rounding are fp32.
//
// Roles of both kernels: warps 0-7 the elementwise part (two warpgroups; warp w has the rows of
// TMEM lane quarter w % 4 and half the columns), warp 8 producer (TMA), warp 9 MMA issuer.
// Steps of consecutive items run on without a drain: the products of a step are issued around
// the one before it, so that the tensor core works while the elementwise part of a step runs.
#include <algorithm>
#include <cstdint>
#include <mutex>

#include "cross.cuh"

namespace ug {
namespace {

__device__ int g_error;                // first wait that ran out since the last status read

constexpr int kWarpProducer = 8, kWarpMma = 9, kWarpAux = 10;

// Slot and wait parity of the n-th use of a ring of N slots.
template <int N>
struct Ring {
  uint32_t n = 0;
  __device__ __forceinline__ uint32_t slot() const { return n % N; }
  __device__ __forceinline__ uint32_t phase() const { return (n / N) & 1; }
};

// At a kernel's end: a wait that ran out.
__device__ __forceinline__ void report(const uint32_t* abort_word) {
  const int code = *reinterpret_cast<const volatile int*>(abort_word);
  if (threadIdx.x == 0 && code != 0) atomicExch(&g_error, code);
}

template <typename T, int D>
__device__ __forceinline__ void zero_half(T* dst) {
#pragma unroll
  for (int q = 0; q < D / 16; ++q) reinterpret_cast<uint4*>(dst)[q] = make_uint4(0, 0, 0, 0);
}

// Visibility of 32 columns as masks of packed pairs: bit 2 c goes to bit c, bit 2 c + 1 to bit 16 + c;
// a pair's mask is then a shift and a byte permutation that repeats the signs of two bytes.
__device__ __forceinline__ uint32_t split_pairs(uint32_t w) {
  uint32_t t;
  t = (w ^ (w >> 1)) & 0x22222222u;
  w ^= t ^ (t << 1);
  t = (w ^ (w >> 2)) & 0x0c0c0c0cu;
  w ^= t ^ (t << 2);
  t = (w ^ (w >> 4)) & 0x00f000f0u;
  w ^= t ^ (t << 4);
  t = (w ^ (w >> 8)) & 0x0000ff00u;
  return w ^ t ^ (t << 8);
}
__device__ __forceinline__ uint32_t pair_mask(uint32_t w, int c) {
  uint32_t m;
  asm("prmt.b32 %0, %1, 0, 0xbb99;" : "=r"(m) : "r"(w << (15 - c)));
  return m;
}

// -lse log2(e), the constant of a row's exponentials; -inf (P = 0) for a row that does not exist
// or has no visible key.
__device__ __forceinline__ float neg_lse2(float lse) { return lse == neg_inf() ? neg_inf() : -lse * 1.4426950408889634f; }

// ---------------------------------------------------------------------------------- dQ
// 512 threads: warps 10 (scrubber: zeroes hidden K rows, which may hold NaN: 0 * NaN), 12-15 (the
// accumulators' way to dq: the elementwise warps are what a step waits for).  delta = do . o comes from
// a kernel before: made by warps 12-15 in here, its code and the other roles' did not fit the
// instruction cache together (156 misses a step), and the pass took 218 us.  Now it takes 119, 826 TF/s,
// and delta 27, 5.7 TB/s, for 4 x 4,096 queries, 512 keys (436, 359 and none in three samples), 24 heads
// of 128; bound by the elementwise warps' chain of loads, exponentials and stores.
// TMEM: S [0,128), dP / dS in two buffers [128,384), dQ [384,384+D).
template <int D>
struct CfgQ {
  static constexpr int TILE = 128 * D * 2;
  static constexpr int NK = D == 128 ? 3 : 5, NV = D == 128 ? 2 : 4;
  static constexpr int DO_OFF = TILE, K_OFF = 2 * TILE, V_OFF = K_OFF + NK * TILE;
  static constexpr int RED_OFF = V_OFF + NV * TILE;            // [2][2][128] floats: halves of a row's sum
  static constexpr int BAR_OFF = RED_OFF + 4 * 128 * 4;
  // full / empty of Q, dO, K (full, scrubbed, empty), V; S ready / read; dP ready; dS ready;
  // accumulator ready / read; halves exchanged.  dP and dS of odd and even steps have barriers of their
  // own: S and dP of step g are issued before dS of step g - 1 is waited for, so that dS of step g may be
  // there by then, and on one barrier that would be a second phase, behind which the first is not seen.
  static constexpr int B_QF = 0, B_QE = 1, B_OF = 2, B_OE = 3, B_KF = 4, B_KS = B_KF + NK, B_KE = B_KS + NK, B_VF = B_KE + NK,
                       B_VE = B_VF + NV, B_SF = B_VE + NV, B_SR = B_SF + 1, B_PF = B_SR + 1, B_DS = B_PF + 2, B_AF = B_DS + 2,
                       B_AE = B_AF + 1, B_XR = B_AE + 1, B_DRAIN = B_XR + 1,
                       NBAR = B_DRAIN + 1;
  static constexpr int MISC_OFF = BAR_OFF + NBAR * 8;
  static constexpr int SMEM = MISC_OFF + 16;
  static_assert(SMEM <= 227 * 1024, "shared memory per CTA exceeds 227 KB");
  static __device__ __forceinline__ uint32_t arrivals(int i) {
    return i == B_SR || i == B_DS || i == B_DS + 1 || i == B_XR ? 8 : (i == B_AE ? 4 : 1);   // elementwise warps; warps 12-15
  }
};
constexpr int kThreadsQ = 512, kRegsLaunchQ = 128, kRegsElemQ = 184, kRegsOtherQ = 72;
static_assert(256 * kRegsElemQ + 256 * kRegsOtherQ <= kThreadsQ * kRegsLaunchQ, "register split exceeds the launch allocation");

struct ItemQ {
  int b, hk, qt, len, n;
  __device__ __forceinline__ ItemQ(const CrossParams& p, int it) {
    const uint32_t u = p.div_q.div(it);
    qt = it - u * p.nqt;
    b = p.div_kv.div(u);
    hk = u - b * p.kv_heads;
    len = cross_len(p, b);
    n = (len + 127) >> 7;
  }
};

template <int D>
__device__ void dq_producer(const CrossMaps& m, const CrossParams& p, uint32_t sbase, const Waiter& wait) {
  using C = CfgQ<D>;
  const uint32_t bar = wait.bar;
  const int q_bytes = p.toks * p.group * D * 2;
  Ring<1> rq, ro;
  Ring<C::NK> rk;
  Ring<C::NV> rv;
  bool ok = true;
  for (int it = blockIdx.x; ok && it < p.total; it += gridDim.x) {
    const ItemQ w(p, it);
    const int n = uniform(w.n);
    const int ahead = it + (int)gridDim.x;
    if (ahead < p.total) {             // (total + a grid stays below 2^31: see the entry point's check)
      const ItemQ a(p, ahead);         // the next item's rows into L2: their slots free late
#pragma unroll
      for (int bx = 0; bx < D / 64; ++bx) {
        tma_prefetch_5d_elect(&m.q, bx * 64, 0, a.qt * p.toks, a.hk, a.b);
        tma_prefetch_5d_elect(&m.d_o, bx * 64, 0, a.qt * p.toks, a.hk, a.b);
      }
    }
    for (int j = 0; j < n; ++j) {
      if (j == 0) {
        if (!(ok = wait.warp(C::B_QE, rq.phase() ^ 1))) break;
        mbar_expect_tx_elect(bar + 8 * C::B_QF, q_bytes);
        load_tile<D>(sbase, &m.q, w.qt * p.toks, w.hk, w.b, bar + 8 * C::B_QF);
        ++rq.n;
      }
      const uint32_t ks = rk.slot(), vs = rv.slot();
      if (!(ok = wait.warp(C::B_KE + ks, rk.phase() ^ 1))) break;
      mbar_expect_tx_elect(bar + 8 * (C::B_KF + ks), C::TILE);
      load_tile<D>(sbase + C::K_OFF + ks * C::TILE, &m.k, j * 128, w.hk, w.b, bar + 8 * (C::B_KF + ks));
      ++rk.n;
      if (j == 0) {
        if (!(ok = wait.warp(C::B_OE, ro.phase() ^ 1))) break;
        mbar_expect_tx_elect(bar + 8 * C::B_OF, q_bytes);
        load_tile<D>(sbase + C::DO_OFF, &m.d_o, w.qt * p.toks, w.hk, w.b, bar + 8 * C::B_OF);
        ++ro.n;
      }
      if (!(ok = wait.warp(C::B_VE + vs, rv.phase() ^ 1))) break;
      mbar_expect_tx_elect(bar + 8 * (C::B_VF + vs), C::TILE);
      load_tile<D>(sbase + C::V_OFF + vs * C::TILE, &m.v, j * 128, w.hk, w.b, bar + 8 * (C::B_VF + vs));
      ++rv.n;
    }
  }
  if (!ok) settle();
}

template <int D>
__device__ void dq_scrub(const CrossParams& p, uint32_t sbase, const Waiter& wait) {
  using C = CfgQ<D>;
  Ring<C::NK> rk;
  for (int it = blockIdx.x; it < p.total; it += gridDim.x) {
    const ItemQ w(p, it);
    for (int j = 0; j < w.n; ++j, ++rk.n) {
      const uint4 vis = cross_words(p, w.b, j, w.len);
      if (!wait.warp(C::B_KF + rk.slot(), rk.phase())) return;
      if (!all_visible(vis)) {
        scrub_rows<D>(sbase + C::K_OFF + rk.slot() * C::TILE, BOX_BYTES, vis, 0, 128);
        fence_async_smem();
      }
      warp_arrive(wait.bar + 8 * (C::B_KS + rk.slot()));
    }
  }
}

// The accumulators' way to dq (zeros where no key is visible).  Four warps, 32 rows each.
template <typename T, int D>
__device__ void dq_store(const CrossParams& p, uint32_t tbase, const Waiter& wait) {
  using C = CfgQ<D>;
  const int r = threadIdx.x & 127, tr = row_tok(p, r), gr = r - tr * p.group;
  const uint32_t tAcc = tbase + ((uint32_t)((threadIdx.x >> 5) & 3) * 32u << 16) + 384;
  uint32_t items = 0;
  for (int it = blockIdx.x; it < p.total; it += gridDim.x) {
    const ItemQ w(p, it);
    const int tok = w.qt * p.toks + tr;
    T* out = nullptr;
    if (tr < p.toks && tok < p.nq)
      out = static_cast<T*>(p.out[0]) + w.b * p.out_st[0][0] + tok * p.out_st[0][1] + (w.hk * p.group + gr) * p.out_st[0][2];
    if (w.n == 0) {
      if (out) {
        zero_half<T, D>(out);
        zero_half<T, D>(out + D / 2);
      }
      continue;
    }
    if (!wait.warp(C::B_AF, items & 1)) return;
    tc_fence_after();
#pragma unroll 1
    for (int ch = 0; ch < D / 32; ++ch) store_piece<T, 32>(tAcc + ch * 32, out ? out + ch * 32 : nullptr, p.scale);
    tc_fence_before();
    warp_arrive(wait.bar + 8 * C::B_AE);
    ++items;
  }
}

template <typename T, int D>
__device__ void dq_mma(const CrossParams& p, uint32_t sbase, uint32_t tbase, const Waiter& wait) {
  using C = CfgQ<D>;
  const uint32_t bar = wait.bar, tAcc = tbase + 384;
  const int kready = p.scrub ? C::B_KS : C::B_KF;
  Ring<1> rq;
  Ring<C::NK> rk;
  Ring<C::NV> rv;
  uint32_t g = 0, items = 0;           // steps and items begun
  bool ok = true, pending = false, pfirst = false, plast = false;
  uint32_t pslot = 0, pitem = 0;
  // one round more than there are items: the last step's product (each product has one place in
  // the code, which the warps of all roles share the instruction cache with)
  for (int it = blockIdx.x; ok; it += gridDim.x) {
    const bool end = it >= p.total;
    const int n = end ? 1 : uniform(ItemQ(p, it).n);
    for (int j = 0; j < n; ++j) {
      if (!end) {
        if (j == 0 && !(ok = wait.warp(C::B_QF, rq.phase()))) break;
        if (!(ok = wait.warp(kready + rk.slot(), rk.phase()))) break;
        if (g > 0 && !(ok = wait.warp(C::B_SR, (g - 1) & 1))) break;
        tc_fence_after();
        mma_scores<T, D>(tbase, sbase, sbase + C::K_OFF + rk.slot() * C::TILE);
        mma_commit_elect(bar + 8 * C::B_SF);
        if (j == n - 1) mma_commit_elect(bar + 8 * C::B_QE);
        if (j == 0 && !(ok = wait.warp(C::B_OF, rq.phase()))) break;
        if (!(ok = wait.warp(C::B_VF + rv.slot(), rv.phase()))) break;
        tc_fence_after();
        // (overwrites dS of step g - 2, which the product issued before has read)
        mma_scores<T, D>(tbase + 128 + 128 * (g & 1), sbase + C::DO_OFF, sbase + C::V_OFF + rv.slot() * C::TILE);
        mma_commit_elect(bar + 8 * (C::B_PF + (g & 1)));
        mma_commit_elect(bar + 8 * (C::B_VE + rv.slot()));
        if (j == n - 1) mma_commit_elect(bar + 8 * C::B_OE);
      }
      if (pending) {                   // dQ += dS K of step g - 1
        if (!(ok = wait.warp(C::B_DS + ((g - 1) & 1), ((g - 1) >> 1) & 1))) break;
        if (pfirst && pitem > 0 && !(ok = wait.warp(C::B_AE, (pitem - 1) & 1))) break;
        tc_fence_after();
        mma_accum<T, D>(tAcc, tbase + 128 + 128 * ((g - 1) & 1), sbase + C::K_OFF + pslot * C::TILE, pfirst);
        mma_commit_elect(bar + 8 * (C::B_KE + pslot));
        if (plast) mma_commit_elect(bar + 8 * C::B_AF);
      }
      if (end) return;
      pending = true;
      pfirst = j == 0;
      plast = j == n - 1;
      pslot = rk.slot();
      pitem = items;
      ++rk.n;
      ++rv.n;
      ++g;
    }
    if (n > 0) {
      ++rq.n;
      ++items;
    }
  }
  mma_commit_elect(bar + 8 * C::B_DRAIN);
  wait.drain(C::B_DRAIN, 0, &g_error);
}

// The elementwise part.  delta comes from do . o, except where all of a row's keys are in one tile:
// there it is sum_j p_j dP_j, without the rounding of o, which matters where few keys share the weight.
template <typename T, int D>
__device__ void dq_elementwise(const CrossParams& p, float* red, uint32_t tbase, const Waiter& wait) {
  using C = CfgQ<D>;
  const uint32_t bar = wait.bar;
  const int half = threadIdx.x >> 7, r = threadIdx.x & 127;
  const uint32_t lane_off = (uint32_t)((threadIdx.x >> 5) & 3) * 32u << 16;
  const uint32_t tS = tbase + lane_off + half * 64, tP = tS + 128;
  const int tok_r = row_tok(p, r), g_r = r - tok_r * p.group;
  const float2 scale2 = make_float2(p.scale_log2, p.scale_log2);
  uint32_t g = 0, xn = 0;
  // lse and delta of this thread's row of an item, fetched an item ahead
  auto row_of = [&](const ItemQ& w) {
    const int tok = w.qt * p.toks + tok_r;
    return tok_r < p.toks && tok < p.nq ? ((int64_t)w.b * p.heads + w.hk * p.group + g_r) * p.nq + tok : (int64_t)-1;
  };
  float lse = neg_inf(), delta = 0.f;
  auto fetch = [&](int it) {
    lse = neg_inf();
    if (it >= p.total) return;
    const ItemQ w(p, it);
    const int64_t row = row_of(w);
    if (row < 0) return;
    lse = __ldg(p.lse + row);
    if (w.n > 1) delta = __ldg(p.delta + row);
  };
  for (int it = blockIdx.x; it < p.total; it += gridDim.x) {
    if (it == blockIdx.x) fetch(it);
    const ItemQ w(p, it);
    const float nl = neg_lse2(lse);
    float nd = -delta;                 // (not set with one key tile)
    fetch(it + gridDim.x);
    const int n = w.n;
    if (n == 0) continue;
    // one visible key has weight one whatever its logit: dS is zero exactly
    const bool zero = w.len == 1 || (p.single && __ldg(p.single + w.b));
    const float2 nl2 = make_float2(nl, nl);
    for (int j = 0; j < n; ++j) {
      const uint4 vis = cross_words(p, w.b, j, w.len);
      const uint32_t w0 = half ? vis.z : vis.x, w1 = half ? vis.w : vis.y;
      uint32_t s[64];
      if (!wait.warp(C::B_SF, g & 1)) return;
      tc_fence_after();
      tmem_ld64_sync(tS, s);
      tc_fence_before();
      warp_arrive(bar + 8 * C::B_SR);
#pragma unroll
      for (int c = 0; c < 32; ++c) {
        const float2 x = ffma2(make_float2(__uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1])), scale2, nl2);
        s[2 * c] = __float_as_uint(ex2(x.x));
        s[2 * c + 1] = __float_as_uint(ex2(x.y));
      }
      if (!wait.warp(C::B_PF + (g & 1), (g >> 1) & 1)) return;
      tc_fence_after();
      uint32_t d[64];
      tmem_ld64_sync(tP + 128 * (g & 1), d);
      const bool part = (w0 & w1) != ~0u;
      if (n == 1) {
        if (part) {                    // whatever hidden keys and values hold
#pragma unroll
          for (int c = 0; c < 64; ++c)
            if (!(((c < 32 ? w0 : w1) >> (c & 31)) & 1u)) s[c] = d[c] = 0u;
        }
        float2 sum = make_float2(0.f, 0.f);
#pragma unroll
        for (int c = 0; c < 32; ++c)
          sum = ffma2(make_float2(__uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1])),
                      make_float2(__uint_as_float(d[2 * c]), __uint_as_float(d[2 * c + 1])), sum);
        // two buffers: the next exchange's writers may be ahead of this one's readers
        float* x = red + (xn & 1) * 256;
        x[half * 128 + r] = sum.x + sum.y;
        warp_arrive(bar + 8 * C::B_XR);
        if (!wait.warp(C::B_XR, xn & 1)) return;
        nd = -(x[r] + x[128 + r]);
        ++xn;
        const int64_t row = row_of(w);
        if (half == 0 && row >= 0) p.delta[row] = -nd;
      }
      const float2 nd2 = make_float2(nd, nd);
      uint32_t pk[32];
#pragma unroll
      for (int c = 0; c < 32; ++c) {
        const float2 x = fmul2(make_float2(__uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1])),
                               fadd2(make_float2(__uint_as_float(d[2 * c]), __uint_as_float(d[2 * c + 1])), nd2));
        pk[c] = pack2<T>(x.x, x.y);
      }
      if (part || zero) {
        const uint32_t m0 = zero ? 0u : split_pairs(w0), m1 = zero ? 0u : split_pairs(w1);
#pragma unroll
        for (int c = 0; c < 32; ++c) pk[c] &= pair_mask(c < 16 ? m0 : m1, c & 15);
      }
      __syncwarp();
      tmem_st32(tP + 128 * (g & 1), pk);
      tmem_wait_st();
      tc_fence_before();
      warp_arrive(bar + 8 * (C::B_DS + (g & 1)));
      ++g;
    }
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreadsQ, 1) cross_dq_kernel(const __grid_constant__ CrossMaps m, const CrossParams p) {
  using C = CfgQ<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  if (sbase & 1023) {                  // the swizzle needs it; the declaration asks for it
    if (threadIdx.x == 0) atomicExch(&g_error, (int)DEV_TIMEOUT_PRODUCER);
    return;
  }
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + C::MISC_OFF);
  const uint32_t bar = sbase + C::BAR_OFF;
  const int warp = uniform(threadIdx.x >> 5);
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NBAR; ++i) mbar_init(bar + 8 * i, C::arrivals(i));
    misc[1] = 0;                       // abort word
    fence_mbar_init();
  }
  if (p.toks * p.group < 128) {        // rows that no copy fills are read by the products
    uint4* q = reinterpret_cast<uint4*>(smem);
    for (int i = threadIdx.x; i < 2 * C::TILE / 16; i += kThreadsQ) q[i] = make_uint4(0, 0, 0, 0);
    fence_async_smem();
  }
  if (warp == kWarpMma) {
    tmem_alloc(smem_u32(misc), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = misc[0];
  Waiter wait{bar, smem_u32(misc + 1), DEV_TIMEOUT_SOFTMAX, (uint32_t)p.timeout_ns};
  if (warp >= 8) {
    regs_shrink<kRegsOtherQ>();
    if (warp == kWarpProducer) {
      wait.code = DEV_TIMEOUT_PRODUCER;
      dq_producer<D>(m, p, sbase, wait);
    } else if (warp == kWarpMma) {
      wait.code = DEV_TIMEOUT_MMA;
      dq_mma<T, D>(p, sbase, uniform(tbase), wait);
    } else if (warp == kWarpAux) {
      if (p.scrub) dq_scrub<D>(p, sbase, wait);
    } else if (warp >= 12) {
      dq_store<T, D>(p, tbase, wait);
    }
  } else {
    regs_grow<kRegsElemQ>();
    dq_elementwise<T, D>(p, reinterpret_cast<float*>(smem + C::RED_OFF), tbase, wait);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  report(misc + 1);
  if (warp == kWarpMma) {
    __syncwarp();
    tmem_dealloc(tbase, 512);
  }
}

// delta = do . o of the queries of samples with more than one key tile (see dq_elementwise).  D / 8
// lanes per row and four rows per lane, so that a warp has 4 KB in flight; bound by the bytes of o
// and do.
template <typename T, int D>
__global__ void __launch_bounds__(256) cross_delta_kernel(const CrossParams p) {
  constexpr int LPR = D / 8, ROWS = 4 * 256 / LPR;     // rows of a block: heads of consecutive queries
  const int64_t first = (int64_t)blockIdx.x * ROWS + threadIdx.x / LPR, total = (int64_t)p.nq * p.heads;
  const int c = threadIdx.x % LPR * 8;
  for (int b = blockIdx.y; b < p.batch; b += gridDim.y) {
    if (cross_len(p, b) <= 128) continue;
    uint4 a[4] = {}, g[4] = {};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t r = first + i * (256 / LPR);
      if (r >= total) break;
      const uint32_t tok = p.div_h.div((uint32_t)r), h = (uint32_t)r - tok * p.heads;
      a[i] = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(p.o) + b * p.o_st[0] + tok * p.o_st[1] + h * p.o_st[2] + c));
      g[i] = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(p.d_o) + b * p.do_st[0] + tok * p.do_st[1] + h * p.do_st[2] + c));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const T* av = reinterpret_cast<const T*>(&a[i]);
      const T* gv = reinterpret_cast<const T*>(&g[i]);
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) s += to_f32(av[e]) * to_f32(gv[e]);
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      const int64_t r = first + i * (256 / LPR);
      if (c == 0 && r < total) {
        const uint32_t tok = p.div_h.div((uint32_t)r), h = (uint32_t)r - tok * p.heads;
        p.delta[((int64_t)b * p.heads + h) * p.nq + tok] = s;
      }
    }
  }
}

// ---------------------------------------------------------------------------------- dK, dV
// 384 threads: warp 10 brings each step's -lse log2(e) and -delta into shared memory.
// TMEM: S^T [0,128), dP^T [128,256), dV [256,256+D), dK [256+D,256+2D).  A warp that holds its dP^T
// in registers writes P^T and dS^T (16 bits, 32 columns each) over it, so that S^T is free as soon
// as it is read and the next S^T is made beside this step's exponentials; with P^T over S^T a step waits
// for its own dV product and the next S^T.  4 x 4,096 queries, 512 keys (436, 359 and none in three
// samples), 24 heads of 128: 132 us, 995 TF/s; tensor pipe about half busy, bound by a step's chain
// of product, exponentials, product.
template <int D>
struct CfgK {
  static constexpr int TILE = 128 * D * 2;
  static constexpr int NQ = D == 128 ? 3 : 4, NO = D == 128 ? 2 : 4, NA = D == 128 ? 2 : 4;
  static constexpr int V_OFF = TILE, Q_OFF = 2 * TILE, DO_OFF = Q_OFF + NQ * TILE;
  static constexpr int AUX_OFF = DO_OFF + NO * TILE;           // [NA][2][128] floats
  static constexpr int BAR_OFF = AUX_OFF + NA * 2 * 128 * 4;
  // full / empty of K, V, Q, dO and the row constants; S ready / read; dP ready; P and dS stored;
  // accumulators ready / read
  static constexpr int B_KF = 0, B_KE = 1, B_VF = 2, B_VE = 3, B_QF = 4, B_QE = B_QF + NQ, B_OF = B_QE + NQ, B_OE = B_OF + NO,
                       B_XF = B_OE + NO, B_XE = B_XF + NA, B_SF = B_XE + NA, B_SR = B_SF + 1, B_PF = B_SR + 1, B_DS = B_PF + 1,
                       B_AF = B_DS + 1, B_AE = B_AF + 1, B_DRAIN = B_AE + 1, NBAR = B_DRAIN + 1;
  static constexpr int MISC_OFF = BAR_OFF + NBAR * 8;
  static constexpr int SMEM = MISC_OFF + 16;
  static_assert(SMEM <= 227 * 1024, "shared memory per CTA exceeds 227 KB");
  static __device__ __forceinline__ uint32_t arrivals(int i) {
    return i == B_SR || i == B_DS || i == B_AE || (i >= B_XE && i < B_XE + NA) ? 8 : 1;   // 8 elementwise warps
  }
};
constexpr int kThreadsK = 384, kRegsLaunchK = 168, kRegsElemK = 208, kRegsOtherK = 80;
static_assert(256 * kRegsElemK + 128 * kRegsOtherK <= kThreadsK * kRegsLaunchK, "register split exceeds the launch allocation");

// Work item: key tiles fastest (neighbours in time share the query tiles in L2), then the split of
// the query tiles, then units.  Query tiles [q0, q1); none when every key is behind `len`.
struct ItemK {
  int b, hk, kt, split, len, q0, q1;
  __device__ __forceinline__ ItemK(const CrossParams& p, int it) {
    const uint32_t nkt = (p.ns + 127) >> 7;
    uint32_t i = p.div_kt.div(it), u = i;
    kt = it - i * nkt;
    split = 0;
    if (p.nsplit > 1) {
      u = p.div_split.div(i);
      split = i - u * p.nsplit;
    }
    b = p.div_kv.div(u);
    hk = u - b * p.kv_heads;
    len = cross_len(p, b);
    // (fewer than 2^24 query tiles, at most 64 splits: 32 bits hold the products)
    q0 = p.div_split.div((uint32_t)p.nqt * split);
    q1 = kt * 128 < len ? (int)p.div_split.div((uint32_t)p.nqt * (split + 1)) : q0;
  }
};

template <int D>
__device__ void dkv_producer(const CrossMaps& m, const CrossParams& p, uint32_t sbase, const Waiter& wait) {
  using C = CfgK<D>;
  const uint32_t bar = wait.bar;
  const int q_bytes = p.toks * p.group * D * 2;
  Ring<1> rk, rv;
  Ring<C::NQ> rq;
  Ring<C::NO> ro;
  bool ok = true;
  for (int it = blockIdx.x; ok && it < p.total; it += gridDim.x) {
    const ItemK w(p, it);
    const int q0 = uniform(w.q0), q1 = uniform(w.q1);
    for (int i = q0; i < q1; ++i) {
      if (i == q0) {
        if (!(ok = wait.warp(C::B_KE, rk.phase() ^ 1))) break;
        mbar_expect_tx_elect(bar + 8 * C::B_KF, C::TILE);
        load_tile<D>(sbase, &m.k, w.kt * 128, w.hk, w.b, bar + 8 * C::B_KF);
        ++rk.n;
      }
      const uint32_t qs = rq.slot(), os = ro.slot();
      if (!(ok = wait.warp(C::B_QE + qs, rq.phase() ^ 1))) break;
      mbar_expect_tx_elect(bar + 8 * (C::B_QF + qs), q_bytes);
      load_tile<D>(sbase + C::Q_OFF + qs * C::TILE, &m.q, i * p.toks, w.hk, w.b, bar + 8 * (C::B_QF + qs));
      ++rq.n;
      if (i == q0) {
        if (!(ok = wait.warp(C::B_VE, rv.phase() ^ 1))) break;
        mbar_expect_tx_elect(bar + 8 * C::B_VF, C::TILE);
        load_tile<D>(sbase + C::V_OFF, &m.v, w.kt * 128, w.hk, w.b, bar + 8 * C::B_VF);
        ++rv.n;
      }
      if (!(ok = wait.warp(C::B_OE + os, ro.phase() ^ 1))) break;
      mbar_expect_tx_elect(bar + 8 * (C::B_OF + os), q_bytes);
      load_tile<D>(sbase + C::DO_OFF + os * C::TILE, &m.d_o, i * p.toks, w.hk, w.b, bar + 8 * (C::B_OF + os));
      ++ro.n;
    }
  }
  if (!ok) settle();
}

// The rows' constants, four rows a lane, fetched two steps before they are stored: a step is shorter
// than a fetch from memory.
template <int D>
__device__ void dkv_rows(const CrossParams& p, float* aux, const Waiter& wait) {
  using C = CfgK<D>;
  struct Rows {
    float nl[4], nd[4];
  };
  const int lane = threadIdx.x & 31;
  auto fetch = [&](const ItemK& w, int i) {
    Rows v;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int r = lane + 32 * k, tr = row_tok(p, r), tok = i * p.toks + tr, h = w.hk * p.group + r - tr * p.group;
      v.nl[k] = neg_inf();
      v.nd[k] = 0.f;
      if (i < w.q1 && tr < p.toks && tok < p.nq) {
        const int64_t row = ((int64_t)w.b * p.heads + h) * p.nq + tok;
        v.nl[k] = __ldg(p.lse + row);
        v.nd[k] = __ldg(p.delta + row);
      }
    }
    return v;
  };
  Ring<C::NA> ra;
  for (int it = blockIdx.x; it < p.total; it += gridDim.x) {
    const ItemK w(p, it);
    Rows a = fetch(w, w.q0), b = fetch(w, w.q0 + 1);
    for (int i = w.q0; i < w.q1; ++i, ++ra.n) {
      const Rows c = fetch(w, i + 2);
      if (!wait.warp(C::B_XE + ra.slot(), ra.phase() ^ 1)) return;
      float* x = aux + ra.slot() * 256;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        x[lane + 32 * k] = neg_lse2(a.nl[k]);
        x[128 + lane + 32 * k] = -a.nd[k];
      }
      warp_arrive(wait.bar + 8 * (C::B_XF + ra.slot()));
      a = b;
      b = c;
    }
  }
}

template <typename T, int D>
__device__ void dkv_mma(const CrossParams& p, uint32_t sbase, uint32_t tbase, const Waiter& wait) {
  using C = CfgK<D>;
  const uint32_t bar = wait.bar, tV = tbase + 256, tK = tbase + 256 + D;
  Ring<1> rk;
  Ring<C::NQ> rq;
  Ring<C::NO> ro;
  uint32_t g = 0, items = 0;
  bool ok = true, pending = false, pfirst = false, plast = false;
  uint32_t pq = 0, po = 0, pitem = 0;
  for (int it = blockIdx.x; ok; it += gridDim.x) {      // (one round more: the last step's products)
    const bool end = it >= p.total;
    const ItemK w(p, end ? 0 : it);
    const int q0 = uniform(w.q0), q1 = end ? q0 + 1 : uniform(w.q1);
    for (int i = q0; i < q1; ++i) {
      const bool first = i == q0, last = i == q1 - 1;
      if (!end) {
        if (first && !(ok = wait.warp(C::B_KF, rk.phase()))) break;
        if (!(ok = wait.warp(C::B_QF + rq.slot(), rq.phase()))) break;
        if (g > 0 && !(ok = wait.warp(C::B_SR, (g - 1) & 1))) break;
        tc_fence_after();
        mma_scores<T, D>(tbase, sbase, sbase + C::Q_OFF + rq.slot() * C::TILE);
        mma_commit_elect(bar + 8 * C::B_SF);
        if (last) mma_commit_elect(bar + 8 * C::B_KE);
      }
      if (pending) {                   // dV += P^T dO and dK += dS^T Q of step g - 1
        if (!(ok = wait.warp(C::B_DS, (g - 1) & 1))) break;
        if (pfirst && pitem > 0 && !(ok = wait.warp(C::B_AE, (pitem - 1) & 1))) break;
        tc_fence_after();
        mma_accum<T, D>(tV, tbase + 128, sbase + C::DO_OFF + po * C::TILE, pfirst);
        mma_commit_elect(bar + 8 * (C::B_OE + po));
        mma_accum<T, D>(tK, tbase + 160, sbase + C::Q_OFF + pq * C::TILE, pfirst);
        mma_commit_elect(bar + 8 * (C::B_QE + pq));
        if (plast) mma_commit_elect(bar + 8 * C::B_AF);
      }
      if (end) return;
      if (first && !(ok = wait.warp(C::B_VF, rk.phase()))) break;
      if (!(ok = wait.warp(C::B_OF + ro.slot(), ro.phase()))) break;
      tc_fence_after();
      // (overwrites P^T and dS^T of step g - 1, which the products issued before have read)
      mma_scores<T, D>(tbase + 128, sbase + C::V_OFF, sbase + C::DO_OFF + ro.slot() * C::TILE);
      mma_commit_elect(bar + 8 * C::B_PF);
      if (last) mma_commit_elect(bar + 8 * C::B_VE);
      pending = true;
      pfirst = first;
      plast = last;
      pq = rq.slot();
      po = ro.slot();
      pitem = items;
      ++rq.n;
      ++ro.n;
      ++g;
    }
    if (q1 > q0) {
      ++rk.n;
      ++items;
    }
  }
  mma_commit_elect(bar + 8 * C::B_DRAIN);
  wait.drain(C::B_DRAIN, 0, &g_error);
}

template <typename T, int D>
__device__ void dkv_elementwise(const CrossParams& p, const float* aux, uint32_t tbase, const Waiter& wait) {
  using C = CfgK<D>;
  const uint32_t bar = wait.bar;
  const int half = threadIdx.x >> 7, r = threadIdx.x & 127;
  const uint32_t lane_off = (uint32_t)((threadIdx.x >> 5) & 3) * 32u << 16;
  const uint32_t tS = tbase + lane_off + half * 64, tP = tS + 128, tAcc = tbase + lane_off + 256 + half * (D / 2);
  const float2 scale2 = make_float2(p.scale_log2, p.scale_log2);
  uint32_t g = 0, items = 0;
  Ring<C::NA> ra;
  T *pend_k = nullptr, *pend_v = nullptr;
  float* pend_part = nullptr;
  bool pend_vis = false;
  for (int it = blockIdx.x;; it += gridDim.x) {
    const bool end = it >= p.total;    // one round more: the last item's accumulators
    if (end && items == 0) return;
    const ItemK w(p, end ? 0 : it);
    const int key = w.kt * 128 + r;
    const uint4 words = cross_words(p, w.b, w.kt, w.len);
    const bool vis = (word_of(words, r >> 5) >> (r & 31)) & 1u;
    T* out_k = static_cast<T*>(p.out[0]) + w.b * p.out_st[0][0] + key * p.out_st[0][1] + w.hk * p.out_st[0][2] + half * (D / 2);
    T* out_v = static_cast<T*>(p.out[1]) + w.b * p.out_st[1][0] + key * p.out_st[1][1] + w.hk * p.out_st[1][2] + half * (D / 2);
    if (!end && !p.part && key < p.ns && !vis) {       // (with partials the join writes these)
      zero_half<T, D>(out_k);
      zero_half<T, D>(out_v);
    }
    if (!end && w.q1 == w.q0) continue;
    const bool zero = w.len == 1 || (p.single && __ldg(p.single + w.b));
    for (int i = w.q0; i < (end ? w.q0 + 1 : w.q1); ++i) {
      if (!end) {
        uint32_t s[64];
        const float4* nl = reinterpret_cast<const float4*>(aux + ra.slot() * 256 + half * 64);
        if (!wait.warp(C::B_XF + ra.slot(), ra.phase())) return;
        if (!wait.warp(C::B_SF, g & 1)) return;
        tc_fence_after();
        tmem_ld64_sync(tS, s);
        tc_fence_before();
        warp_arrive(bar + 8 * C::B_SR);
        uint32_t pk[32], dk[32];
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const float4 l = nl[c];
          const float2 a = ffma2(make_float2(__uint_as_float(s[4 * c]), __uint_as_float(s[4 * c + 1])), scale2, make_float2(l.x, l.y));
          const float2 b = ffma2(make_float2(__uint_as_float(s[4 * c + 2]), __uint_as_float(s[4 * c + 3])), scale2, make_float2(l.z, l.w));
          s[4 * c] = __float_as_uint(ex2(a.x));
          s[4 * c + 1] = __float_as_uint(ex2(a.y));
          s[4 * c + 2] = __float_as_uint(ex2(b.x));
          s[4 * c + 3] = __float_as_uint(ex2(b.y));
          pk[2 * c] = vis ? pack2<T>(__uint_as_float(s[4 * c]), __uint_as_float(s[4 * c + 1])) : 0u;
          pk[2 * c + 1] = vis ? pack2<T>(__uint_as_float(s[4 * c + 2]), __uint_as_float(s[4 * c + 3])) : 0u;
        }
        if (!wait.warp(C::B_PF, g & 1)) return;
        tc_fence_after();
        const float4* nd = nl + 32;
        uint32_t d[64];
        tmem_ld64_sync(tP, d);
        tmem_st32(tP, pk);
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const float4 l = nd[c];
          const int k = 4 * c;
          const float2 a = fmul2(make_float2(__uint_as_float(s[k]), __uint_as_float(s[k + 1])),
                                 fadd2(make_float2(__uint_as_float(d[k]), __uint_as_float(d[k + 1])), make_float2(l.x, l.y)));
          const float2 b = fmul2(make_float2(__uint_as_float(s[k + 2]), __uint_as_float(s[k + 3])),
                                 fadd2(make_float2(__uint_as_float(d[k + 2]), __uint_as_float(d[k + 3])), make_float2(l.z, l.w)));
          dk[2 * c] = vis && !zero ? pack2<T>(a.x, a.y) : 0u;
          dk[2 * c + 1] = vis && !zero ? pack2<T>(b.x, b.y) : 0u;
        }
        __syncwarp();
        tmem_st32(tP + 32, dk);
        tmem_wait_st();
        tc_fence_before();
        warp_arrive(bar + 8 * C::B_DS);
        warp_arrive(bar + 8 * (C::B_XE + ra.slot()));
        ++ra.n;
        ++g;
      }
      // the accumulators of the item before: dV, dK rows, or their fp32 partials [2][128][D]
      if (i == w.q0 && items > 0) {
        if (!wait.warp(C::B_AF, (items - 1) & 1)) return;
        tc_fence_after();
        if (p.part) {
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int ch = 0; ch < D / 64; ++ch) {
              uint32_t o[32];
              __syncwarp();
              tmem_ld32_sync(tAcc + t * D + ch * 32, o);
              if (!pend_vis) continue;
              uint4* dst = reinterpret_cast<uint4*>(pend_part + t * 128 * D + ch * 32);
#pragma unroll
              for (int q = 0; q < 8; ++q) dst[q] = make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
            }
        } else {
          store_piece<T, D / 2>(tAcc, pend_vis ? pend_v : nullptr, 1.0f);
          store_piece<T, D / 2>(tAcc + D, pend_vis ? pend_k : nullptr, p.scale);
        }
        tc_fence_before();
        warp_arrive(bar + 8 * C::B_AE);
      }
    }
    if (end) return;
    ++items;
    pend_k = out_k;
    pend_v = out_v;
    pend_vis = vis;
    if (p.part) pend_part = p.part + ((int64_t)it * 2 * 128 + r) * D + half * (D / 2);
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreadsK, 1) cross_dkv_kernel(const __grid_constant__ CrossMaps m, const CrossParams p) {
  using C = CfgK<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  if (sbase & 1023) {
    if (threadIdx.x == 0) atomicExch(&g_error, (int)DEV_TIMEOUT_PRODUCER);
    return;
  }
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + C::MISC_OFF);
  const uint32_t bar = sbase + C::BAR_OFF;
  float* aux = reinterpret_cast<float*>(smem + C::AUX_OFF);
  const int warp = uniform(threadIdx.x >> 5);
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NBAR; ++i) mbar_init(bar + 8 * i, C::arrivals(i));
    misc[1] = 0;                       // abort word
    fence_mbar_init();
  }
  if (p.toks * p.group < 128) {
    uint4* q = reinterpret_cast<uint4*>(smem + C::Q_OFF);
    for (int i = threadIdx.x; i < (C::NQ + C::NO) * C::TILE / 16; i += kThreadsK) q[i] = make_uint4(0, 0, 0, 0);
    fence_async_smem();
  }
  if (warp == kWarpMma) {
    tmem_alloc(smem_u32(misc), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = misc[0];
  Waiter wait{bar, smem_u32(misc + 1), DEV_TIMEOUT_SOFTMAX, (uint32_t)p.timeout_ns};
  if (warp >= 8) {
    regs_shrink<kRegsOtherK>();
    if (warp == kWarpProducer) {
      wait.code = DEV_TIMEOUT_PRODUCER;
      dkv_producer<D>(m, p, sbase, wait);
    } else if (warp == kWarpMma) {
      wait.code = DEV_TIMEOUT_MMA;
      dkv_mma<T, D>(p, sbase, uniform(tbase), wait);
    } else if (warp == kWarpAux) {
      dkv_rows<D>(p, aux, wait);
    }
  } else {
    regs_grow<kRegsElemK>();
    dkv_elementwise<T, D>(p, aux, tbase, wait);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  report(misc + 1);
  if (warp == kWarpMma) {
    __syncwarp();
    tmem_dealloc(tbase, 512);
  }
}

// dK and dV of every key from the splits' partials, added in split order (nsplit = 0: no queries,
// zeros).  One warp per key and tensor.
template <typename T, int D>
__global__ void __launch_bounds__(256) cross_dkv_join_kernel(const CrossParams p) {
  const int64_t r = ((int64_t)blockIdx.x * 8 + (threadIdx.x >> 5)) >> 1;
  const int t = (threadIdx.x >> 5) & 1, lane = threadIdx.x & 31;     // t: 0 dV, 1 dK
  if (r >= (int64_t)p.units * p.ns) return;
  const int key = (int)(r % p.ns), u = (int)(r / p.ns), b = u / p.kv_heads, hk = u - b * p.kv_heads;
  const int nkt = (p.ns + 127) >> 7, kt = key >> 7;
  const uint4 words = cross_words(p, b, kt, cross_len(p, b));
  const bool vis = (word_of(words, (key >> 5) & 3) >> (key & 31)) & 1u;
  float s[D / 32] = {};
  if (vis)
    for (int i = 0; i < p.nsplit; ++i) {
      float v[D / 32];
      load_f32<float, D / 32>(p.part + ((((int64_t)u * p.nsplit + i) * nkt + kt) * 256 + t * 128 + (key & 127)) * D + lane * (D / 32), v);
#pragma unroll
      for (int c = 0; c < D / 32; ++c) s[c] += v[c];
    }
#pragma unroll
  for (int c = 0; c < D / 32; ++c) s[c] *= t ? p.scale : 1.0f;
  const int o = t ? 0 : 1;
  store_f32<T, D / 32>(static_cast<T*>(p.out[o]) + b * p.out_st[o][0] + key * p.out_st[o][1] + hk * p.out_st[o][2] + lane * (D / 32), s);
}

// Launches `kernel`, whose register split is sound only if it has `regs` registers at launch.
template <typename Tag, typename K>
cudaError_t launch(K kernel, int regs, int threads, int smem, const CrossMaps& m, const CrossParams& p, int grid, cudaStream_t s) {
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
      cudaFuncAttributes fa;
      if ((e = cudaFuncGetAttributes(&fa, kernel)) != cudaSuccess) return e;
      if (fa.numRegs != regs) return cudaErrorInvalidConfiguration;
      if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess) return e;
      attr_set[dev] = true;
    }
  }
  kernel<<<grid, threads, smem, s>>>(m, p);
  return cudaGetLastError();
}

template <typename T, int D> struct TagQ {};
template <typename T, int D> struct TagK {};

template <typename T, int D>
cudaError_t launch_dq(const CrossMaps& m, const CrossParams& p, int grid, cudaStream_t s) {
  if (p.ns > 128) {
    constexpr int kRows = 4 * 256 / (D / 8);
    const dim3 blocks((unsigned)(((int64_t)p.nq * p.heads + kRows - 1) / kRows), std::min(p.batch, 65535));
    cross_delta_kernel<T, D><<<blocks, 256, 0, s>>>(p);
  }
  return launch<TagQ<T, D>>(cross_dq_kernel<T, D>, kRegsLaunchQ, kThreadsQ, CfgQ<D>::SMEM, m, p, grid, s);
}
template <typename T, int D>
cudaError_t launch_dkv(const CrossMaps& m, const CrossParams& p, int grid, cudaStream_t s) {
  if (p.total > 0) {
    const cudaError_t e = launch<TagK<T, D>>(cross_dkv_kernel<T, D>, kRegsLaunchK, kThreadsK, CfgK<D>::SMEM, m, p, grid, s);
    if (e != cudaSuccess || p.nsplit == 1) return e;
  }
  cross_dkv_join_kernel<T, D><<<(unsigned)(((int64_t)p.units * p.ns * 2 + 7) / 8), 256, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cross_dq(const CrossMaps& m, const CrossParams& p, int dtype, int D, int grid, cudaStream_t s) {
  if (dtype == 0) return D == 128 ? launch_dq<__nv_bfloat16, 128>(m, p, grid, s) : launch_dq<__nv_bfloat16, 64>(m, p, grid, s);
  return D == 128 ? launch_dq<__half, 128>(m, p, grid, s) : launch_dq<__half, 64>(m, p, grid, s);
}

cudaError_t launch_cross_dkv(const CrossMaps& m, const CrossParams& p, int dtype, int D, int grid, cudaStream_t s) {
  if (dtype == 0) return D == 128 ? launch_dkv<__nv_bfloat16, 128>(m, p, grid, s) : launch_dkv<__nv_bfloat16, 64>(m, p, grid, s);
  return D == 128 ? launch_dkv<__half, 128>(m, p, grid, s) : launch_dkv<__half, 64>(m, p, grid, s);
}

cudaError_t cross_bwd_status(int* code, cudaStream_t s) { return read_clear_error(&g_error, code, s); }

}  // namespace ug
