// Cross attention forward for sm_100a (tcgen05 + TMEM + TMA): o = softmax(scale q k^T) v with the
// running maximum and sum of each row, and the row's log-sum-exp.
//
// CTA organisation (one persistent CTA per SM, 384 threads = 3 warpgroups), the same as the joint
// attention's:
//   warps 0-3, 4-7  softmax of query tile 0 / 1 of the item (thread = row = TMEM lane)
//   warp  8         producer: TMA loads of Q (per item) and of K, V tiles in stages
//   warp  9         MMA issuer: S = Q K^T and O += P V (P from TMEM); owns TMEM
//   warp  10        scrubber: zeroes the V rows of hidden keys, which may hold NaN (0 * NaN)
// TMEM (512 columns): S0 [0,128), S1 [128,256), O0 [256,256+D), O1 [256+D, 256+2D); P (16 bits,
// packed in pairs) overwrites the first 64 columns of its S block.
// Stage j of an item with n key tiles holds V(j-1) (j > 0) and K(j) (j < n), what step j reads.
#include <cstdint>
#include <mutex>

#include "cross.cuh"

namespace ug {
namespace {

__device__ int g_error;                // first wait that ran out since the last status read

template <int D>
struct Cfg {
  static constexpr int BOXES = D / 64;
  static constexpr int BOX_BYTES = 128 * 64 * 2;
  static constexpr int TILE_BYTES = 128 * D * 2;
  static constexpr int NS = D == 128 ? 4 : 8;      // tile slots
  static constexpr int NSTG = NS / 2;              // stages in flight (two tiles each)
  static constexpr int KV_OFF = 2 * TILE_BYTES;
  static constexpr int OUT_OFF = KV_OFF + NS * TILE_BYTES;      // 8 warps x 32 rows x 128 bytes
  static constexpr int BAR_OFF = OUT_OFF + 8 * 4096;
  // Q full / empty, stage full / scrubbed / empty, S ready, P ready, O ready (per query tile), drain
  static constexpr int B_QF = 0, B_QE = 1, B_KVF = 2, B_KVS = B_KVF + NSTG, B_KVE = B_KVS + NSTG,
                       B_SF = B_KVE + NSTG, B_PF = B_SF + 2, B_OF = B_PF + 2, B_DRAIN = B_OF + 2,
                       NBAR = B_DRAIN + 1;
  static constexpr int MISC_OFF = BAR_OFF + NBAR * 8;           // TMEM base, abort flag
  static constexpr int SMEM_BYTES = MISC_OFF + 16 + 1024;       // + slack for 1024-byte alignment
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory per CTA exceeds 227 KB");
  static __device__ __forceinline__ uint32_t v_slot(uint32_t g) { return 2 * g; }
  static __device__ __forceinline__ uint32_t k_slot(uint32_t g) { return 2 * g + 1; }
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr uint32_t O_COL = 256;
};

constexpr int kThreads = 384;
constexpr int kRegsLaunch = 168;      // per thread at launch: 65536 / 384, rounded down to 8
constexpr int kRegsSoftmax = 224;
constexpr int kRegsControl = 56;
static_assert(2 * 128 * kRegsSoftmax + 128 * kRegsControl <= kThreads * kRegsLaunch,
              "register split exceeds the launch allocation");
constexpr int kWarpProducer = 8, kWarpMma = 9, kWarpScrub = 10;
constexpr uint64_t kDrainNs = 50ull * 1000 * 1000;   // bounded drain on the abort path

// Work item `it`: split fastest, then query tiles, then units, so that neighbours in time share
// keys and values in L2.
struct Item {
  int b, hk, qt0, ntile, split, len, k0, k1;
  __device__ __forceinline__ Item(const CrossParams& p, int it) {
    uint32_t i = it, u;
    split = 0;
    if (p.nsplit > 1) {
      i = p.div_split.div(it);
      split = it - i * p.nsplit;
    }
    u = p.div_q.div(i);
    qt0 = (i - u * p.nitem_q) * p.per_item;
    b = p.div_kv.div(u);
    hk = u - b * p.kv_heads;
    ntile = min(p.per_item, p.nqt - qt0);
    len = cross_len(p, b);
    split_range(len, split, p.nsplit, k0, k1);
  }
};

template <int D>
__device__ void producer_role(const CrossMaps& m, const CrossParams& p, uint32_t sbase, volatile int* abort_flag) {
  using C = Cfg<D>;
  const uint32_t sKV = sbase + C::KV_OFF, bar = sbase + C::BAR_OFF;
  const int q_bytes = p.toks * p.group * D * 2;
  uint32_t st = 0, qi = 0;
  bool ok = true;
  auto wait = [&](int b, uint32_t par) {
    return mbar_wait(bar + 8 * b, par, abort_flag, &g_error, DEV_TIMEOUT_PRODUCER, p.timeout_ns);
  };
  for (int it = blockIdx.x; ok && it < p.total; it += gridDim.x) {
    const Item w(p, it);
    const int n = w.k1 - w.k0;
    if (n == 0) continue;
    if (!wait(C::B_QE, (qi & 1) ^ 1)) { ok = false; break; }
    mbar_expect_tx(bar + 8 * C::B_QF, w.ntile * q_bytes);
    for (int t = 0; t < w.ntile; ++t)
#pragma unroll
      for (int bx = 0; bx < C::BOXES; ++bx)
        tma_load_5d(sbase + t * C::TILE_BYTES + bx * C::BOX_BYTES, &m.q, bx * 64, 0, (w.qt0 + t) * p.toks, w.hk, w.b,
                    bar + 8 * C::B_QF);
    ++qi;
    for (int j = 0; j <= n; ++j) {
      const uint32_t g = st % C::NSTG, ph = (st / C::NSTG) & 1;
      if (!wait(C::B_KVE + g, ph ^ 1)) { ok = false; break; }
      const uint32_t fb = bar + 8 * (C::B_KVF + g);
      mbar_expect_tx(fb, (j > 0 ? C::TILE_BYTES : 0) + (j < n ? C::TILE_BYTES : 0));
      ++st;
#pragma unroll
      for (int bx = 0; bx < C::BOXES; ++bx) {
        if (j > 0)
          tma_load_5d(sKV + C::v_slot(g) * C::TILE_BYTES + bx * C::BOX_BYTES, &m.v, bx * 64, 0,
                      (w.k0 + j - 1) * 128, w.hk, w.b, fb);
        if (j < n)
          tma_load_5d(sKV + C::k_slot(g) * C::TILE_BYTES + bx * C::BOX_BYTES, &m.k, bx * 64, 0, (w.k0 + j) * 128,
                      w.hk, w.b, fb);
      }
    }
  }
  if (!ok) {
    // wait (bounded) for the copies in flight: none may land after this CTA exits
    for (uint32_t g = st >= (uint32_t)C::NSTG ? st - C::NSTG : 0; g < st; ++g)
      mbar_wait(bar + 8 * (C::B_KVF + g % C::NSTG), (g / C::NSTG) & 1, nullptr, &g_error, DEV_TIMEOUT_DRAIN, kDrainNs);
    if (qi > 0) mbar_wait(bar + 8 * C::B_QF, (qi - 1) & 1, nullptr, &g_error, DEV_TIMEOUT_DRAIN, kDrainNs);
  }
}

// One warp, only when hidden keys exist below ns: stage by stage, zeroes the hidden rows of V
// and passes the stage on.
template <int D>
__device__ void scrub_role(const CrossParams& p, uint32_t sbase, volatile int* abort_flag) {
  using C = Cfg<D>;
  const uint32_t sKV = sbase + C::KV_OFF, bar = sbase + C::BAR_OFF;
  uint32_t st = 0;
  for (int it = blockIdx.x; it < p.total; it += gridDim.x) {
    const Item w(p, it);
    const int n = w.k1 - w.k0;
    if (n == 0) continue;
    for (int j = 0; j <= n; ++j, ++st) {
      const uint32_t g = st % C::NSTG;
      const uint4 vis = j > 0 ? cross_words(p, w.b, w.k0 + j - 1, w.len) : make_uint4(~0u, ~0u, ~0u, ~0u);
      const bool ok = mbar_wait(bar + 8 * (C::B_KVF + g), (st / C::NSTG) & 1, abort_flag, &g_error,
                                DEV_TIMEOUT_PRODUCER, p.timeout_ns);
      if (!__all_sync(0xffffffffu, ok)) return;
      if (!all_visible(vis)) {
        scrub_rows<D>(sKV + C::v_slot(g) * C::TILE_BYTES, C::BOX_BYTES, vis, 0, 128);
        fence_async_smem();
      }
      __syncwarp();
      if ((threadIdx.x & 31) == 0) mbar_arrive(bar + 8 * (C::B_KVS + g));
    }
  }
}

template <typename T, int D>
__device__ void mma_role(const CrossParams& p, uint32_t sbase, uint32_t tbase, volatile int* abort_flag) {
  using C = Cfg<D>;
  constexpr uint32_t hi = desc_hi_sw128(1024);
  constexpr uint32_t idS = idesc_half<T>(128, 128, 0), idO = idesc_half<T>(128, D, 1);
  const uint32_t sKV = sbase + C::KV_OFF, bar = sbase + C::BAR_OFF;
  const int ready = p.scrub ? C::B_KVS : C::B_KVF;
  uint32_t st = 0, qi = 0, pc[2] = {0, 0};
  bool ok = true;
  auto wait = [&](int b, uint32_t par) {
    return __all_sync(0xffffffffu, mbar_wait(bar + 8 * b, par, abort_flag, &g_error, DEV_TIMEOUT_MMA, p.timeout_ns));
  };
  for (int it = blockIdx.x; ok && it < p.total; it += gridDim.x) {
    const Item w(p, it);
    const int n = uniform(w.k1 - w.k0), ntile = uniform(w.ntile);
    if (n == 0) continue;
    if (!wait(C::B_QF, qi & 1)) { ok = false; break; }
    ++qi;
    tc_fence_after();
    for (int j = 0; j <= n && ok; ++j) {
      const uint32_t g = st % C::NSTG;
      if (!wait(ready + g, (st / C::NSTG) & 1)) { ok = false; break; }
      tc_fence_after();
      const uint32_t vlo = desc_lo(sKV + C::v_slot(g) * C::TILE_BYTES, C::BOX_BYTES);
      const uint32_t klo = desc_lo(sKV + C::k_slot(g) * C::TILE_BYTES, 16);
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        if (t >= ntile) break;
        if (j > 0) {
          if (!wait(C::B_PF + t, pc[t] & 1)) { ok = false; break; }
          ++pc[t];
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_ts_elect(tbase + C::O_COL + D * t, tbase + 128 * t + kk * 8, vlo + kk * (2048 >> 4), hi, idO,
                     (j > 1 || kk > 0) ? 1u : 0u);
        }
        if (j < n) {
          const uint32_t qlo = desc_lo(sbase + t * C::TILE_BYTES, 16);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = ((kk / 4) * C::BOX_BYTES + (kk % 4) * 32) >> 4;
            mma_ss_elect(tbase + 128 * t, qlo + off, klo + off, hi, idS, kk > 0 ? 1u : 0u);
          }
          mma_commit_elect(bar + 8 * (C::B_SF + t));
        } else {
          mma_commit_elect(bar + 8 * (C::B_OF + t));
        }
      }
      if (!ok) break;
      mma_commit_elect(bar + 8 * (C::B_KVE + g));
      if (j == n - 1) mma_commit_elect(bar + 8 * C::B_QE);
      ++st;
    }
  }
  if (!ok) {
    mma_commit_elect(bar + 8 * C::B_DRAIN);
    mbar_wait(bar + 8 * C::B_DRAIN, 0, nullptr, &g_error, DEV_TIMEOUT_DRAIN, kDrainNs);
  }
}

// Exponentials of one S row at the running max mu (log2 units): the pair (s[2c], s[2c+1]) is
// replaced by its packed 16-bit P in s[c] (the tensor core's operand type; the row sum adds the
// unrounded fp32 values).  Returns the row sum of this tile's P.
template <typename T>
__device__ __forceinline__ float exp_row(uint32_t (&s)[128], float scale, float mu) {
  const float2 scale2 = make_float2(scale, scale), nmu2 = make_float2(-mu, -mu);
  float2 ls[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) ls[i] = make_float2(0.f, 0.f);
#pragma unroll
  for (int c2 = 0; c2 < 64; ++c2) {
    float2 x = ffma2(make_float2(__uint_as_float(s[2 * c2]), __uint_as_float(s[2 * c2 + 1])), scale2, nmu2);
    x.x = ex2(x.x);
    x.y = ex2(x.y);
    ls[c2 & 3] = fadd2(ls[c2 & 3], x);
    s[c2] = pack2<T>(x.x, x.y);
  }
  const float2 l2 = fadd2(fadd2(ls[0], ls[1]), fadd2(ls[2], ls[3]));
  return l2.x + l2.y;
}

__device__ __forceinline__ void mask_row(uint32_t (&s)[128], const uint4& w) {
#pragma unroll
  for (int c = 0; c < 128; ++c)
    if (!((word_of(w, c >> 5) >> (c & 31)) & 1u)) s[c] = 0xff800000u;   // -inf
}

// Multiplies the O accumulator row (TMEM) by f, 32 columns at a time.
template <int D>
__device__ __forceinline__ void rescale_o(uint32_t tO, float f) {
#pragma unroll 1
  for (int ch = 0; ch < D / 32; ++ch) {
    uint32_t o[32];
    tmem_ld32_sync(tO + ch * 32, o);
#pragma unroll
    for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
    tmem_st32(tO + ch * 32, o);
  }
}

template <typename T, int D>
__device__ void softmax_role(const CrossParams& p, uint8_t* smem, uint32_t sbase, uint32_t tbase, volatile int* abort_flag) {
  using C = Cfg<D>;
  const uint32_t bar = sbase + C::BAR_OFF;
  const int t = threadIdx.x >> 7, r = threadIdx.x & 127;
  const uint32_t lane_off = (uint32_t)((threadIdx.x >> 5) & 3) * 32u << 16;
  const uint32_t tS = tbase + lane_off + (uint32_t)(t * 128);
  const uint32_t tO = tbase + lane_off + C::O_COL + (uint32_t)(t * D);
  const float scale = p.scale_log2;
  const int tok_r = row_tok(p, r), g_r = r - tok_r * p.group;
  uint8_t* out = smem + C::OUT_OFF + (threadIdx.x >> 5) * 4096;
  uint32_t sc = 0, oc = 0;
  for (int it = blockIdx.x; it < p.total; it += gridDim.x) {
    const Item w(p, it);
    if (t >= w.ntile) continue;
    const int n = w.k1 - w.k0, qt = w.qt0 + t;
    const int tok = qt * p.toks + tok_r, h = w.hk * p.group + g_r;
    const bool real = tok_r < p.toks && tok < p.nq;
    float m = neg_inf(), lsum = 0.f;
    for (int j = 0; j < n; ++j) {
      const uint4 vis = cross_words(p, w.b, w.k0 + j, w.len);
      const bool part_tile = !all_visible(vis);
      const bool ok = mbar_wait(bar + 8 * (C::B_SF + t), sc & 1, abort_flag, &g_error, DEV_TIMEOUT_SOFTMAX, p.timeout_ns);
      if (!__all_sync(0xffffffffu, ok)) return;
      ++sc;
      tc_fence_after();
      uint32_t s[128];
      tmem_ld128_sync(tS, s);
      if (part_tile) mask_row(s, vis);
      if (__any_sync(0xffffffffu, m == neg_inf())) {
        // a row without a running max yet: take the tile's first
        float mx4[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) mx4[i] = neg_inf();
#pragma unroll
        for (int c = 0; c < 128; c += 8) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            mx4[i] = fmax3(mx4[i], __uint_as_float(s[c + 2 * i]), __uint_as_float(s[c + 2 * i + 1]));
        }
        const float mx = fmax3(fmaxf(mx4[0], mx4[1]), mx4[2], mx4[3]);
        const float mnew = fmaxf(m, mx * scale);
        // lazy rescale: a running max stays unless it grew by more than 2^8 (the division by the
        // row sum makes the result exact for any max)
        const bool need = m != neg_inf() && mnew > m + 8.0f;
        if (__any_sync(0xffffffffu, need)) {
          const float f = need ? ex2(m - mnew) : 1.0f;
          if (need) lsum *= f;
          __syncwarp();
          rescale_o<D>(tO, f);
        }
        if (m == neg_inf() || need) m = mnew;
        lsum += exp_row<T>(s, scale, m == neg_inf() ? 0.f : m);
      } else {
        // every row has a running max: take the exponentials at it without a tile max; a tile
        // sum above 2^12 (fp16 P still holds it) is redone at the exact max
        float part = exp_row<T>(s, scale, m);
        if (__any_sync(0xffffffffu, !(part <= 4096.0f))) {
          float mx = neg_inf();
#pragma unroll 1
          for (int ch = 0; ch < 4; ++ch) {
            uint32_t c32[32];
            tmem_ld32_sync(tS + ch * 32, c32);
            const uint32_t mwc = word_of(vis, ch);
#pragma unroll
            for (int c = 0; c < 32; c += 2) {
              const float a = ((mwc >> c) & 1u) ? __uint_as_float(c32[c]) : neg_inf();
              const float b = ((mwc >> (c + 1)) & 1u) ? __uint_as_float(c32[c + 1]) : neg_inf();
              mx = fmax3(mx, a, b);
            }
          }
          const float mnew = fmaxf(m, mx * scale);
          const float f = ex2(m - mnew);
          lsum *= f;
          m = mnew;
          __syncwarp();
          rescale_o<D>(tO, f);
          tmem_ld128_sync(tS, s);
          if (part_tile) mask_row(s, vis);
          part = exp_row<T>(s, scale, m);
        }
        lsum += part;
      }
      __syncwarp();
      tmem_st64(tS, s);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if ((threadIdx.x & 31) == 0) mbar_arrive(bar + 8 * (C::B_PF + t));
    }
    if (n > 0) {
      const bool ok = mbar_wait(bar + 8 * (C::B_OF + t), oc & 1, abort_flag, &g_error, DEV_TIMEOUT_SOFTMAX, p.timeout_ns);
      if (!__all_sync(0xffffffffu, ok)) return;
      ++oc;
      tc_fence_after();
      __syncwarp();
    }
    const float inv = lsum > 0.f ? 1.0f / lsum : (lsum == 0.f ? 0.f : lsum);   // NaN stays NaN
    const float lse2 = lsum == 0.f ? neg_inf() : m + log2f(lsum);
    float* prow = nullptr;
    T* orow = nullptr;
    if (real) {
      if (p.part) {
        // split items: [unit][query tile][split] blocks of part_rows x (D floats), then the
        // log-sum-exps (base 2)
        const int64_t blk = ((int64_t)(w.b * p.kv_heads + w.hk) * p.nqt + qt) * p.nsplit + w.split;
        prow = p.part + blk * p.part_rows * D + (int64_t)r * D;
        p.part[(int64_t)p.units * p.nqt * p.nsplit * p.part_rows * D + blk * p.part_rows + r] = lse2;
      } else {
        orow = static_cast<T*>(p.out[0]) + w.b * p.out_st[0][0] + tok * p.out_st[0][1] + h * p.out_st[0][2];
        if (p.lse) p.lse[((int64_t)w.b * p.heads + h) * p.nq + tok] = lse2 * 0.6931471805599453f;
      }
    }
    if (n == 0) {
      // nothing visible: zeros (a split partial is marked by its log-sum-exp alone)
      if (orow) {
#pragma unroll
        for (int c = 0; c < D / 8; ++c) reinterpret_cast<uint4*>(orow)[c] = make_uint4(0, 0, 0, 0);
      }
      continue;
    }
    // a row without a visible key has O = 0 products of P = 0: inv = 0 keeps it zero
    if (p.part) {
#pragma unroll
      for (int ch = 0; ch < D / 32; ++ch) {
        uint32_t o[32];
        __syncwarp();
        tmem_ld32_sync(tO + ch * 32, o);               // warp-wide: every lane loads
        if (!prow) continue;
        float4* dst = reinterpret_cast<float4*>(prow + ch * 32);
#pragma unroll
        for (int q = 0; q < 8; ++q)
          dst[q] = make_float4(__uint_as_float(o[4 * q + 0]) * inv, __uint_as_float(o[4 * q + 1]) * inv,
                               __uint_as_float(o[4 * q + 2]) * inv, __uint_as_float(o[4 * q + 3]) * inv);
      }
    } else {
      store_rows<T, D>(tO, out, orow, inv);
    }
    tc_fence_before();
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1)
    cross_fwd_kernel(const __grid_constant__ CrossMaps m, const CrossParams p) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar = sbase + C::BAR_OFF;
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + C::MISC_OFF);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 1);
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NBAR; ++i)
      mbar_init(bar + 8 * i, i == C::B_PF || i == C::B_PF + 1 ? 4 : 1);   // P: one arrive per softmax warp
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (p.toks * p.group < 128) {
    // query rows that no copy fills are read by the products: keep them zero
    uint4* q = reinterpret_cast<uint4*>(smem);
    for (int i = threadIdx.x; i < 2 * C::TILE_BYTES / 16; i += kThreads) q[i] = make_uint4(0, 0, 0, 0);
    fence_async_smem();
  }
  if (warp == kWarpMma) {
    tmem_alloc(smem_u32(misc), C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = misc[0];
  if (warp >= 8) {
    regs_shrink<kRegsControl>();
    if (warp == kWarpProducer) {
      if (lane == 0) producer_role<D>(m, p, sbase, abort_flag);
    } else if (warp == kWarpMma) {
      mma_role<T, D>(p, sbase, uniform(tbase), abort_flag);
    } else if (warp == kWarpScrub && p.scrub) {
      scrub_role<D>(p, sbase, abort_flag);
    }
  } else {
    regs_grow<kRegsSoftmax>();
    softmax_role<T, D>(p, smem, sbase, tbase, abort_flag);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kWarpMma) {
    __syncwarp();
    tmem_dealloc(tbase, C::TMEM_COLS);
  }
}

template <typename T, int D>
cudaError_t launch(const CrossMaps& m, const CrossParams& p, int grid, cudaStream_t s) {
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
      // the register split is sound only if the kernel launches with kRegsLaunch registers
      cudaFuncAttributes fa;
      if ((e = cudaFuncGetAttributes(&fa, cross_fwd_kernel<T, D>)) != cudaSuccess) return e;
      if (fa.numRegs != kRegsLaunch) return cudaErrorInvalidConfiguration;
      e = cudaFuncSetAttribute(cross_fwd_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::SMEM_BYTES);
      if (e != cudaSuccess) return e;
      attr_set[dev] = true;
    }
  }
  cross_fwd_kernel<T, D><<<grid, kThreads, Cfg<D>::SMEM_BYTES, s>>>(m, p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cross_fwd(const CrossMaps& m, const CrossParams& p, int dtype, int D, int grid, cudaStream_t s) {
  if (dtype == 0) return D == 128 ? launch<__nv_bfloat16, 128>(m, p, grid, s) : launch<__nv_bfloat16, 64>(m, p, grid, s);
  return D == 128 ? launch<__half, 128>(m, p, grid, s) : launch<__half, 64>(m, p, grid, s);
}

cudaError_t cross_fwd_status(int* code, cudaStream_t s) { return read_clear_error(&g_error, code, s); }

}  // namespace ug
