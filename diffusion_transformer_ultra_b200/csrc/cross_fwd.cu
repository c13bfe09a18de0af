// Cross attention forward for sm_100a (tcgen05 + TMEM + TMA): o = softmax(scale q k^T) v with the
// running maximum and sum of each row, and the row's log-sum-exp.
//
// CTA organisation (one persistent CTA per SM, 512 threads = 4 warpgroups):
//   warps 0-3, 4-7  softmax of query tile 0 / 1 of the item (thread = row = TMEM lane)
//   warp  8         producer: TMA loads of Q (per item) and of K, V tiles in stages
//   warp  9         MMA issuer: S = Q K^T and O += P V (P from TMEM); owns TMEM
//   warp  10        scrubber: zeroes the V rows of hidden keys, which may hold NaN (0 * NaN)
//   warps 12-15     output: O from TMEM to memory, beside the next item's first softmax.  An encoder's
//                   states are a few key tiles (4 for 512), so items are short: with this in the
//                   softmax warps it took 5,000 of an item's 19,000 cycles.
// 65,536 queries x 512 keys x 24 heads of 128: 415 us, 993 TF/s, in a burst of calls; in a loop of seconds
// 484 us, 852 TF/s, where the power limit holds the clock at 1,612 of 1,965 MHz.  A tile's chain of product,
// exponentials and product bounds it, two tiles to a CTA against each other (TMEM has no room for a third S
// at this head size), and items are short: one key tile in four is an item's first, whose S is read twice
// (maximum, exponentials), and Q has one buffer.
// TMEM (512 columns): S0 [0,128), S1 [128,256), O0 [256,256+D), O1 [256+D, 256+2D); P (16 bits,
// packed in pairs, 64 columns in 32) overwrites the first and third quarter of its S block.
#include <cstdint>
#include <mutex>

#include "cross.cuh"

namespace ug {
namespace {

__device__ int g_error;                // first wait that ran out since the last status read

template <int D>
struct Cfg {
  static constexpr int TILE_BYTES = 128 * D * 2;
  static constexpr int NS = D == 128 ? 4 : 8;      // tile slots
  static constexpr int NSTG = NS / 2;              // stages in flight (two tiles each)
  static constexpr int KV_OFF = 2 * TILE_BYTES;
  static constexpr int INV_OFF = KV_OFF + NS * TILE_BYTES;      // [2 items][2 tiles][128] floats: 1 / row sum
  static constexpr int BAR_OFF = INV_OFF + 4 * 128 * 4;
  // Q full / empty, stage full / scrubbed / empty, S ready, P ready (the last one of an item: 1 / row
  // sums too), O ready / read (each per query tile), drain
  static constexpr int B_QF = 0, B_QE = 1, B_KVF = 2, B_KVS = B_KVF + NSTG, B_KVE = B_KVS + NSTG,
                       B_SF = B_KVE + NSTG, B_PF = B_SF + 2, B_OF = B_PF + 2, B_OE = B_OF + 2, B_DRAIN = B_OE + 2,
                       NBAR = B_DRAIN + 1;
  static constexpr int MISC_OFF = BAR_OFF + NBAR * 8;           // TMEM base, abort word
  static constexpr int SMEM_BYTES = MISC_OFF + 16;
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory per CTA exceeds 227 KB");
  static __device__ __forceinline__ uint32_t arrivals(int i) { return i >= B_PF && i < B_DRAIN && i != B_OF && i != B_OF + 1 ? 4 : 1; }
  static __device__ __forceinline__ uint32_t v_slot(uint32_t g) { return 2 * g; }
  static __device__ __forceinline__ uint32_t k_slot(uint32_t g) { return 2 * g + 1; }
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr uint32_t O_COL = 256;
};

constexpr int kThreads = 512;
constexpr int kRegsLaunch = 128;      // per thread at launch: 65536 / 512
constexpr int kRegsSoftmax = 200;
constexpr int kRegsControl = 56;
static_assert(2 * 128 * kRegsSoftmax + 2 * 128 * kRegsControl <= kThreads * kRegsLaunch,
              "register split exceeds the launch allocation");
constexpr int kWarpProducer = 8, kWarpMma = 9, kWarpScrub = 10;

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

// Steps of a CTA's items, one key tile each, items without visible keys left out.  A stage of the
// pipeline belongs to a pair of consecutive steps: it holds V of the one and K of the other, so that
// the next item's first S is made right behind an item's last product.
struct Step {
  int it, b, hk, qt0, ntile, tile, len;   // key tile of the step, visible keys of its sample
  bool on, first, last;
};
struct Walk {
  Step s;
  int j, n, k0;
  __device__ __forceinline__ void item(const CrossParams& p, int it) {
    for (;; it += gridDim.x) {
      s.it = it;
      s.on = it < p.total;
      if (!s.on) return;
      const Item w(p, it);
      n = uniform(w.k1 - w.k0);
      if (n == 0) continue;
      k0 = uniform(w.k0);
      s.len = uniform(w.len);
      s.b = w.b;
      s.hk = w.hk;
      s.qt0 = w.qt0;
      s.ntile = w.ntile;
      j = -1;
      next_tile();
      return;
    }
  }
  __device__ __forceinline__ void next_tile() {
    ++j;
    s.tile = k0 + j;
    s.first = j == 0;
    s.last = j == n - 1;
  }
  __device__ __forceinline__ void next(const CrossParams& p) {
    if (s.last) item(p, s.it + gridDim.x);
    else next_tile();
  }
};

template <int D>
__device__ void producer_role(const CrossMaps& m, const CrossParams& p, uint32_t sbase, const Waiter& wait) {
  using C = Cfg<D>;
  const uint32_t sKV = sbase + C::KV_OFF, bar = wait.bar;
  const int q_bytes = p.toks * p.group * D * 2;
  uint32_t st = 0, qi = 0;
  Walk cur;
  Step prev;
  prev.on = false;
  cur.item(p, blockIdx.x);
  for (; cur.s.on || prev.on; ++st) {
    if (cur.s.on && cur.s.first) {
      if (!wait.warp(C::B_QE, (qi & 1) ^ 1)) break;
      mbar_expect_tx_elect(bar + 8 * C::B_QF, cur.s.ntile * q_bytes);
      for (int t = 0; t < cur.s.ntile; ++t)
        load_tile<D>(sbase + t * C::TILE_BYTES, &m.q, (cur.s.qt0 + t) * p.toks, cur.s.hk, cur.s.b, bar + 8 * C::B_QF);
      ++qi;
    }
    const uint32_t g = st % C::NSTG, fb = bar + 8 * (C::B_KVF + g);
    if (!wait.warp(C::B_KVE + g, ((st / C::NSTG) & 1) ^ 1)) break;
    mbar_expect_tx_elect(fb, (prev.on ? C::TILE_BYTES : 0) + (cur.s.on ? C::TILE_BYTES : 0));
    if (prev.on) load_tile<D>(sKV + C::v_slot(g) * C::TILE_BYTES, &m.v, prev.tile * 128, prev.hk, prev.b, fb);
    if (cur.s.on) load_tile<D>(sKV + C::k_slot(g) * C::TILE_BYTES, &m.k, cur.s.tile * 128, cur.s.hk, cur.s.b, fb);
    prev = cur.s;
    if (cur.s.on) cur.next(p);
  }
  if (cur.s.on || prev.on) settle();
}

// One warp, only when hidden keys exist below ns: stage by stage, zeroes the hidden rows of V
// and passes the stage on.
template <int D>
__device__ void scrub_role(const CrossParams& p, uint32_t sbase, const Waiter& wait) {
  using C = Cfg<D>;
  uint32_t st = 0;
  Walk cur;
  Step prev;
  prev.on = false;
  cur.item(p, blockIdx.x);
  for (; cur.s.on || prev.on; ++st) {
    const uint32_t g = st % C::NSTG;
    const uint4 vis = prev.on ? cross_words(p, prev.b, prev.tile, prev.len) : make_uint4(~0u, ~0u, ~0u, ~0u);
    if (!wait.warp(C::B_KVF + g, (st / C::NSTG) & 1)) return;
    if (!all_visible(vis)) {
      scrub_rows<D>(sbase + C::KV_OFF + C::v_slot(g) * C::TILE_BYTES, BOX_BYTES, vis, 0, 128);
      fence_async_smem();
    }
    warp_arrive(wait.bar + 8 * (C::B_KVS + g));
    prev = cur.s;
    if (cur.s.on) cur.next(p);
  }
}

template <typename T, int D>
__device__ void mma_role(const CrossParams& p, uint32_t sbase, uint32_t tbase, const Waiter& wait) {
  using C = Cfg<D>;
  const uint32_t sKV = sbase + C::KV_OFF, bar = wait.bar;
  const int ready = p.scrub ? C::B_KVS : C::B_KVF;
  uint32_t st = 0, qi = 0, pc[2] = {0, 0}, oc[2] = {0, 0};   // P's read, items begun (per query tile)
  bool ok = true;
  Walk cur;
  Step prev;
  prev.on = false;
  cur.item(p, blockIdx.x);
  for (; cur.s.on || prev.on; ++st) {
    const uint32_t g = st % C::NSTG;
    const bool on = cur.s.on;
    if (!(ok = wait.warp(ready + g, (st / C::NSTG) & 1))) break;
    const uint32_t v = sKV + C::v_slot(g) * C::TILE_BYTES, k = sKV + C::k_slot(g) * C::TILE_BYTES;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      if (prev.on && t < prev.ntile) {
        if (!(ok = wait.warp(C::B_PF + t, pc[t] & 1))) break;
        ++pc[t];
        if (prev.first) {
          if (oc[t] > 0 && !(ok = wait.warp(C::B_OE + t, (oc[t] - 1) & 1))) break;
          ++oc[t];
        }
        tc_fence_after();
        mma_accum<T, D>(tbase + C::O_COL + D * t, tbase + 128 * t, v, prev.first);
        if (prev.last) mma_commit_elect(bar + 8 * (C::B_OF + t));
      }
      if (on && t < cur.s.ntile) {
        if (t == 0 && cur.s.first && !(ok = wait.warp(C::B_QF, qi & 1))) break;
        tc_fence_after();
        mma_scores<T, D>(tbase + 128 * t, sbase + t * C::TILE_BYTES, k);
        mma_commit_elect(bar + 8 * (C::B_SF + t));
      }
    }
    if (!ok) break;
    mma_commit_elect(bar + 8 * (C::B_KVE + g));
    if (on && cur.s.last) {
      mma_commit_elect(bar + 8 * C::B_QE);
      ++qi;
    }
    prev = cur.s;
    if (on) cur.next(p);
  }
  if (!ok) {
    mma_commit_elect(bar + 8 * C::B_DRAIN);
    wait.drain(C::B_DRAIN, 0, &g_error);
  }
}

// Exponentials of 64 columns of an S row at the running max mu (log2 units): the pairs' packed 16-bit P
// (the tensor core's operand type; the row sum adds the unrounded fp32 values).  Returns their sum.
template <typename T>
__device__ __forceinline__ float exp_half(const uint32_t (&s)[64], uint32_t (&pk)[32], float scale, float mu) {
  const float2 scale2 = make_float2(scale, scale), nmu2 = make_float2(-mu, -mu);
  float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
  for (int c = 0; c < 32; ++c) {
    float2 x = ffma2(make_float2(__uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1])), scale2, nmu2);
    x.x = ex2(x.x);
    x.y = ex2(x.y);
    ls[c & 1] = fadd2(ls[c & 1], x);
    pk[c] = pack2<T>(x.x, x.y);
  }
  const float2 l2 = fadd2(ls[0], ls[1]);
  return l2.x + l2.y;
}

// 64 columns of an S row, hidden ones as -inf.
__device__ __forceinline__ void load_half(uint32_t tmem, uint32_t (&s)[64], bool part, uint32_t w0, uint32_t w1) {
  tmem_ld64_sync(tmem, s);
  if (!part) return;
#pragma unroll
  for (int c = 0; c < 64; ++c)
    if (!(((c < 32 ? w0 : w1) >> (c & 31)) & 1u)) s[c] = 0xff800000u;
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

// Block of a split item's query tile among the partial results: [unit][query tile][split].
__device__ __forceinline__ int64_t part_block(const CrossParams& p, const Item& w, int qt) {
  return ((int64_t)(w.b * p.kv_heads + w.hk) * p.nqt + qt) * p.nsplit + w.split;
}

template <typename T, int D>
__device__ void softmax_role(const CrossParams& p, float* inv_s, uint32_t tbase, const Waiter& wait) {
  using C = Cfg<D>;
  const uint32_t bar = wait.bar;
  const int t = threadIdx.x >> 7, r = threadIdx.x & 127;
  const uint32_t lane_off = (uint32_t)((threadIdx.x >> 5) & 3) * 32u << 16;
  const uint32_t tS = tbase + lane_off + (uint32_t)(t * 128);
  const uint32_t tO = tbase + lane_off + C::O_COL + (uint32_t)(t * D);
  const float scale = p.scale_log2;
  const int tok_r = row_tok(p, r), g_r = r - tok_r * p.group;
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
      if (!wait.warp(C::B_SF + t, sc & 1)) return;
      ++sc;
      tc_fence_after();
      // With a running max the exponentials are taken at it without a look at the tile's max; a tile
      // sum above 2^12 (fp16 P still holds it), and a row without a max yet, take the max first.  A
      // running max stays unless it grew by more than 2^8: the division by the row sum makes the
      // result exact for any max.
      bool exact = __any_sync(0xffffffffu, m == neg_inf());
      float part;
      uint32_t pa[32], pb[32];
      for (;;) {
        uint32_t s[64];
        if (exact) {
          float mx = neg_inf();
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            __syncwarp();
            load_half(tS + 64 * h, s, part_tile, h ? vis.z : vis.x, h ? vis.w : vis.y);
            float mx4[4] = {neg_inf(), neg_inf(), neg_inf(), neg_inf()};
#pragma unroll
            for (int c = 0; c < 64; c += 8)
#pragma unroll
              for (int i = 0; i < 4; ++i) mx4[i] = fmax3(mx4[i], __uint_as_float(s[c + 2 * i]), __uint_as_float(s[c + 2 * i + 1]));
            mx = fmax3(mx, fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
          }
          const float mnew = fmaxf(m, mx * scale);
          const bool need = m != neg_inf() && mnew > m + 8.0f;
          if (__any_sync(0xffffffffu, need)) {
            const float f = need ? ex2(m - mnew) : 1.0f;
            lsum *= f;
            __syncwarp();
            rescale_o<D>(tO, f);
          }
          if (m == neg_inf() || need) m = mnew;
        }
        const float mu = m == neg_inf() ? 0.f : m;
        part = 0.f;
#pragma unroll 1                       // (one copy of this code: all roles share the instruction cache)
        for (int h = 0; h < 2; ++h) {
          __syncwarp();
          load_half(tS + 64 * h, s, part_tile, h ? vis.z : vis.x, h ? vis.w : vis.y);
          part += exp_half<T>(s, pb, scale, mu);
          if (h == 0) {
#pragma unroll
            for (int c = 0; c < 32; ++c) pa[c] = pb[c];
          }
        }
        if (exact || !__any_sync(0xffffffffu, !(part <= 4096.0f))) break;
        exact = true;
      }
      lsum += part;
      __syncwarp();
      tmem_st32(tS, pa);
      tmem_st32(tS + 64, pb);
      if (j == n - 1)                  // for the output warps; NaN stays NaN
        inv_s[((oc & 1) * 2 + t) * 128 + r] = lsum > 0.f ? 1.0f / lsum : (lsum == 0.f ? 0.f : lsum);
      tmem_wait_st();
      tc_fence_before();
      warp_arrive(bar + 8 * (C::B_PF + t));
    }
    const float lse2 = lsum == 0.f ? neg_inf() : m + log2f(lsum);
    if (n > 0) ++oc;
    if (real) {
      if (p.part) p.part[(int64_t)p.units * p.nqt * p.nsplit * p.part_rows * D + part_block(p, w, qt) * p.part_rows + r] = lse2;
      else if (p.lse) p.lse[((int64_t)w.b * p.heads + h) * p.nq + tok] = lse2 * 0.6931471805599453f;
    }
  }
}

// O of the items' query tiles, divided by the row sums: to o, or as fp32 partials of split items
// (whose log-sum-exp alone marks one without a visible key).
template <typename T, int D>
__device__ void output_role(const CrossParams& p, const float* inv_s, uint32_t tbase, const Waiter& wait) {
  using C = Cfg<D>;
  const int r = threadIdx.x & 127, tok_r = row_tok(p, r), g_r = r - tok_r * p.group;
  const uint32_t tO = tbase + ((uint32_t)((threadIdx.x >> 5) & 3) * 32u << 16) + C::O_COL;
  uint32_t oc[2] = {0, 0};
  for (int it = blockIdx.x; it < p.total; it += gridDim.x) {
    const Item w(p, it);
#pragma unroll 1
    for (int t = 0; t < w.ntile; ++t) {
      const int qt = w.qt0 + t, tok = qt * p.toks + tok_r;
      const bool real = tok_r < p.toks && tok < p.nq;
      T* row = nullptr;
      if (real && !p.part)
        row = static_cast<T*>(p.out[0]) + w.b * p.out_st[0][0] + tok * p.out_st[0][1] + (w.hk * p.group + g_r) * p.out_st[0][2];
      if (w.k1 == w.k0) {              // nothing visible: zeros
        if (row) {
#pragma unroll 1
          for (int c = 0; c < D / 8; ++c) reinterpret_cast<uint4*>(row)[c] = make_uint4(0, 0, 0, 0);
        }
        continue;
      }
      const uint32_t n = t ? oc[1]++ : oc[0]++;
      if (!wait.warp(C::B_OF + t, n & 1)) return;
      tc_fence_after();
      // a row without a visible key has O = 0 products of P = 0: inv = 0 keeps it zero
      const float inv = inv_s[((n & 1) * 2 + t) * 128 + r];
      if (p.part) {
        float* dst = p.part + (part_block(p, w, qt) * p.part_rows + r) * D;
#pragma unroll 1
        for (int ch = 0; ch < D / 32; ++ch) {
          uint32_t o[32];
          __syncwarp();
          tmem_ld32_sync(tO + t * D + ch * 32, o);
          if (!real) continue;
#pragma unroll
          for (int q = 0; q < 8; ++q)
            reinterpret_cast<float4*>(dst + ch * 32)[q] =
                make_float4(__uint_as_float(o[4 * q + 0]) * inv, __uint_as_float(o[4 * q + 1]) * inv,
                            __uint_as_float(o[4 * q + 2]) * inv, __uint_as_float(o[4 * q + 3]) * inv);
        }
      } else {
#pragma unroll 1
        for (int ch = 0; ch < D / 32; ++ch) store_piece<T, 32>(tO + t * D + ch * 32, row ? row + ch * 32 : nullptr, inv);
      }
      tc_fence_before();
      warp_arrive(wait.bar + 8 * (C::B_OE + t));
    }
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1)
    cross_fwd_kernel(const __grid_constant__ CrossMaps m, const CrossParams p) {
  using C = Cfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  if (sbase & 1023) {                  // the swizzle needs it; the declaration asks for it
    if (threadIdx.x == 0) atomicExch(&g_error, (int)DEV_TIMEOUT_PRODUCER);
    return;
  }
  const uint32_t bar = sbase + C::BAR_OFF;
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + C::MISC_OFF);
  float* inv_s = reinterpret_cast<float*>(smem + C::INV_OFF);
  const int warp = uniform(threadIdx.x >> 5);
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NBAR; ++i) mbar_init(bar + 8 * i, C::arrivals(i));
    misc[1] = 0;                       // abort word
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
  Waiter wait{bar, smem_u32(misc + 1), DEV_TIMEOUT_SOFTMAX, (uint32_t)p.timeout_ns};
  if (warp >= 8) {
    regs_shrink<kRegsControl>();
    if (warp == kWarpProducer) {
      wait.code = DEV_TIMEOUT_PRODUCER;
      producer_role<D>(m, p, sbase, wait);
    } else if (warp == kWarpMma) {
      wait.code = DEV_TIMEOUT_MMA;
      mma_role<T, D>(p, sbase, uniform(tbase), wait);
    } else if (warp == kWarpScrub) {
      if (p.scrub) scrub_role<D>(p, sbase, wait);
    } else if (warp >= 12) {
      output_role<T, D>(p, inv_s, tbase, wait);
    }
  } else {
    regs_grow<kRegsSoftmax>();
    softmax_role<T, D>(p, inv_s, tbase, wait);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (threadIdx.x == 0 && misc[1] != 0) atomicExch(&g_error, (int)misc[1]);
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
