// Layer norm over the last dimension, forward and backward, with one weight for every row or
// one per sample (the modulation of a diffusion transformer).
//
//   mu = sum(x) / C,  r = (sum((x - mu)^2) / C + eps)^-1/2,  xh = (x - mu) r
//   y  = xh w' + b,   w' = w, or 1 + w (plus_one), or 1 without a weight
//   g  = dy w',       dx = r (g - sum(g) / C - xh sum(g xh) / C)
//   dw = sum over rows of dy xh,   db = sum over rows of dy
//
// Both passes are bound by HBM: x is read and y written once (x, dy read and dx written once).
// A row belongs to a group of as many warps as give each lane 16 elements (32 in the widest rows), so
// that the lane's part of the weight and bias stays in registers from row to row.  Rows come by bulk
// copies, several ahead, into shared memory (a persistent block per multiprocessor has up to 200 KB of
// them in flight), and from there to registers, so that the variance takes a second pass over registers
// (no cancellation of sum(x^2) against mu^2).  A copy covers the 16-byte pieces that hold the row, so
// that a row may start anywhere; one that does not start on four elements is then worked on element by
// element.  All sums are fp32, the arithmetic is on pairs.
// With the loads out of the way a row is one chain of dependent steps, and what the chain holds sets the
// pace: a warp of its own issues the copies, and a row group of the forward pass takes two rows at a
// time, whose sums share the shuffles and barriers.  For 70,144 x 2,048 bf16 with fp32 weights that
// takes 150 us; a row group that issues its own copies 158; a row to a block, loads straight to
// registers, 151; and the kernel for such rows below, 122 (a copy of the same bytes takes 94).
//
// The weight's gradient: a block of the backward pass walks a run of rows of one sample (of the
// whole batch with a shared weight), keeps its columns' sums in registers, and writes them once
// to the caller's workspace; a second kernel adds the runs in a fixed order.  No atomics: the
// same inputs give the same bits.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "cross.cuh"
#include "device.h"
#include "elem.cuh"
#include "kernels.h"
#include "nvtx_range.h"
#include "ptx.cuh"
#include "ultragen.h"

namespace ug {
namespace {

constexpr int kMaxCols = 16384;

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
  int64_t total;           // rows of all samples, below 2^31: a row plus a step of the walk fits 32 unsigned bits
  int rows, C;             // rows per sample
  FastDiv div_rows;        // by rows
  int64_t w_batch;         // C with a weight per sample, else 0
  int runs_per_group;      // runs of a sample (of everything with a shared weight)
  int64_t group_rows;      // rows of a sample (of everything with a shared weight)
  int warps;               // warps of a row
  int wide;                // forward: norm_wide_kernel
  int at_once;             // rows of a block at a time
  int slots, slot_bytes;   // rows in flight per row group; bytes of one tensor's row in a slot
  float plus, inv_c, eps;
};

// Threads of a row, and the sums over them: a warp's own, or through shared memory behind a named
// barrier of the row's warps.  `red` is double-buffered: whoever writes a buffer again has passed the
// barrier of the sum between, which its readers had to reach first.
template <bool MULTI>
struct Row {
  int t, threads, group;               // this thread's place in the row, threads of a row, row of the block
  float2* red;                         // [2][32], one entry per warp of the block
  int flip;
  __device__ __forceinline__ Row(const NormArgs& p, float2* smem) : red(smem), flip(0) {
    const int warp = threadIdx.x >> 5;
    group = MULTI ? warp / p.warps : warp;
    threads = MULTI ? p.warps * 32 : 32;
    t = threadIdx.x - group * threads;
  }
  __device__ __forceinline__ float2 sum(float2 x, int warps) {
    x.x = warp_sum(x.x);
    x.y = warp_sum(x.y);
    if (!MULTI) return x;
    const int lane = threadIdx.x & 31;
    float2* buf = red + flip * 32 + group * warps;
    flip ^= 1;
    if (lane == 0) buf[t >> 5] = x;
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(threads) : "memory");
    x = make_float2(0.f, 0.f);
    for (int q = 0; q < warps; q += 4) {
      float2 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = q + i < warps ? buf[q + i] : make_float2(0.f, 0.f);
      x = fadd2(x, fadd2(fadd2(v[0], v[1]), fadd2(v[2], v[3])));
    }
    return x;
  }
};

__device__ int g_error;                // a wait that ran out since the last status read

constexpr uint32_t kWaitNs = 2000u * 1000 * 1000;

// The rows of one row group on their way through shared memory: `slots` slots of N tensors' rows each.
template <typename T, int N>
struct Ring {
  uint32_t bar, abort_word;            // barriers of this group's slots: full, then empty
  uint8_t* buf;
  int slots, slot_bytes, row_bytes, slot;
  uint32_t phase;
  __device__ __forceinline__ Ring(const NormArgs& p, int group, uint64_t* bars, uint8_t* smem, uint32_t* abort)
      : bar(smem_u32(bars + 2 * group * p.slots)), abort_word(smem_u32(abort)),
        buf(smem + (int64_t)group * p.slots * N * p.slot_bytes), slots(p.slots), slot_bytes(p.slot_bytes),
        row_bytes(p.C * (int)sizeof(T)), slot(0), phase(0) {}
  // One thread: the 16-byte pieces that hold the rows at src[0 .. N) into slot `to`.
  __device__ __forceinline__ void issue(int to, const T* const (&src)[N]) const {
    uint32_t bytes[N], total = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint32_t off = (uint32_t)(uintptr_t)src[i] & 15u;
      bytes[i] = (off + row_bytes + 15) & ~15u;
      total += bytes[i];
    }
    mbar_expect_tx(bar + 8 * to, total);
#pragma unroll
    for (int i = 0; i < N; ++i)
      bulk_load(smem_u32(buf + (to * N + i) * slot_bytes), reinterpret_cast<const uint8_t*>((uintptr_t)src[i] & ~(uintptr_t)15),
                bytes[i], bar + 8 * to);
  }
  __device__ __forceinline__ bool wait() const {
    return __all_sync(0xffffffffu, mbar_wait_short(bar + 8 * slot, phase, abort_word, DEV_TIMEOUT_PRODUCER, kWaitNs));
  }
  // Row i of the current slot, whose source is src.
  __device__ __forceinline__ const T* row(int i, const T* src) const {
    return reinterpret_cast<const T*>(buf + (slot * N + i) * slot_bytes + ((uint32_t)(uintptr_t)src & 15u));
  }
  // The current slot may be written again (one thread, when all of the row have read it).
  __device__ __forceinline__ void release(int s) const { mbar_arrive(bar + 8 * (slots + s)); }
  // The producer's side: waits until the current slot is free.
  __device__ __forceinline__ bool wait_free() const {
    return mbar_wait_short(bar + 8 * (slots + slot), phase ^ 1, abort_word, DEV_TIMEOUT_PRODUCER, kWaitNs);
  }
  __device__ __forceinline__ void next() {
    if (++slot == slots) {
      slot = 0;
      phase ^= 1;
    }
  }
};

// Barriers of a block's slots (at most kBars / 2 slots in all).
constexpr int kBars = 256;
__device__ __forceinline__ void init_bars(uint64_t* bars, uint32_t* abort, int n) {
  for (int i = threadIdx.x; i < n; i += blockDim.x) mbar_init(smem_u32(bars + i), 1);
  if (threadIdx.x == 0) *abort = 0;
  fence_mbar_init();
  __syncthreads();
}
// At the end of a warp's work, whichever its role: the producer may be done long before a row's wait runs out.
__device__ __forceinline__ void report(const uint32_t* abort) {
  const int code = *reinterpret_cast<const volatile int*>(abort);
  if (code == 0) return;
  if ((threadIdx.x & 31) == 0) atomicExch(&g_error, code);
  settle();
}

// A piece: four elements of a row, as 32-bit words (kept as such: element by element, the compiler
// takes 16-bit types apart and together again).
template <typename T>
struct Raw {
  uint32_t w[sizeof(T)];
};
template <typename T>
__device__ __forceinline__ void pairs(const Raw<T>& v, float2 (&out)[2]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if constexpr (sizeof(T) == 4) out[i] = make_float2(__uint_as_float(v.w[2 * i]), __uint_as_float(v.w[2 * i + 1]));
    else if constexpr (std::is_same<T, __half>::value) out[i] = __half22float2(*reinterpret_cast<const __half2*>(&v.w[i]));
    else out[i] = make_float2(__uint_as_float(v.w[i] << 16), __uint_as_float(v.w[i] & 0xffff0000u));
  }
}
template <typename T>
__device__ __forceinline__ void unpairs(Raw<T>& v, const float2 (&in)[2]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if constexpr (sizeof(T) == 4) {
      v.w[2 * i] = __float_as_uint(in[i].x);
      v.w[2 * i + 1] = __float_as_uint(in[i].y);
    } else {
      v.w[i] = pack2<T>(in[i].x, in[i].y);
    }
  }
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// The words as values the compiler knows nothing about.
template <typename T>
__device__ __forceinline__ void opaque(Raw<T>& v) {
#pragma unroll
  for (int i = 0; i < (int)sizeof(T); ++i) asm volatile("" : "+r"(v.w[i]));
}

// A lane's pieces of a row.  Warp q of the row has the span of 128 NV columns from 128 NV q; its piece k
// is four columns in a row, 128 k + 4 lane, where rows start on four elements (CONTIG; C is then a
// multiple of four), else 128 k + lane + 32 e.  The offsets within the span are constants, and only the
// row's last warp (`full` false) looks at the row's end.
template <bool CONTIG, int NV>
struct Span {
  int col, C;                          // this lane's first column
  bool full;
  __device__ __forceinline__ Span(int t, int C_) : C(C_) {
    const int first = (t >> 5) * (NV * 128);
    col = first + (CONTIG ? 4 : 1) * (t & 31);
    full = first + NV * 128 <= C;
  }
  static __device__ constexpr int offset(int k, int e) { return k * 128 + (CONTIG ? e : 32 * e); }
  __device__ __forceinline__ bool has(int k, int e) const { return full || col + offset(k, e) < C; }
  // From shared memory, which may be read behind the row's end: zeros there.
  template <typename T>
  __device__ __forceinline__ void load_row(const T* row, Raw<T> (&v)[NV]) const {
    const T* p = row + col;
#pragma unroll
    for (int k = 0; k < NV; ++k) v[k] = words(p + offset(k, 0), [&](int e) { return offset(0, e); });
    if (full) return;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[k].w[e] = has(k, e) ? v[k].w[e] : 0u;
      } else {
#pragma unroll
        for (int i = 0; i < 2; ++i)
          v[k].w[i] &= (has(k, 2 * i) ? 0xffffu : 0u) | (has(k, 2 * i + 1) ? 0xffff0000u : 0u);
      }
    }
  }
  // From global memory: some elements of the row behind its end.
  template <typename T>
  __device__ __forceinline__ Raw<T> load_any(const T* row, int k) const {
    const int c = col + offset(k, 0);
    if (CONTIG) return words(row + min(c, C - 4), [](int e) { return e; });
    return words(row, [&](int e) { return min(c + 32 * e, C - 1); });
  }
  template <typename T>
  __device__ __forceinline__ void store(T* row, int k, const Raw<T>& v) const {
    T* p = row + col + offset(k, 0);
    if constexpr (CONTIG && sizeof(T) == 4) {
      if (has(k, 0)) *reinterpret_cast<uint4*>(p) = make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]);
    } else if constexpr (CONTIG) {
      if (has(k, 0)) *reinterpret_cast<uint2*>(p) = make_uint2(v.w[0], v.w[1]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (!has(k, e)) continue;
        if constexpr (sizeof(T) == 4) reinterpret_cast<uint32_t*>(p)[32 * e] = v.w[e];
        else reinterpret_cast<uint16_t*>(p)[32 * e] = (uint16_t)(v.w[e >> 1] >> (16 * (e & 1)));
      }
    }
  }

 private:
  template <typename T, typename At>
  static __device__ __forceinline__ Raw<T> words(const T* p, At at) {
    Raw<T> v;
    if constexpr (CONTIG && sizeof(T) == 4) {
      const uint4 u = *reinterpret_cast<const uint4*>(p);
      v.w[0] = u.x;
      v.w[1] = u.y;
      v.w[2] = u.z;
      v.w[3] = u.w;
    } else if constexpr (CONTIG) {
      const uint2 u = *reinterpret_cast<const uint2*>(p);
      v.w[0] = u.x;
      v.w[1] = u.y;
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int e = 0; e < 4; ++e) v.w[e] = reinterpret_cast<const uint32_t*>(p)[at(e)];
    } else {
      const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
      for (int i = 0; i < 2; ++i) v.w[i] = h[at(2 * i)] | (uint32_t)h[at(2 * i + 1)] << 16;
    }
    return v;
  }
};

// One block walks the rows [r0, r1) of run blockIdx.x, its row groups in turn.
template <typename T, typename W, bool CONTIG, int NV, bool MULTI>
__global__ void __launch_bounds__(NV == 8 ? 544 : 512) norm_fwd_kernel(const NormArgs p) {
  __shared__ float2 red[64];
  __shared__ uint64_t bars[kBars];
  __shared__ uint32_t abort_word;
  extern __shared__ __align__(16) uint8_t smem[];
  init_bars(bars, &abort_word, 2 * p.at_once * p.slots);
  const uint32_t first = blockIdx.x * p.at_once, r1 = (uint32_t)p.total, step = gridDim.x * p.at_once;
  if (threadIdx.x >= p.at_once * p.warps * 32) {             // producer warp: a lane to a row group
    const int group = threadIdx.x & 31;
    if (group < p.at_once) {
      Ring<T, 1> ring(p, group, bars, smem, &abort_word);
      for (uint32_t row = first + group; row < r1; row += step, ring.next()) {
        if (!ring.wait_free()) break;
        const uint32_t s = p.div_rows.div(row), i = row - s * p.rows;
        const T* src[1] = {static_cast<const T*>(p.x) + s * p.x_batch + i * p.x_row};
        ring.issue(ring.slot, src);
      }
    }
    __syncwarp();
    report(&abort_word);
    return;
  }
  Row<MULTI> me(p, red);
  const Span<CONTIG, NV> at(me.t, p.C);
  Ring<T, 1> ring(p, me.group, bars, smem, &abort_word);
  const uint32_t r0 = first + me.group;
  float2 w[NV][2], b[NV][2];
  int64_t loaded = -1;                 // whose weight these are
  // Two rows at a time, whose sums share the shuffles and barriers: a row alone is one long chain of
  // them.  (Rows of two samples with a weight each go one by one.)
  for (uint32_t row = r0; row < r1;) {
    uint32_t at_row[2] = {row, row + step};
    uint32_t smp[2] = {p.div_rows.div(row), 0};
    bool two = at_row[1] < r1;
    if (two) smp[1] = p.div_rows.div(at_row[1]);
    two = two && (p.w_batch == 0 || smp[1] == smp[0]);
    const int64_t weight = smp[0] * p.w_batch;
    if (weight != loaded) {
      loaded = weight;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        w[k][0] = w[k][1] = both(1.f);
        b[k][0] = b[k][1] = both(0.f);
        if (p.w) {
          pairs<W>(at.load_any(static_cast<const W*>(p.w) + loaded, k), w[k]);
#pragma unroll
          for (int e = 0; e < 2; ++e) w[k][e] = fadd2(w[k][e], both(p.plus));
        }
        if (p.b) pairs<W>(at.load_any(static_cast<const W*>(p.b) + loaded, k), b[k]);
      }
    }
    float2 v[2][NV][2], sum[2] = {both(0.f), both(0.f)};
    int slot[2] = {0, 0};
    bool ok = true;                    // (after a wait that ran out the rows' barriers are still kept)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      if (r == 1 && !two) break;
      const T* x = ring.row(0, static_cast<const T*>(p.x) + smp[r] * p.x_batch + (at_row[r] - smp[r] * p.rows) * p.x_row);
      ok = ring.wait() && ok;
      Raw<T> raw[NV];
      at.load_row(x, raw);
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        pairs<T>(raw[k], v[r][k]);
        sum[r] = fadd2(sum[r], fadd2(v[r][k][0], v[r][k][1]));
      }
      slot[r] = ring.slot;
      ring.next();
    }
    float2 mean = me.sum(make_float2(sum[0].x + sum[0].y, sum[1].x + sum[1].y), p.warps);
    mean = make_float2(mean.x * p.inv_c, mean.y * p.inv_c);
    if (me.t == 0) {                   // every thread of the rows has read their slots
      ring.release(slot[0]);
      if (two) ring.release(slot[1]);
    }
    float2 sq[2] = {both(0.f), both(0.f)};
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      if (r == 1 && !two) break;
      const float2 nm = both(r ? -mean.y : -mean.x);
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int e = 0; e < 2; ++e) v[r][k][e] = fadd2(v[r][k][e], nm);
      if (!at.full) {                  // the zeros behind the row stay zeros
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            v[r][k][e].x = at.has(k, 2 * e) ? v[r][k][e].x : 0.f;
            v[r][k][e].y = at.has(k, 2 * e + 1) ? v[r][k][e].y : 0.f;
          }
      }
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int e = 0; e < 2; ++e) sq[r] = ffma2(v[r][k][e], v[r][k][e], sq[r]);
    }
    const float2 var = me.sum(make_float2(sq[0].x + sq[0].y, sq[1].x + sq[1].y), p.warps);
    const float2 rs = make_float2(1.0f / sqrtf(var.x * p.inv_c + p.eps), 1.0f / sqrtf(var.y * p.inv_c + p.eps));
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      if (!ok || (r == 1 && !two)) break;
      const float rstd = r ? rs.y : rs.x;
      T* y = static_cast<T*>(p.y) + smp[r] * p.y_batch + (at_row[r] - smp[r] * p.rows) * p.y_row;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
#pragma unroll
        for (int e = 0; e < 2; ++e) v[r][k][e] = ffma2(fmul2(v[r][k][e], both(rstd)), w[k][e], b[k][e]);
        Raw<T> out;
        unpairs<T>(out, v[r][k]);
        at.store(y, k, out);
      }
      if (me.t == 0) {
        if (p.mean) p.mean[at_row[r]] = r ? mean.y : mean.x;
        if (p.rstd) p.rstd[at_row[r]] = rstd;
      }
    }
    row += two ? 2 * step : step;
  }
  report(&abort_word);
}

// The forward pass of rows of more than 512 contiguous 16-bit elements, up to 2,048: a warp to a row, so
// that no barrier joins its sums, two rows at a time.  A lane keeps its elements as they were read (64 at
// most) and converts them for each of the three passes; the weight and bias, too many for registers,
// come from L1, once for both rows.
template <typename T, typename W, int NV>
__global__ void __launch_bounds__(512) norm_wide_kernel(const NormArgs p) {
  __shared__ uint64_t bars[kBars];
  __shared__ uint32_t abort_word;
  extern __shared__ __align__(16) uint8_t smem[];
  init_bars(bars, &abort_word, 2 * p.at_once * p.slots);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t first = blockIdx.x * p.at_once, r1 = (uint32_t)p.total, step = gridDim.x * p.at_once;
  if (warp == p.at_once) {             // producer warp: a lane to a row group
    if (lane < p.at_once) {
      Ring<T, 1> ring(p, lane, bars, smem, &abort_word);
      for (uint32_t row = first + lane; row < r1; row += step, ring.next()) {
        if (!ring.wait_free()) break;
        const uint32_t s = p.div_rows.div(row), i = row - s * p.rows;
        const T* src[1] = {static_cast<const T*>(p.x) + s * p.x_batch + i * p.x_row};
        ring.issue(ring.slot, src);
      }
    }
    __syncwarp();
    report(&abort_word);
    return;
  }
  Ring<T, 1> ring(p, warp, bars, smem, &abort_word);
  const Span<true, NV> at(lane, p.C);
  const float2 plus = both(p.w ? p.plus : 1.f);
  for (uint32_t row = first + warp; row < r1;) {
    uint32_t smp[2] = {p.div_rows.div(row), 0};
    bool two = row + step < r1;
    if (two) smp[1] = p.div_rows.div(row + step);
    two = two && (p.w_batch == 0 || smp[1] == smp[0]);
    Raw<T> v[2][NV];
    float2 sum[2] = {both(0.f), both(0.f)};
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      if (r == 1 && !two) break;
      const uint32_t i = row + r * step - smp[r] * p.rows;
      if (!ring.wait()) {
        report(&abort_word);
        return;
      }
      at.load_row(ring.row(0, static_cast<const T*>(p.x) + smp[r] * p.x_batch + i * p.x_row), v[r]);
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        float2 f[2];
        pairs<T>(v[r][k], f);
        sum[r] = fadd2(sum[r], fadd2(f[0], f[1]));
      }
      __syncwarp();
      if (lane == 0) ring.release(ring.slot);
      ring.next();
    }
    float mean[2], rstd[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) mean[r] = warp_sum(sum[r].x + sum[r].y) * p.inv_c;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const float2 nm = both(-mean[r]);
      float2 sq = both(0.f);
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        opaque(v[r][k]);               // convert again instead of keeping fp32 copies
        float2 f[2];
        pairs<T>(v[r][k], f);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float2 d = fadd2(f[e], nm);
          if (!at.full && !at.has(k, 0)) d = both(0.f);      // the zeros behind the row stay zeros
          sq = ffma2(d, d, sq);
        }
      }
      rstd[r] = sq.x + sq.y;
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) rstd[r] = 1.0f / sqrtf(warp_sum(rstd[r]) * p.inv_c + p.eps);
    const W* w = static_cast<const W*>(p.w) + smp[0] * p.w_batch;
    const W* b = static_cast<const W*>(p.b) + smp[0] * p.w_batch;
    T* y[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) y[r] = static_cast<T*>(p.y) + smp[r] * p.y_batch + (int64_t)(row + r * step - smp[r] * p.rows) * p.y_row;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      float2 wv[2] = {both(0.f), both(0.f)}, bv[2] = {both(0.f), both(0.f)};
      if (p.w) pairs<W>(at.load_any(w, k), wv);
      if (p.b) pairs<W>(at.load_any(b, k), bv);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        if (r == 1 && !two) break;
        opaque(v[r][k]);
        float2 f[2];
        pairs<T>(v[r][k], f);
#pragma unroll
        for (int e = 0; e < 2; ++e)
          f[e] = ffma2(fmul2(fadd2(f[e], both(-mean[r])), both(rstd[r])), fadd2(wv[e], plus), bv[e]);
        Raw<T> out;
        unpairs<T>(out, f);
        at.store(y[r], k, out);
      }
    }
    if (lane < (two ? 2 : 1)) {
      if (p.mean) p.mean[row + lane * step] = lane ? mean[1] : mean[0];
      if (p.rstd) p.rstd[row + lane * step] = lane ? rstd[1] : rstd[0];
    }
    row += two ? 2 * step : step;
  }
  report(&abort_word);
}

// The same walk; the columns' sums of dy xh and dy stay in registers.
template <typename T, typename W, bool CONTIG, int NV, bool MULTI>
__global__ void __launch_bounds__(NV == 8 ? 544 : 512) norm_bwd_kernel(const NormArgs p) {
  __shared__ float2 red[64];
  __shared__ uint64_t bars[kBars];
  __shared__ uint32_t abort_word;
  extern __shared__ __align__(16) uint8_t smem[];
  init_bars(bars, &abort_word, 2 * p.at_once * p.slots);
  const int64_t group = blockIdx.x / p.runs_per_group, run = blockIdx.x - group * p.runs_per_group;
  const uint32_t first = (uint32_t)(group * p.group_rows + p.group_rows * run / p.runs_per_group);
  const uint32_t r1 = (uint32_t)(group * p.group_rows + p.group_rows * (run + 1) / p.runs_per_group);
  if (threadIdx.x >= p.at_once * p.warps * 32) {             // producer warp: a lane to a row group
    const int g = threadIdx.x & 31;
    if (g < p.at_once) {
      Ring<T, 2> ring(p, g, bars, smem, &abort_word);
      for (uint32_t row = first + g; row < r1; row += p.at_once, ring.next()) {
        if (!ring.wait_free()) break;
        const uint32_t s = p.div_rows.div(row), i = row - s * p.rows;
        const T* src[2] = {static_cast<const T*>(p.x) + s * p.x_batch + i * p.x_row,
                           static_cast<const T*>(p.dy) + s * p.dy_batch + i * p.dy_row};
        ring.issue(ring.slot, src);
      }
    }
    __syncwarp();
    report(&abort_word);
    if (p.part) {                      // the barriers of the sums below
      __syncthreads();
      if (p.at_once > 1) __syncthreads();
    }
    return;
  }
  Row<MULTI> me(p, red);
  const Span<CONTIG, NV> at(me.t, p.C);
  Ring<T, 2> ring(p, me.group, bars, smem, &abort_word);
  const uint32_t r0 = first + me.group;
  float2 dw[NV][2], db[NV][2], w[NV][2];
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      dw[k][e] = db[k][e] = both(0.f);
      w[k][e] = both(1.f);
    }
  if (p.w) {                           // a run's rows share their weight
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      pairs<W>(at.load_any(static_cast<const W*>(p.w) + group * p.w_batch, k), w[k]);
#pragma unroll
      for (int e = 0; e < 2; ++e) w[k][e] = fadd2(w[k][e], both(p.plus));
    }
  }
  float mean = 0.f, rstd = 0.f;        // of the next row
  if (r0 < r1) {
    mean = __ldg(p.mean + r0);
    rstd = __ldg(p.rstd + r0);
  }
  for (uint32_t row = r0; row < r1; row += p.at_once, ring.next()) {
    const uint32_t s = p.div_rows.div(row), i = row - s * p.rows;
    const T* x = ring.row(0, static_cast<const T*>(p.x) + s * p.x_batch + i * p.x_row);
    const T* dy = ring.row(1, static_cast<const T*>(p.dy) + s * p.dy_batch + i * p.dy_row);
    const float2 nm = both(-mean), rs = both(rstd);
    if (row + p.at_once < r1) {
      mean = __ldg(p.mean + row + p.at_once);
      rstd = __ldg(p.rstd + row + p.at_once);
    }
    const bool ok = ring.wait();       // (after one that ran out the rows' barriers are still kept)
    float2 xh[NV][2], g[NV][2], a = both(0.f), b = both(0.f);
    Raw<T> rx[NV], rg[NV];
    at.load_row(x, rx);
    at.load_row(dy, rg);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      pairs<T>(rx[k], xh[k]);
      pairs<T>(rg[k], g[k]);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        xh[k][e] = fmul2(fadd2(xh[k][e], nm), rs);
        dw[k][e] = ffma2(g[k][e], xh[k][e], dw[k][e]);
        db[k][e] = fadd2(db[k][e], g[k][e]);
        g[k][e] = fmul2(g[k][e], w[k][e]);
        a = fadd2(a, g[k][e]);
        b = ffma2(g[k][e], xh[k][e], b);
      }
    }
    const float2 ab = me.sum(make_float2(a.x + a.y, b.x + b.y), p.warps);
    if (me.t == 0) ring.release(ring.slot);     // every thread of the row has read its slot
    if (!ok) continue;
    const float2 am = both(-ab.x * p.inv_c), bm = both(-ab.y * p.inv_c);
    T* dx = static_cast<T*>(p.y) + s * p.y_batch + i * p.y_row;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
#pragma unroll
      for (int e = 0; e < 2; ++e) g[k][e] = fmul2(rs, ffma2(xh[k][e], bm, fadd2(g[k][e], am)));
      Raw<T> out;
      unpairs<T>(out, g[k]);
      at.store(dx, k, out);
    }
  }
  report(&abort_word);
  if (!p.part) return;
  // the row groups hold sums of the same columns: side by side in the slots' memory, then added in order
  float* out = p.part + (int64_t)blockIdx.x * 2 * p.C;
  float* acc = reinterpret_cast<float*>(smem);           // [at_once][2][C]
  float* mine = p.at_once > 1 ? acc + (int64_t)me.group * 2 * p.C : out;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (!at.has(k, e)) continue;
      const int c = at.col + at.offset(k, e);
      mine[c] = e & 1 ? dw[k][e / 2].y : dw[k][e / 2].x;
      mine[p.C + c] = e & 1 ? db[k][e / 2].y : db[k][e / 2].x;
    }
  if (p.at_once == 1) return;
  __syncthreads();
  for (int c = threadIdx.x; c < 2 * p.C; c += blockDim.x - 32) {
    float t = acc[c];
    for (int q = 1; q < p.at_once; ++q) t += acc[(int64_t)q * 2 * p.C + c];
    out[c] = t;
  }
}

// Adds the runs of a group: block (32 columns, 32 lanes of runs), grid (columns / 32, groups, 2).
template <typename O>
__global__ void __launch_bounds__(1024) norm_reduce_kernel(const float* part, int C, int runs, O* dw, O* db) {
  O* out = blockIdx.z ? db : dw;
  if (!out) return;
  __shared__ float acc[32][33];
  const int c = blockIdx.x * 32 + threadIdx.x;
  const int64_t g = blockIdx.y;
  float s = 0.f;
  if (c < C)
    for (int r = threadIdx.y; r < runs; r += 32) s += part[((g * runs + r) * 2 + blockIdx.z) * C + c];
  acc[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  // warp y adds column y's 32 lanes, in the order of a fixed tree
  s = warp_sum(acc[threadIdx.x][threadIdx.y]);
  const int col = blockIdx.x * 32 + threadIdx.y;
  if (threadIdx.x == 0 && col < C) out[g * C + col] = from_f32<O>(s);
}

// How a row is spread: its warps, and its pieces of four elements per lane, four at most (eight where 15
// warps would not hold the row).
struct Spread {
  int warps, nv;
};
Spread spread(int C) {
  const int most = C <= 7680 ? 4 : 8, pieces = (C + 3) / 4;
  const int warps = (pieces + 32 * most - 1) / (32 * most);
  return {warps, (pieces + 32 * warps - 1) / (32 * warps)};
}

constexpr int kSmem = 200 * 1024;      // shared memory for the slots of a block at most
constexpr int kSlack = 4096;           // the row's last warp reads its whole span, up to 1,024 elements

// Rows of a block at a time (15 warps and the producer, one block per multiprocessor: 512 threads leave
// 128 registers to each), and the rows in flight behind each: as many as fit, 8 at most.  The backward pass's groups
// leave their sums in the same memory.
void plan_block(NormArgs& a, bool bwd, int elem, int64_t rows_per_block) {
  const int tensors = bwd ? 2 : 1;
  a.slot_bytes = (a.C * elem + 31) & ~15;                  // a row that starts anywhere
  a.at_once = std::max(1, 15 / a.warps);                   // (the widest rows: 16 warps and the producer)
  a.at_once = (int)std::max<int64_t>(1, std::min<int64_t>(a.at_once, rows_per_block));
  a.at_once = std::min(a.at_once, std::max(1, kSmem / (tensors * a.slot_bytes)));
  if (bwd) a.at_once = std::min(a.at_once, std::max(1, kSmem / (2 * a.C * (int)sizeof(float))));
  // (a wide row's weight needs room in L1)
  a.slots = std::max(1, std::min(a.wide ? 2 : 8, kSmem / (a.at_once * tensors * a.slot_bytes)));
}
int smem_bytes(const NormArgs& a, bool bwd) {
  const int ring = a.at_once * a.slots * (bwd ? 2 : 1) * a.slot_bytes + kSlack;
  return std::max(ring, bwd && a.at_once > 1 ? a.at_once * 2 * a.C * (int)sizeof(float) : 0);
}

// Runs of a group in the backward pass: one block per multiprocessor, no more than rows.
int runs_of(int64_t group_rows, int64_t groups, int sms) {
  return (int)std::max<int64_t>(1, std::min(std::max<int64_t>(1, sms / groups), group_rows));
}

// (The limit is the most that any call takes, set once: one that followed the call's own size could be
// lowered by another thread's call before this one's launch.)
template <auto kernel>
cudaError_t launch_one(int blocks, int threads, int smem, const NormArgs& a, cudaStream_t st) {
  static OncePerDevice limit;
  const cudaError_t e = limit([] { return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem + kSlack); });
  if (e != cudaSuccess) return e;
  kernel<<<blocks, threads, smem, st>>>(a);
  return cudaGetLastError();
}

template <typename T, typename W>
cudaError_t launch_wide(const NormArgs& a, int blocks, cudaStream_t st) {
  const int threads = 32 * (a.at_once + 1), smem = smem_bytes(a, false);
  if (a.C <= 1024) return launch_one<norm_wide_kernel<T, W, 8>>(blocks, threads, smem, a, st);
  if (a.C <= 1536) return launch_one<norm_wide_kernel<T, W, 12>>(blocks, threads, smem, a, st);
  return launch_one<norm_wide_kernel<T, W, 16>>(blocks, threads, smem, a, st);
}

template <typename T, typename W, bool CONTIG, int NV>
cudaError_t launch_nv(bool bwd, const NormArgs& a, int blocks, cudaStream_t st) {
  const int threads = 32 * (a.warps * a.at_once + 1), smem = smem_bytes(a, bwd);
  if (!bwd)
    return a.warps > 1 ? launch_one<norm_fwd_kernel<T, W, CONTIG, NV, true>>(blocks, threads, smem, a, st)
                       : launch_one<norm_fwd_kernel<T, W, CONTIG, NV, false>>(blocks, threads, smem, a, st);
  return a.warps > 1 ? launch_one<norm_bwd_kernel<T, W, CONTIG, NV, true>>(blocks, threads, smem, a, st)
                     : launch_one<norm_bwd_kernel<T, W, CONTIG, NV, false>>(blocks, threads, smem, a, st);
}

template <typename T, typename W, bool CONTIG>
cudaError_t launch_pieces(bool bwd, const NormArgs& a, int nv, int blocks, cudaStream_t st) {
  return nv <= 1   ? launch_nv<T, W, CONTIG, 1>(bwd, a, blocks, st)
         : nv <= 2 ? launch_nv<T, W, CONTIG, 2>(bwd, a, blocks, st)
         : nv <= 3 ? launch_nv<T, W, CONTIG, 3>(bwd, a, blocks, st)
         : nv <= 4 ? launch_nv<T, W, CONTIG, 4>(bwd, a, blocks, st)
                   : launch_nv<T, W, CONTIG, 8>(bwd, a, blocks, st);
}

template <typename T, typename W>
cudaError_t launch_norm(bool bwd, bool contig, const NormArgs& a, int nv, int blocks, cudaStream_t st) {
  if constexpr (sizeof(T) == 2)
    if (a.wide) return launch_wide<T, W>(a, blocks, st);
  return contig ? launch_pieces<T, W, true>(bwd, a, nv, blocks, st) : launch_pieces<T, W, false>(bwd, a, nv, blocks, st);
}

cudaError_t dispatch(bool bwd, int dtype, int wdtype, bool contig, const NormArgs& a, int nv, int blocks, cudaStream_t st) {
  const bool wf = wdtype == ULTRAGEN_F32;
  if (dtype == ULTRAGEN_BF16)
    return wf ? launch_norm<__nv_bfloat16, float>(bwd, contig, a, nv, blocks, st)
              : launch_norm<__nv_bfloat16, __nv_bfloat16>(bwd, contig, a, nv, blocks, st);
  if (dtype == ULTRAGEN_F16)
    return wf ? launch_norm<__half, float>(bwd, contig, a, nv, blocks, st)
              : launch_norm<__half, __half>(bwd, contig, a, nv, blocks, st);
  return launch_norm<float, float>(bwd, contig, a, nv, blocks, st);
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

// Whether a tensor with strides (row, batch) at `p` is all of another at `q`: the same elements at the same
// places, so that an output may replace it, or has no element in common with its first.
bool same_or_apart(const ultragen_norm_t* n, const void* p, int64_t row, int64_t batch, const void* q, int64_t qrow, int64_t qbatch) {
  return p != q || ((n->rows == 1 || row == qrow) && (n->batch == 1 || batch == qbatch));
}

// Whether an operand's rows start on `bytes`.
bool starts_on(const void* p, int64_t row, int64_t batch, int bytes, int dtype) {
  const int e = elem_size(dtype);
  return p == nullptr || ((uintptr_t)p % bytes == 0 && row * e % bytes == 0 && batch * e % bytes == 0);
}

NormArgs args_of(const ultragen_norm_t* n) {
  NormArgs a = {};
  a.total = (int64_t)n->batch * n->rows;
  a.rows = n->rows;
  a.div_rows = FastDiv((uint32_t)std::max(1, n->rows));
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

// Whether every row, and every sample's weight, starts on four elements.
bool contiguous_pieces(const ultragen_norm_t* n, const void* x, const void* dy, const void* y, const void* w,
               const void* b) {
  const int e = 4 * elem_size(n->dtype), we = 4 * elem_size(n->wdtype);
  const int64_t wb = n->per_sample ? n->cols : 0;
  return n->cols % 4 == 0 && starts_on(x, n->x_row, n->x_batch, e, n->dtype) &&
         starts_on(dy, n->dy_row, n->dy_batch, e, n->dtype) &&
         starts_on(y, n->y_row, n->y_batch, e, n->dtype) && starts_on(w, wb, wb, we, n->wdtype) &&
         starts_on(b, wb, wb, we, n->wdtype);
}

int status_of(cudaError_t e) { return e == cudaSuccess ? ULTRAGEN_OK : ULTRAGEN_ERR_CUDA; }

}  // namespace

cudaError_t norm_status(int* code, cudaStream_t s) { return read_clear_error(&g_error, code, s); }

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
  if (!same_or_apart(n, y, n->y_row, n->y_batch, x, n->x_row, n->x_batch) || begins_at(y, {weight, bias, mean, rstd}) ||
      begins_at(mean, {rstd}))
    return ULTRAGEN_ERR_INVALID_ARG;
  int dev;
  if ((st = current_device(&dev)) != ULTRAGEN_OK) return st;
  NormArgs a = args_of(n);
  a.x = x;
  a.w = weight;
  a.b = bias;
  a.y = y;
  a.mean = mean;
  a.rstd = rstd;
  const bool contig = contiguous_pieces(n, x, nullptr, y, weight, bias);
  Spread sp = spread(n->cols);
  // A warp to a row where every warp has several; with fewer, warps that share a row are sooner done.  In us,
  // by a warp to a row and by warps that share one: rows of 2,048, 4,736 of them 15.1 and 13.7, 9,472 (the
  // border) 25.3 and 23.5, 20,000 43.7 and 45.7, 70,144 113 and 150; rows of 516, 8.9 and 7.1, 12.2 and 11.4,
  // 18.9 and 20.2, 55 and 62.  768, 1,024 and 1,536 columns lie between, with 4 to 11% lost at the border.
  a.wide = contig && n->dtype != ULTRAGEN_F32 && n->cols > 512 && n->cols <= 2048 && a.total >= 64 * (int64_t)sm_count();
  if (a.wide) sp.warps = 1;
  a.warps = sp.warps;
  plan_block(a, false, elem_size(n->dtype), (a.total + sm_count() - 1) / sm_count());
  const int64_t blocks = std::min<int64_t>((a.total + a.at_once - 1) / a.at_once, sm_count());
  return status_of(dispatch(false, n->dtype, n->wdtype, contig, a, sp.nv, (int)blocks,
                            reinterpret_cast<cudaStream_t>(stream)));
}

int ultragen_layer_norm_backward_workspace(const ultragen_norm_t* n, size_t* bytes) {
  int st = check(n);
  if (st != ULTRAGEN_OK) return st;
  if (!bytes) return ULTRAGEN_ERR_INVALID_ARG;
  const NormArgs a = args_of(n);
  const int64_t groups = n->per_sample ? n->batch : 1;
  *bytes = a.total == 0 ? 0 : (size_t)groups * runs_of(a.group_rows, groups, sm_count()) * 2 * n->cols * sizeof(float);
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
  if (!same_or_apart(n, dx, n->y_row, n->y_batch, x, n->x_row, n->x_batch) ||
      !same_or_apart(n, dx, n->y_row, n->y_batch, dy, n->dy_row, n->dy_batch) ||
      begins_at(dx, {weight, mean, rstd, dweight, dbias}) || begins_at(dweight, {dbias}))
    return ULTRAGEN_ERR_INVALID_ARG;
  if ((st = current_device(&dev)) != ULTRAGEN_OK) return st;
  const bool contig = contiguous_pieces(n, x, dy, dx, weight, nullptr);
  const Spread sp = spread(n->cols);
  a.warps = sp.warps;
  a.runs_per_group = runs_of(a.group_rows, groups, sm_count());
  plan_block(a, true, elem_size(n->dtype), (a.group_rows + a.runs_per_group - 1) / a.runs_per_group);
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
  st = status_of(dispatch(true, n->dtype, n->wdtype, contig, a, sp.nv, (int)(groups * a.runs_per_group), s));
  if (st != ULTRAGEN_OK || !a.part) return st;
  const dim3 grid((n->cols + 31) / 32, (unsigned)groups, 2), block(32, 32);
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
