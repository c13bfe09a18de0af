// Layer norm over the last dimension, forward and backward, with one weight for every row or
// one per sample (the modulation of a diffusion transformer).
//
//   mu = sum(x) / C,  r = (sum((x - mu)^2) / C + eps)^-1/2,  xh = (x - mu) r
//   y  = xh w' + b,   w' = w, or 1 + w (plus_one), or 1 without a weight
//   g  = dy w',       dx = r (g - sum(g) / C - xh sum(g xh) / C)
//   dw = sum over rows of dy xh,   db = sum over rows of dy
//
// Both passes are bound by HBM: x is read and y written once (x, dy read and dx written once).
// A row belongs to one warp up to 2,048 elements of 16 bits (1,024 of 32; the backward pass, which
// keeps the weight's gradient too, fewer), else to a group of warps.  Its rows come by bulk copies,
// several ahead, into shared memory (a persistent block per multiprocessor has up to 200 KB of them in
// flight), and from there to registers, as they were read, so that the variance takes a second pass
// over registers (no cancellation of sum(x^2) against mu^2).  A copy covers the 16-byte pieces that
// hold the row, so that a row may start anywhere; one that does not start on four elements is then
// worked on element by element.  All sums are fp32.
// With the loads ahead of time the instructions and the weight's way from L1 set the pace: arithmetic
// is on pairs, and a lane's piece is four elements, so that a warp's fp32 weights are one contiguous
// 512-byte load.  (With pieces of eight, whose fp32 weights a warp reads in halves of 32-byte sectors,
// and scalar arithmetic, the forward pass took 150 instead of 1XX us for 70,144 x 2,048 bf16.)
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
  int64_t total;           // rows of all samples
  int rows, C;             // rows per sample
  FastDiv div_rows;        // by rows
  int64_t w_batch;         // C with a weight per sample, else 0
  int runs_per_group;      // runs of a sample (of everything with a shared weight)
  int64_t group_rows;      // rows of a sample (of everything with a shared weight)
  int warps;               // warps of a row
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
    x = lane < warps ? buf[lane] : make_float2(0.f, 0.f);
    x.x = warp_sum(x.x);
    x.y = warp_sum(x.y);
    return x;
  }
};

__device__ int g_error;                // a wait that ran out since the last status read

constexpr uint32_t kWaitNs = 2000u * 1000 * 1000;

// The rows of one row group on their way through shared memory: `slots` slots of N tensors' rows each.
template <typename T, int N>
struct Ring {
  uint32_t bar, abort_word;            // barriers of this group's slots
  uint8_t* buf;
  int slots, slot_bytes, row_bytes, slot;
  uint32_t phase;
  __device__ __forceinline__ Ring(const NormArgs& p, int group, uint64_t* bars, uint8_t* smem, uint32_t* abort)
      : bar(smem_u32(bars + group * p.slots)), abort_word(smem_u32(abort)),
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
  __device__ __forceinline__ void next() {
    if (++slot == slots) {
      slot = 0;
      phase ^= 1;
    }
  }
};

// Barriers of a block's slots (at most kBars in all).
constexpr int kBars = 128;
__device__ __forceinline__ void init_bars(uint64_t* bars, uint32_t* abort, int n) {
  for (int i = threadIdx.x; i < n; i += blockDim.x) mbar_init(smem_u32(bars + i), 1);
  if (threadIdx.x == 0) *abort = 0;
  fence_mbar_init();
  __syncthreads();
}
__device__ __forceinline__ void report(const uint32_t* abort) {
  const int code = *reinterpret_cast<const volatile int*>(abort);
  if (code == 0) return;
  if ((threadIdx.x & 31) == 0) atomicExch(&g_error, code);
  settle();
}

// The vector's registers as values the compiler knows nothing about.
template <typename T>
__device__ __forceinline__ void opaque(Vec<T, 4>& v) {
#pragma unroll
  for (int i = 0; i < (int)sizeof(T); ++i) asm volatile("" : "+r"(reinterpret_cast<uint32_t*>(&v)[i]));
}

// A piece: four elements of a row, as fp32 pairs.
template <typename T>
__device__ __forceinline__ void pairs(const Vec<T, 4>& v, float2 (&out)[2]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if constexpr (sizeof(T) == 4) {
      out[i] = make_float2(v.v[2 * i], v.v[2 * i + 1]);
    } else if constexpr (std::is_same<T, __half>::value) {
      out[i] = __half22float2(reinterpret_cast<const __half2*>(&v)[i]);
    } else {
      const uint32_t w = reinterpret_cast<const uint32_t*>(&v)[i];
      out[i] = make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
  }
}
template <typename T>
__device__ __forceinline__ void unpairs(Vec<T, 4>& v, const float2 (&in)[2]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if constexpr (sizeof(T) == 4) {
      v.v[2 * i] = in[i].x;
      v.v[2 * i + 1] = in[i].y;
    } else {
      reinterpret_cast<uint32_t*>(&v)[i] = pack2<T>(in[i].x, in[i].y);
    }
  }
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// Piece k of thread t of a row's `threads`: columns 4 (t + k threads) and on where rows start on four
// elements (CONTIG; C is then a multiple of four), else t + (4 k + e) threads, element by element.
template <bool CONTIG>
struct Piece {
  int col, step, C;
  __device__ __forceinline__ Piece(int t, int k, int threads, int C_)
      : col(CONTIG ? (t + k * threads) * 4 : t + 4 * k * threads), step(CONTIG ? 1 : threads), C(C_) {}
  __device__ __forceinline__ bool any() const { return col < C; }
  __device__ __forceinline__ int at(int e) const { return col + e * step; }
  __device__ __forceinline__ bool has(int e) const { return CONTIG || at(e) < C; }
  template <typename T>
  __device__ __forceinline__ Vec<T, 4> load(const T* p) const {   // zeros behind the row
    Vec<T, 4> v{};
    if (CONTIG) {
      if (any()) v = *reinterpret_cast<const Vec<T, 4>*>(p + col);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (has(e)) v.v[e] = p[at(e)];
    }
    return v;
  }
  template <typename T>
  __device__ __forceinline__ void store(T* p, const Vec<T, 4>& v) const {
    if (CONTIG) {
      if (any()) *reinterpret_cast<Vec<T, 4>*>(p + col) = v;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (has(e)) p[at(e)] = v.v[e];
    }
  }
};

template <typename T, typename W, bool CONTIG, int NV, bool MULTI>
__global__ void __launch_bounds__(512) norm_fwd_kernel(const NormArgs p) {
  __shared__ float2 red[64];
  __shared__ uint64_t bars[kBars];
  __shared__ uint32_t abort_word;
  extern __shared__ __align__(16) uint8_t smem[];
  init_bars(bars, &abort_word, p.at_once * p.slots);
  Row<MULTI> me(p, red);
  Ring<T, 1> ring(p, me.group, bars, smem, &abort_word);
  const int64_t first = (int64_t)blockIdx.x * p.at_once + me.group, step = (int64_t)gridDim.x * p.at_once;
  auto source = [&](int64_t row) {
    const uint32_t s = p.div_rows.div((uint32_t)row), i = (uint32_t)row - s * p.rows;
    return static_cast<const T*>(p.x) + s * p.x_batch + i * p.x_row;
  };
  if (me.t == 0)
    for (int k = 0; k < p.slots && first + k * step < p.total; ++k) {
      const T* src[1] = {source(first + k * step)};
      ring.issue(k, src);
    }
  for (int64_t row = first; row < p.total; row += step, ring.next()) {
    const uint32_t s = p.div_rows.div((uint32_t)row), i = (uint32_t)row - s * p.rows;
    const T* x = ring.row(0, static_cast<const T*>(p.x) + s * p.x_batch + i * p.x_row);
    const bool ok = ring.wait();       // (after one that ran out the rows' barriers are still kept)
    Vec<T, 4> v[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) v[k] = Piece<CONTIG>(me.t, k, me.threads, p.C).load(x);
    float2 sum[2] = {both(0.f), both(0.f)};
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      float2 f[2];
      pairs<T>(v[k], f);
#pragma unroll
      for (int e = 0; e < 2; ++e) sum[e & 1] = fadd2(sum[e & 1], f[e]);
    }
    sum[0] = fadd2(sum[0], sum[1]);
    const float mean = me.sum(make_float2(sum[0].x + sum[0].y, 0.f), p.warps).x * p.inv_c;
    if (me.t == 0 && ok && row + p.slots * step < p.total) {     // every thread of the row has read its slot
      const T* src[1] = {source(row + p.slots * step)};
      ring.issue(ring.slot, src);
    }
    const float2 nm = both(-mean);
    float2 sq[2] = {both(0.f), both(0.f)};
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      opaque(v[k]);                    // convert again instead of keeping fp32 copies
      const Piece<CONTIG> at(me.t, k, me.threads, p.C);
      if (!at.any()) continue;
      float2 f[2];
      pairs<T>(v[k], f);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float2 d = fadd2(f[e], nm);
        if (!at.has(2 * e)) d.x = 0.f;
        if (!at.has(2 * e + 1)) d.y = 0.f;
        sq[e & 1] = ffma2(d, d, sq[e & 1]);
      }
    }
    sq[0] = fadd2(sq[0], sq[1]);
    const float rstd = 1.0f / sqrtf(me.sum(make_float2(sq[0].x + sq[0].y, 0.f), p.warps).x * p.inv_c + p.eps);
    if (!ok) continue;
    T* y = static_cast<T*>(p.y) + s * p.y_batch + i * p.y_row;
    const W* w = p.w ? static_cast<const W*>(p.w) + s * p.w_batch : nullptr;
    const W* b = p.b ? static_cast<const W*>(p.b) + s * p.w_batch : nullptr;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      opaque(v[k]);
      const Piece<CONTIG> at(me.t, k, me.threads, p.C);
      if (!at.any()) continue;
      float2 f[2], wv[2], bv[2];
      pairs<T>(v[k], f);
      if (w) pairs<W>(at.load(w), wv);
      if (b) pairs<W>(at.load(b), bv);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        f[e] = fmul2(fadd2(f[e], nm), both(rstd));
        f[e] = ffma2(f[e], w ? fadd2(wv[e], both(p.plus)) : both(1.0f), b ? bv[e] : both(0.f));
      }
      unpairs<T>(v[k], f);
      at.store(y, v[k]);
    }
    if (me.t == 0) {
      if (p.mean) p.mean[row] = mean;
      if (p.rstd) p.rstd[row] = rstd;
    }
  }
  report(&abort_word);
}

// One block walks the rows [r0, r1) of run blockIdx.x, its row groups in turn.
template <typename T, typename W, bool CONTIG, int NV, bool MULTI>
__global__ void __launch_bounds__(512) norm_bwd_kernel(const NormArgs p) {
  __shared__ float2 red[64];
  __shared__ uint64_t bars[kBars];
  __shared__ uint32_t abort_word;
  extern __shared__ __align__(16) uint8_t smem[];
  init_bars(bars, &abort_word, p.at_once * p.slots);
  Row<MULTI> me(p, red);
  Ring<T, 2> ring(p, me.group, bars, smem, &abort_word);
  const int64_t group = blockIdx.x / p.runs_per_group;
  const int64_t run = blockIdx.x - group * p.runs_per_group;
  const int64_t r0 = group * p.group_rows + p.group_rows * run / p.runs_per_group;
  const int64_t r1 = group * p.group_rows + p.group_rows * (run + 1) / p.runs_per_group;
  float2 dw[NV][2], db[NV][2];
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int e = 0; e < 2; ++e) dw[k][e] = db[k][e] = both(0.f);
  auto issue = [&](int slot, int64_t row) {
    const uint32_t s = p.div_rows.div((uint32_t)row), i = (uint32_t)row - s * p.rows;
    const T* src[2] = {static_cast<const T*>(p.x) + s * p.x_batch + i * p.x_row,
                       static_cast<const T*>(p.dy) + s * p.dy_batch + i * p.dy_row};
    ring.issue(slot, src);
  };
  if (me.t == 0)
    for (int k = 0; k < p.slots && r0 + me.group + k * p.at_once < r1; ++k) issue(k, r0 + me.group + k * p.at_once);
  float mean = 0.f, rstd = 0.f;        // of the next row
  if (r0 + me.group < r1) {
    mean = __ldg(p.mean + r0 + me.group);
    rstd = __ldg(p.rstd + r0 + me.group);
  }
  for (int64_t row = r0 + me.group; row < r1; row += p.at_once, ring.next()) {
    const uint32_t s = p.div_rows.div((uint32_t)row), i = (uint32_t)row - s * p.rows;
    const T* x = ring.row(0, static_cast<const T*>(p.x) + s * p.x_batch + i * p.x_row);
    const T* dy = ring.row(1, static_cast<const T*>(p.dy) + s * p.dy_batch + i * p.dy_row);
    const W* w = p.w ? static_cast<const W*>(p.w) + s * p.w_batch : nullptr;
    const float2 nm = both(-mean), rs = both(rstd), plus = both(p.plus);
    if (row + p.at_once < r1) {
      mean = __ldg(p.mean + row + p.at_once);
      rstd = __ldg(p.rstd + row + p.at_once);
    }
    const bool ok = ring.wait();       // (after one that ran out the rows' barriers are still kept)
    Vec<T, 4> xv[NV], gv[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const Piece<CONTIG> at(me.t, k, me.threads, p.C);
      xv[k] = at.load(x);
      gv[k] = at.load(dy);
    }
    float2 a = both(0.f), b = both(0.f);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const Piece<CONTIG> at(me.t, k, me.threads, p.C);
      if (!at.any()) continue;
      float2 xf[2], gf[2], wv[2];
      pairs<T>(xv[k], xf);
      pairs<T>(gv[k], gf);
      if (w) pairs<W>(at.load(w), wv);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float2 xh = fmul2(fadd2(xf[e], nm), rs);
        dw[k][e] = ffma2(gf[e], xh, dw[k][e]);
        db[k][e] = fadd2(db[k][e], gf[e]);
        const float2 g = w ? fmul2(gf[e], fadd2(wv[e], plus)) : gf[e];
        a = fadd2(a, g);
        b = ffma2(g, xh, b);
      }
    }
    const float2 ab = me.sum(make_float2(a.x + a.y, b.x + b.y), p.warps);
    if (me.t == 0 && ok && row + (int64_t)p.slots * p.at_once < r1) issue(ring.slot, row + (int64_t)p.slots * p.at_once);
#pragma unroll
    for (int k = 0; k < NV; ++k) {     // convert again below instead of keeping fp32 copies
      opaque(xv[k]);
      opaque(gv[k]);
    }
    const float2 am = both(-ab.x * p.inv_c), bm = both(-ab.y * p.inv_c);
    if (!ok) continue;
    T* dx = static_cast<T*>(p.y) + s * p.y_batch + i * p.y_row;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const Piece<CONTIG> at(me.t, k, me.threads, p.C);
      if (!at.any()) continue;
      float2 xf[2], gf[2], wv[2];
      pairs<T>(xv[k], xf);
      pairs<T>(gv[k], gf);
      if (w) pairs<W>(at.load(w), wv);       // (again: cheaper than keeping g in fp32)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float2 xh = fmul2(fadd2(xf[e], nm), rs);
        const float2 g = w ? fmul2(gf[e], fadd2(wv[e], plus)) : gf[e];
        xf[e] = fmul2(rs, ffma2(xh, bm, fadd2(g, am)));
      }
      unpairs<T>(gv[k], xf);
      at.store(dx, gv[k]);
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
  for (int k = 0; k < NV; ++k) {
    const Piece<CONTIG> at(me.t, k, me.threads, p.C);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (at.at(e) >= p.C) continue;
      mine[at.at(e)] = e & 1 ? dw[k][e / 2].y : dw[k][e / 2].x;
      mine[p.C + at.at(e)] = e & 1 ? db[k][e / 2].y : db[k][e / 2].x;
    }
  }
  if (p.at_once == 1) return;
  __syncthreads();
  for (int c = threadIdx.x; c < 2 * p.C; c += blockDim.x) {
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

// How a row is spread: its warps and its pieces of four elements per lane, at most 16 of 16 bits and 8 of
// 32 bits or not contiguous; in the backward pass, with two sums beside each element, 6 and 4.  The
// widest rows take 8, so that 16 warps hold them.
struct Spread {
  int warps, nv;
};
Spread spread(bool bwd, bool contig, int C, int elem) {
  const bool light = contig && elem == 2;
  const int most = !bwd ? (light ? 16 : 8) : (C <= 8192 ? (light ? 6 : 4) : 8);
  const int pieces = (C + 3) / 4;
  const int warps = (pieces + 32 * most - 1) / (32 * most);
  return {warps, (pieces + 32 * warps - 1) / (32 * warps)};
}

constexpr int kSmem = 200 * 1024;      // dynamic shared memory of a block at most

// Rows of a block at a time (16 warps, one block per multiprocessor; named barriers give 15 groups of
// warps), and the rows in flight behind each: as many as fit, 8 at most.  The backward pass's groups
// leave their sums in the same memory.
void plan_block(NormArgs& a, bool bwd, int elem, int64_t rows_per_block) {
  const int tensors = bwd ? 2 : 1;
  a.slot_bytes = (a.C * elem + 31) & ~15;                  // a row that starts anywhere
  a.at_once = a.warps > 1 ? std::min(15, 16 / a.warps) : 16;
  a.at_once = (int)std::max<int64_t>(1, std::min<int64_t>(a.at_once, rows_per_block));
  a.at_once = std::min(a.at_once, std::max(1, kSmem / (tensors * a.slot_bytes)));
  if (bwd) a.at_once = std::min(a.at_once, std::max(1, kSmem / (2 * a.C * (int)sizeof(float))));
  a.slots = std::max(1, std::min(8, kSmem / (a.at_once * tensors * a.slot_bytes)));
}
int smem_bytes(const NormArgs& a, bool bwd) {
  const int ring = a.at_once * a.slots * (bwd ? 2 : 1) * a.slot_bytes;
  return std::max(ring, bwd && a.at_once > 1 ? a.at_once * 2 * a.C * (int)sizeof(float) : 0);
}

// Runs of a group in the backward pass: one block per multiprocessor, no more than rows.
int runs_of(int64_t group_rows, int64_t groups, int sms) {
  return (int)std::max<int64_t>(1, std::min(std::max<int64_t>(1, sms / groups), group_rows));
}

template <typename K>
cudaError_t launch_one(K kernel, int blocks, int threads, int smem, const NormArgs& a, cudaStream_t st) {
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  kernel<<<blocks, threads, smem, st>>>(a);
  return cudaGetLastError();
}

template <typename T, typename W, bool CONTIG, int NV>
cudaError_t launch_nv(bool bwd, const NormArgs& a, int blocks, cudaStream_t st) {
  const int threads = 32 * a.warps * a.at_once, smem = smem_bytes(a, bwd);
  if (!bwd)
    return a.warps > 1 ? launch_one(norm_fwd_kernel<T, W, CONTIG, NV, true>, blocks, threads, smem, a, st)
                       : launch_one(norm_fwd_kernel<T, W, CONTIG, NV, false>, blocks, threads, smem, a, st);
  if constexpr (NV <= 8)                                   // (no more: see spread)
    return a.warps > 1 ? launch_one(norm_bwd_kernel<T, W, CONTIG, NV, true>, blocks, threads, smem, a, st)
                       : launch_one(norm_bwd_kernel<T, W, CONTIG, NV, false>, blocks, threads, smem, a, st);
  return cudaErrorInvalidValue;
}

template <typename T, typename W, bool CONTIG>
cudaError_t launch_pieces(bool bwd, const NormArgs& a, int nv, int blocks, cudaStream_t st) {
  return nv <= 2    ? launch_nv<T, W, CONTIG, 2>(bwd, a, blocks, st)
         : nv <= 4  ? launch_nv<T, W, CONTIG, 4>(bwd, a, blocks, st)
         : nv <= 6  ? launch_nv<T, W, CONTIG, 6>(bwd, a, blocks, st)
         : nv <= 8  ? launch_nv<T, W, CONTIG, 8>(bwd, a, blocks, st)
         : nv <= 12 ? launch_nv<T, W, CONTIG, 12>(bwd, a, blocks, st)
                    : launch_nv<T, W, CONTIG, 16>(bwd, a, blocks, st);
}

template <typename T, typename W>
cudaError_t launch_norm(bool bwd, bool contig, const NormArgs& a, int nv, int blocks, cudaStream_t st) {
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
  const Spread sp = spread(false, contig, n->cols, elem_size(n->dtype));
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
  if ((st = current_device(&dev)) != ULTRAGEN_OK) return st;
  const bool contig = contiguous_pieces(n, x, dy, dx, weight, nullptr);
  const Spread sp = spread(true, contig, n->cols, elem_size(n->dtype));
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
