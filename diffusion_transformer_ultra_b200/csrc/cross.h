// Cross attention: what its entry points (cross_attention.cu) and its kernels (cross_fwd.cu,
// cross_bwd.cu) share.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "kernels.h"

namespace ug {

// Query rows are packed by key/value head: row tok * group + g of a unit (sample b, key/value
// head hk) is query tok of head hk * group + g, so that heads which share keys and values also
// share their tiles.  A 128-row query tile holds `toks` = 128 / group whole queries; the rows
// behind them (group not a divisor of 128) stay zero.
struct CrossParams {
  int batch, nq, ns, heads, kv_heads, group, toks;
  int group_inv;                   // ceil(2^16 / group): r / group = (r * group_inv) >> 16 for r < 128
  int units, nqt;                  // batch * kv_heads; query tiles per unit
  int total;                       // work items of the launch
  int per_item;                    // query tiles of an item (1 or 2)
  FastDiv div_h, div_kv, div_q, div_kt, div_split;   // by heads, kv_heads, items along the queries, key tiles, nsplit
  int nitem_q;                     // items along a unit's queries: ceil(nqt / per_item)
  int nsplit;                      // items along its keys (backward: along its queries)
  float scale, scale_log2;         // scale, scale * log2(e)
  const int32_t* lens;             // [batch], or null
  const uint32_t* words;           // [batch][word_tiles * 4] visibility bits, or null
  const int32_t* single;           // [batch] 1: exactly one key is visible (with words)
  int word_tiles;                  // 128-key tiles of the bit words
  int scrub;                       // hidden keys exist below ns: their rows are zeroed in shared memory
  // tensors written or read by threads: base and batch, row, head strides (elements)
  void* out[3];                    // forward: o; dQ kernel: dq; dK/dV kernel: dk, dv
  int64_t out_st[3][3];
  const void* o;                   // backward: o and do of the rows, for delta
  const void* d_o;
  int64_t o_st[3], do_st[3];
  float* lse;                      // [batch][heads][nq]; forward: output or null, backward: input
  float* delta;                    // backward: [batch][heads][nq] do . o
  float* part;                     // partial results of split items (null: nsplit == 1)
  int part_rows;                   // rows stored per (unit, query tile, split)
  unsigned long long timeout_ns;
};

struct CrossMaps {
  CUtensorMap q, k, v, d_o;
};

// Keys [0, len) of sample b may be visible.
__host__ __device__ inline int cross_clamp_len(int len, int ns) { return len < 0 ? 0 : (len > ns ? ns : len); }

cudaError_t launch_cross_fwd(const CrossMaps& m, const CrossParams& p, int dtype, int D, int grid, cudaStream_t s);
cudaError_t launch_cross_dq(const CrossMaps& m, const CrossParams& p, int dtype, int D, int grid, cudaStream_t s);
cudaError_t launch_cross_dkv(const CrossMaps& m, const CrossParams& p, int dtype, int D, int grid, cudaStream_t s);
// Device error words of the kernels: read and cleared, in stream order; waits for `s`.
cudaError_t cross_fwd_status(int* code, cudaStream_t s);
cudaError_t cross_bwd_status(int* code, cudaStream_t s);
cudaError_t norm_status(int* code, cudaStream_t s);
// Reads `symbol` (a device int) after the work of `s`, and clears it if it is set.
cudaError_t read_clear_error(const void* symbol, int* code, cudaStream_t s);

}  // namespace ug
