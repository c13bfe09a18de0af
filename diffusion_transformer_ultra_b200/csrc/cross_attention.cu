// Cross attention of one sequence's queries over another's keys and values, forward and backward:
//   s_ij = scale q_i . k_j over the visible keys j,  lse_i = log(sum_j exp(s_ij)),
//   p_ij = exp(s_ij - lse_i),  o_i = sum_j p_ij v_j
//   delta_i = do_i . o_i,  ds_ij = p_ij (do_i . v_j - delta_i)
//   dq_i = scale sum_j ds_ij k_j,  dk_j = scale sum_i ds_ij q_i,  dv_j = sum_i p_ij do_i
// This file holds the entry points, the schedules, and the small kernels beside the tensor-core ones
// (cross_fwd.cu, cross_bwd.cu): the bit words of a key mask and the join of split query rows.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "adapter.h"
#include "cross.cuh"
#include "device.h"
#include "elem.cuh"
#include "kernels.h"
#include "nvtx_range.h"
#include "ultragen.h"

namespace ug {
namespace {

// Bit words of the visible keys of each sample (mask and length), and whether exactly one is.
// One block per sample.
__global__ void __launch_bounds__(256) mask_words_kernel(const uint8_t* mask, const int32_t* lens, int ns, int word_tiles,
                                                         uint32_t* words, int32_t* single) {
  const int b = blockIdx.x, lane = threadIdx.x & 31;
  const int len = lens ? cross_clamp_len(lens[b], ns) : ns;
  __shared__ int seen;
  if (threadIdx.x == 0) seen = 0;
  __syncthreads();
  int mine = 0;
  for (int w = threadIdx.x >> 5; w < word_tiles * 4; w += 8) {
    const int j = w * 32 + lane;
    const uint32_t bits = __ballot_sync(0xffffffffu, j < len && mask[(int64_t)b * ns + j] != 0);
    if (lane == 0) words[(int64_t)b * word_tiles * 4 + w] = bits;
    mine += __popc(bits);
  }
  if (lane == 0) atomicAdd(&seen, mine);
  __syncthreads();
  if (threadIdx.x == 0) single[b] = seen == 1;
}

// Joins the partial results of split items: with per-split log-sum-exps L_s (base 2) and outputs
// O_s, L = log2(sum_s 2^L_s) and o = sum_s 2^(L_s - L) O_s, added in split order.  One warp per
// query row; a split without a visible key (L_s = -inf) holds no O and is skipped.
template <typename T, int D>
__global__ void __launch_bounds__(256) cross_join_kernel(const CrossParams p) {
  const int64_t r = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (r >= (int64_t)p.batch * p.heads * p.nq) return;
  const int lane = threadIdx.x & 31;
  const int i = (int)(r % p.nq), h = (int)(r / p.nq % p.heads), b = (int)(r / p.nq / p.heads);
  const int hk = h / p.group, qt = i / p.toks, row = (i - qt * p.toks) * p.group + (h - hk * p.group);
  const int64_t blk = ((int64_t)(b * p.kv_heads + hk) * p.nqt + qt) * p.nsplit;
  const float* lse = p.part + (int64_t)p.units * p.nqt * p.nsplit * p.part_rows * D + row;
  float top = neg_inf();
  for (int s = 0; s < p.nsplit; ++s) top = fmaxf(top, lse[(blk + s) * p.part_rows]);
  float o[D / 32] = {}, sum = 0.f;
  for (int s = 0; s < p.nsplit; ++s) {
    const float l = lse[(blk + s) * p.part_rows];
    if (l == neg_inf()) continue;
    const float f = exp2f(l - top);            // NaN (a NaN row) passes through
    sum += f;
    float v[D / 32];
    load_f32<float, D / 32>(p.part + ((blk + s) * p.part_rows + row) * D + lane * (D / 32), v);
#pragma unroll
    for (int c = 0; c < D / 32; ++c) o[c] += f * v[c];
  }
  const float inv = sum == 0.f ? 0.f : 1.0f / sum;
#pragma unroll
  for (int c = 0; c < D / 32; ++c) o[c] *= inv;
  store_f32<T, D / 32>(static_cast<T*>(p.out[0]) + b * p.out_st[0][0] + i * p.out_st[0][1] + h * p.out_st[0][2] +
                           lane * (D / 32), o);
  if (p.lse && lane == 0) p.lse[r] = sum == 0.f ? neg_inf() : (top + log2f(sum)) * 0.6931471805599453f;
}

int check(const ultragen_cross_t* c) {
  if (!c || c->batch < 0 || c->nq < 0 || c->ns < 0 || c->heads < 1 || c->kv_heads < 1) return ULTRAGEN_ERR_INVALID_ARG;
  if (c->heads % c->kv_heads != 0 || !std::isfinite(c->scale) || !(c->scale > 0.f)) return ULTRAGEN_ERR_INVALID_ARG;
  if (c->dtype != ULTRAGEN_BF16 && c->dtype != ULTRAGEN_F16) return ULTRAGEN_ERR_UNSUPPORTED;
  if (c->head_dim != 64 && c->head_dim != 128) return ULTRAGEN_ERR_UNSUPPORTED;
  if (c->heads / c->kv_heads > 128) return ULTRAGEN_ERR_UNSUPPORTED;
  if ((int64_t)c->batch * c->heads * ((int64_t)std::max(c->nq, c->ns) + 128) > 0x7fffffffLL) return ULTRAGEN_ERR_UNSUPPORTED;
  return ULTRAGEN_OK;
}

int status_of(cudaError_t e) { return e == cudaSuccess ? ULTRAGEN_OK : ULTRAGEN_ERR_CUDA; }

// Bytes of the workspace's parts, each a multiple of 16: bit words and single flags of a key mask,
// then (backward) delta, then the partial results of split items.
struct Layout {
  size_t words, single, delta, part;
  size_t total() const { return words + single + delta + part; }
};
size_t pad16(size_t n) { return (n + 15) & ~size_t(15); }

// Schedule of the forward pass.  A work item is one or two query tiles (two share each key tile)
// times a range of the key tiles.  Splitting the keys pays when the items would not fill the
// multiprocessors: the cost of nsplit is taken as the rounds of items, each of its key tiles and
// about two tiles' time for its query load and epilogue, plus about six for the join kernel.
void schedule(const ultragen_cross_t* c, int sms, CrossParams& p) {
  p.units = c->batch * c->kv_heads;
  p.group = c->heads / c->kv_heads;
  p.toks = 128 / p.group;
  p.group_inv = (65536 + p.group - 1) / p.group;
  p.nqt = (c->nq + p.toks - 1) / p.toks;
  const int kt = std::max(1, (c->ns + 127) / 128);
  p.per_item = (int64_t)p.units * ((p.nqt + 1) / 2) >= sms && p.nqt > 1 ? 2 : 1;
  p.nitem_q = (p.nqt + p.per_item - 1) / p.per_item;
  const int64_t items = (int64_t)p.units * p.nitem_q;
  int64_t best = 0;
  p.nsplit = 1;
  for (int n = 1; n <= std::min(kt, 64); ++n) {
    const int64_t cost = (items * n + sms - 1) / sms * ((kt + n - 1) / n + 2) + (n > 1 ? 6 : 0);
    if (n == 1 || cost < best) {
      best = cost;
      p.nsplit = n;
    }
  }
  p.total = (int)(items * p.nsplit);
  p.div_q = FastDiv((uint32_t)std::max(1, p.nitem_q));
  p.div_split = FastDiv((uint32_t)p.nsplit);
  p.part_rows = p.nqt == 1 ? p.group * c->nq : 128;
}

Layout mask_layout(const ultragen_cross_t* c) {
  Layout l = {};
  if (c->masked) {
    l.words = (size_t)c->batch * ((c->ns + 127) / 128) * 16;
    l.single = pad16((size_t)c->batch * 4);
  }
  return l;
}

Layout forward_layout(const ultragen_cross_t* c, CrossParams& p) {
  schedule(c, sm_count(), p);
  Layout l = mask_layout(c);
  if (p.nsplit > 1) l.part = pad16((size_t)p.units * p.nqt * p.nsplit * p.part_rows * (c->head_dim + 1) * 4);
  return l;
}

// Schedule of the dK/dV kernel: an item is a key tile and a range of the query tiles.  The ranges
// are split when the key tiles alone would not fill the multiprocessors evenly: the cost is taken
// as the rounds of items, each of its query tiles and about two tiles' time to begin and end; a
// split adds the fp32 partials' way through memory, about one tile's time per item on top, and
// about three for the join kernel.
Layout backward_layout(const ultragen_cross_t* c, CrossParams& p) {
  const int sms = sm_count();
  p.units = c->batch * c->kv_heads;
  p.group = c->heads / c->kv_heads;
  p.toks = 128 / p.group;
  p.group_inv = (65536 + p.group - 1) / p.group;
  p.nqt = (c->nq + p.toks - 1) / p.toks;
  const int64_t tiles = (int64_t)p.units * ((c->ns + 127) / 128);
  int64_t best = 0;
  p.nsplit = p.nqt > 0 ? 1 : 0;
  for (int n = 1; n <= std::min(p.nqt, 64); ++n) {
    const int64_t cost = (tiles * n + sms - 1) / sms * ((p.nqt + n - 1) / n + (n > 1 ? 3 : 2)) + (n > 1 ? 3 : 0);
    if (n == 1 || cost < best) {
      best = cost;
      p.nsplit = n;
    }
  }
  p.total = (int)(tiles * p.nsplit);
  p.div_q = FastDiv((uint32_t)std::max(1, p.nqt));
  p.div_kt = FastDiv((uint32_t)std::max(1, (c->ns + 127) / 128));
  p.div_split = FastDiv((uint32_t)std::max(1, p.nsplit));
  Layout l = mask_layout(c);
  l.delta = pad16((size_t)c->batch * c->heads * c->nq * 4);
  if (p.nsplit > 1) l.part = (size_t)p.total * 2 * 128 * c->head_dim * 4;
  return l;
}

// Tensor map of [batch, rows, kv_heads * group, D] as (element, head in group, row, key/value
// head, batch) with [64 elements x group x rows_box] boxes and the 128-byte swizzle: a box lands
// as group * rows_box rows of 128 bytes.  Rows behind the tensor's last land as zeros.
int make_map(CUtensorMap* m, const void* base, const int64_t st[3], int dtype, int batch, int rows, int kv_heads,
             int group, int D, int rows_box) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return ULTRAGEN_ERR_CUDA;
  const cuuint64_t dims[5] = {(cuuint64_t)D, (cuuint64_t)group, (cuuint64_t)rows, (cuuint64_t)kv_heads, (cuuint64_t)batch};
  const cuuint64_t strides[4] = {(cuuint64_t)st[2] * 2, (cuuint64_t)st[1] * 2, (cuuint64_t)st[2] * group * 2,
                                 (cuuint64_t)st[0] * 2};
  const cuuint32_t box[5] = {64, (cuuint32_t)group, (cuuint32_t)rows_box, 1, 1};
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  const CUresult r = fn(m, dtype == ULTRAGEN_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 5,
                        const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? ULTRAGEN_OK : ULTRAGEN_ERR_CUDA;
}

constexpr unsigned long long kTimeoutNs = 2000ull * 1000 * 1000;   // limit of every device-side wait

// Pointers and strides on 16-byte boundaries.
bool aligned(const void* p, const int64_t st[3]) {
  return ((uintptr_t)p & 15u) == 0 && st[0] % 8 == 0 && st[1] % 8 == 0 && st[2] % 8 == 0 && st[0] >= 0 && st[1] >= 0 &&
         st[2] >= 0;
}

// The parameters that both passes share.
void common(const ultragen_cross_t* c, const int32_t* lens, const uint8_t* mask, const Layout& l, void* ws, CrossParams& p) {
  p.batch = c->batch;
  p.nq = c->nq;
  p.ns = c->ns;
  p.heads = c->heads;
  p.kv_heads = c->kv_heads;
  p.div_h = FastDiv((uint32_t)c->heads);
  p.div_kv = FastDiv((uint32_t)c->kv_heads);
  p.scale = c->scale;
  p.scale_log2 = (float)(c->scale * 1.4426950408889634);
  p.lens = lens;
  p.word_tiles = (c->ns + 127) / 128;
  p.words = mask ? static_cast<const uint32_t*>(ws) : nullptr;
  p.single = mask ? reinterpret_cast<const int32_t*>(static_cast<uint8_t*>(ws) + l.words) : nullptr;
  p.scrub = (lens || mask) ? 1 : 0;
  p.timeout_ns = kTimeoutNs;
}

cudaError_t pack_mask(const ultragen_cross_t* c, const int32_t* lens, const uint8_t* mask, const CrossParams& p,
                      cudaStream_t s) {
  mask_words_kernel<<<c->batch, 256, 0, s>>>(mask, lens, c->ns, p.word_tiles, const_cast<uint32_t*>(p.words),
                                            const_cast<int32_t*>(p.single));
  return cudaGetLastError();
}

}  // namespace

cudaError_t read_clear_error(const void* symbol, int* code, cudaStream_t s) {
  const int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbolAsync(code, symbol, sizeof(int), 0, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e == cudaSuccess && *code) {
    e = cudaMemcpyToSymbolAsync(symbol, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  }
  return e;
}

}  // namespace ug

using namespace ug;

extern "C" {

int ultragen_cross_attention_workspace(const ultragen_cross_t* c, int backward, size_t* bytes) {
  int st = check(c);
  if (st != ULTRAGEN_OK) return st;
  if (!bytes || (backward != 0 && backward != 1)) return ULTRAGEN_ERR_INVALID_ARG;
  CrossParams p = {};
  if (c->batch == 0) *bytes = 0;
  else if (backward) *bytes = backward_layout(c, p).total();
  else *bytes = c->nq == 0 ? 0 : forward_layout(c, p).total();
  return ULTRAGEN_OK;
}

int ultragen_cross_attention(const ultragen_cross_t* c, const void* q, const void* k, const void* v,
                             const int32_t* kv_lens, const uint8_t* key_mask, void* o, float* lse,
                             void* workspace, size_t workspace_bytes, ultragen_stream_t stream) {
  ug::NvtxRange nvtx_range("ultragen_cross_attention");
  int st = check(c);
  if (st != ULTRAGEN_OK) return st;
  if (c->batch == 0 || c->nq == 0) return ULTRAGEN_OK;
  if (!q || !o || (c->ns > 0 && (!k || !v)) || (key_mask && !c->masked)) return ULTRAGEN_ERR_INVALID_ARG;
  if (!aligned(q, c->stride[0]) || !aligned(o, c->stride[3])) return ULTRAGEN_ERR_INVALID_ARG;
  if (c->ns > 0 && (!aligned(k, c->stride[1]) || !aligned(v, c->stride[2]))) return ULTRAGEN_ERR_INVALID_ARG;
  // o may be q: an item reads its query tiles whole before it writes their rows
  if (begins_at(o, {k, v, lse, workspace}) || (o == q && !std::equal(c->stride[0], c->stride[0] + 3, c->stride[3])))
    return ULTRAGEN_ERR_INVALID_ARG;
  if (c->ns == 0) key_mask = nullptr;
  CrossParams p = {};
  const Layout l = forward_layout(c, p);
  if (l.total() > 0 && (!workspace || workspace_bytes < l.total() || ((uintptr_t)workspace & 15u))) return ULTRAGEN_ERR_INVALID_ARG;
  int dev;
  if ((st = current_device(&dev)) != ULTRAGEN_OK) return st;
  common(c, kv_lens, key_mask, l, workspace, p);
  p.out[0] = o;
  std::copy(c->stride[3], c->stride[3] + 3, p.out_st[0]);
  p.lse = lse;
  p.part = l.part ? reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + l.words + l.single) : nullptr;
  alignas(64) CrossMaps m;
  std::memset(&m, 0, sizeof(m));
  if ((st = make_map(&m.q, q, c->stride[0], c->dtype, c->batch, c->nq, c->kv_heads, p.group, c->head_dim, p.toks))) return st;
  if (c->ns > 0 &&
      ((st = make_map(&m.k, k, c->stride[1], c->dtype, c->batch, c->ns, c->kv_heads, 1, c->head_dim, 128)) ||
       (st = make_map(&m.v, v, c->stride[2], c->dtype, c->batch, c->ns, c->kv_heads, 1, c->head_dim, 128))))
    return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (key_mask && (st = status_of(pack_mask(c, kv_lens, key_mask, p, s)))) return st;
  if ((st = status_of(launch_cross_fwd(m, p, c->dtype, c->head_dim, std::min(p.total, sm_count()), s)))) return st;
  if (p.nsplit == 1) return ULTRAGEN_OK;
  const unsigned blocks = (unsigned)(((int64_t)c->batch * c->heads * c->nq + 7) / 8);
  if (c->dtype == ULTRAGEN_BF16) {
    if (c->head_dim == 128) cross_join_kernel<__nv_bfloat16, 128><<<blocks, 256, 0, s>>>(p);
    else cross_join_kernel<__nv_bfloat16, 64><<<blocks, 256, 0, s>>>(p);
  } else {
    if (c->head_dim == 128) cross_join_kernel<__half, 128><<<blocks, 256, 0, s>>>(p);
    else cross_join_kernel<__half, 64><<<blocks, 256, 0, s>>>(p);
  }
  return status_of(cudaGetLastError());
}

int ultragen_operator_status(ultragen_stream_t stream) {
  int dev, st, code = 0;
  if ((st = current_device(&dev)) != ULTRAGEN_OK) return st;
  int back = 0;
  if ((st = status_of(cross_fwd_status(&code, reinterpret_cast<cudaStream_t>(stream))))) return st;
  if ((st = status_of(cross_bwd_status(&back, reinterpret_cast<cudaStream_t>(stream))))) return st;
  int proj = 0, norm = 0;
  if ((st = status_of(adapter_status(&proj, reinterpret_cast<cudaStream_t>(stream))))) return st;
  if ((st = status_of(norm_status(&norm, reinterpret_cast<cudaStream_t>(stream))))) return st;
  return code || back || proj || norm ? ULTRAGEN_ERR_TIMEOUT : ULTRAGEN_OK;
}

int ultragen_cross_attention_backward(const ultragen_cross_t* c, const void* d_o, const void* q, const void* k,
                                      const void* v, const void* o, const float* lse, const int32_t* kv_lens,
                                      const uint8_t* key_mask, void* dq, void* dk, void* dv, void* workspace,
                                      size_t workspace_bytes, ultragen_stream_t stream) {
  ug::NvtxRange nvtx_range("ultragen_cross_attention_backward");
  int st = check(c);
  if (st != ULTRAGEN_OK) return st;
  if (c->batch == 0) return ULTRAGEN_OK;
  if (c->nq > 0 && (!d_o || !q || !o || !lse || !dq)) return ULTRAGEN_ERR_INVALID_ARG;
  if (c->ns > 0 && (!k || !v || !dk || !dv)) return ULTRAGEN_ERR_INVALID_ARG;
  const int64_t(*sd)[3] = c->stride;
  if (c->nq > 0 && (!aligned(q, sd[0]) || !aligned(o, sd[3]) || !aligned(d_o, sd[4]) || !aligned(dq, sd[5])))
    return ULTRAGEN_ERR_INVALID_ARG;
  if (c->ns > 0 && (!aligned(k, sd[1]) || !aligned(v, sd[2]) || !aligned(dk, sd[6]) || !aligned(dv, sd[7])))
    return ULTRAGEN_ERR_INVALID_ARG;
  if (key_mask && !c->masked) return ULTRAGEN_ERR_INVALID_ARG;
  // dq is written before the pass that makes dk and dv reads q, k, v and do; those are read for every key tile
  if (begins_at(dq, {q, k, v, d_o, dk, dv, lse, workspace}) || begins_at(dk, {q, d_o, dv, workspace}) ||
      begins_at(dv, {q, d_o, workspace}))
    return ULTRAGEN_ERR_INVALID_ARG;
  if (c->ns == 0) key_mask = nullptr;
  CrossParams p = {};
  const Layout l = backward_layout(c, p);
  if (l.total() > 0 && (!workspace || workspace_bytes < l.total() || ((uintptr_t)workspace & 15u))) return ULTRAGEN_ERR_INVALID_ARG;
  int dev;
  if ((st = current_device(&dev)) != ULTRAGEN_OK) return st;
  common(c, kv_lens, key_mask, l, workspace, p);
  p.o = o;
  p.d_o = d_o;
  std::copy(sd[3], sd[3] + 3, p.o_st);
  std::copy(sd[4], sd[4] + 3, p.do_st);
  p.lse = const_cast<float*>(lse);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.delta = reinterpret_cast<float*>(ws + l.words + l.single);
  alignas(64) CrossMaps m;
  std::memset(&m, 0, sizeof(m));
  if (c->nq > 0 &&
      ((st = make_map(&m.q, q, sd[0], c->dtype, c->batch, c->nq, c->kv_heads, p.group, c->head_dim, p.toks)) ||
       (st = make_map(&m.d_o, d_o, sd[4], c->dtype, c->batch, c->nq, c->kv_heads, p.group, c->head_dim, p.toks))))
    return st;
  if (c->ns > 0 &&
      ((st = make_map(&m.k, k, sd[1], c->dtype, c->batch, c->ns, c->kv_heads, 1, c->head_dim, 128)) ||
       (st = make_map(&m.v, v, sd[2], c->dtype, c->batch, c->ns, c->kv_heads, 1, c->head_dim, 128))))
    return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (key_mask && (st = status_of(pack_mask(c, kv_lens, key_mask, p, s)))) return st;
  if (c->nq > 0) {
    CrossParams pq = p;
    pq.nsplit = 1;
    pq.total = p.units * p.nqt;
    pq.out[0] = dq;
    std::copy(sd[5], sd[5] + 3, pq.out_st[0]);
    if ((st = status_of(launch_cross_dq(m, pq, c->dtype, c->head_dim, std::min(pq.total, sm_count()), s)))) return st;
  }
  if (c->ns == 0) return ULTRAGEN_OK;
  p.out[0] = dk;
  p.out[1] = dv;
  std::copy(sd[6], sd[6] + 3, p.out_st[0]);
  std::copy(sd[7], sd[7] + 3, p.out_st[1]);
  p.part = l.part ? reinterpret_cast<float*>(ws + l.words + l.single + l.delta) : nullptr;
  return status_of(launch_cross_dkv(m, p, c->dtype, c->head_dim, std::min(p.total, sm_count()), s));
}

}  // extern "C"
