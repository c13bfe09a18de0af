// Cross attention of one sequence's queries over another's keys and values, forward and backward:
//   s_ij = scale q_i . k_j over the visible keys j,  lse_i = log(sum_j exp(s_ij)),
//   p_ij = exp(s_ij - lse_i),  o_i = sum_j p_ij v_j
//   delta_i = do_i . o_i,  ds_ij = p_ij (do_i . v_j - delta_i)
//   dq_i = scale sum_j ds_ij k_j,  dk_j = scale sum_i ds_ij q_i,  dv_j = sum_i p_ij do_i
// One warp per row; the lanes share the head dimension.  Hidden keys are never read.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "elem.cuh"
#include "kernels.h"
#include "nvtx_range.h"
#include "ultragen.h"

namespace ug {
namespace {

struct CrossArgs {
  const void* p[8];             // q, k, v, o, do, dq, dk, dv
  int64_t st[8][3];             // batch, row and head strides
  float* lse;
  const int32_t* lens;
  const uint8_t* mask;
  int batch, nq, ns, heads, kv_heads, group;
  float scale;
};

template <typename T>
__device__ __forceinline__ T* at(const CrossArgs& a, int which, int b, int64_t row, int h) {
  return const_cast<T*>(static_cast<const T*>(a.p[which])) + b * a.st[which][0] + row * a.st[which][1] +
         h * a.st[which][2];
}

__device__ __forceinline__ int visible_len(const CrossArgs& a, int b) {
  return a.lens ? max(0, min(a.ns, a.lens[b])) : a.ns;
}
__device__ __forceinline__ bool hidden(const CrossArgs& a, int b, int j) {
  return a.mask && !a.mask[(int64_t)b * a.ns + j];
}

template <typename T, int D>
__device__ __forceinline__ void load_row(const T* p, float (&v)[D / 32]) {
#pragma unroll
  for (int c = 0; c < D / 32; ++c) v[c] = to_f32(p[(threadIdx.x & 31) + 32 * c]);
}
template <int D>
__device__ __forceinline__ float dot(const float (&a)[D / 32], const float (&b)[D / 32]) {
  float s = 0.f;
#pragma unroll
  for (int c = 0; c < D / 32; ++c) s += a[c] * b[c];
  return warp_sum(s);
}

template <typename T, int D>
__global__ void __launch_bounds__(256) cross_fwd_kernel(const CrossArgs a) {
  const int64_t r = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (r >= (int64_t)a.batch * a.heads * a.nq) return;
  const int i = r % a.nq, h = r / a.nq % a.heads, b = r / a.nq / a.heads;
  float q[D / 32], o[D / 32] = {}, t[D / 32];
  load_row<T, D>(at<T>(a, 0, b, i, h), q);
  float m = -INFINITY, l = 0.f;
  const int len = visible_len(a, b);
  for (int j = 0; j < len; ++j) {
    if (hidden(a, b, j)) continue;
    load_row<T, D>(at<T>(a, 1, b, j, h / a.group), t);
    const float s = a.scale * dot<D>(q, t);
    load_row<T, D>(at<T>(a, 2, b, j, h / a.group), t);
    const float mn = fmaxf(m, s), f = expf(m - mn), p = expf(s - mn);
    l = l * f + p;
    m = mn;
#pragma unroll
    for (int c = 0; c < D / 32; ++c) o[c] = o[c] * f + p * t[c];
  }
  T* out = at<T>(a, 3, b, i, h);
  const float inv = l > 0.f ? 1.0f / l : 0.f;
#pragma unroll
  for (int c = 0; c < D / 32; ++c) out[(threadIdx.x & 31) + 32 * c] = from_f32<T>(o[c] * inv);
  if (a.lse && (threadIdx.x & 31) == 0) a.lse[r] = l > 0.f ? m + logf(l) : -INFINITY;
}

template <typename T, int D>
__global__ void __launch_bounds__(256) cross_dq_kernel(const CrossArgs a) {
  const int64_t r = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (r >= (int64_t)a.batch * a.heads * a.nq) return;
  const int i = r % a.nq, h = r / a.nq % a.heads, b = r / a.nq / a.heads;
  float q[D / 32], g[D / 32], dq[D / 32] = {}, t[D / 32], v[D / 32];
  load_row<T, D>(at<T>(a, 0, b, i, h), q);
  load_row<T, D>(at<T>(a, 4, b, i, h), g);
  load_row<T, D>(at<T>(a, 3, b, i, h), t);
  const float delta = dot<D>(g, t), lse = a.lse[r];
  const int len = lse == -INFINITY ? 0 : visible_len(a, b);
  for (int j = 0; j < len; ++j) {
    if (hidden(a, b, j)) continue;
    load_row<T, D>(at<T>(a, 1, b, j, h / a.group), t);
    load_row<T, D>(at<T>(a, 2, b, j, h / a.group), v);
    const float ds = expf(a.scale * dot<D>(q, t) - lse) * (dot<D>(g, v) - delta) * a.scale;
#pragma unroll
    for (int c = 0; c < D / 32; ++c) dq[c] += ds * t[c];
  }
  T* out = at<T>(a, 5, b, i, h);
#pragma unroll
  for (int c = 0; c < D / 32; ++c) out[(threadIdx.x & 31) + 32 * c] = from_f32<T>(dq[c]);
}

template <typename T, int D>
__global__ void __launch_bounds__(256) cross_dkv_kernel(const CrossArgs a) {
  const int64_t r = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (r >= (int64_t)a.batch * a.kv_heads * a.ns) return;
  const int j = r % a.ns, hk = r / a.ns % a.kv_heads, b = r / a.ns / a.kv_heads;
  float k[D / 32] = {}, v[D / 32] = {}, dk[D / 32] = {}, dv[D / 32] = {}, q[D / 32], g[D / 32], t[D / 32];
  if (j < visible_len(a, b) && !hidden(a, b, j)) {
    load_row<T, D>(at<T>(a, 1, b, j, hk), k);
    load_row<T, D>(at<T>(a, 2, b, j, hk), v);
    for (int h = hk * a.group; h < (hk + 1) * a.group; ++h)
      for (int i = 0; i < a.nq; ++i) {
        load_row<T, D>(at<T>(a, 0, b, i, h), q);
        load_row<T, D>(at<T>(a, 4, b, i, h), g);
        load_row<T, D>(at<T>(a, 3, b, i, h), t);
        const float p = expf(a.scale * dot<D>(q, k) - a.lse[((int64_t)b * a.heads + h) * a.nq + i]);
        const float ds = p * (dot<D>(g, v) - dot<D>(g, t)) * a.scale;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          dk[c] += ds * q[c];
          dv[c] += p * g[c];
        }
      }
  }
  T* ok = at<T>(a, 6, b, j, hk);
  T* ov = at<T>(a, 7, b, j, hk);
#pragma unroll
  for (int c = 0; c < D / 32; ++c) {
    ok[(threadIdx.x & 31) + 32 * c] = from_f32<T>(dk[c]);
    ov[(threadIdx.x & 31) + 32 * c] = from_f32<T>(dv[c]);
  }
}

int check(const ultragen_cross_t* c) {
  if (!c || c->batch < 0 || c->nq < 0 || c->ns < 0 || c->heads < 1 || c->kv_heads < 1) return ULTRAGEN_ERR_INVALID_ARG;
  if (c->heads % c->kv_heads != 0 || !std::isfinite(c->scale)) return ULTRAGEN_ERR_INVALID_ARG;
  if (c->dtype != ULTRAGEN_BF16 && c->dtype != ULTRAGEN_F16) return ULTRAGEN_ERR_UNSUPPORTED;
  if (c->head_dim != 64 && c->head_dim != 128) return ULTRAGEN_ERR_UNSUPPORTED;
  if (c->heads / c->kv_heads > 128) return ULTRAGEN_ERR_UNSUPPORTED;
  if ((int64_t)c->batch * c->heads * ((int64_t)std::max(c->nq, c->ns) + 128) > 0x7fffffffLL) return ULTRAGEN_ERR_UNSUPPORTED;
  return ULTRAGEN_OK;
}

CrossArgs args_of(const ultragen_cross_t* c, const int32_t* lens, const uint8_t* mask) {
  CrossArgs a = {};
  for (int t = 0; t < 8; ++t)
    for (int d = 0; d < 3; ++d) a.st[t][d] = c->stride[t][d];
  a.lens = lens;
  a.mask = mask;
  a.batch = c->batch;
  a.nq = c->nq;
  a.ns = c->ns;
  a.heads = c->heads;
  a.kv_heads = c->kv_heads;
  a.group = c->heads / c->kv_heads;
  a.scale = c->scale;
  return a;
}

int status_of(cudaError_t e) { return e == cudaSuccess ? ULTRAGEN_OK : ULTRAGEN_ERR_CUDA; }

template <typename T, int D>
cudaError_t forward(const CrossArgs& a, cudaStream_t s) {
  const int64_t n = (int64_t)a.batch * a.heads * a.nq;
  if (n) cross_fwd_kernel<T, D><<<(unsigned)((n + 7) / 8), 256, 0, s>>>(a);
  return cudaGetLastError();
}
template <typename T, int D>
cudaError_t backward(const CrossArgs& a, cudaStream_t s) {
  const int64_t n = (int64_t)a.batch * a.heads * a.nq, m = (int64_t)a.batch * a.kv_heads * a.ns;
  if (n) cross_dq_kernel<T, D><<<(unsigned)((n + 7) / 8), 256, 0, s>>>(a);
  if (m) cross_dkv_kernel<T, D><<<(unsigned)((m + 7) / 8), 256, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace
}  // namespace ug

using namespace ug;

extern "C" {

int ultragen_cross_attention_workspace(const ultragen_cross_t* c, int backward, size_t* bytes) {
  int st = check(c);
  if (st != ULTRAGEN_OK) return st;
  if (!bytes || (backward != 0 && backward != 1)) return ULTRAGEN_ERR_INVALID_ARG;
  *bytes = 0;
  return ULTRAGEN_OK;
}

int ultragen_cross_attention(const ultragen_cross_t* c, const void* q, const void* k, const void* v,
                             const int32_t* kv_lens, const uint8_t* key_mask, void* o, float* lse,
                             void* workspace, size_t workspace_bytes, ultragen_stream_t stream) {
  ug::NvtxRange nvtx_range("ultragen_cross_attention");
  int st = check(c);
  if (st != ULTRAGEN_OK) return st;
  if (c->batch == 0 || c->nq == 0) return ULTRAGEN_OK;
  if (!q || !o || (c->ns > 0 && (!k || !v))) return ULTRAGEN_ERR_INVALID_ARG;
  int dev;
  if ((st = current_device(&dev)) != ULTRAGEN_OK) return st;
  (void)workspace;
  (void)workspace_bytes;
  CrossArgs a = args_of(c, kv_lens, key_mask);
  const void* ptrs[8] = {q, k, v, o, nullptr, nullptr, nullptr, nullptr};
  std::copy(ptrs, ptrs + 8, a.p);
  a.lse = lse;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (c->dtype == ULTRAGEN_BF16)
    return status_of(c->head_dim == 128 ? forward<__nv_bfloat16, 128>(a, s) : forward<__nv_bfloat16, 64>(a, s));
  return status_of(c->head_dim == 128 ? forward<__half, 128>(a, s) : forward<__half, 64>(a, s));
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
  int dev;
  if ((st = current_device(&dev)) != ULTRAGEN_OK) return st;
  (void)workspace;
  (void)workspace_bytes;
  CrossArgs a = args_of(c, kv_lens, key_mask);
  const void* ptrs[8] = {q, k, v, o, d_o, dq, dk, dv};
  std::copy(ptrs, ptrs + 8, a.p);
  a.lse = const_cast<float*>(lse);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (c->dtype == ULTRAGEN_BF16)
    return status_of(c->head_dim == 128 ? backward<__nv_bfloat16, 128>(a, s) : backward<__nv_bfloat16, 64>(a, s));
  return status_of(c->head_dim == 128 ? backward<__half, 128>(a, s) : backward<__half, 64>(a, s));
}

}  // extern "C"
