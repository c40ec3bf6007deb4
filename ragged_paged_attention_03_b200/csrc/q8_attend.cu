// q8_attend.cu -- attention over the 8-bit paged cache (rpa_q8_attend).
//
// The simple form: one warp per (query row, query head) walks the visible
// keys with a running maximum and sum.
#include <cmath>
#include <cuda_runtime.h>

#include <algorithm>

#include "host_common.h"
#include "q8_common.cuh"
#include "q8_host.h"
#include "rpa.h"

namespace rpa {
namespace q8 {
namespace {

struct AttendArgs {
  const void *q;
  Cache c;
  Lengths len;
  const int32_t *page_table;
  uint32_t *err;
  void *out;
  float *lse;
  int32_t hq, hkv, p, p_shift, num_pages, max_pages, causal;
  float scale;
};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float v, float *p) { *p = v; }
__device__ __forceinline__ void from_f(float v, __nv_bfloat16 *p) { *p = __float2bfloat16_rn(v); }

template <typename T, int D>
__global__ void __launch_bounds__(256) simple_kernel(const AttendArgs a) {
  constexpr int E = D / 32;
  const int n = checked_seqs(a.len);
  if (n < 0) {
    if (blockIdx.x == 0 && threadIdx.x == 0) raise(a.err, RPA_DEV_BAD_LENGTHS);
    return;
  }
  if (n == 0) return;
  const int lane = threadIdx.x & 31;
  const int G = a.hq / a.hkv;
  const int64_t tasks = (int64_t)a.len.cu[n] * a.hq;
  const int64_t step = (int64_t)gridDim.x * (blockDim.x / 32);
  for (int64_t w = (int64_t)blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32; w < tasks; w += step) {
    const int t = (int)(w / a.hq), h = (int)(w % a.hq), hk = h / G;
    const int s = seq_of(a.len.cu, n, t);
    const int kv = a.len.kv[s];
    const int last = kv - a.len.cu[s + 1] + t;      // kv_len - q_len + i
    const int nvis = a.causal ? max(0, last + 1) : kv;
    const T *q = static_cast<const T *>(a.q) + (size_t)w * D + lane * E;
    float qv[E], acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      qv[e] = to_f(q[e]);
      acc[e] = 0.f;
    }
    float m = -INFINITY, l = 0.f;
    for (int j = 0; j < nvis; ++j) {
      const int page = a.page_table[(size_t)s * a.max_pages + (j >> a.p_shift)];
      const bool ok = page >= 0 && page < a.num_pages;
      if (!ok && lane == 0) raise(a.err, RPA_DEV_BAD_PAGE);
      const int slot = j & (a.p - 1);
      const size_t off = (((size_t)(ok ? page : 0) * a.p + slot) * a.hkv + hk) * D + lane * E;
      const size_t so = ((size_t)(ok ? page : 0) * a.hkv + hk) * a.p + slot;
      const float ks = ok ? scale_value(a.c.ks[so]) : 0.f;
      const float vs = ok ? scale_value(a.c.vs[so]) : 0.f;
      float kf[E], vf[E];
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const float2 kk = __half22float2(from_e4m3x2(*reinterpret_cast<const uint16_t *>(a.c.k + off + e)));
        const float2 vv = __half22float2(from_e4m3x2(*reinterpret_cast<const uint16_t *>(a.c.v + off + e)));
        kf[e] = ok ? kk.x : 0.f; kf[e + 1] = ok ? kk.y : 0.f;
        vf[e] = ok ? vv.x : 0.f; vf[e + 1] = ok ? vv.y : 0.f;
      }
      float dot = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) dot = fmaf(qv[e], kf[e], dot);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
      const float x = dot * ks * a.scale + vs * 0.f;   // a NaN row of K or V is NaN for whoever sees it
      const float m_new = fmaxf(m, x);
      const float alpha = m == m_new ? 1.f : expf(m - m_new);
      const float p = m_new == -INFINITY && x == x ? 0.f : expf(x - (m_new == -INFINITY ? 0.f : m_new));
      l = l * alpha + p;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = fmaf(p * vs, vf[e], acc[e] * alpha);
      m = m_new;
    }
    T *out = static_cast<T *>(a.out) + (size_t)w * D + lane * E;
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int e = 0; e < E; ++e) from_f(nvis > 0 ? acc[e] * inv : 0.f, &out[e]);
    if (a.lse != nullptr && lane == 0) a.lse[w] = nvis > 0 ? (m == -INFINITY ? 0.f : m) + logf(l) : -INFINITY;
  }
}

}  // namespace
}  // namespace q8
}  // namespace rpa

using namespace rpa;

extern "C" RPA_API int rpa_q8_workspace_size(const rpa_dims *dims, int32_t max_seqs, int32_t max_q_len,
                                             int64_t *bytes) {
  if (bytes == nullptr) return RPA_ERR_INVALID_ARG;
  *bytes = 0;
  const int rc = validate_dims(dims);
  if (rc) return rc;
  if (max_seqs < 0 || max_q_len < 0) return RPA_ERR_INVALID_ARG;
  *bytes = 256;
  return RPA_OK;
}

extern "C" RPA_API int rpa_q8_attend(const void *q, const rpa_q8_cache *cache, const int32_t *page_table,
                                     const int32_t *cu_q_lens, const int32_t *kv_lens, const int32_t *num_seqs,
                                     int32_t max_seqs, int32_t max_q_len, float scale, int32_t causal, void *out,
                                     float *lse, const rpa_dims *dims, void *workspace, int64_t workspace_bytes,
                                     uint32_t *dev_flags, void *stream_ptr) {
  using namespace rpa::q8;
  cudaStream_t stream = (cudaStream_t)stream_ptr;
  if (!(scale > 0.f) || !std::isfinite(scale)) return RPA_ERR_INVALID_ARG;
  int rc = validate_dims(dims);
  if (rc) return rc;
  if (max_seqs < 0 || max_q_len < 0) return RPA_ERR_INVALID_ARG;
  if (max_seqs == 0 || max_q_len == 0 || dims->total_q_tokens == 0) return RPA_OK;
  if (!q || !cache || !cache->k_codes || !cache->v_codes || !cache->k_scales || !cache->v_scales || !page_table ||
      !cu_q_lens || !kv_lens || !num_seqs || !out || !workspace)
    return RPA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(out) || !aligned16(cache->k_codes) || !aligned16(cache->v_codes))
    return RPA_ERR_INVALID_ARG;
  int64_t need = 0;
  rc = rpa_q8_workspace_size(dims, max_seqs, max_q_len, &need);
  if (rc) return rc;
  if (workspace_bytes < need || reinterpret_cast<uintptr_t>(workspace) % 256 != 0) return RPA_ERR_WORKSPACE;
  AttendArgs a{};
  a.q = q;
  a.c = cache_of(cache);
  a.len = lengths_of(cu_q_lens, kv_lens, num_seqs, max_seqs, dims, max_q_len, false);
  a.page_table = page_table;
  a.err = dev_flags;
  a.out = out;
  a.lse = lse;
  a.hq = dims->num_q_heads;
  a.hkv = dims->num_kv_heads;
  a.p = dims->page_size;
  a.p_shift = log2_of(dims->page_size);
  a.num_pages = dims->num_pages;
  a.max_pages = dims->max_pages_per_seq;
  a.causal = causal ? 1 : 0;
  a.scale = scale;
  const int64_t warps = (int64_t)dims->total_q_tokens * a.hq;
  const unsigned grid = (unsigned)std::min<int64_t>((warps + 7) / 8, 148 * 64);
#define RPA_Q8_SIMPLE(DD)                                                               \
  case DD:                                                                              \
    if (dims->dtype == RPA_F32) simple_kernel<float, DD><<<grid, 256, 0, stream>>>(a);  \
    else simple_kernel<__nv_bfloat16, DD><<<grid, 256, 0, stream>>>(a);                 \
    break;
  switch (dims->head_dim) {
    RPA_Q8_SIMPLE(64)
    RPA_Q8_SIMPLE(128)
    RPA_Q8_SIMPLE(256)
    default: return RPA_ERR_UNSUPPORTED;
  }
#undef RPA_Q8_SIMPLE
  return cudaGetLastError() == cudaSuccess ? RPA_OK : RPA_ERR_CUDA;
}
