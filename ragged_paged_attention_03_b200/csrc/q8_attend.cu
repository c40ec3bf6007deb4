// q8_attend.cu -- rpa_q8_attend: attention over the 8-bit paged cache; checks,
// workspace and the choice of kernels.
#include <cmath>
#include <cuda_runtime.h>

#include <algorithm>

#include "host_common.h"
#include "q8_host.h"
#include "q8_kernels.h"
#include "rpa.h"

namespace rpa {
namespace q8 {
namespace {

// A sequence of at most this many rows per KV head (new tokens times G) reads its
// keys once in the row-group kernel.
constexpr int kRowsPerGroup = 16;

struct AttendLayout {
  int32_t q_limit;             // longest q_len of the row-group kernel; longer ones are the chunk kernel's
  bool chunk;                  // the chunk kernel is launched too
  int64_t rows, parts, total;  // byte offsets
};

AttendLayout attend_layout(const rpa_dims &d, int32_t max_seqs, int32_t max_q) {
  AttendLayout w{};
  w.q_limit = chunk_takes(d) ? std::max(1, kRowsPerGroup / (d.num_q_heads / d.num_kv_heads)) : INT32_MAX;
  w.chunk = max_q > w.q_limit;
  const int32_t q = std::min(max_q, w.q_limit);
  const int R = rows_per_group(d, q);
  w.rows = 0;
  w.parts = w.total = rows_layout(rows_grid(d, max_seqs, q, R), R, d.head_dim).total;
  if (w.chunk) w.total += chunk_layout(chunk_grid(d, max_seqs, max_q), d.head_dim).total;
  return w;
}

// Everything before the lengths: RPA_OK and *go, or a code.
int check_call(const rpa_dims *d, int32_t max_seqs, int32_t max_q) {
  const int rc = validate_dims(d);
  if (rc) return rc;
  if (max_seqs < 0 || max_q < 0) return RPA_ERR_INVALID_ARG;
  // rows of the pool are TMA coordinates, one past the last included
  if ((int64_t)d->num_pages * d->page_size > INT32_MAX - 1024) return RPA_ERR_UNSUPPORTED;
  return RPA_OK;
}

}  // namespace
}  // namespace q8
}  // namespace rpa

using namespace rpa;

extern "C" RPA_API int rpa_q8_workspace_size(const rpa_dims *dims, int32_t max_seqs, int32_t max_q_len,
                                             int64_t *bytes) {
  if (bytes == nullptr) return RPA_ERR_INVALID_ARG;
  *bytes = 0;
  const int rc = rpa::q8::check_call(dims, max_seqs, max_q_len);
  if (rc) return rc;
  *bytes = max_seqs == 0 || max_q_len == 0 || dims->total_q_tokens == 0
               ? 256
               : rpa::q8::attend_layout(*dims, max_seqs, max_q_len).total;
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
  const int rc = check_call(dims, max_seqs, max_q_len);
  if (rc) return rc;
  if (max_seqs == 0 || max_q_len == 0 || dims->total_q_tokens == 0) return RPA_OK;
  if (!q || !cache || !cache->k_codes || !cache->v_codes || !cache->k_scales || !cache->v_scales || !page_table ||
      !cu_q_lens || !kv_lens || !num_seqs || !out || !workspace)
    return RPA_ERR_INVALID_ARG;
  if (!aligned32(q) || !aligned32(out) || !aligned16(cache->k_codes) || !aligned16(cache->v_codes) ||
      !aligned16(cache->k_scales) || !aligned16(cache->v_scales))
    return RPA_ERR_INVALID_ARG;
  const AttendLayout w = attend_layout(*dims, max_seqs, max_q_len);
  if (workspace_bytes < w.total || reinterpret_cast<uintptr_t>(workspace) % 256 != 0) return RPA_ERR_WORKSPACE;
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
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  cudaError_t e = cudaSuccess;
  for (const bool join : {false, true}) {
    if (e == cudaSuccess) e = launch_rows(a, *dims, max_seqs, max_q_len, w.q_limit, ws + w.rows, join, stream);
    if (e == cudaSuccess && w.chunk)
      e = launch_chunk(a, *dims, max_seqs, max_q_len, w.q_limit, ws + w.parts, join, stream);
  }
  return e == cudaSuccess ? RPA_OK : RPA_ERR_CUDA;
}
