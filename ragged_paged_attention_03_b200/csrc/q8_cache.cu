// q8_cache.cu -- quantising new K/V rows into the 8-bit paged cache
// (rpa_q8_write) and reading cached rows back (rpa_q8_read).
//
// Both are one pass over the rows and bound by memory: a row of D values
// moves D * sizeof(T) + D + 1 bytes.  D / 16 neighbouring lanes share a row,
// each with 16 of its values in 16-byte pieces that stay in registers between
// the row's maximum (shuffles among those lanes) and the rounding, so every
// value is read once; K and V of a row are in flight together.
#include <algorithm>
#include <cuda_runtime.h>

#include "host_common.h"
#include "q8_common.cuh"
#include "q8_host.h"
#include "rpa.h"

namespace rpa {
namespace q8 {
namespace {

constexpr int kThreads = 256;
constexpr int kCuCap = 1024;   // sequences whose offsets are kept in shared memory

struct IoArgs {
  void *k, *v;                 // [T, Hkv, D] rows outside the cache
  Cache c;
  Lengths len;
  const int32_t *page_table;
  uint32_t *err;
  int32_t hkv, p, p_shift, num_pages, max_pages;
};

// 16 bytes of T as fp32 values and back (rounded to nearest-even).
template <typename T> struct Piece;
template <> struct Piece<float> {
  static constexpr int E = 4;
  static __device__ __forceinline__ void unpack(const uint4 &u, float (&f)[4]) {
    f[0] = __uint_as_float(u.x); f[1] = __uint_as_float(u.y);
    f[2] = __uint_as_float(u.z); f[3] = __uint_as_float(u.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
};
template <> struct Piece<__nv_bfloat16> {
  static constexpr int E = 8;
  static __device__ __forceinline__ void unpack(const uint4 &u, float (&f)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(f[2 * i + 1]), "f"(f[2 * i]));
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

template <typename T, int D, bool WRITE>
__global__ void __launch_bounds__(kThreads) io_kernel(const IoArgs a) {
  constexpr int E = Piece<T>::E;      // values per 16-byte piece
  constexpr int NP = 16 / E;          // pieces per lane
  constexpr int LPR = D / 16;         // lanes per row
  __shared__ int32_t s_cu[kCuCap + 1];
  const int n = checked_seqs(a.len);
  if (n < 0) {
    if (blockIdx.x == 0 && threadIdx.x == 0) raise(a.err, RPA_DEV_BAD_LENGTHS);
    return;
  }
  if (n == 0) return;
  const int32_t *cu = a.len.cu;
  if (n <= kCuCap) {
    for (int i = threadIdx.x; i <= n; i += kThreads) s_cu[i] = a.len.cu[i];
    __syncthreads();
    cu = s_cu;
  }
  const int64_t rows = (int64_t)cu[n] * a.hkv;
  const int sub = threadIdx.x % LPR;
  const int64_t step = (int64_t)gridDim.x * (kThreads / LPR);
  // a row's lanes are neighbours in one warp and leave the loop together
  const unsigned lanes = LPR == 32 ? 0xffffffffu : ((1u << LPR) - 1u) << ((threadIdx.x & 31) / LPR * LPR);
  for (int64_t r = (int64_t)blockIdx.x * (kThreads / LPR) + threadIdx.x / LPR; r < rows; r += step) {
    const int t = (int)(r / a.hkv);
    const int h = (int)(r - (int64_t)t * a.hkv);
    const size_t row = (size_t)r * D + sub * E;
    uint4 x[2][NP];
    if (WRITE) {
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        x[0][i] = __ldcs(reinterpret_cast<const uint4 *>(static_cast<const T *>(a.k) + row + i * (LPR * E)));
        x[1][i] = __ldcs(reinterpret_cast<const uint4 *>(static_cast<const T *>(a.v) + row + i * (LPR * E)));
      }
    }
    const int s = seq_of(cu, n, t);
    const int pos = a.len.kv[s] - cu[s + 1] + t;   // kv_len - q_len + (t - cu[s])
    const int page = a.page_table[(size_t)s * a.max_pages + (pos >> a.p_shift)];
    const bool ok = page >= 0 && page < a.num_pages;
    if (!ok && sub == 0) raise(a.err, RPA_DEV_BAD_PAGE);
    const int slot = pos & (a.p - 1);
    const size_t crow = (((size_t)(ok ? page : 0) * a.p + slot) * a.hkv + h) * D + sub * E;
    const size_t srow = ((size_t)(ok ? page : 0) * a.hkv + h) * a.p + slot;
    if (WRITE) {
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        float f[NP][E];
        uint32_t amax = 0;
        // |x| as integers: ordered like the values, with infinities and NaN on top
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          Piece<T>::unpack(x[kv][i], f[i]);
#pragma unroll
          for (int j = 0; j < E; ++j) amax = max(amax, __float_as_uint(f[i][j]) & 0x7fffffffu);
        }
#pragma unroll
        for (int o = 1; o < LPR; o <<= 1) amax = max(amax, __shfl_xor_sync(lanes, amax, o));
        const uint32_t code = scale_code(amax);
        const float inv = code == kScaleNan ? 0.f : inverse_scale(code);
        if (!ok) continue;
        uint8_t *dst = (kv ? a.c.v : a.c.k) + crow;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          uint32_t w[E / 4];
#pragma unroll
          for (int j = 0; j < E / 4; ++j)
            w[j] = code == kScaleNan ? 0u : to_e4m3x2(f[i][4 * j] * inv, f[i][4 * j + 1] * inv) |
                                                (to_e4m3x2(f[i][4 * j + 2] * inv, f[i][4 * j + 3] * inv) << 16);
          if (E == 8) *reinterpret_cast<uint2 *>(dst + i * (LPR * E)) = make_uint2(w[0], w[E / 4 - 1]);
          else *reinterpret_cast<uint32_t *>(dst + i * (LPR * E)) = w[0];
        }
        if (sub == 0) (kv ? a.c.vs : a.c.ks)[srow] = (uint8_t)code;
      }
    } else {
      uint2 c[2][NP];
      uint32_t sc[2];
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const uint8_t *src = (kv ? a.c.v : a.c.k) + crow;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          if (E == 8) c[kv][i] = *reinterpret_cast<const uint2 *>(src + i * (LPR * E));
          else c[kv][i].x = *reinterpret_cast<const uint32_t *>(src + i * (LPR * E));
        }
        sc[kv] = (kv ? a.c.vs : a.c.ks)[srow];
      }
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        // a page outside the pool reads as zeros
        const float scale = ok ? scale_value(sc[kv]) : 0.f;
        T *dst = static_cast<T *>(kv ? a.v : a.k) + row;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          float f[E];
#pragma unroll
          for (int j = 0; j < E / 4; ++j) {
            float g[4];
            e4m3x4_to_f32(j == 0 ? c[kv][i].x : c[kv][i].y, g);
#pragma unroll
            for (int e = 0; e < 4; ++e) f[4 * j + e] = ok ? g[e] * scale : 0.f;
          }
          __stcs(reinterpret_cast<uint4 *>(dst + i * (LPR * E)), Piece<T>::pack(f));
        }
      }
    }
  }
}

template <bool WRITE>
int io_call(void *k, void *v, const rpa_q8_cache *cache, const int32_t *page_table, const int32_t *cu,
            const int32_t *kv, const int32_t *num_seqs, int32_t max_seqs, const rpa_dims *d, uint32_t *dev_flags,
            cudaStream_t stream) {
  int rc = validate_dims(d);
  if (rc) return rc;
  if (max_seqs < 0) return RPA_ERR_INVALID_ARG;
  if (max_seqs == 0 || d->total_q_tokens == 0) return RPA_OK;
  if (!k || !v || !cache || !cache->k_codes || !cache->v_codes || !cache->k_scales || !cache->v_scales ||
      !page_table || !cu || !kv || !num_seqs)
    return RPA_ERR_INVALID_ARG;
  if (!aligned16(k) || !aligned16(v) || !aligned16(cache->k_codes) || !aligned16(cache->v_codes) ||
      !aligned16(cache->k_scales) || !aligned16(cache->v_scales))
    return RPA_ERR_INVALID_ARG;
  IoArgs a{};
  a.k = k;
  a.v = v;
  a.c = cache_of(cache);
  a.len = lengths_of(cu, kv, num_seqs, max_seqs, d, -1, true);
  a.page_table = page_table;
  a.err = dev_flags;
  a.hkv = d->num_kv_heads;
  a.p = d->page_size;
  a.p_shift = log2_of(d->page_size);
  a.num_pages = d->num_pages;
  a.max_pages = d->max_pages_per_seq;
  // enough blocks to fill 148 SMs at 8 blocks each; longer batches loop
  const int64_t rows = (int64_t)d->total_q_tokens * d->num_kv_heads;
  const int64_t per = kThreads / (d->head_dim / 16);
  const unsigned grid = (unsigned)std::min<int64_t>((rows + per - 1) / per, 148 * 8);
#define RPA_Q8_IO(DD)                                                                                \
  case DD:                                                                                           \
    if (d->dtype == RPA_F32) io_kernel<float, DD, WRITE><<<grid, kThreads, 0, stream>>>(a);          \
    else io_kernel<__nv_bfloat16, DD, WRITE><<<grid, kThreads, 0, stream>>>(a);                      \
    break;
  switch (d->head_dim) {
    RPA_Q8_IO(64)
    RPA_Q8_IO(128)
    RPA_Q8_IO(256)
    default: return RPA_ERR_UNSUPPORTED;
  }
#undef RPA_Q8_IO
  return cudaGetLastError() == cudaSuccess ? RPA_OK : RPA_ERR_CUDA;
}

}  // namespace
}  // namespace q8
}  // namespace rpa

extern "C" RPA_API int rpa_q8_write(const void *k_new, const void *v_new, const rpa_q8_cache *cache,
                                    const int32_t *page_table, const int32_t *cu_q_lens, const int32_t *kv_lens,
                                    const int32_t *num_seqs, int32_t max_seqs, const rpa_dims *dims,
                                    uint32_t *dev_flags, void *stream) {
  return rpa::q8::io_call<true>(const_cast<void *>(k_new), const_cast<void *>(v_new), cache, page_table, cu_q_lens,
                                kv_lens, num_seqs, max_seqs, dims, dev_flags, (cudaStream_t)stream);
}

extern "C" RPA_API int rpa_q8_read(void *k_out, void *v_out, const rpa_q8_cache *cache, const int32_t *page_table,
                                   const int32_t *cu_lens, const int32_t *kv_lens, const int32_t *num_seqs,
                                   int32_t max_seqs, const rpa_dims *dims, uint32_t *dev_flags, void *stream) {
  return rpa::q8::io_call<false>(k_out, v_out, cache, page_table, cu_lens, kv_lens, num_seqs, max_seqs, dims,
                                 dev_flags, (cudaStream_t)stream);
}
