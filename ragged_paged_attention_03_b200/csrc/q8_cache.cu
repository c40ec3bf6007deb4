// q8_cache.cu -- quantising new K/V rows into the 8-bit paged cache
// (rpa_q8_write) and reading cached rows back (rpa_q8_read).
//
// Both are one pass over the rows and bound by memory: a row of D values
// moves D * sizeof(T) + D + 1 bytes.  D / 16 neighbouring lanes share a row, each
// with 16 values next to each other: 32-byte loads or stores of T (two for fp32) and
// 16-byte ones of codes.  The values stay in registers between the row's maximum
// (shuffles among those lanes) and the rounding, so every value is read once; K and V of
// a row are in flight together.  A warp's rows are neighbouring tokens of one head, so
// that their scales, single bytes, share a sector, and neighbouring warps take the
// heads, so that together they read what lies together.
//
// Measured, launch included: 16,384 tokens of 8 heads, D 128, bf16, written in 20.5 us
// (4.9 TB/s, 0.75 of a plain copy's rate) and a context of about that size read in 19.6 us;
// below a few thousand rows a call costs its launch (3.0 us in a graph).  The write issues in
// 67 % of its slots: maxima, products and conversions, not the memory, set the rest.
#include <algorithm>
#include <cuda_runtime.h>

#include "host_common.h"
#include "ptx.cuh"
#include "q8_common.cuh"
#include "q8_host.h"
#include "rpa.h"

namespace rpa {
namespace q8 {
namespace {

constexpr int kThreads = 256;
constexpr int kLenCap = 512;    // sequences whose lengths are kept in shared memory
// Blocks of 256 threads that an SM holds: 6 with 16-bit rows (40 registers a thread), 4 with
// fp32 ones, whose 32 values a thread take 64 registers.  The grid is no larger than that.
template <typename T> constexpr int kBlocks = sizeof(T) == 2 ? 6 : 4;

struct IoArgs {
  void *k, *v;                 // [T, Hkv, D] rows outside the cache
  Cache c;
  Lengths len;
  const int32_t *page_table;
  uint32_t *err;
  int32_t hkv, p, p_shift, num_pages, max_pages;
};

// 16 values of T next to each other, as 32-bit words.
template <typename T> constexpr int kWords = 4 * (int)sizeof(T);
template <typename T>
__device__ __forceinline__ void load16(const T *p, uint32_t (&w)[kWords<T>]) {
#pragma unroll
  for (int i = 0; i < kWords<T>; i += 8)
    asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3]), "=r"(w[i + 4]), "=r"(w[i + 5]),
                   "=r"(w[i + 6]), "=r"(w[i + 7])
                 : "l"(reinterpret_cast<const uint32_t *>(p) + i));
}
template <typename T>
__device__ __forceinline__ void store16(T *p, const uint32_t (&w)[kWords<T>]) {
#pragma unroll
  for (int i = 0; i < kWords<T>; i += 8)
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(reinterpret_cast<uint32_t *>(p) + i),
                 "r"(w[i]), "r"(w[i + 1]), "r"(w[i + 2]), "r"(w[i + 3]), "r"(w[i + 4]), "r"(w[i + 5]), "r"(w[i + 6]),
                 "r"(w[i + 7])
                 : "memory");
}
// The fp32 bits of the largest |x|: compared as integers, with infinities and NaN on top,
// or two bf16 at a time (a NaN stays).
__device__ __forceinline__ uint32_t absmax(const uint32_t (&w)[16]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = max(m, w[i] & 0x7fffffffu);
  return m;
}
__device__ __forceinline__ uint32_t absmax(const uint32_t (&w)[8]) {
  uint32_t m = ptx::absmax_bf16x2(w[0], w[1]);
#pragma unroll
  for (int i = 2; i < 8; ++i) m = ptx::absmax_bf16x2(m, w[i]);
  return max((m << 16) & 0x7fff0000u, m & 0x7fff0000u);
}
// Values 2 i and 2 i + 1 of the 16 as an fp32 pair, and back.
__device__ __forceinline__ uint64_t pair(const uint32_t (&w)[16], int i) {
  return ptx::f2_pack(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
}
__device__ __forceinline__ uint64_t pair(const uint32_t (&w)[8], int i) {
  return ptx::f2_pack(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}
__device__ __forceinline__ void put(uint32_t (&w)[16], int i, uint64_t p) {
  float a, b;
  ptx::f2_unpack(p, a, b);
  w[2 * i] = __float_as_uint(a);
  w[2 * i + 1] = __float_as_uint(b);
}
__device__ __forceinline__ void put(uint32_t (&w)[8], int i, uint64_t p) {
  float a, b;
  ptx::f2_unpack(p, a, b);
  w[i] = ptx::pack_bf16(a, b);
}

template <typename T, int D, bool WRITE>
__global__ void __launch_bounds__(kThreads, kBlocks<T>) io_kernel(const IoArgs a) {
  constexpr int LPR = D / 16;         // lanes per row
  constexpr int RW = 32 / LPR;        // rows (tokens) per warp
  __shared__ int32_t s_cu[kLenCap + 1], s_kv[kLenCap];
  // The lengths, checked, and in shared memory where they fit.  Where the arrays fit, in one pass
  // that reads them beside the count (entries past it lie within the arrays and are dropped):
  // one latency instead of three.
  const int32_t *cu = a.len.cu, *kv = a.len.kv;
  int n;
  if (a.len.max_seqs <= kLenCap) {
    constexpr int PER = kLenCap / kThreads;
    int c0[PER], c1[PER], k[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int i = threadIdx.x + j * kThreads;
      if (i < a.len.max_seqs) c0[j] = cu[i], c1[j] = cu[i + 1], k[j] = kv[i];
    }
    n = *a.len.num_seqs;
    int bad = n < 0 || n > a.len.max_seqs;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int i = threadIdx.x + j * kThreads;
      if (bad || i >= n) continue;
      bad |= breaks(a.len, n, i, c0[j], c1[j], k[j]);
      s_cu[i] = c0[j];
      s_kv[i] = k[j];
      if (i == n - 1) s_cu[n] = c1[j];
    }
    if (__syncthreads_or(bad)) n = -1;
    cu = s_cu;
    kv = s_kv;
  } else {
    n = checked_seqs(a.len);
    if (n >= 0 && n <= kLenCap) {
      for (int i = threadIdx.x; i <= n; i += kThreads) {
        s_cu[i] = cu[i];
        if (i < n) s_kv[i] = kv[i];
      }
      __syncthreads();
      cu = s_cu;
      kv = s_kv;
    }
  }
  if (n < 0) {
    if (blockIdx.x == 0 && threadIdx.x == 0) raise(a.err, RPA_DEV_BAD_LENGTHS);
    return;
  }
  if (n == 0) return;
  const int total = cu[n];
  const int lane = threadIdx.x & 31, sub = lane % LPR;
  // a row's lanes are neighbours in one warp and take the same way
  const unsigned lanes = LPR == 32 ? 0xffffffffu : ((1u << LPR) - 1u) << (lane / LPR * LPR);
  // the warp's tasks: RW tokens of one head each, `step` tasks apart; divided once
  const int step = (int)gridDim.x * (kThreads / 32), step_g = step / a.hkv, step_h = step - step_g * a.hkv;
  const int first = (int)blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
  int tg = first / a.hkv, h = first - tg * a.hkv, s = 0;
  for (; (int64_t)tg * RW < total; tg += step_g, h += step_h) {
    if (h >= a.hkv) {
      h -= a.hkv;
      if ((int64_t)++tg * RW >= total) break;
    }
    const int t = tg * RW + lane / LPR;
    if (t >= total) continue;
    const size_t row = ((size_t)t * a.hkv + h) * D + sub * 16;
    uint32_t x[2][kWords<T>];
    if (WRITE) {
      load16(static_cast<const T *>(a.k) + row, x[0]);
      load16(static_cast<const T *>(a.v) + row, x[1]);
    }
    if (t < cu[s] || t >= cu[s + 1]) s = seq_of(cu, n, t);    // mostly the sequence of the task before
    const int pos = kv[s] - cu[s + 1] + t;         // kv_len - q_len + (t - cu[s])
    const int page = a.page_table[(size_t)s * a.max_pages + (pos >> a.p_shift)];
    const bool ok = page >= 0 && page < a.num_pages;
    if (!ok && sub == 0) raise(a.err, RPA_DEV_BAD_PAGE);
    const int slot = pos & (a.p - 1);
    const size_t crow = (((size_t)(ok ? page : 0) * a.p + slot) * a.hkv + h) * D + sub * 16;
    const size_t srow = ((size_t)(ok ? page : 0) * a.hkv + h) * a.p + slot;
    if (WRITE) {
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        uint32_t amax = absmax(x[v]);
#pragma unroll
        for (int o = 1; o < LPR; o <<= 1) amax = max(amax, __shfl_xor_sync(lanes, amax, o));
        const uint32_t code = scale_code(amax);
        const float inv = code == kScaleNan ? 0.f : inverse_scale(code);
        if (!ok) continue;
        const uint64_t inv2 = ptx::f2_pack(inv, inv);
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float f[4];
          ptx::f2_unpack(ptx::f2_mul(pair(x[v], 2 * i), inv2), f[0], f[1]);
          ptx::f2_unpack(ptx::f2_mul(pair(x[v], 2 * i + 1), inv2), f[2], f[3]);
          w[i] = to_e4m3x2(f[0], f[1]) | (to_e4m3x2(f[2], f[3]) << 16);
        }
        if (code >= kScaleTop) {
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] = code == kScaleNan ? 0u : below_2_128(w[i]);
        }
        *reinterpret_cast<uint4 *>((v ? a.c.v : a.c.k) + crow) = make_uint4(w[0], w[1], w[2], w[3]);
        if (sub == 0) (v ? a.c.vs : a.c.ks)[srow] = (uint8_t)code;
      }
    } else {
      uint4 c[2];
      uint32_t sc[2];
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        c[v] = *reinterpret_cast<const uint4 *>((v ? a.c.v : a.c.k) + crow);
        sc[v] = (v ? a.c.vs : a.c.ks)[srow];
      }
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        // a page outside the pool reads as zeros
        const float scale = ok ? scale_value(sc[v]) : 0.f;
        const uint64_t scale2 = ptx::f2_pack(scale, scale);
        const uint32_t w[4] = {c[v].x, c[v].y, c[v].z, c[v].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float g[4];
          e4m3x4_to_f32(ok ? w[i] : 0u, g);
          put(x[v], 2 * i, ptx::f2_mul(ptx::f2_pack(g[0], g[1]), scale2));
          put(x[v], 2 * i + 1, ptx::f2_mul(ptx::f2_pack(g[2], g[3]), scale2));
        }
        store16(static_cast<T *>(v ? a.v : a.k) + row, x[v]);
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
  if (!aligned32(k) || !aligned32(v) || !aligned16(cache->k_codes) || !aligned16(cache->v_codes) ||
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
  // as many blocks as the 148 SMs hold at once; longer batches loop
  const int64_t per = (512 / d->head_dim) * (kThreads / 32);     // rows of a block's warps
  const int64_t rows = ((int64_t)d->total_q_tokens + 31) / 32 * 32 * d->num_kv_heads;
  const unsigned grid = (unsigned)std::min<int64_t>((rows + per - 1) / per, 148 * (d->dtype == RPA_F32 ? kBlocks<float> : kBlocks<__nv_bfloat16>));
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
