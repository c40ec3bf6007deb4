// q8_common.cuh -- what the kernels on the 8-bit K/V cache share: the format's
// arithmetic, and the device-side view and checks of a call's lengths.
//
// Format.  A row x of D values (one token, one KV head) is stored as D e4m3
// codes and one scale 2^e:  e is the smallest integer >= -127 with
// max|x| <= 448 * 2^e (448 is e4m3's largest value; e = 0 for a row of
// zeros), and code_d = x_d * 2^-e rounded to nearest-even.  The scale is
// a power of two so that x_d * 2^-e is exact and the code is one well-defined
// rounding (half a step: relative 2^-4, or absolute 2^-10 * 2^e below 2^-6):
// every machine writes the same bits.  e4m3 codes carry an exponent of their
// own, so a finer scale would not make them more precise, only use the last
// fraction of a binade at the top.  The scale is stored as the byte e + 127
// (e8m0); 255 is NaN and marks a row that held an infinity or a NaN, whose codes
// are zeros: a stored code is never NaN.  At the largest scale, 2^120, codes stop at 240: the next one,
// 256, would stand for 2^128, an infinity in both row types (240 is within half a step, 2^-4, of every
// finite value that would round to it).
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "rpa.h"

namespace rpa {
namespace q8 {

constexpr uint32_t kScaleOne = 127;
constexpr uint32_t kScaleNan = 255;
constexpr uint32_t kScaleTop = 247;   // 2^120, the largest of a finite row

struct Cache {
  uint8_t *k, *v;     // codes [num_pages, P, Hkv, D]
  uint8_t *ks, *vs;   // scales [num_pages, Hkv, P]
};

// The lengths of one call, in device memory.
struct Lengths {
  const int32_t *cu, *kv, *num_seqs;
  int32_t max_seqs;
  int32_t T;          // rows of the token arrays
  int32_t cap;        // max_pages_per_seq * P, saturated
  int32_t max_q;      // longest allowed q_len; < 0: any
  int32_t self;       // 1: every sequence needs kv_len >= q_len
};

__device__ __forceinline__ void raise(uint32_t *err, uint32_t bits) {
  if (err != nullptr) atomicOr(err, bits);
}

// 1 if sequence s of n, whose tokens are x0 .. x1 - 1, breaks a rule.
__device__ __forceinline__ int breaks(const Lengths &a, int n, int s, int x0, int x1, int kv) {
  const int64_t ql = (int64_t)x1 - x0;
  return ql < 0 || kv < 0 || kv > a.cap || (a.max_q >= 0 && ql > a.max_q) || (a.self && kv < ql) ||
         (s == 0 && x0 != 0) || (s == n - 1 && x1 > a.T);
}

// Checks the lengths by every thread of the block (a read of the whole list:
// kernels that run many blocks share it through L2).  Returns the number of
// sequences, or -1 (uniform in the block) when a rule is broken.  Contains
// block barriers.
__device__ __forceinline__ int checked_seqs(const Lengths &a) {
  const int n = *a.num_seqs;
  int bad = n < 0 || n > a.max_seqs;
  if (!bad) {
    for (int s = threadIdx.x; s < n; s += blockDim.x) bad |= breaks(a, n, s, a.cu[s], a.cu[s + 1], a.kv[s]);
  }
  return __syncthreads_or(bad) ? -1 : n;
}

// A CTA's run in a list of blocks of work, the sequences' blocks in order: runs are
// equal, the first total % ctas of them one block longer.
struct Start {
  int n;           // sequences; < 0: the lengths break a rule
  int s;           // the sequence of the run's first block,
  int64_t off;     // that block's place within it,
  int64_t count;   // the run's blocks (0: none; s and off are not set)
};

// Checks the lengths, as checked_seqs does, and finds the CTA's run; blocks(q_len, kv_len)
// is a sequence's number of blocks.  By all NT threads, uniform in the block; scan: shared
// memory for 2 * NT / 32 + 2 words.  Up to NT sequences take one pass: their lengths are
// read beside the count (entries past it lie within the arrays and are dropped).
template <int NT, class F>
__device__ __forceinline__ Start find_start(const Lengths &a, int cta, int ctas, int64_t *scan, F blocks) {
  constexpr int NW = NT / 32;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int c0 = 0, c1 = 0, kv = 0;
  if (tid < a.max_seqs) {
    c0 = a.cu[tid];
    c1 = a.cu[tid + 1];
    kv = a.kv[tid];
  }
  const int n = *a.num_seqs;
  int bad = n < 0 || n > a.max_seqs;
  auto check = [&](int s, int x0, int x1, int k) { bad |= breaks(a, n, s, x0, x1, k); };
  auto warp_scan = [&](int64_t v) -> int64_t {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    return v;
  };
  int64_t b = 0, rest = 0;
  if (!bad && tid < n) {
    check(tid, c0, c1, kv);
    if (!bad) b = blocks(c1 - c0, kv);
  }
  if (n > NT)
    for (int s = tid + NT; !bad && s < n; s += NT) {
      const int x0 = a.cu[s], x1 = a.cu[s + 1], k = a.kv[s];
      check(s, x0, x1, k);
      if (!bad) rest += blocks(x1 - x0, k);
    }
  int64_t incl = warp_scan(b);
  if (lane == 31) scan[warp] = incl;
  rest = n > NT ? warp_scan(rest) : 0;
  if (lane == 31) scan[NW + warp] = rest;
  if (__syncthreads_or(bad)) return Start{-1, 0, 0, 0};
  int64_t excl = incl - b, tile = 0, total = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    if (w < warp) excl += scan[w];
    tile += scan[w];
    total += scan[w] + scan[NW + w];
  }
  const int64_t per = total / ctas, extra = total - per * ctas;
  const int64_t first = per * cta + (cta < extra ? cta : extra);
  Start r{n, 0, 0, per + (cta < extra ? 1 : 0)};
  if (r.count == 0) return r;
  if (first >= excl && first < excl + b) {
    scan[2 * NW] = tid;
    scan[2 * NW + 1] = first - excl;
  }
  int64_t before = tile;
  for (int s0 = NT; first >= before; s0 += NT) {   // uniform; only with more than NT sequences
    const int s = s0 + tid;
    b = s < n ? blocks(a.cu[s + 1] - a.cu[s], a.kv[s]) : 0;
    incl = warp_scan(b);
    __syncthreads();                               // the sums of the round before have been read
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    excl = before + incl - b;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      if (w < warp) excl += scan[w];
      before += scan[w];
    }
    if (first >= excl && first < excl + b) {
      scan[2 * NW] = s;
      scan[2 * NW + 1] = first - excl;
    }
  }
  __syncthreads();
  r.s = (int)scan[2 * NW];
  r.off = scan[2 * NW + 1];
  return r;
}

// The sequence that holds token t: the largest s in [0, n) with cu[s] <= t.
__device__ __forceinline__ int seq_of(const int32_t *cu, int n, int t) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (cu[mid] <= t) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Scale byte of a row whose largest |x| has the fp32 bits `amax`.
__device__ __forceinline__ uint32_t scale_code(uint32_t amax) {
  if (amax >= 0x7f800000u) return kScaleNan;
  if (amax == 0) return kScaleOne;
  // amax = f * 2^k, f in [1, 2); 448 = 1.75 * 2^8: e = k - 8, one more when
  // f > 1.75.  Subnormal amax lands below the clamp.
  const int k = (int)(amax >> 23) - 127;
  const int e = k - 8 + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0);
  return (uint32_t)(max(e, -127) + 127);
}
// 2^-e for a scale byte that is not NaN (e <= 120, so this is a normal number).
__device__ __forceinline__ float inverse_scale(uint32_t code) { return __uint_as_float((254u - code) << 23); }
// 2^e, NaN for 255.
__device__ __forceinline__ float scale_value(uint32_t code) {
  return __uint_as_float(code == 0 ? 0x00400000u : code == kScaleNan ? 0x7fffffffu : code << 23);
}

// Two fp32 values to e4m3 (nearest-even), `lo` in the low byte.
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// Four codes at the scale kScaleTop: 256 becomes 240, of either sign.
__device__ __forceinline__ uint32_t below_2_128(uint32_t v) {
  return v - (__vcmpeq4(v & 0x7f7f7f7fu, 0x78787878u) & 0x01010101u);
}
// Two e4m3 codes (low 16 bits) to fp16 (exact).
__device__ __forceinline__ __half2 from_e4m3x2(uint32_t v) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)v));
  return *reinterpret_cast<__half2 *>(&r);
}
__device__ __forceinline__ void e4m3x4_to_f32(uint32_t v, float (&f)[4]) {
  const float2 a = __half22float2(from_e4m3x2(v)), b = __half22float2(from_e4m3x2(v >> 16));
  f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y;
}

}  // namespace q8
}  // namespace rpa
