// q8_chunk_kernel.cu -- attention over the 8-bit cache for chunks of query rows
// (bf16): bound by the tensor cores and the softmax.
//
// Mathematics.  The query rows of one KV head, row = token i * G + head g, are
// the M side (a KV head's G query heads share every key tile); S = Q K^T and
// O += P V are fp16 MMAs with fp32 accumulators and an online softmax in fp32
// (log2 domain, lazily rescaled).  fp16 and not bf16: one instruction turns two
// e4m3 codes into fp16 (64 a clock and SM measured, against 32 for the shifts and
// masks that make bf16 of them), and P has 11 bits instead of 8.  Ranges are
// kept by powers of two, which are exact:
//   K tile:  code * 2^(ek - ekb), ekb the largest K scale of the 128 keys (but for rows of
//            zeros); the factor 2^ekb joins the row's score factor;
//   V tile:  code * 2^(ev - evb) the same way; P of the block carries 2^(evb - evr)
//            in its exponent, evr the row's own reference, moved (with a rescale of
//            the row's O) when its contributions pass it by more than 2^6;
//   both exact while the tile's scales lie within 2^15 of each other.  A "wide" tile,
//            whose scales do not, holds the bare codes, and the softmax warps apply the
//            scales in fp32, key by key, from global memory (slow, and rare: rows of
//            one sequence, zeros aside, that differ in size by more than 30,000 times);
//   Q row:   q * 2^-eq, as the cache's rows are scaled, so every value is exact
//            down to 2^-25 of the row's largest and within 2^-33 of that below;
//   P:       2^5 at the row's largest weight times its tile's V scale (up to 2^11 while the
//            rescale is put off), so it has 11 bits down to 2^-19 of that and counts
//            down to 2^-29.  Keys whose V rows are zeros do not set this unit.
// A token whose K or V row is NaN gets a NaN key and a zero value: its column is
// NaN for the rows that see it, and a masked column is dropped whatever it holds.
//
// Split of the work: as in the row-group kernel, the blocks of all items (two
// 128-row tiles of one sequence and KV head) are one list, cut into equal runs,
// one per CTA; runs that begin or end inside an item leave partial results that
// combine_kernel joins.
//
// Roles (512 threads of at most 128 registers).  Every hot loop is short and
// rolled: with five kinds of warps on an SM the unrolled forms (a row's 128 scores in
// registers) were bound by instruction fetch, at a third of this speed.
// Measured (Hq 32, Hkv 8, D 128): 8 prompts of 2048 tokens 402 us (684 TFLOP/s of the causal
// products), 4 chunks of 512 behind contexts of some thousands 194 us (725 TFLOP/s); D 256 (Hq 16,
// Hkv 4), 4 prompts of 4096 tokens 940 us (585 TFLOP/s).  A block of
// 128 keys takes 4,200 to 4,900 clocks where its MMAs need 2,048: the conversion of its K and V takes
// the converters 4,200 (1,250 each, the rest waits that are over when they are looked at), a
// softmax step 2,000 to 2,500 of which the exponentials are 650 to 1,200, by whether both
// tiles' are at theirs; the tensor pipe is active 35 % of the time, the issue slots 51 %.
//   warps 0-3, 4-7  softmax and output of tile 0 and 1 (one row per thread); they
//                   also turn their tile's Q, landed by TMA as bf16, into scaled
//                   fp16 in place
//   warps 8-11      keys and values: code tiles, landed by TMA, into swizzled fp16 tiles
//   warps 12, 15    MMA issue of tile 0 and 1 (warp 12 owns TMEM).  One warp for both
//                   took 4,500 clocks for a step of the two tiles, waits that
//                   were over included, and held everything else up
//   warp 13         walks the run: writes its segments down for the others; TMA of Q
//   warp 14         TMA of the code tiles; the scales of their keys as fp16 factors; looks
//                   for rows of zeros among those of scale 2^0 (8 prompts of 2048 tokens take
//                   480 us where every row has that scale, 780 us with a V row of zeros in every block)
// TMEM (512 columns): S/P of tile 0 (two buffers of 64 keys) | of tile 1 | O of
// tile 0 | O of tile 1.
#include <cuda.h>
#include <math.h>

#include <algorithm>

#include "ptx.cuh"
#include "q8_common.cuh"
#include "q8_kernels.h"
#include "tma.h"

namespace rpa {
namespace q8 {
namespace {

constexpr int kThreads = 512;
constexpr int BM = 128;             // rows of a tile
constexpr int HN = 64;              // keys of a step
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescale = 6.0f;    // lazy rescale of O: weights reach 2^(6 + kBase)
constexpr int kBase = 5;
constexpr int kWide = 15;           // a tile whose scales spread further is "wide"
constexpr int kLift = 24;           // weights whose V rows are zeros pass the units of O by 2^kLift at most
constexpr int kWideBit = 1 << 16;   // in the published ekb / evb
constexpr int kZeroBit = 1 << 17;   // in the published evb: the tile has V rows of zeros
constexpr int kExpWords = 6;        // published of a block: ekb, evb, V rows of zeros (word k: keys 4 i + k)
constexpr int kExpSlots = 8;
constexpr int kSegSlots = 4;

template <int D>
struct Shape {
  // head_dim 256: one tile, and blocks of 64 keys instead of 128 (TMEM holds one O of 256
  // columns beside the scores, shared memory half as many keys)
  static constexpr int NT = D == 256 ? 1 : 2;              // tiles of an item
  static constexpr int BN = D == 256 ? 64 : 128;           // keys of a block
  static constexpr int SPB = BN / HN;                      // steps of a block
  static constexpr int ROWS = NT * BM;
  static constexpr int NSK = D == 64 ? 4 : 2, NSV = NSK;   // fp16 tiles
  static constexpr int NST = D == 64 ? 4 : 2;              // code tiles: K, V, K, V, ...
  static constexpr int kHalves = D / 64;
  static constexpr int kQBytes = kHalves * BM * 128;
  static constexpr int kKVBytes = kHalves * BN * 128;
  static constexpr int kCodes = BN * D;
  static constexpr int kData = NT * kQBytes + (NSK + NSV) * kKVBytes + NST * kCodes;
  static constexpr int kSmem = 1024 + kData + 2048;
  static constexpr uint32_t kTmemCols = 512, kColO = NT * 128;
};

struct Bars {
  uint64_t q_full[2], q_empty[2], qc_full[2];
  uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4];
  uint64_t c_full[4], c_empty[4];
  uint64_t f_full[2], f_empty[2];
  uint64_t e_full[kExpSlots];
  uint64_t s_full[2][2], p_full[2][2], pv_done[2][2], o_free[2];   // [tile][S buffer]
  uint64_t seg_full[kSegSlots], seg_empty[kSegSlots];
  uint64_t drain[2];
};

// One item's part of the CTA's run, written by warp 13 for the others.
struct Seg {
  int32_t seq, hk, item, b0;
  int32_t blocks;                // blocks to run; < 0: the end of the run
  int32_t nt[2], rows[2];        // steps and rows of each tile
  int32_t q0, row0;              // first token of the sequence, of the item within it
  int32_t kv, q_len;
  int32_t whole;                 // the item begins and ends here
  int32_t pad[2];
};
template <int NT> constexpr int kSegUsers = NT + 1 + 4 + 4 * NT;   // warps that release a slot: MMA, TMA of codes, converters, softmax

static_assert(1024 + sizeof(Bars) + kExpWords * kExpSlots * 4 + kSegSlots * sizeof(Seg) + 8 <= 2048, "control block");

struct PartHead {
  int32_t seq, hk, item, begin;
};

struct Args {
  AttendArgs a;
  int32_t q_limit;       // sequences of at most this many new tokens are another kernel's
  int32_t tpt;           // tokens per tile: 128 / G
  PartHead *heads;       // [ctas]
  float2 *ml;            // [2 * ctas][ROWS] maximum (log2), sum
  float4 *o;             // [2 * ctas][D / 4][ROWS]
};

// sum over i in [0, n) of floor((a i + b) / M), a, b >= 0: by the quotients and
// remainders of a and b, which leaves floor((a' i + b') / M) with a', b' < M; its sum
// repeats every M terms.
template <int M>
__device__ __forceinline__ int64_t floor_sum(int64_t n, int64_t a, int64_t b) {
  int64_t sum = (a / M) * (n * (n - 1) / 2) + (b / M) * n;
  const int ar = (int)(a % M), br = (int)(b % M);
  const int64_t turns = n / M;
  const int rest = (int)(n % M);
  // i = M j + k: floor((ar i + br) / M) = ar j + floor((ar k + br) / M)
  int64_t whole = 0, part = 0;
  if (turns > 0)
#pragma unroll 1
    for (int k = 0; k < M; ++k) whole += (ar * k + br) / M;
#pragma unroll 1
  for (int k = 0; k < rest; ++k) part += (ar * k + br) / M;
  return sum + turns * whole + (int64_t)ar * M * (turns * (turns - 1) / 2) + part + (int64_t)ar * turns * rest;
}

// The items of one sequence and KV head.  Item i holds tokens [i TT, (i + 1) TT)
// and sees the first end(i) keys; it has max(1, ceil(end / BN)) blocks.  In the list
// that is cut into runs an item counts kItemCost blocks more, at its front: its Q and its
// output take 12,000 clocks beside 5,000 a block, and runs of equal blocks took 370 to 467 us
// where they held 9 and 22 items.
constexpr int kItemCost = 2;
template <int BN>
struct SeqItems {
  int q_len, kv, TT, causal, items;
  __device__ __forceinline__ int end_of(int tokens) const {   // keys that token `tokens - 1` sees
    return causal ? min(kv, max(0, kv - q_len + tokens)) : kv;
  }
  __device__ __forceinline__ int blocks_of(int item) const {
    return max(1, (end_of(min(q_len, (item + 1) * TT)) + BN - 1) / BN);
  }
  // blocks of items [0, n), kItemCost included
  __device__ __forceinline__ int64_t before(int n) const {
    if (n <= 0) return 0;
    if (!causal) return (int64_t)n * (max(1, (kv + BN - 1) / BN) + kItemCost);
    const int whole = min(n, q_len / TT);            // items with all their tokens
    const int64_t c = (int64_t)kv - q_len;
    // the first items whose last token sees no key have one block
    const int64_t none = c >= 0 ? 0 : min((int64_t)whole, -c / TT);
    int64_t sum = none;
    if (whole > none) sum += floor_sum<BN>(whole - none, TT, c + (none + 1) * TT + BN - 1);
    if (n > whole) sum += blocks_of(n - 1);
    return sum + (int64_t)n * kItemCost;
  }
};
template <int D>
__device__ __forceinline__ SeqItems<Shape<D>::BN> seq_items(int q_len, int kv, const Args &g) {
  SeqItems<Shape<D>::BN> w;
  w.q_len = q_len;
  w.kv = kv;
  w.TT = Shape<D>::NT * g.tpt;
  w.causal = g.a.causal;
  w.items = q_len > g.q_limit ? (q_len + w.TT - 1) / w.TT : 0;
  return w;
}

// The CTA's run of blocks, one segment per item it touches.
template <int D>
struct Run {
  static constexpr int SPB = Shape<D>::SPB;
  const Args *g;
  int n, s, hk, item, blk;       // blk: place in the item, kItemCost included
  int64_t left;
  SeqItems<Shape<D>::BN> w;
  int q0, row0, b0, b1, nb;      // of the current segment: first token of the item, its blocks
  int nt[2];                     // steps (64 keys) of the segment that tile t takes part in
  int rows[2];                   // rows of tile t

  __device__ __forceinline__ void load() {
    q0 = g->a.len.cu[s];
    w = seq_items<D>(g->a.len.cu[s + 1] - q0, g->a.len.kv[s], *g);
  }
  __device__ __forceinline__ bool next() {
    if (left <= 0) return false;
    while (item >= w.items) {
      item = 0;
      if (w.items == 0 || ++hk >= g->a.hkv) {
        hk = 0;
        if (++s >= n) return false;
        load();
      }
    }
    row0 = item * w.TT;
    nb = w.blocks_of(item);
    const int end = nb + kItemCost, stop = (int)(left < end - blk ? blk + left : end);
    b0 = max(0, blk - kItemCost);
    b1 = max(0, stop - kItemCost);
    left -= stop - blk;
    blk = 0;
    ++item;
    if (b1 <= b0) return false;    // the run ends before the item's first block
    const int G = g->a.hq / g->a.hkv;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int tok = t < Shape<D>::NT ? min(g->tpt, max(0, w.q_len - row0 - t * g->tpt)) : 0;
      rows[t] = tok * G;
      const int vis = tok == 0 ? 0 : max(1, (w.end_of(row0 + t * g->tpt + tok) + HN - 1) / HN);
      nt[t] = max(0, min(SPB * b1, vis) - SPB * b0);
    }
    return true;
  }
  __device__ __forceinline__ int blocks() const { return (max(nt[0], nt[1]) + SPB - 1) / SPB; }
};

// 2^(e - top) as fp16 bits (0 below fp16's range; a byte of no key may lie above
// top: 1), NaN if `nan`.
__device__ __forceinline__ uint32_t half_factor(int e, int top, bool nan) {
  const int d = min(e - top, 0);
  return nan ? 0x7fffu : d >= -14 ? (uint32_t)(15 + d) << 10 : d >= -24 ? 1u << (24 + d) : 0u;
}
__device__ __forceinline__ uint32_t mul_h2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t codes_h2(uint32_t v) {
  const __half2 h = from_e4m3x2(v);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// A row's running maximum (log2), the sum of its weights (2^kBase per unit weight), and the units of its O.
struct RowSum {
  float m, l;
  float evf;                     // log2 of the row's largest contribution so far, less m,
  int evr;                       // rounded up: O is in units of 2^(m + evr - kBase)
};
// A step of a softmax warp: 64 keys of a tile.
struct Step {
  uint32_t tS, tO;               // the scores, which P replaces, and O in TMEM
  uint64_t *pv_done;             // of the step before
  uint32_t pv_parity;
  int first;                     // of a segment: there is no O yet
  int lim;                       // keys that the row sees
  int ek, ev;                    // the block's K and V scales
  float sc;                      // score factor
  volatile int *abort_flag;
  uint32_t *err;
};

// Moves m (and the units of O, evr) to what the step needs: mx its largest score, my its
// largest score with the V scale, relative to 2^ev.
template <int D>
__device__ __forceinline__ bool take_max(RowSum &r, const Step &st, float mx, float my) {
  const float m_new = fmaxf(r.m, mx);
  // contributions of the row may pass the units of O by 2^kRescale
  const bool need = m_new > r.m + kRescale || my + (float)(st.ev - r.evr) > r.m + kRescale;
  if (__any_sync(0xffffffffu, need)) {
    // O must be complete up to the step before.  (A barrier for each S buffer: the
    // scores of step j came behind PV(j - 2), so the PV before on this one is over and
    // its parity is not ambiguous.)
    if (!st.first && !wait_warp(st.pv_done, st.pv_parity, st.abort_flag, st.err)) return false;
    ptx::tc_fence_after();
    // The new units: the larger of the old ones and the block's largest contribution (a row
    // that has seen nothing has no old ones), relative to 2^m and with their fraction: whole
    // octaves taken from the whole ones of the time before would gain up to one each time, and
    // every row of the warp comes by whenever one of them needs it
    const float was = r.m == -INFINITY ? -INFINITY : r.evf + (r.m - m_new);
    if (m_new != -INFINITY) r.evf = fmaxf(was, (my - m_new) + (float)st.ev);
    const int evn = (int)ceilf(r.evf);
    const float am = r.m == -INFINITY ? 0.f : ptx::ex2(r.m - m_new);
    const float alpha = r.m == -INFINITY ? 0.f : ptx::ex2((r.m - m_new) + (float)(r.evr - evn));
    if (!st.first) {
#pragma unroll 1
      for (int cc = 0; cc < D / 32; ++cc) {
        uint32_t o[32];
        ptx::tmem_ld32(st.tO + cc * 32, o);
        ptx::tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
        ptx::tmem_st32(st.tO + cc * 32, o);
      }
    }
    r.l *= am;
    r.m = m_new;
    r.evr = evn;
  }
  return true;
}

// The step of a tile whose values carry their scales.  No key's contribution has a score above `most`.
template <int D>
__device__ __forceinline__ bool tile_step(RowSum &r, const Step &st, float most) {
  uint32_t x[HN];
  ptx::tmem_ld32(st.tS, *reinterpret_cast<uint32_t(*)[32]>(&x[0]));
  ptx::tmem_ld32(st.tS + 32, *reinterpret_cast<uint32_t(*)[32]>(&x[32]));
  ptx::tmem_ld_wait();
  if (__any_sync(0xffffffffu, st.lim < HN)) {
#pragma unroll
    for (int i = 0; i < HN; ++i) x[i] = i < st.lim ? x[i] : 0xff800000u;
  }
  float mq[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) mq[q] = fmaxf(__uint_as_float(x[2 * q]), __uint_as_float(x[2 * q + 1]));
#pragma unroll
  for (int i = 8; i < HN; i += 8)
#pragma unroll
    for (int q = 0; q < 4; ++q)
      mq[q] = ptx::fmax3(mq[q], __uint_as_float(x[i + 2 * q]), __uint_as_float(x[i + 2 * q + 1]));
  const float mx = ptx::fmax3(mq[0], mq[1], fmaxf(mq[2], mq[3])) * st.sc;
  // (not fminf: a row of the tile that is no query holds anything, and NaN must not pass for `most`)
  if (!take_max<D>(r, st, mx, most < mx ? most : mx)) return false;
  // values more than 2^64 below the row's units count as that small (the sum
  // needs the weights above fp32's underflow)
  const int dv = max(st.ev - r.evr, -64);
  const float shift = (r.m == -INFINITY ? 0.f : -r.m) + (float)(kBase + dv);
  const uint64_t scale2 = ptx::f2_pack(st.sc, st.sc);
  const uint64_t shift2 = ptx::f2_pack(shift, shift);
  uint64_t sp2[4] = {0, 0, 0, 0};
  uint32_t pk[HN / 2];
#pragma unroll
  for (int i = 0; i < HN; i += 2) {
    float a0, a1;
    ptx::f2_unpack(ptx::f2_fma(ptx::f2_pack(__uint_as_float(x[i]), __uint_as_float(x[i + 1])), scale2, shift2), a0, a1);
    const float p0 = ptx::ex2(a0), p1 = ptx::ex2(a1);
    sp2[(i >> 1) & 3] = ptx::f2_add(sp2[(i >> 1) & 3], ptx::f2_pack(p0, p1));
    pk[i >> 1] = ptx::pack_f16_sat(p0, p1);
  }
  ptx::tmem_st32(st.tS, pk);
  float sp[8];
#pragma unroll
  for (int k = 0; k < 4; ++k) ptx::f2_unpack(sp2[k], sp[2 * k], sp[2 * k + 1]);
  const float sum = ((sp[0] + sp[1]) + (sp[2] + sp[3])) + ((sp[4] + sp[5]) + (sp[6] + sp[7]));
  r.l += sum * ptx::ex2((float)-dv);            // weights of this step carry 2^dv
  return true;
}

// The steps of blocks that are marked, with V rows of zeros or scales far apart.  Functions of their
// own and not inlined: such blocks are rare, and the softmax warps' loop is bound by its code's size
// too (with them in line 8 prompts of 2048 tokens took 4 % longer).
struct MarkedSum {
  RowSum r;
  int ok;
};

// V rows of zeros among the step's keys: bit i of word k (from bit `shift` on) is key 4 i + k.  Such a
// key's weight counts in the sum but not for the units of O: it may pass them, and is cut off at
// fp16's largest value, which its zeros take to nothing.  By up to 2^kLift: exp2's argument, in which a
// weight's distance from the unit is added, keeps 2^-20 of a weight up to there (2^-18 at 2^100), and the other
// weights keep 11 bits down to 2^-43 of such a key's.
template <int D>
__device__ __noinline__ MarkedSum zeros_step(RowSum r, const Step st, const int *words, int shift) {
  uint32_t z[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) z[k] = (uint32_t)words[k] >> shift;
  float mx = -INFINITY, my = -INFINITY;
#pragma unroll 1
  for (int c = 0; c < HN; c += 8) {
    uint32_t v[8];
    ptx::tmem_ld8(st.tS + c, v, 0);
    ptx::tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float y = c + i < st.lim ? __uint_as_float(v[i]) : -INFINITY;
      mx = fmaxf(mx, y);
      my = fmaxf(my, (z[i & 3] >> (i / 4)) & 1 ? -INFINITY : y);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) z[k] >>= 2;
  }
  const bool ok = tile_step<D>(r, st, fmaxf(my * st.sc, mx * st.sc - kLift));
  return MarkedSum{r, ok};
}

// A wide tile, whose codes carry no scale.
struct Wide {
  const int *e;                  // what is published of the block
  int shift;                     // the step's place in its words
  int key0, end;                 // the step's first key; the keys that the row sees
  const int32_t *pt;
  const uint8_t *ks, *vs;
  int hk, hkv, p, p_shift, num_pages;
};
template <int D>
__device__ __noinline__ MarkedSum wide_step(RowSum r, const Step st, const Wide b) {
  const int lim = st.lim;
  const bool wide_k = (b.e[0] & kWideBit) != 0, wide_v = (b.e[1] & kWideBit) != 0, zeros = (b.e[1] & kZeroBit) != 0;
  uint32_t z[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) z[k] = zeros ? (uint32_t)b.e[2 + k] >> b.shift : 0u;
  // the scale byte of key i, -1 if it is not seen or its page is outside the pool
  auto scale_byte = [&](const uint8_t *src, int i) -> int {
    const int pos = b.key0 + i;
    const int pg = pos < b.end ? b.pt[pos >> b.p_shift] : -1;
    if (pg < 0 || pg >= b.num_pages) return -1;
    return src[((size_t)pg * b.hkv + b.hk) * b.p + (pos & (b.p - 1))];
  };
  auto score = [&](uint32_t v, int i) -> float {
    if (i >= lim) return -INFINITY;
    const int d = wide_k ? min(scale_byte(b.ks, i) - st.ek, 0) : 0;   // > 0: a NaN key, NaN already
    return __uint_as_float(v) * (d < -126 ? 0.f : __uint_as_float((uint32_t)(127 + d) << 23)) * st.sc;
  };
  // V scale of key i relative to `ref`; the tile's own where its values carry theirs
  auto rel_ev = [&](int i, int ref) -> float { return (float)((wide_v ? scale_byte(b.vs, i) : st.ev) - ref); };
  float mx = -INFINITY, my = -INFINITY;
#pragma unroll 1
  for (int c = 0; c < HN; c += 8) {
    uint32_t v[8];
    ptx::tmem_ld8(st.tS + c, v, 0);
    ptx::tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float y = score(v[i], c + i);
      mx = fmaxf(mx, y);
      if (!((z[i & 3] >> (c / 4 + i / 4)) & 1)) my = fmaxf(my, y + rel_ev(c + i, st.ev));
    }
  }
  if (!take_max<D>(r, st, mx, fmaxf(my, mx - 300.f))) return MarkedSum{r, 0};
  // the sum of the bare weights; P with each key's scale
  const float shift = (r.m == -INFINITY ? 0.f : -r.m) + (float)kBase;
  float sum = 0.f;
#pragma unroll 1
  for (int c = 0; c < HN; c += 8) {
    uint32_t v[8], pk[4];
    ptx::tmem_ld8(st.tS + c, v, 0);
    ptx::tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const float y0 = score(v[i], c + i) + shift;
      const float y1 = score(v[i + 1], c + i + 1) + shift;
      sum += ptx::ex2(y0) + ptx::ex2(y1);
      pk[i / 2] = ptx::pack_f16_sat(ptx::ex2(y0 + rel_ev(c + i, r.evr)), ptx::ex2(y1 + rel_ev(c + i + 1, r.evr)));
    }
    ptx::tmem_st4(st.tS + c / 2, pk);            // behind what has been read
  }
  r.l += sum;
  return MarkedSum{r, 1};
}

// Bytes of v that are the scale 2^0.
__device__ __forceinline__ uint32_t has_one(uint32_t v) {
  const uint32_t x = v ^ (kScaleOne * 0x01010101u);
  return (x - 0x01010101u) & ~x & 0x80808080u;
}
// Which of a lane's four keys, at most `keys` of them, hold rows of zeros (of either sign): bit k is
// the K row of key k, bit 4 + k its V row.  Byte k of ks and vs are their scales; their codes are `at`
// + k * stride.  By the format a row of zeros has the scale 2^0, so only such rows are looked
// through.  Not inlined: rare.
template <int D>
__device__ __noinline__ uint32_t zero_rows(const uint8_t *k_codes, const uint8_t *v_codes, size_t at, size_t stride,
                                           uint32_t ks, uint32_t vs, int keys) {
  auto some = [](const uint4 &v) { return ((v.x | v.y | v.z | v.w) & 0x7f7f7f7fu) != 0; };
  auto row = [&](int i) { return (i < 4 ? k_codes : v_codes) + at + (i & 3) * stride; };
  uint32_t mask = 0;
  uint4 first[8];                                 // one latency
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const bool look = (i & 3) < keys && (((i < 4 ? ks : vs) >> (8 * (i & 3))) & 255u) == kScaleOne;
    first[i] = look ? *reinterpret_cast<const uint4 *>(row(i)) : make_uint4(1, 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (!some(first[i])) mask |= 1u << i;
#pragma unroll 1
  for (uint32_t left = mask; left != 0; left &= left - 1) {   // the rest of those: one each
    const int i = __ffs((int)left) - 1;
    bool any = false;
#pragma unroll
    for (int q = 16; q < D; q += 16) any |= some(*reinterpret_cast<const uint4 *>(row(i) + q));
    if (any) mask &= ~(1u << i);
  }
  return mask;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_v, const Args g) {
  using S = Shape<D>;
  constexpr int NSK = S::NSK, NSV = S::NSV, NT = S::NT, BN = S::BN, SPB = S::SPB;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  extern __shared__ uint8_t smem_raw[];
  uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t *sQ = base;
  uint8_t *sK = sQ + NT * S::kQBytes;
  uint8_t *sV = sK + NSK * S::kKVBytes;
  uint8_t *sC = sV + NSV * S::kKVBytes;
  uint16_t *s_fac = reinterpret_cast<uint16_t *>(base + S::kData);   // [2][K, V][128] factors of a block's keys
  Bars *bars = reinterpret_cast<Bars *>(s_fac + 2 * 2 * BN);
  int64_t *s_scan = reinterpret_cast<int64_t *>(s_fac);          // [2 * 16 + 2], before the factors
  int *s_exp = reinterpret_cast<int *>(bars + 1);             // [kExpSlots][kExpWords]
  Seg *s_seg = reinterpret_cast<Seg *>(s_exp + kExpWords * kExpSlots);   // [kSegSlots]
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(s_seg + kSegSlots);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

  const AttendArgs &a = g.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x, ctas = gridDim.x;
  const int G = a.hq / a.hkv;
  uint32_t *err = a.err;

  // This kernel may begin while the call's row-group kernels, queued before it, still run.
  // It reads nothing of theirs (and they began behind everything queued before the call),
  // but what the stream holds next counts on them: every CTA waits for them as it ends.
  auto finish = [] { asm volatile("griddepcontrol.wait;" ::: "memory"); };
  // ---- this CTA's run of blocks
  const Start start = find_start<kThreads>(a.len, cta, ctas, s_scan, [&](int q_len, int kv) {
    const auto w = seq_items<D>(q_len, kv, g);
    return w.before(w.items) * a.hkv;
  });
  if (start.count == 0) {
    if (start.n < 0 && cta == 0 && tid == 0) raise(err, RPA_DEV_BAD_LENGTHS);
    if (tid == 0) g.heads[cta].begin = 0;
    finish();
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&bars->q_full[i], 1);
      ptx::mbar_init(&bars->q_empty[i], 1);
      ptx::mbar_init(&bars->qc_full[i], 128);
      for (int k = 0; k < 2; ++k) {
        ptx::mbar_init(&bars->s_full[i][k], 1);
        ptx::mbar_init(&bars->p_full[i][k], 128);
        ptx::mbar_init(&bars->pv_done[i][k], 1);
      }
      ptx::mbar_init(&bars->o_free[i], 128);
    }
    for (int i = 0; i < 4; ++i) {
      ptx::mbar_init(&bars->k_full[i], 128);
      ptx::mbar_init(&bars->k_empty[i], NT);
      ptx::mbar_init(&bars->v_full[i], 128);
      ptx::mbar_init(&bars->v_empty[i], NT);
    }
    for (int i = 0; i < 4; ++i) {
      ptx::mbar_init(&bars->c_full[i], 1);
      ptx::mbar_init(&bars->c_empty[i], 128);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&bars->f_full[i], 1);
      ptx::mbar_init(&bars->f_empty[i], 4);
    }
    for (int i = 0; i < kExpSlots; ++i) ptx::mbar_init(&bars->e_full[i], 1);
    for (int i = 0; i < kSegSlots; ++i) {
      ptx::mbar_init(&bars->seg_full[i], 1);
      ptx::mbar_init(&bars->seg_empty[i], kSegUsers<S::NT>);
    }
    ptx::mbar_init(&bars->drain[0], 1);
    ptx::mbar_init(&bars->drain[1], 1);
    *abort_flag = 0;
    ptx::fence_barrier_init();
  }
  if (warp == 12) {
    ptx::tmem_alloc(tmem_slot, S::kTmemCols);
    ptx::tmem_relinquish();
  }
  if (tid == 13 * 32) ptx::tma_prefetch_desc(&tm_q);
  if (tid == 14 * 32) {
    ptx::tma_prefetch_desc(&tm_k);
    ptx::tma_prefetch_desc(&tm_v);
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // the next segment of the run, or nullptr at its end (or after an abort)
  int segs = 0;
  auto next_seg = [&]() -> const Seg * {
    const int slot = segs % kSegSlots;
    if (!wait_warp(&bars->seg_full[slot], (uint32_t)((segs / kSegSlots) & 1), abort_flag, err)) return nullptr;
    return s_seg[slot].blocks < 0 ? nullptr : &s_seg[slot];
  };
  auto done_seg = [&]() {
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(&bars->seg_empty[segs % kSegSlots]);
    ++segs;
  };

  if (warp >= 12) {
    if (warp == 13) {
      // --------------------------------------------- the run, TMA of Q
      Run<D> run;
      run.g = &g;
      run.n = start.n;
      run.s = start.s;
      run.left = start.count;
      run.load();
      {
        // the KV head, the item (the largest with before(item) <= off) and the block in it:
        // by halves while that saves steps, then item by item
        const int64_t one = run.w.before(run.w.items);
        run.hk = (int)(start.off / one);
        const int64_t off = start.off - run.hk * one;
        int lo = 0, hi = run.w.items - 1;
        while (hi - lo > 32) {
          const int mid = (lo + hi + 1) >> 1;
          if (run.w.before(mid) <= off) lo = mid; else hi = mid - 1;
        }
        int64_t at = lo > 0 ? run.w.before(lo) : 0;
        for (int nb; lo < hi && at + (nb = run.w.blocks_of(lo) + kItemCost) <= off; ++lo) at += nb;
        run.item = lo;
        run.blk = (int)(off - at);
      }
      const uint64_t once = ptx::l2_evict_first_policy();
      int uses0 = 0, uses1 = 0;
      const uint32_t bytes = (uint32_t)(S::kHalves * 128 * g.tpt * G);
      bool ok = true;
      for (bool more = true; ok && more; ++segs) {
        const int slot = segs % kSegSlots;
        if (segs >= kSegSlots &&
            !wait_warp(&bars->seg_empty[slot], (uint32_t)(((segs / kSegSlots) & 1) ^ 1), abort_flag, err))
          break;
        more = run.next();
        if (lane == 0) {
          Seg d{};
          d.blocks = -1;
          if (more)
            d = Seg{run.s, run.hk, run.item - 1, run.b0, run.blocks(), {run.nt[0], run.nt[1]},
                    {run.rows[0], run.rows[1]}, run.q0, run.row0, run.w.kv, run.w.q_len,
                    run.b0 == 0 && run.b1 == run.nb ? 1 : 0, {0, 0}};
          s_seg[slot] = d;
          ptx::mbar_arrive(&bars->seg_full[slot]);
        }
        __syncwarp();
        for (int t = 0; t < NT; ++t) {
          if (!ok || !more || (t ? run.nt[1] : run.nt[0]) == 0) continue;
          const int u = t ? uses1 : uses0;
          if (u > 0) ok = wait_warp(&bars->q_empty[t], (uint32_t)((u - 1) & 1), abort_flag, err);
          if (!ok) continue;
          ptx::mbar_arrive_expect_tx_elect(&bars->q_full[t], bytes);
          for (int h = 0; h < S::kHalves; ++h)
            ptx::tma_load_3d_hint_elect(sQ + t * S::kQBytes + h * BM * 128, &tm_q, &bars->q_full[t], h * 64,
                                        run.hk * G, run.q0 + run.row0 + t * g.tpt, once);
          if (t) ++uses1; else ++uses0;
        }
      }
      // queued copies land before the CTA ends
      if (uses0 > 0) ptx::mbar_wait(&bars->q_full[0], (uint32_t)((uses0 - 1) & 1));
      if (uses1 > 0) ptx::mbar_wait(&bars->q_full[1], (uint32_t)((uses1 - 1) & 1));
      __syncwarp();
    } else if (warp == 14) {
      // ----------------------------------- TMA of the codes, the scales
      const int br = a.p < BN ? a.p : BN;
      const int nload = BN / br;
      int gb = 0;
      bool ok = true;
      auto queue = [&](int v, bool load, uint32_t bytes, int hk, int row) -> bool {
        const int use = 2 * gb + v, st = use % S::NST;
        if (use >= S::NST && !wait_warp(&bars->c_empty[st], (uint32_t)(((use / S::NST) & 1) ^ 1), abort_flag, err))
          return false;
        ptx::mbar_arrive_expect_tx_elect(&bars->c_full[st], bytes);
        __syncwarp();
        if (load) ptx::tma_load_3d(sC + st * S::kCodes + lane * br * D, v ? &tm_v : &tm_k, &bars->c_full[st], 0, hk, row);
        __syncwarp();
        return true;
      };
      int queued = 0;                    // code tiles
      while (ok) {
        const Seg *sg = next_seg();
        if (sg == nullptr) break;
        const int blocks = sg->blocks, b0 = sg->b0, kv = sg->kv, hk = sg->hk;
        const int32_t *pt = a.page_table + (size_t)sg->seq * a.max_pages;
        done_seg();
        // pages as the table has them: of the box this lane queues, and of the lane's
        // keys 4 lane .. + 3 (-1: no key)
        auto page_at = [&](int j, int pos, bool use) -> int { return use && j < blocks && pos < kv ? pt[pos >> a.p_shift] : -1; };
        auto box_page = [&](int j) -> int { return page_at(j, (b0 + j) * BN + lane * br, lane < nload); };
        auto key_page = [&](int j) -> int { return page_at(j, (b0 + j) * BN + lane * 4, lane < BN / 4); };
        auto scales_of = [&](int j, int pg, const uint8_t *src) -> uint32_t {
          if ((unsigned)pg >= (unsigned)a.num_pages) return 0;
          const int pos = (b0 + j) * BN + lane * 4;
          return *reinterpret_cast<const uint32_t *>(src + ((size_t)pg * a.hkv + hk) * a.p + (pos & (a.p - 1)));
        };
        int box_next = box_page(0), pg = key_page(0);
        uint32_t ks = scales_of(0, pg, a.c.ks), vs = scales_of(0, pg, a.c.vs);
        for (int j = 0; ok && j < blocks; ++j, ++gb) {
          const int page = box_next;
          box_next = box_page(j + 1);
          const int pgn = key_page(j + 1);
          const int pos = (b0 + j) * BN + lane * br;
          const bool load = lane < nload && pos < kv;
          int row = page * a.p + (pos & (a.p - 1));
          if (load && (unsigned)page >= (unsigned)a.num_pages) {
            raise(err, RPA_DEV_BAD_PAGE);
            row = a.num_pages * a.p;       // outside the tensor: the copy fills zeros
          }
          const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, load)) * (uint32_t)(br * D);
          ok = queue(0, load, bytes, hk, row);
          if (!ok) break;
          ++queued;
          const uint32_t ksn = scales_of(j + 1, pgn, a.c.ks), vsn = scales_of(j + 1, pgn, a.c.vs);
          // Rows of zeros have a scale that says nothing of their size: they do not count for the block's
          // scales (their bytes become 255 here), and the softmax warps are told of the V rows.
          uint32_t real = 15, zero_bit = 0;              // real: keys whose NaN scales are that
          if (__builtin_expect(__any_sync(0xffffffffu, (has_one(ks) | has_one(vs)) != 0), 0)) {
            const int lpos = (b0 + j) * BN + lane * 4, keys = (unsigned)pg < (unsigned)a.num_pages ? kv - lpos : 0;
            const size_t stride = (size_t)a.hkv * D;
            const size_t at = keys > 0 ? ((size_t)pg * a.p + (lpos & (a.p - 1))) * stride + (size_t)hk * D : 0;
            const uint32_t zero = zero_rows<D>(a.c.k, a.c.v, at, stride, ks, vs, keys);
            real = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              if (((ks >> (8 * k)) & 255u) == kScaleNan || ((vs >> (8 * k)) & 255u) == kScaleNan) real |= 1u << k;
              if ((zero >> k) & 1) ks |= 255u << (8 * k);
              if ((zero >> (4 + k)) & 1) vs |= 255u << (8 * k);
              const uint32_t word = __ballot_sync(0xffffffffu, (zero >> (4 + k)) & 1);
              if (word != 0) zero_bit = kZeroBit;
              // free, as below
              if (lane == 0) s_exp[(gb % kExpSlots) * kExpWords + 2 + k] = (int)word;
            }
          }
          // the block's largest and smallest scales over the keys it has; NaN scales mark the key
          uint32_t nans = 0;
          int ek = 0, ev = 0, ek0 = 255, ev0 = 255;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const bool key = (unsigned)pg < (unsigned)a.num_pages && (b0 + j) * BN + lane * 4 + k < kv;
            const int k8 = (ks >> (8 * k)) & 255u, v8 = (vs >> (8 * k)) & 255u;
            if (key && (k8 == (int)kScaleNan || v8 == (int)kScaleNan)) nans |= 1u << k;
            if (key && k8 != (int)kScaleNan) ek = max(ek, k8), ek0 = min(ek0, k8);
            if (key && v8 != (int)kScaleNan) ev = max(ev, v8), ev0 = min(ev0, v8);
          }
          nans &= real;
          ek = __reduce_max_sync(0xffffffffu, ek);
          ev = __reduce_max_sync(0xffffffffu, ev);
          const bool wk = ek - __reduce_min_sync(0xffffffffu, ek0) > kWide;
          const bool wv = ev - __reduce_min_sync(0xffffffffu, ev0) > kWide;
          const int fs = gb & 1;
          if (gb >= 2) ok = wait_warp(&bars->f_empty[fs], (uint32_t)(((gb >> 1) & 1) ^ 1), abort_flag, err);
          if (!ok) break;
          uint32_t fk[4], fv[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const bool nan = (nans >> k) & 1;
            fk[k] = half_factor(wk ? ek : (int)((ks >> (8 * k)) & 255u), ek, nan);
            // a NaN key's weight is NaN where it is seen; its values count as zeros elsewhere
            fv[k] = nan ? 0u : half_factor(wv ? ev : (int)((vs >> (8 * k)) & 255u), ev, false);
          }
          uint2 *dst = reinterpret_cast<uint2 *>(s_fac + fs * 2 * BN) + lane;
          if (lane < BN / 4) dst[0] = make_uint2(fk[0] | (fk[1] << 16), fk[2] | (fk[3] << 16));
          if (lane < BN / 4) dst[BN / 4] = make_uint2(fv[0] | (fv[1] << 16), fv[2] | (fv[3] << 16));
          if (lane == 0) {
            // free: the K tile of block gb - 1 is converted, so QK of block gb - 5 or a later one
            // is done for both tiles, and was issued behind the P of every block before it
            s_exp[(gb % kExpSlots) * kExpWords] = ek | (wk ? kWideBit : 0);
            s_exp[(gb % kExpSlots) * kExpWords + 1] = ev | (wv ? kWideBit : 0) | (int)zero_bit;
          }
          __syncwarp();
          if (lane == 0) {
            ptx::mbar_arrive(&bars->f_full[fs]);
            ptx::mbar_arrive(&bars->e_full[gb % kExpSlots]);
          }
          ok = queue(1, load, bytes, hk, row);
          if (!ok) break;
          ++queued;
          pg = pgn;
          ks = ksn;
          vs = vsn;
        }
      }
      // queued copies land before the CTA ends
      if (lane == 0)
        for (int k = queued - S::NST < 0 ? 0 : queued - S::NST; k < queued; ++k)
          ptx::mbar_wait(&bars->c_full[k % S::NST], (uint32_t)((k / S::NST) & 1));
      __syncwarp();
    } else if (warp == 12 || NT == 2) {
      // ------------------------------------------------- MMA of one tile
      // A tile's scores of step n go to its S buffer n & 1, where P of step n replaces them;
      // QK(n + 2) follows PV(n) into the same buffer, so a tile's softmax has the scores of
      // step n + 1 while PV(n) and QK(n + 2) run.  MMAs of one thread execute in order.
      const int t = warp == 12 ? 0 : 1;
      const uint64_t dq = ptx::umma_desc_sw128(ptx::smem_u32(sQ) + t * S::kQBytes, 16, 1024);
      const uint64_t dk0 = ptx::umma_desc_sw128(ptx::smem_u32(sK), 16, 1024);
      const uint64_t dv0 = ptx::umma_desc_sw128(ptx::smem_u32(sV), BN * 128, 1024);
      const uint32_t tS0 = tmem + t * 128, tO = tmem + S::kColO + t * D;
      constexpr uint32_t idesc_qk = ptx::umma_idesc_f16(128, HN, false), idesc_pv = ptx::umma_idesc_f16(128, D, true);
      int gb = 0, gt = 0, ep = 0;
      bool ok = true;
      while (ok) {
        const Seg *sg = next_seg();
        if (sg == nullptr) break;
        const int nt = sg->nt[t], nb = sg->blocks;
        done_seg();
#pragma unroll 1
        for (int vn = -2; vn < SPB * nb; ++vn) {
          const int kn = vn + 2;
          if (vn >= 0) {
            // (a block's tiles are waited for, and released, by both warps, whichever tile uses
            // them: an arrival of one warp must not count for the next block in the slot)
            const int st = (gb + vn / SPB) % NSV;
            if (vn % SPB == 0 && !wait_warp(&bars->v_full[st], (uint32_t)(((gb + vn / SPB) / NSV) & 1), abort_flag, err)) {
              ok = false;
              break;
            }
            if (vn < nt) {
              const int buf = (gt + vn) & 1;
              // O is overwritten by the segment's first PV: it must have been read
              if (vn == 0 && ep > 0) ok = wait_warp(&bars->o_free[t], (uint32_t)((ep - 1) & 1), abort_flag, err);
              ok = ok && wait_warp(&bars->p_full[t][buf], (uint32_t)(((gt + vn) >> 1) & 1), abort_flag, err);
              if (!ok) break;
              ptx::tc_fence_after();
              ptx::umma_ts_x4_elect(tO, tS0 + buf * HN, dv0 + (uint64_t)((st * S::kKVBytes + (vn % SPB) * HN * 128) >> 4),
                                    idesc_pv, vn > 0 ? 1u : 0u);
              ptx::umma_commit_elect(&bars->pv_done[t][buf]);
            }
            if (vn % SPB == SPB - 1) ptx::umma_commit_elect(&bars->v_empty[st]);
          }
          const int st = (gb + kn / SPB) % NSK;
          if (kn % SPB == 0 && kn < SPB * nb) {
            ok = wait_warp(&bars->k_full[st], (uint32_t)(((gb + kn / SPB) / NSK) & 1), abort_flag, err);
            if (ok && kn == 0 && nt > 0) ok = wait_warp(&bars->qc_full[t], (uint32_t)(ep & 1), abort_flag, err);
            if (!ok) break;
            ptx::tc_fence_after();
          }
          if (kn < nt) {
            const int buf = (gt + kn) & 1;
            const uint64_t dk = dk0 + (uint64_t)((st * S::kKVBytes + (kn % SPB) * HN * 128) >> 4);
#pragma unroll
            for (int h = 0; h < S::kHalves; ++h)
              ptx::umma_ss_x4_elect(tS0 + buf * HN, dq + (uint64_t)((h * BM * 128) >> 4),
                                    dk + (uint64_t)((h * BN * 128) >> 4), idesc_qk, h > 0 ? 1u : 0u);
            ptx::umma_commit_elect(&bars->s_full[t][buf]);
            if (kn + 1 == nt) ptx::umma_commit_elect(&bars->q_empty[t]);
          }
          if (kn % SPB == SPB - 1 && kn < SPB * nb) ptx::umma_commit_elect(&bars->k_empty[st]);
        }
        gb += nb;
        gt += nt;
        ep += nt > 0 ? 1 : 0;
      }
      ptx::umma_commit_elect(&bars->drain[t]);
      ptx::mbar_wait(&bars->drain[t], 0);
      __syncwarp();
    }
  } else if (warp >= 8) {
    // ------------------------------------------------- keys and values
    // D / 16 lanes share a row, 16 codes each; a lane's NU rows are neighbours, so their
    // factors are one load
    constexpr int LPR = D / 16, NU = BN / (32 / LPR) / 4;
    const int cw = warp - 8, lrow = lane / LPR, lcol = lane % LPR;
    const int row0 = lrow * (4 * NU) + cw * NU;
    // the two 16-byte chunks of a lane's values, in the order that hits no bank twice
    const int swp = D == 64 ? lrow & 1 : (lcol >> 2) & 1;
    const int c0 = 2 * (lcol & 3) + swp, c1 = c0 ^ 1;
    const uint32_t src0 = (uint32_t)(row0 * D + lcol * 16 + swp * 8);
    const uint32_t dst0 = (uint32_t)((lcol >> 2) * BN * 128 + row0 * 128);
    const int x0 = c0 ^ (row0 & 7), x1 = c1 ^ (row0 & 7);      // NU rows from row0 on: row & 7 = (row0 & 7) | i
    int gb = 0;
    bool ok = true;
    while (ok) {
      const Seg *sg = next_seg();
      if (sg == nullptr) break;
      const int blocks = sg->blocks;
      int keys = sg->kv - sg->b0 * BN;
      done_seg();
      for (int j = 0; ok && j < blocks; ++j, ++gb, keys -= BN) {
        ok = wait_warp(&bars->f_full[gb & 1], (uint32_t)((gb >> 1) & 1), abort_flag, err);
        if (!ok) break;
        const int st = gb % NSK;
#pragma unroll 1
        for (int v = 0; v < 2; ++v) {
          const int use = 2 * gb + v, cs = use % S::NST;
          const uint16_t *fac = s_fac + (gb & 1) * 2 * BN + v * BN + row0;
          ok = gb < NSK || wait_warp(v ? &bars->v_empty[st] : &bars->k_empty[st], (uint32_t)(((gb / NSK) & 1) ^ 1),
                                     abort_flag, err);
          ok = ok && wait_warp(&bars->c_full[cs], (uint32_t)((use / S::NST) & 1), abort_flag, err);
          if (!ok) break;
          const uint8_t *src = sC + cs * S::kCodes + src0;
          uint8_t *dst = (v ? sV : sK) + st * S::kKVBytes + dst0;
          // two rows at a time: eight were 8 KB of code, which the caches did not hold beside the
          // softmax's (8 prompts of 2048 tokens 475 us, with two 444)
#pragma unroll 2
          for (int i = 0; i < NU; ++i) {
            uint2 a0 = *reinterpret_cast<const uint2 *>(src + i * D);
            uint2 a1 = *reinterpret_cast<const uint2 *>(src + i * D + (swp ? -8 : 8));
            const uint32_t f = __byte_perm((uint32_t)fac[i], 0u, 0x1010);
            *reinterpret_cast<uint4 *>(dst + i * 128 + ((x0 ^ i) << 4)) =
                make_uint4(mul_h2(codes_h2(a0.x), f), mul_h2(codes_h2(a0.x >> 16), f),
                           mul_h2(codes_h2(a0.y), f), mul_h2(codes_h2(a0.y >> 16), f));
            *reinterpret_cast<uint4 *>(dst + i * 128 + ((x1 ^ i) << 4)) =
                make_uint4(mul_h2(codes_h2(a1.x), f), mul_h2(codes_h2(a1.x >> 16), f),
                           mul_h2(codes_h2(a1.y), f), mul_h2(codes_h2(a1.y >> 16), f));
          }
          // rows without a key, which no copy filled or whose page holds anything: zeros
          if (keys < BN)
#pragma unroll 1
            for (int i = 0; i < NU; ++i)
              if (row0 + i >= keys) {
                *reinterpret_cast<uint4 *>(dst + i * 128 + ((x0 ^ i) << 4)) = make_uint4(0, 0, 0, 0);
                *reinterpret_cast<uint4 *>(dst + i * 128 + ((x1 ^ i) << 4)) = make_uint4(0, 0, 0, 0);
              }
          ptx::fence_proxy_async_smem();
          ptx::mbar_arrive(v ? &bars->v_full[st] : &bars->k_full[st]);
          ptx::mbar_arrive(&bars->c_empty[cs]);
        }
        __syncwarp();                     // the other lanes have read their factors too
        if (lane == 0) ptx::mbar_arrive(&bars->f_empty[gb & 1]);
      }
    }
  } else if (warp < 4 * NT) {
    // ------------------------------------------------------ softmax, output
    const int t = warp >> 2, row = tid & 127;
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t tO = lane_base + S::kColO + (uint32_t)(t * D);
    const int tok = row / G, head = row - tok * G;
    const float f = a.scale * kLog2e;
    int gb = 0, gt = 0, eq = 0;                       // blocks, steps and Q tiles so far
    bool ok = true;
    // this row's view of a segment
    struct View {
      int nt, nb, b0, hk, end;                        // end: keys the row sees
      bool mine, whole;
      const int32_t *pt;
      size_t slot, at;                                // place of a part; the row in out and lse
      float qf;                                       // score factor of the row
    };
    // Takes the next segment and makes scaled fp16 of its Q, landed as bf16, in place
    // (the row is this thread's); false at the end of the run.
    auto take = [&](View &c) -> bool {
      const Seg *sg = next_seg();
      if (sg == nullptr) return false;
      c.nt = sg->nt[t];
      c.nb = sg->blocks;
      c.b0 = sg->b0;
      c.hk = sg->hk;
      c.mine = row < sg->rows[t];
      c.whole = sg->whole != 0;
      c.pt = a.page_table + (size_t)sg->seq * a.max_pages;
      c.slot = 2 * (size_t)cta + (c.b0 > 0 ? 0 : 1);
      if (segs == 0 && tid == 0) g.heads[cta] = PartHead{sg->seq, sg->hk, sg->item, sg->b0};
      const int tk = sg->row0 + t * g.tpt + tok;      // token within the sequence
      c.end = !c.mine ? 0 : !a.causal ? sg->kv : min(sg->kv, max(0, sg->kv - sg->q_len + tk + 1));
      c.at = (size_t)(sg->q0 + tk) * a.hq + sg->hk * G + head;
      done_seg();
      if (c.nt == 0) return true;
      if (!wait_warp(&bars->q_full[t], (uint32_t)(eq & 1), abort_flag, err)) {
        ok = false;
        return false;
      }
      ++eq;
      uint8_t *q = sQ + t * S::kQBytes + row * 128;
      uint32_t big = 0;                               // largest |q| of the even and the odd values (NaN stays)
#pragma unroll 1
      for (int h = 0; h < S::kHalves; ++h)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint4 u = *reinterpret_cast<const uint4 *>(q + h * BM * 128 + ((i ^ (row & 7)) << 4));
          big = ptx::absmax_bf16x2(ptx::absmax_bf16x2(big, u.x), ptx::absmax_bf16x2(u.y, ptx::absmax_bf16x2(u.z, u.w)));
        }
      const uint32_t code = scale_code(max((big << 16) & 0x7fff0000u, big & 0x7fff0000u));
      const float inv = code == kScaleNan ? 0.f : inverse_scale(code);
      c.qf = scale_value(code) * f;
#pragma unroll 1
      for (int h = 0; h < S::kHalves; ++h)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          uint4 *p = reinterpret_cast<uint4 *>(q + h * BM * 128 + ((i ^ (row & 7)) << 4));
          const uint4 u = *p;
          uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int k = 0; k < 4; ++k)
            w[k] = ptx::pack_f16(__uint_as_float(w[k] << 16) * inv, __uint_as_float(w[k] & 0xffff0000u) * inv);
          *p = make_uint4(w[0], w[1], w[2], w[3]);
        }
      ptx::fence_proxy_async_smem();
      ptx::mbar_arrive(&bars->qc_full[t]);
      return true;
    };
    View c{};
    bool have = take(c);
    if (!have && tid == 0) g.heads[cta].begin = 0;   // a run without a block
    while (have && ok) {
      if (c.nt == 0) {
        // no block of this segment is seen by the tile: an empty part
        if (!c.whole && c.mine) g.ml[c.slot * S::ROWS + t * 128 + row] = make_float2(-INFINITY, 0.f);
        gb += c.nb;
        have = take(c);
        continue;
      }
      const int nt = c.nt, b0 = c.b0, hk = c.hk, end = c.end;
      const int32_t *pt = c.pt;
      const float qf = c.qf;
      int ek = 0, ev = 0;
      int marks = 0;                                  // of the block: kWideBit, kZeroBit
      RowSum r{-INFINITY, 0.f, 0.f, 0};
      for (int j = 0; j < nt; ++j) {                  // steps
        const int blk = gb + j / SPB, eslot = blk % kExpSlots, buf = (gt + j) & 1;
        const uint32_t tS = lane_base + (uint32_t)(t * 128 + buf * HN);
        if (j % SPB == 0) {                           // a new block's scales
          // (A tile that skipped blocks cannot come by here eight blocks early, when the barrier's
          // parity would pass: tile 0 skips one block at most, at a run's begin; tile 1's Q is
          // loaded behind tile 0's, which waits for every QK of the segment before.)
          ok = wait_warp(&bars->e_full[eslot], (uint32_t)((blk / kExpSlots) & 1), abort_flag, err);
          ek = s_exp[eslot * kExpWords];
          ev = s_exp[eslot * kExpWords + 1];
          marks = ek | ev;
          ek &= 255;
          ev &= 255;
        }
        ok = ok && wait_warp(&bars->s_full[t][buf], (uint32_t)(((gt + j) >> 1) & 1), abort_flag, err);
        if (!ok) break;
        const int key0 = b0 * BN + j * HN;            // the step's first key
        ptx::tc_fence_after();
        // never 0, which would make NaN of a masked score
        float sc = qf * scale_value((uint32_t)ek);
        if (sc < 1e-37f) sc = 1e-37f;
        const Step st{tS, tO, &bars->pv_done[t][buf ^ 1], (uint32_t)(((gt + j - 1) >> 1) & 1), j == 0,
                      min(HN, end - key0), ek, ev, sc, abort_flag, err};
        if (__builtin_expect(marks < kWideBit, 1)) {
          ok = tile_step<D>(r, st, INFINITY);
        } else {
          const int *e = s_exp + eslot * kExpWords;
          const int shift = j % SPB * (HN / 4);
          const MarkedSum ms = marks & kWideBit
                                   ? wide_step<D>(r, st, Wide{e, shift, key0, end, pt, a.c.ks, a.c.vs, hk, a.hkv, a.p,
                                                              a.p_shift, a.num_pages})
                                   : zeros_step<D>(r, st, e + 2, shift);
          r = ms.r;
          ok = ms.ok != 0;
        }
        if (!ok) break;
        ptx::tmem_st_wait();
        ptx::tc_fence_before();
        ptx::mbar_arrive(&bars->p_full[t][buf]);
      }
      if (!ok) break;
      gb += c.nb;
      gt += nt;
      // the next segment's Q before this one's output: its first scores are computed meanwhile
      View next{};
      have = take(next);
      if (!ok) break;
      if (!wait_warp(&bars->pv_done[t][(gt - 1) & 1], (uint32_t)(((gt - 1) >> 1) & 1), abort_flag, err)) {
        ok = false;
        break;
      }
      ptx::tc_fence_after();
      if (end == 0) {                                 // sees no key, whatever its q holds
        r.l = 0.f;
        r.m = -INFINITY;
      }
      // O / l is in units of 2^(evr - 127), which may be below ex2's smallest; a part keeps O in them
      const float unit = r.evr < 64 ? ptx::ex2((float)(r.evr - 63)) * 0x1p-64f : ptx::ex2((float)(r.evr - 127));
      const float mul = end == 0 ? 0.f : !c.whole ? unit : r.l == 0.f ? 0.f : unit / r.l;
      const uint64_t mul2 = ptx::f2_pack(mul, mul);
      const bool blank = __any_sync(0xffffffffu, end == 0);   // a row of the warp sees no key: its O is dropped
      const uint64_t once = ptx::l2_evict_first_policy();
#pragma unroll 1
      for (int cc = 0; cc < D; cc += 32) {
        uint32_t ov[32];
        ptx::tmem_ld32(tO + cc, ov);
        ptx::tmem_ld_wait();
        if (cc + 32 == D) {
          ptx::tc_fence_before();
          ptx::mbar_arrive(&bars->o_free[t]);
        }
        float o[32];
#pragma unroll
        for (int i = 0; i < 32; i += 2)
          ptx::f2_unpack(ptx::f2_mul(ptx::f2_pack(__uint_as_float(ov[i]), __uint_as_float(ov[i + 1])), mul2), o[i], o[i + 1]);
        if (blank) {
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = end == 0 ? 0.f : o[i];
        }
        if (!c.mine) continue;
        if (c.whole) {
          // whole 32-byte sectors: a row is this thread's, its neighbours' are far away
          uint32_t *out = reinterpret_cast<uint32_t *>(static_cast<__nv_bfloat16 *>(a.out) + c.at * D + cc);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint32_t o2[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) o2[k] = ptx::pack_bf16(o[16 * i + 2 * k], o[16 * i + 2 * k + 1]);
            ptx::st_global_hint8(out + 8 * i, o2, once);
          }
        } else {
          float4 *po = g.o + (c.slot * (D / 4) + cc / 4) * S::ROWS + t * 128 + row;
#pragma unroll
          for (int i = 0; i < 8; ++i) po[i * S::ROWS] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
        }
      }
      if (c.mine) {
        if (!c.whole)
          g.ml[c.slot * S::ROWS + t * 128 + row] = make_float2(r.m, r.l);
        else if (a.lse != nullptr)
          a.lse[c.at] = r.l == 0.f ? -INFINITY : ((r.m == -INFINITY ? 0.f : r.m) + log2f(r.l) - kBase) * kLn2;
      }
      c = next;
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == 12) ptx::tmem_dealloc(tmem, S::kTmemCols);
  finish();
}

// Joins the parts of an item that several runs share (see the row-group
// kernel's).  A block joins 16 of an item's rows, 16 lanes a row.
template <int D>
__global__ void __launch_bounds__(256) combine_kernel(const Args g) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int ROWS = Shape<D>::ROWS, PER = ROWS / 16;      // blocks per item
  const int i = blockIdx.x / PER, ctas = gridDim.x / PER;
  const PartHead h = g.heads[i];
  if (h.begin <= 0) return;
  auto same = [&](const PartHead &p) { return p.begin > 0 && p.seq == h.seq && p.hk == h.hk && p.item == h.item; };
  if (same(g.heads[i - 1])) return;
  const AttendArgs &a = g.a;
  const int G = a.hq / a.hkv;
  const int q0 = a.len.cu[h.seq], q_len = a.len.cu[h.seq + 1] - q0;
  const int r = (blockIdx.x % PER) * 16 + (threadIdx.x & 15), t = r >> 7, row = r & 127;
  const int tok = row / G, tk = (Shape<D>::NT * h.item + t) * g.tpt + tok;
  if (tok >= g.tpt || tk >= q_len) return;
  int end = i + 1;
  while (end < ctas && same(g.heads[end])) ++end;
  const int parts = end - i + 1;
  auto slot = [&](int k) { return (size_t)(k == 0 ? 2 * (i - 1) + 1 : 2 * (i + k - 1)); };
  float M = -INFINITY, l = 0.f;
  for (int k = 0; k < parts; ++k) M = fmaxf(M, g.ml[slot(k) * ROWS + r].x);
  constexpr int NC = D / 64;                 // float4 pieces per thread
  const int c0 = threadIdx.x >> 4;
  float4 acc[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
  for (int k = 0; k < parts; ++k) {
    const float2 ml = g.ml[slot(k) * ROWS + r];
    float4 v[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) v[c] = g.o[(slot(k) * (D / 4) + c * 16 + c0) * ROWS + r];
    if (ml.y == 0.f) continue;               // saw no key: nothing there
    const float wt = ml.x == M ? 1.f : ptx::ex2((ml.x == -INFINITY ? 0.f : ml.x) - (M == -INFINITY ? 0.f : M));
    l = fmaf(wt, ml.y, l);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      acc[c].x = fmaf(wt, v[c].x, acc[c].x);
      acc[c].y = fmaf(wt, v[c].y, acc[c].y);
      acc[c].z = fmaf(wt, v[c].z, acc[c].z);
      acc[c].w = fmaf(wt, v[c].w, acc[c].w);
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const size_t at = (size_t)(q0 + tk) * a.hq + h.hk * G + row % G;
  __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out) + at * D;
#pragma unroll
  for (int c = 0; c < NC; ++c)
    *reinterpret_cast<uint2 *>(out + (c * 16 + c0) * 4) =
        make_uint2(ptx::pack_bf16(acc[c].x * inv, acc[c].y * inv), ptx::pack_bf16(acc[c].z * inv, acc[c].w * inv));
  if (c0 == 0 && a.lse != nullptr)
    a.lse[at] = l == 0.f ? -INFINITY : ((M == -INFINITY ? 0.f : M) + log2f(l) - kBase) * kLn2;
}

template <int D>
cudaError_t launch_t(const AttendArgs &a, int q_limit, int total_q, int grid, uint8_t *ws, bool join,
                     cudaStream_t stream) {
  using S = Shape<D>;
  Args g{};
  g.a = a;
  g.q_limit = q_limit;
  const int G = a.hq / a.hkv;
  g.tpt = BM / G;
  const ChunkLayout w = chunk_layout(grid, D);
  g.heads = reinterpret_cast<PartHead *>(ws + w.heads);
  g.ml = reinterpret_cast<float2 *>(ws + w.ml);
  g.o = reinterpret_cast<float4 *>(ws + w.o);
  if (join) {
    if (grid == 1) return cudaSuccess;
    return launch_behind(combine_kernel<D>, S::ROWS / 16 * grid, 256, 0, stream, g);
  }
  CUtensorMap tk, tv;
  const uint64_t cdims[3] = {(uint64_t)D, (uint64_t)a.hkv, (uint64_t)a.num_pages * a.p};
  const uint64_t cstrides[2] = {(uint64_t)D, (uint64_t)a.hkv * D};
  const uint32_t cbox[3] = {(uint32_t)D, 1, (uint32_t)(a.p < S::BN ? a.p : S::BN)};
  if (!make_tmap_u8_3d(&tk, a.c.k, cdims, cstrides, cbox, false) ||
      !make_tmap_u8_3d(&tv, a.c.v, cdims, cstrides, cbox, false))
    return cudaErrorInvalidValue;
  // a tile of Q: the G heads of tpt tokens, token-major
  CUtensorMap tq;
  const uint64_t dims[3] = {(uint64_t)D, (uint64_t)a.hq, (uint64_t)total_q};
  const uint64_t strides[2] = {(uint64_t)D * 2, (uint64_t)a.hq * D * 2};
  const uint32_t box[3] = {64, (uint32_t)G, (uint32_t)g.tpt};
  if (!make_tmap_bf16_3d(&tq, a.q, dims, strides, box, true)) return cudaErrorInvalidValue;
  auto kern = chunk_kernel<D>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
  if (e != cudaSuccess) return e;
  return launch_behind(kern, grid, kThreads, S::kSmem, stream, tq, tk, tv, g);
}

}  // namespace

bool chunk_takes(const rpa_dims &d) { return d.dtype == RPA_BF16; }

// Rows of an item and keys of a block (Shape's).
static int item_tiles(int D) { return D == 256 ? Shape<256>::NT : Shape<128>::NT; }
static int block_keys(int D) { return D == 256 ? Shape<256>::BN : Shape<128>::BN; }

int chunk_grid(const rpa_dims &d, int32_t max_seqs, int32_t max_q) {
  const int64_t cap = (int64_t)d.max_pages_per_seq * d.page_size;
  const int TT = item_tiles(d.head_dim) * (BM / (d.num_q_heads / d.num_kv_heads)), BN = block_keys(d.head_dim);
  const int64_t seqs = std::min<int64_t>(max_seqs, d.total_q_tokens);
  const double most = (double)seqs * d.num_kv_heads * (double)((max_q + TT - 1) / TT) * (double)((cap + BN - 1) / BN);
  return (int)std::max(1.0, std::min(most, 148.0));
}

ChunkLayout chunk_layout(int grid, int D) {
  ChunkLayout w;
  auto up = [](int64_t x) { return (x + 255) / 256 * 256; };
  w.heads = 0;
  w.ml = up((int64_t)grid * sizeof(PartHead));
  const int64_t rows = (int64_t)grid * 2 * item_tiles(D) * BM;
  w.o = up(w.ml + rows * 8);
  w.total = up(w.o + rows * D * 4);
  return w;
}

cudaError_t launch_chunk(const AttendArgs &a, const rpa_dims &d, int32_t max_seqs, int32_t max_q, int32_t q_limit,
                         uint8_t *ws, bool join, cudaStream_t stream) {
  const int grid = chunk_grid(d, max_seqs, max_q);
  switch (d.head_dim) {
    case 64: return launch_t<64>(a, q_limit, d.total_q_tokens, grid, ws, join, stream);
    case 128: return launch_t<128>(a, q_limit, d.total_q_tokens, grid, ws, join, stream);
    case 256: return launch_t<256>(a, q_limit, d.total_q_tokens, grid, ws, join, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace q8
}  // namespace rpa
