// q8_rows_kernel.cu -- attention over the 8-bit cache for few query rows per
// KV head (single tokens, a few tokens, and every fp32 call): bound by reading
// the cache once.
//
// Mathematics.  A group of R query rows of one KV head (rows are the pairs
// (token i, head g), row = i * G + g) runs over blocks of 128 keys with the
// keys on the M side of the tensor cores, so that the codes are used as they lie
// in the cache, never converted:
//   S^T[128 keys x R] = K Q^T      A = K codes, K-major, straight from TMA
//   O^T[D x R]       += V^T P^T    A = V codes, M-major, the same
// in kind::f8f6f4, whose B operand must be 8 bits too.  Q and the weights P
// are therefore written as sums of e4m3 parts, part i scaled by 16^i:
// the remainder of a rounding is exact in fp32 and half a step at most, so that n parts
// are off by 2^-(5 n - 1) of the value, while their last one is not below e4m3's smallest:
//   bf16 I/O: 2 parts of Q (exact for values down to 2^-12 of the row's largest |q|, within
//             2^-21 of that below), 4 of P (2^-19; weights down to 2^-30 of the row's largest
//             count, so a long flat tail behind one large weight keeps its sum);
//   fp32 I/O: 6 parts of both (five would hold 24 bits of the larger values).
// The parts are columns of the same MMA (N = parts * R, whose time below
// N = 64 is that of reading A), and their products are joined in fp32.
// Scales: a key's K scale multiplies its score and its V scale its weight; one
// thread owns one key, so both are a scalar of that thread.  A weight with its V
// scale, exp2(x + ev), is taken relative to the largest of its row and block
// (times 256) before the rounding to parts: keys that a row does not see, whose
// weight is small, or whose V row is zeros, do not coarsen it however large their scales are.
// Softmax: running maximum and sum in fp32 (log2 domain).  Each block's product
// O^T is read from TMEM into fp32 registers, which are rescaled when the
// maximum moves: no read-modify-write of TMEM and no wait between blocks.
//
// Split of the work: the blocks of every (sequence, row group) of one KV head
// in a row are one list, cut into equal runs, one per CTA (every SM gets the
// same number of blocks whatever the lengths).  A CTA computes its run from the
// lengths in device memory, so there is no planning launch.  The CTAs of all
// heads with the same run are neighbours: they read the rows of a token, which lie
// side by side, at about the same time.  A run may begin and
// end inside a group: those partial results go to the workspace and
// combine_kernel, queued with programmatic dependent launch, joins them
// in the order of the keys (the same bits every time).
//
// Warps: 0-3 the parts of Q (a row each at a time; one warp for all of them took
// 12,000 clocks for 16 rows, more than many a group's keys), softmax, weights and
// output (thread = key of the block, then row of O^T), 4 TMA of K and V tiles,
// 5 MMA issue, 6 the scales (cp.async).  4 and 6 run ahead across groups through
// rings in shared memory.
//
// Measured: 128 single tokens behind 1024 to 8192 keys (Hq 32, Hkv 8, D 128) 158 to 168 us by the
// card, 5.9 to 6.2 TB/s of the cache's bytes, 0.90 to 0.95 of a plain copy's rate (986 MB read where 985 are needed); contexts up to
// 131072 at D 256 315 to 320 us, 6.7 to 6.8 TB/s.  fp32 single tokens of the same lengths run at 5.3 TB/s; every
// 8 fp32 rows of a KV head pass over its keys once more (4 chunks of 512 behind contexts 2.3 ms).
#include <cuda.h>
#include <limits.h>
#include <math.h>

#include <algorithm>

#include "ptx.cuh"
#include "q8_common.cuh"
#include "q8_kernels.h"
#include "tma.h"

namespace rpa {
namespace q8 {
namespace {

constexpr int kThreads = 224;
constexpr int BN = 128;               // keys per block
constexpr int kScaleSlots = 8;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kPartStep = 1.f / 16.f;

template <typename T> struct Parts;
template <> struct Parts<__nv_bfloat16> { static constexpr int Q = 2, P = 4; };
template <> struct Parts<float> { static constexpr int Q = 6, P = 6; };

constexpr int round_up(int x, int m) { return (x + m - 1) / m * m; }
constexpr int pow2_cols(int x) { return x <= 32 ? 32 : x <= 64 ? 64 : x <= 128 ? 128 : x <= 256 ? 256 : 512; }

template <typename T, int D, int R>
struct Shape {
  static constexpr int NQ = Parts<T>::Q, NP = Parts<T>::P;
  static constexpr int CQ = NQ * R, CP = NP * R;                 // columns in use
  static constexpr int NQpad = round_up(CQ, 16), NPpad = round_up(CP, 16);
  static constexpr int RC = R < 8 ? R : 8;                       // rows read from TMEM at a time
  static constexpr int W = D == 64 ? 64 : 128;                   // bytes of a tile row
  static constexpr int CT = D / W;                               // column tiles
  static constexpr int kTile = BN * D;                           // K or V codes of a block
  static constexpr int kQBuf = NQpad * D;
  static constexpr int kPBuf = NPpad * BN;
  static constexpr int kFixed = 1024 + kQBuf + 2 * kPBuf + kScaleSlots * 2 * BN + 2816;
  static constexpr int kTmem = pow2_cols(2 * NQpad + 2 * NPpad * CT);
  // CTAs per SM: three where their TMEM, registers and two-slot rings fit
  static constexpr int kSmMax = 227 * 1024;
  static constexpr int fits(int ctas, int ns) {
    return ctas * (kFixed + 2 * ns * kTile + 1024) <= kSmMax && ctas * kTmem <= 512 ? 1 : 0;
  }
  static constexpr int CTAS = R <= 4 && fits(3, 2) ? 3 : fits(2, 2) ? 2 : 1;
  static constexpr int slots() {
    int ns = 2;
    while (ns < 8 && fits(CTAS, ns + 1)) ++ns;
    return ns;
  }
  static constexpr int NS = slots();
  static constexpr int kSmem = kFixed + 2 * NS * kTile;
  static_assert(fits(1, 2) == 1, "shape does not fit");
};

struct Bars {
  uint64_t k_full[8], k_empty[8], v_full[8], v_empty[8];
  uint64_t s_full[2], p_full[2], pv_full[2];
  uint64_t q_full;
  uint64_t sc_full[kScaleSlots], sc_empty[kScaleSlots];
  uint64_t x_full[2], l_full;    // the softmax warps' maxima and sums are in shared memory
  uint64_t drain;
};

// A partial result of a group: its CTA's run begins or ends inside the group.
struct PartHead {
  int32_t seq, hk, grp, begin;   // begin: first block of the run in the group (> 0: joined by the combine)
};

struct Args {
  AttendArgs a;
  int32_t q_limit;               // longer sequences are another kernel's
  PartHead *heads;               // [ctas]
  float *ml;                     // [2 * ctas][R][2] running maximum (log2) and sum
  float *o;                      // [2 * ctas][R][D] unnormalised
};

// Blocks of one sequence: groups of R rows per KV head, each of nb blocks (a
// sequence without keys has one, empty, so that its rows are written).  In the list
// that is cut into runs a group counts kGroupCost blocks more, at its front: making Q's
// parts and writing the output took 6,000 to 9,000 clocks beside 1,200 to 3,000 a block, and
// without it the CTAs with many short groups took twice the average.
constexpr int kGroupCost = 2;
struct SeqWork {
  int groups, nb;
  __device__ __forceinline__ int64_t blocks() const { return (int64_t)groups * (nb + kGroupCost); }
};
template <int R>
__device__ __forceinline__ SeqWork seq_work(int q_len, int kv_len, int G, int q_limit) {
  SeqWork w;
  w.groups = q_len > q_limit ? 0 : (q_len * G + R - 1) / R;
  w.nb = max(1, (kv_len + BN - 1) / BN);
  return w;
}

// The CTA's run of blocks as segments, one per group it touches.
template <int R>
struct Run {
  const AttendArgs *a;
  int n, G, q_limit;
  int hk, s, grp_next, blk;      // blk: place in the group, kGroupCost included
  int64_t left;
  // the current segment
  int q0, q_len, kv, grp, nb, b0, b1;

  __device__ __forceinline__ bool next() {
    if (left <= 0) return false;
    SeqWork w;
    while (true) {
      if (s >= n) return false;
      q0 = a->len.cu[s];
      q_len = a->len.cu[s + 1] - q0;
      kv = a->len.kv[s];
      w = seq_work<R>(q_len, kv, G, q_limit);
      if (grp_next < w.groups) break;
      ++s;
      grp_next = 0;
    }
    nb = w.nb;
    grp = grp_next++;
    const int end = nb + kGroupCost, stop = (int)(left < end - blk ? blk + left : end);
    b0 = max(0, blk - kGroupCost);
    b1 = max(0, stop - kGroupCost);
    left -= stop - blk;
    blk = 0;
    return b1 > b0;          // a run's end before a group's first block is no segment
  }
  // the segment's last block that any row sees, plus one (>= b0)
  __device__ __forceinline__ int last_block() const {
    const int rho = min((grp + 1) * R, q_len * G) - 1;
    const int end = a->causal ? min(kv, max(0, kv - q_len + rho / G + 1)) : kv;
    const int vis = max(1, (end + BN - 1) / BN);
    return max(b0, min(b1, vis));
  }
};

__device__ __forceinline__ float joined(float m) { return m == -INFINITY ? 0.f : m; }

// Largest of the warp's values (a NaN is passed over, as fmaxf does).
__device__ __forceinline__ float warp_max(float x) {
  float m;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(x));
  return m;
}

// sum_p 16^-p x part p of RC rows; part p of a row is R columns after part p - 1.
template <int NP, int R, int RC>
__device__ __forceinline__ void join_parts(uint32_t taddr, float (&sum)[RC]) {
  uint32_t v[NP * RC];
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    if constexpr (RC == 8) ptx::tmem_ld8(taddr + p * R, v, p * RC);
    else ptx::tmem_ld4(taddr + p * R, v, p * RC);
  }
  ptx::tmem_ld_wait();
#pragma unroll
  for (int r = 0; r < RC; ++r) {
    sum[r] = __uint_as_float(v[(NP - 1) * RC + r]);
#pragma unroll
    for (int p = NP - 2; p >= 0; --p) sum[r] = fmaf(sum[r], kPartStep, __uint_as_float(v[p * RC + r]));
  }
}

template <typename T, int D, int R>
__global__ void __launch_bounds__(kThreads, (Shape<T, D, R>::CTAS))
    rows_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const Args g) {
  using S = Shape<T, D, R>;
  constexpr int NS = S::NS;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  extern __shared__ uint8_t smem_raw[];
  uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t *sK = base;
  uint8_t *sV = sK + NS * S::kTile;
  uint8_t *sQ = sV + NS * S::kTile;
  uint8_t *sP = sQ + S::kQBuf;                             // two buffers
  uint8_t *sSc = sP + 2 * S::kPBuf;                        // [slot][K, V][128]
  Bars *bars = reinterpret_cast<Bars *>(sSc + kScaleSlots * 2 * BN);
  float *s_qf = reinterpret_cast<float *>(bars + 1);       // [2][16] row factors
  int *s_end = reinterpret_cast<int *>(s_qf + 32);         // [2][16] keys each row sees
  long long *s_at = reinterpret_cast<long long *>(s_end + 32);   // [2][16] the rows' places in out, -1: none
  float *s_max = reinterpret_cast<float *>(s_at + 32);    // [2][4][16 + 16] warps' maxima of x, x + ev
  float *s_l = reinterpret_cast<float *>(s_max + 256);       // [4][16]
  float *s_ml = s_l + 64;                                  // [16][2] maximum and sum of a finished group
  int64_t *s_scan = reinterpret_cast<int64_t *>(s_ml + 32); // [2 * 8 + 2]
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(s_scan + 18);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

  const AttendArgs &a = g.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int ctas = gridDim.x / a.hkv;           // of one head
  const int hk = blockIdx.x % a.hkv, cta = blockIdx.x / a.hkv;
  const int place = hk * ctas + cta;            // in the lists of partial results
  const int G = a.hq / a.hkv;

  // ---- this CTA's run of blocks
  const Start start = find_start<kThreads>(a.len, cta, ctas, s_scan, [&](int q_len, int kv) {
    return seq_work<R>(q_len, kv, G, g.q_limit).blocks();
  });
  if (start.count == 0) {
    if (start.n < 0 && blockIdx.x == 0 && tid == 0) raise(a.err, RPA_DEV_BAD_LENGTHS);
    if (tid == 0) g.heads[place].begin = 0;
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      ptx::mbar_init(&bars->k_full[i], 1);
      ptx::mbar_init(&bars->k_empty[i], 1);
      ptx::mbar_init(&bars->v_full[i], 1);
      ptx::mbar_init(&bars->v_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&bars->s_full[i], 1);
      ptx::mbar_init(&bars->p_full[i], 128);
      ptx::mbar_init(&bars->pv_full[i], 1);
    }
    for (int i = 0; i < kScaleSlots; ++i) {
      ptx::mbar_init(&bars->sc_full[i], 32);
      ptx::mbar_init(&bars->sc_empty[i], 128);
    }
    ptx::mbar_init(&bars->q_full, 128);
    ptx::mbar_init(&bars->x_full[0], 4);
    ptx::mbar_init(&bars->x_full[1], 4);
    ptx::mbar_init(&bars->l_full, 4);
    ptx::mbar_init(&bars->drain, 1);
    *abort_flag = 0;
    ptx::fence_barrier_init();
  }
  if (warp == 5) {
    ptx::tmem_alloc(tmem_slot, S::kTmem);
    ptx::tmem_relinquish();
  }
  if (tid == 128) {
    ptx::tma_prefetch_desc(&tm_k);
    ptx::tma_prefetch_desc(&tm_v);
  }
  // columns that no part fills are zeros
  if (S::NQpad > S::CQ)
    for (int i = tid; i < S::kQBuf / 16; i += kThreads) reinterpret_cast<uint4 *>(sQ)[i] = make_uint4(0, 0, 0, 0);
  ptx::fence_proxy_async_smem();
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t tS = tmem, tO = tmem + 2 * S::NQpad;

  Run<R> run;
  run.a = &a;
  run.n = start.n;
  run.G = G;
  run.q_limit = g.q_limit;
  run.hk = hk;
  run.s = start.s;
  {
    const int nb = seq_work<R>(1, a.len.kv[start.s], G, INT_MAX).nb;
    run.grp_next = (int)(start.off / (nb + kGroupCost));
    run.blk = (int)(start.off - (int64_t)run.grp_next * (nb + kGroupCost));
  }
  run.left = start.count;

  if (warp == 4) {
    // ------------------------------------------------------------ TMA
    const uint64_t once = ptx::l2_evict_first_policy();
    const int br = a.p < BN ? a.p : BN;
    const int nseg = BN / br;
    const uint32_t seg_bytes = (uint32_t)(br * D);
    int gb = 0;
    int queued[2] = {0, 0};                // K and V tiles: a wait that gives up may leave them unequal
    bool ok = true;
    while (ok && run.next()) {
      const int last = run.last_block();
      const int32_t *pt = a.page_table + (size_t)run.s * a.max_pages;
      auto page_of = [&](int b) -> int {
        const int pos = b * BN + lane * br;
        return lane < nseg && b < last && pos < run.kv ? pt[pos >> a.p_shift] : -1;
      };
      int next_page = page_of(run.b0);
      for (int b = run.b0; b < last; ++b, ++gb) {
        const int page = next_page;
        next_page = page_of(b + 1);
        const int pos = b * BN + lane * br;
        const bool load = lane < nseg && pos < run.kv;
        int row = page * a.p + (pos & (a.p - 1));
        if (load && (page < 0 || page >= a.num_pages)) {
          raise(a.err, RPA_DEV_BAD_PAGE);
          row = a.num_pages * a.p;      // outside the tensor: the copy fills zeros
        }
        const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, load)) * seg_bytes;
        const int st = gb % NS;
        const uint32_t ph = (uint32_t)((gb / NS) & 1);
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          uint64_t *full = kv ? &bars->v_full[st] : &bars->k_full[st];
          uint64_t *empty = kv ? &bars->v_empty[st] : &bars->k_empty[st];
          uint8_t *dst = (kv ? sV : sK) + st * S::kTile + lane * br * S::W;
          if (gb >= NS && !wait_warp(empty, ph ^ 1u, abort_flag, a.err)) {
            ok = false;
            break;
          }
          ptx::mbar_arrive_expect_tx_elect(full, bytes);
          __syncwarp();
          if (load)
#pragma unroll
            for (int c = 0; c < S::CT; ++c)
              ptx::tma_load_3d_hint(dst + c * BN * S::W, kv ? &tm_v : &tm_k, full, c * S::W, run.hk, row, once);
          __syncwarp();
          ++queued[kv];
        }
        if (!ok) break;
      }
    }
    // every queued copy lands before the CTA ends
    if (lane == 0)
#pragma unroll
      for (int kv = 0; kv < 2; ++kv)
        for (int k = max(0, queued[kv] - NS); k < queued[kv]; ++k)
          ptx::mbar_wait(kv ? &bars->v_full[k % NS] : &bars->k_full[k % NS], (uint32_t)((k / NS) & 1));
    __syncwarp();
  } else if (warp == 5) {
    // ------------------------------------------------------------ MMA
    constexpr uint32_t idesc_qk = ptx::umma_idesc_e4m3(128, S::NQpad, false, false);
    constexpr uint32_t idesc_pv = ptx::umma_idesc_e4m3(128, S::NPpad, true, true);
    constexpr uint32_t sw = S::W == 128 ? 2 : 4;
    const uint64_t dk0 = ptx::umma_desc(ptx::smem_u32(sK), 16, 8 * S::W, sw);
    const uint64_t dq0 = ptx::umma_desc(ptx::smem_u32(sQ), 16, 8 * S::W, sw);
    // head_dim 64: rows 64..127 of M read the same 64 values (LBO 0); their lanes are not used
    const uint64_t dv0 = ptx::umma_desc(ptx::smem_u32(sV), 0, 8 * S::W, sw);
    const uint64_t dp0 = ptx::umma_desc(ptx::smem_u32(sP), 128, BN * 16, 0);
    int gb = 0, seg = 0;
    bool ok = true;
    // QK of block `blk` (ring position)
    auto qk = [&](int blk) -> bool {
      const int st = blk % NS;
      if (!wait_warp(&bars->k_full[st], (uint32_t)((blk / NS) & 1), abort_flag, a.err)) return false;
      ptx::tc_fence_after();
#pragma unroll
      for (int k = 0; k < D / 32; ++k) {
        const int c = k * 32 / S::W, kk = k * 32 % S::W;
        ptx::umma_ss_e4m3_elect(tS + (blk & 1) * S::NQpad,
                                dk0 + (uint64_t)((st * S::kTile + c * BN * S::W + kk) >> 4),
                                dq0 + (uint64_t)((c * S::NQpad * S::W + kk) >> 4), idesc_qk, k > 0);
      }
      ptx::umma_commit_elect(&bars->s_full[blk & 1]);
      ptx::umma_commit_elect(&bars->k_empty[st]);
      return true;
    };
    auto pv = [&](int blk) -> bool {
      const int st = blk % NS;
      if (!wait_warp(&bars->p_full[blk & 1], (uint32_t)((blk >> 1) & 1), abort_flag, a.err)) return false;
      if (!wait_warp(&bars->v_full[st], (uint32_t)((blk / NS) & 1), abort_flag, a.err)) return false;
      ptx::tc_fence_after();
#pragma unroll
      for (int c = 0; c < S::CT; ++c)
#pragma unroll
        for (int k = 0; k < BN / 32; ++k)
          ptx::umma_ss_e4m3_elect(tO + ((blk & 1) * S::CT + c) * S::NPpad,
                                  dv0 + (uint64_t)((st * S::kTile + c * BN * S::W + k * 32 * S::W) >> 4),
                                  dp0 + (uint64_t)(((blk & 1) * S::kPBuf + k * 32 * 16) >> 4), idesc_pv, k > 0);
      ptx::umma_commit_elect(&bars->pv_full[blk & 1]);
      ptx::umma_commit_elect(&bars->v_empty[st]);
      return true;
    };
    // Within a segment QK runs one block ahead of PV.  The S buffer of QK(b) was read
    // before P(b - 2) was published, which PV(b - 2), issued earlier, waited for; the O and
    // P buffers of PV(b) are free once P(b) is published (the softmax threads read PV(b - 2)
    // before that).  The next segment's Q comes when this one's last PV has been read.
    while (ok && run.next()) {
      const int last = run.last_block();
      if (last == run.b0) continue;
      ok = wait_warp(&bars->q_full, (uint32_t)(seg & 1), abort_flag, a.err);
      for (int b = run.b0; ok && b < last; ++b, ++gb) {
        ok = qk(gb);
        if (ok && b > run.b0) ok = pv(gb - 1);
      }
      if (ok) ok = pv(gb - 1);
      ++seg;
    }
    ptx::umma_commit_elect(&bars->drain);
    ptx::mbar_wait(&bars->drain, 0);
    __syncwarp();
  } else if (warp == 6) {
    // ------------------------------------------------------ the scales
    int gb = 0;
    bool ok = true;
    while (ok && run.next()) {
      const int last = run.last_block();
      const int32_t *pt = a.page_table + (size_t)run.s * a.max_pages;
      auto page_of = [&](int b) -> int {
        const int pos = b * BN + lane * 4;
        return b < last && pos < run.kv ? pt[pos >> a.p_shift] : -1;
      };
      int next_page = page_of(run.b0);
      for (int b = run.b0; b < last; ++b, ++gb) {
        const int page = next_page;
        next_page = page_of(b + 1);
        const int slot = gb % kScaleSlots;
        if (gb >= kScaleSlots &&
            !wait_warp(&bars->sc_empty[slot], (uint32_t)(((gb / kScaleSlots) & 1) ^ 1), abort_flag, a.err)) {
          ok = false;
          break;
        }
        const int pos = b * BN + lane * 4;
        uint8_t *dst = sSc + slot * 2 * BN + lane * 4;
        if (pos < run.kv && page >= 0 && page < a.num_pages) {
          const size_t src = ((size_t)page * a.hkv + run.hk) * a.p + (pos & (a.p - 1));
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(ptx::smem_u32(dst)), "l"(a.c.ks + src)
                       : "memory");
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(ptx::smem_u32(dst + BN)), "l"(a.c.vs + src)
                       : "memory");
          asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(
                           ptx::smem_u32(&bars->sc_full[slot]))
                       : "memory");
        } else {
          *reinterpret_cast<uint32_t *>(dst) = 0;
          *reinterpret_cast<uint32_t *>(dst + BN) = 0;
          ptx::mbar_arrive(&bars->sc_full[slot]);
        }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else {
    // -------------------------------------- softmax, weights, output
    const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
    int gb = 0, seg = 0;
    bool ok = true;
    bool head_written = false;
    constexpr int E = D / 32, RW = R / 4;   // values per lane of a row, rows per warp
    // The parts of the current segment's query rows, and the rows' factors, places and
    // key counts.  (The scores of the segment before have been read, so Q is free.)
    auto prepare = [&]() {
      constexpr int NW = E * (int)sizeof(T) / 4;      // words per lane and row
      uint32_t raw[RW][NW];
      int qb = (seg & 1) * 16;
#pragma unroll
      for (int k = 0; k < RW; ++k) {                  // every row's loads first: one latency
        const int r = warp + 4 * k, rho = run.grp * R + r, i = rho / G;
        const bool row_ok = i < run.q_len;
        const size_t at = ((size_t)(run.q0 + i) * a.hq + hk * G + (rho - i * G)) * D;
        const uint32_t *src = reinterpret_cast<const uint32_t *>(static_cast<const T *>(a.q) + at) + lane * NW;
        if constexpr (NW == 1) {
          raw[k][0] = row_ok ? src[0] : 0u;
        } else if constexpr (NW == 2) {
          const uint2 v = row_ok ? *reinterpret_cast<const uint2 *>(src) : make_uint2(0, 0);
          raw[k][0] = v.x;
          raw[k][1] = v.y;
        } else {
#pragma unroll
          for (int w = 0; w < NW; w += 4) {
            const uint4 v = row_ok ? *reinterpret_cast<const uint4 *>(src + w) : make_uint4(0, 0, 0, 0);
            raw[k][w] = v.x;
            raw[k][w + 1] = v.y;
            raw[k][w + 2] = v.z;
            raw[k][w + 3] = v.w;
          }
        }
        if (lane == 0) {
          s_at[qb + r] = row_ok ? (long long)at : -1;
          s_end[qb + r] = !row_ok ? 0 : a.causal ? min(run.kv, max(0, run.kv - run.q_len + i + 1)) : run.kv;
        }
      }
      const int d0 = lane * E, c = d0 / S::W, dd = d0 % S::W;
#pragma unroll
      for (int k = 0; k < RW; ++k) {
        const int r = warp + 4 * k;
        float x[E];
        uint32_t amax = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          if constexpr (sizeof(T) == 4) x[e] = __uint_as_float(raw[k][e]);
          else x[e] = __uint_as_float(e & 1 ? raw[k][e / 2] & 0xffff0000u : raw[k][e / 2] << 16);
          amax = max(amax, __float_as_uint(x[e]) & 0x7fffffffu);
        }
        amax = __reduce_max_sync(0xffffffffu, amax);
        const uint32_t code = scale_code(amax);
        const float inv = code == kScaleNan ? 0.f : inverse_scale(code);
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] = code == kScaleNan ? 0.f : x[e] * inv;
        // part p of the row: row p * R + r of the K-major tile, 16-byte chunks swizzled
#pragma unroll
        for (int p = 0; p < S::NQ; ++p) {
          const int row = p * R + r, sz = S::W == 128 ? row & 7 : (row >> 1) & 3;
          uint8_t *dst = sQ + c * S::NQpad * S::W + row * S::W + (((dd >> 4) ^ sz) << 4) + (dd & 15);
          uint32_t word[(E + 3) / 4] = {};
#pragma unroll
          for (int e = 0; e < E; e += 2) {
            const uint32_t v = to_e4m3x2(x[e], x[e + 1]);
            word[e / 4] |= v << (8 * (e & 2));
            if (p + 1 < S::NQ) {
              const float2 b = __half22float2(from_e4m3x2(v));
              x[e] = (x[e] - b.x) * 16.f;
              x[e + 1] = (x[e + 1] - b.y) * 16.f;
            }
          }
          if constexpr (E == 2) *reinterpret_cast<uint16_t *>(dst) = (uint16_t)word[0];
          else if constexpr (E == 4) *reinterpret_cast<uint32_t *>(dst) = word[0];
          else *reinterpret_cast<uint2 *>(dst) = make_uint2(word[0], word[E / 4 - 1]);
        }
        if (lane == 0) s_qf[qb + r] = scale_value(code) * (a.scale * kLog2e);
      }
      ptx::fence_proxy_async_smem();
      ptx::mbar_arrive(&bars->q_full);
    };
    bool have = run.next();
    if (have && run.last_block() > run.b0) prepare();
    while (ok && have) {
      const int last = run.last_block();
      float m[R], l[R], o[S::CT][R];    // o is in units of exp2(m)
      float F[R];                       // what the pending block's O^T counts in units of exp2(m)
#pragma unroll
      for (int r = 0; r < R; ++r) {
        m[r] = -INFINITY;
        l[r] = F[r] = 0.f;
#pragma unroll
        for (int c = 0; c < S::CT; ++c) o[c][r] = 0.f;
      }
      // joins block blk's product, in units of the maxima before `al` moved them, into o
      auto take_pv = [&](int blk, const float (&al)[R]) -> bool {
        if (!wait_warp(&bars->pv_full[blk & 1], (uint32_t)((blk >> 1) & 1), abort_flag, a.err)) return false;
        ptx::tc_fence_after();
#pragma unroll
        for (int c = 0; c < S::CT; ++c)
#pragma unroll
          for (int r0 = 0; r0 < R; r0 += S::RC) {
            float sum[S::RC];
            join_parts<S::NP, R, S::RC>(tO + lane_base + ((blk & 1) * S::CT + c) * S::NPpad + r0, sum);
#pragma unroll
            for (int r = 0; r < S::RC; ++r) o[c][r0 + r] = fmaf(sum[r], F[r0 + r], o[c][r0 + r]) * al[r0 + r];
          }
        ptx::tc_fence_before();
        return true;
      };
      if (last > run.b0) {
        // (the other warps' factors and counts too)
        if (!wait_warp(&bars->q_full, (uint32_t)(seg & 1), abort_flag, a.err)) break;
        const float *qf = s_qf + (seg & 1) * 16;
        const int *ends = s_end + (seg & 1) * 16;
        int all = run.kv;               // keys that every row of the group sees
#pragma unroll
        for (int r = 0; r < R; ++r) all = min(all, ends[r]);
        for (int b = run.b0; b < last; ++b, ++gb) {
          const int slot = gb % kScaleSlots;
          const int par = gb & 1;
          if (!wait_warp(&bars->sc_full[slot], (uint32_t)((gb / kScaleSlots) & 1), abort_flag, a.err)) {
            ok = false;
            break;
          }
          const int pos = b * BN + tid;
          const bool key = pos < run.kv;
          uint32_t kc = sSc[slot * 2 * BN + tid], vc = sSc[slot * 2 * BN + BN + tid];
          ptx::mbar_arrive(&bars->sc_empty[slot]);
          // NaN of either scale makes the score NaN for the rows that see the key
          const float kf = scale_value(kc) + (vc == kScaleNan ? NAN : 0.f);
          // A V row of zeros adds nothing, so its scale must not set the unit of the block's weights
          // (a key of most of the weight, whose row is zeros, would leave the others no bits).  The
          // format gives such rows the scale 2^0, or the smallest one: only those are looked through.
          bool zero = key && (vc == kScaleOne || vc == 0);
          if (__any_sync(0xffffffffu, zero)) {
            const int st = gb % NS;
            if (!wait_warp(&bars->v_full[st], (uint32_t)((gb / NS) & 1), abort_flag, a.err)) {
              ok = false;
              break;
            }
            const uint8_t *row = sV + st * S::kTile + tid * S::W;
#pragma unroll 1
            for (int q = 0; zero && q < D / 16; ++q) {
              const int c = q * 16 / S::W, i = (q + tid) % (S::W / 16);   // lanes start at different banks
              const uint4 v = *reinterpret_cast<const uint4 *>(row + c * BN * S::W + i * 16);
              zero = ((v.x | v.y | v.z | v.w) & 0x7f7f7f7fu) == 0;
            }
          }
          const float ev = zero ? -INFINITY : key && vc != kScaleNan ? (float)((int)vc - 127) : 0.f;
          if (!wait_warp(&bars->s_full[par], (uint32_t)((gb >> 1) & 1), abort_flag, a.err)) {
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          float x[R];
#pragma unroll
          for (int r0 = 0; r0 < R; r0 += S::RC) {
            float sum[S::RC];
            join_parts<S::NQ, R, S::RC>(tS + lane_base + par * S::NQpad + r0, sum);
#pragma unroll
            for (int r = 0; r < S::RC; ++r) x[r0 + r] = sum[r] * (qf[r0 + r] * kf);
          }
          if (b * BN + BN > all) {
#pragma unroll
            for (int r = 0; r < R; ++r)
              if (pos >= ends[r]) x[r] = -INFINITY;
          }
          // maxima of the block: warp, then the four warps through shared memory
          float *wm = s_max + par * 128;
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const float mx = warp_max(x[r]), my = warp_max(x[r] + ev);
            if (lane == 0) {
              wm[warp * 32 + r] = mx;
              wm[warp * 32 + 16 + r] = my;
            }
          }
          if (lane == 0) ptx::mbar_arrive(&bars->x_full[par]);
          if (!wait_warp(&bars->x_full[par], (uint32_t)((gb >> 1) & 1), abort_flag, a.err)) {
            ok = false;
            break;
          }
          float w[R], al[R], Fn[R];
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const float mb = fmaxf(fmaxf(wm[r], wm[32 + r]), fmaxf(wm[64 + r], wm[96 + r]));
            // -inf where the row sees nothing of the block: its weights are zeros then, and so is
            // what they count (joined(yb) in its place would be 2^-m, which overflows for low scores)
            const float yb = fmaxf(fmaxf(wm[16 + r], wm[48 + r]), fmaxf(wm[80 + r], wm[112 + r]));
            const float mn = fmaxf(m[r], mb);
            al[r] = m[r] == mn ? 1.f : ptx::ex2(m[r] - mn);
            m[r] = mn;
            l[r] = l[r] * al[r] + ptx::ex2(x[r] - joined(mn));
            w[r] = ptx::ex2((x[r] + (8.f - joined(yb))) + ev);
            Fn[r] = ptx::ex2(yb - joined(mn) - 8.f);
          }
          uint32_t pw[S::CP / 4];
#pragma unroll
          for (int p = 0; p < S::NP; ++p) {
#pragma unroll
            for (int r = 0; r < R; r += 4) {
              const uint32_t lo = to_e4m3x2(w[r], w[r + 1]), hi = to_e4m3x2(w[r + 2], w[r + 3]);
              pw[(p * R + r) / 4] = lo | (hi << 16);
              if (p + 1 < S::NP) {
                const float2 bl = __half22float2(from_e4m3x2(lo)), bh = __half22float2(from_e4m3x2(hi));
                w[r] = (w[r] - bl.x) * 16.f;
                w[r + 1] = (w[r + 1] - bl.y) * 16.f;
                w[r + 2] = (w[r + 2] - bh.x) * 16.f;
                w[r + 3] = (w[r + 3] - bh.y) * 16.f;
              }
            }
          }
          uint8_t *dst = sP + par * S::kPBuf + tid * 16;
#pragma unroll
          for (int i = 0; i < S::NPpad / 16; ++i) {
            uint32_t q4[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) q4[j] = i * 4 + j < S::CP / 4 ? pw[i * 4 + j < S::CP / 4 ? i * 4 + j : 0] : 0u;
            *reinterpret_cast<uint4 *>(dst + i * BN * 16) = make_uint4(q4[0], q4[1], q4[2], q4[3]);
          }
          // V rows without a key hold whatever the page or the slot held: zeros
          if (b * BN + BN > run.kv) {
            const int st = gb % NS;
            if (!wait_warp(&bars->v_full[st], (uint32_t)((gb / NS) & 1), abort_flag, a.err)) {
              ok = false;
              break;
            }
            if (!key)
#pragma unroll
              for (int c = 0; c < S::CT; ++c)
#pragma unroll
                for (int q = 0; q < S::W / 16; ++q)
                  *reinterpret_cast<uint4 *>(sV + st * S::kTile + c * BN * S::W + tid * S::W + q * 16) =
                      make_uint4(0, 0, 0, 0);
          }
          ptx::fence_proxy_async_smem();
          ptx::tc_fence_before();
          ptx::mbar_arrive(&bars->p_full[par]);
          if (b > run.b0 && !take_pv(gb - 1, al)) {
            ok = false;
            break;
          }
#pragma unroll
          for (int r = 0; r < R; ++r) F[r] = Fn[r];
        }
        float one[R];
#pragma unroll
        for (int r = 0; r < R; ++r) one[r] = 1.f;
        if (!ok || !take_pv(gb - 1, one)) {
          ok = false;
          break;
        }
        // row sums of the 128 keys' threads
#pragma unroll
        for (int r = 0; r < R; ++r) {
#pragma unroll
          for (int off = 16; off > 0; off >>= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], off);
          if (lane == 0) s_l[warp * 16 + r] = l[r];
        }
        if (lane == 0) ptx::mbar_arrive(&bars->l_full);
        if (!wait_warp(&bars->l_full, (uint32_t)(seg & 1), abort_flag, a.err)) {
          ok = false;
          break;
        }
        // (s_l is written again only behind the next segment's first x_full)
#pragma unroll
        for (int r = 0; r < R; ++r) l[r] = (s_l[r] + s_l[16 + r]) + (s_l[32 + r] + s_l[48 + r]);
      }
      const bool whole = run.b0 == 0 && run.b1 == run.nb;
      // 2 * place: the run begins inside the group; 2 * place + 1: it begins with it
      const size_t slot = 2 * (size_t)place + (run.b0 > 0 ? 0 : 1);
      if (!head_written && tid == 0) g.heads[place] = PartHead{run.s, hk, run.grp, run.b0};
      head_written = true;
      // the next segment's Q before this one's output: its first scores are computed meanwhile
      const long long *at = s_at + (seg & 1) * 16;    // (a whole group has been prepared)
      if (last > run.b0) ++seg;
      have = run.next();
      if (have && run.last_block() > run.b0) prepare();
      if (tid == 0) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
          s_ml[2 * r] = m[r];
          s_ml[2 * r + 1] = l[r];
        }
      }
      if (whole) {
        T *out = static_cast<T *>(a.out) + tid;
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const long long row = at[r];
          const float inv = l[r] == 0.f ? 0.f : ptx::rcp(l[r]);
          if (row >= 0)
#pragma unroll
            for (int c = 0; c < S::CT; ++c)
              if (D >= 128 || tid < D) store(out + row + c * 128, o[c][r] * inv);
        }
      } else {
        float *po = g.o + slot * (R * D) + tid;
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int c = 0; c < S::CT; ++c)
            if (D >= 128 || tid < D) po[r * D + c * 128] = o[c][r];
      }
      if (warp == 0) {
        __syncwarp();
        if (lane < R) {
          const float mr = s_ml[2 * lane], lr = s_ml[2 * lane + 1];
          if (!whole) {
            g.ml[(slot * R + lane) * 2] = mr;
            g.ml[(slot * R + lane) * 2 + 1] = lr;
          } else if (a.lse != nullptr && at[lane] >= 0) {
            a.lse[at[lane] / D] = lr == 0.f ? -INFINITY : (joined(mr) + log2f(lr)) * kLn2;
          }
        }
        __syncwarp();
      }
    }
    if (!head_written && tid == 0) g.heads[place].begin = 0;
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == 5) ptx::tmem_dealloc(tmem, S::kTmem);
}

// Joins the partial results of one group.  Block i: the group that the run at
// place i begins inside, if it is the first to do so; its parts are slot
// 2 (i - 1) + 1, where the run before began the group, then 2 j of i and every
// following place whose run begins inside the same group.  D / 4 lanes take a row; where
// there are more lanes than rows, several share a row's parts.
constexpr int kJoinThreads = 1024;
template <typename T, int D, int R>
__global__ void __launch_bounds__(kJoinThreads) combine_kernel(const Args g) {
  constexpr int L = D / 4, W = kJoinThreads / L, SL = W / R;   // lanes of a row, rows at once, shares of a row
  static_assert(SL >= 1 && SL * R == W, "rows of a group");
  __shared__ float s_o[W][D];
  __shared__ float s_l[W];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int i = blockIdx.x, places = gridDim.x, tid = threadIdx.x;
  const PartHead h = g.heads[i];
  if (h.begin <= 0) return;
  auto same = [&](const PartHead &p) { return p.begin > 0 && p.seq == h.seq && p.hk == h.hk && p.grp == h.grp; };
  if (same(g.heads[i - 1])) return;
  const AttendArgs &a = g.a;
  const int G = a.hq / a.hkv;
  const int q0 = a.len.cu[h.seq], q_len = a.len.cu[h.seq + 1] - q0;
  int end = i + 1;
  while (end < places && same(g.heads[end])) ++end;
  const int parts = end - i + 1;
  const int li = tid % L, wi = tid / L, r = wi % R, sl = wi / R;
  auto slot = [&](int k) { return ((size_t)(k == 0 ? 2 * (i - 1) + 1 : 2 * (i + k - 1))) * R + r; };
  // the maximum of the row's parts, by every lane
  float M = -INFINITY;
  for (int k = 0; k < parts; ++k) M = fmaxf(M, g.ml[slot(k) * 2]);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float l = 0.f;
#pragma unroll 2
  for (int k = sl; k < parts; k += SL) {
    const float mk = g.ml[slot(k) * 2], lk = g.ml[slot(k) * 2 + 1];
    const float4 v = *reinterpret_cast<const float4 *>(g.o + slot(k) * D + li * 4);
    if (lk == 0.f) continue;               // saw no key: nothing there
    const float wt = mk == M ? 1.f : ptx::ex2(joined(mk) - joined(M));
    acc.x = fmaf(wt, v.x, acc.x);
    acc.y = fmaf(wt, v.y, acc.y);
    acc.z = fmaf(wt, v.z, acc.z);
    acc.w = fmaf(wt, v.w, acc.w);
    l = fmaf(wt, lk, l);
  }
  *reinterpret_cast<float4 *>(&s_o[wi][li * 4]) = acc;
  if (li == 0) s_l[wi] = l;
  __syncthreads();
  for (int e = tid; e < R * D; e += kJoinThreads) {
    const int row = e / D, d = e % D, rho = h.grp * R + row;
    if (rho >= q_len * G) continue;
    float v = 0.f, sum = 0.f;
#pragma unroll
    for (int w = 0; w < SL; ++w) {
      v += s_o[w * R + row][d];
      sum += s_l[w * R + row];
    }
    const size_t at = (size_t)(q0 + rho / G) * a.hq + h.hk * G + rho % G;
    store(static_cast<T *>(a.out) + at * D + d, sum == 0.f ? 0.f : v / sum);
    if (d == 0 && a.lse != nullptr) {
      float mm = -INFINITY;
      for (int k = 0; k < parts; ++k)
        mm = fmaxf(mm, g.ml[(((size_t)(k == 0 ? 2 * (i - 1) + 1 : 2 * (i + k - 1))) * R + row) * 2]);
      a.lse[at] = sum == 0.f ? -INFINITY : (joined(mm) + log2f(sum)) * kLn2;
    }
  }
}

template <typename T, int D, int R>
cudaError_t launch_t(const AttendArgs &a, int q_limit, int grid, uint8_t *ws, bool join, cudaStream_t stream) {
  using S = Shape<T, D, R>;
  Args g{};
  g.a = a;
  g.q_limit = q_limit;
  const RowsLayout w = rows_layout(grid, R, D);
  g.heads = reinterpret_cast<PartHead *>(ws + w.heads);
  g.ml = reinterpret_cast<float *>(ws + w.ml);
  g.o = reinterpret_cast<float *>(ws + w.o);
  if (join) {
    if (grid == a.hkv) return cudaSuccess;   // one run per head: nothing is split
    return launch_behind(combine_kernel<T, D, R>, grid, kJoinThreads, 0, stream, g);
  }
  CUtensorMap tk, tv;
  const uint64_t dims[3] = {(uint64_t)D, (uint64_t)a.hkv, (uint64_t)a.num_pages * a.p};
  const uint64_t strides[2] = {(uint64_t)D, (uint64_t)a.hkv * D};
  const uint32_t box[3] = {(uint32_t)S::W, 1, (uint32_t)(a.p < BN ? a.p : BN)};
  if (!make_tmap_u8_3d(&tk, a.c.k, dims, strides, box, true) || !make_tmap_u8_3d(&tv, a.c.v, dims, strides, box, true))
    return cudaErrorInvalidValue;
  auto kern = rows_kernel<T, D, R>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
  if (e != cudaSuccess) return e;
  kern<<<grid, kThreads, S::kSmem, stream>>>(tk, tv, g);
  return cudaGetLastError();
}

template <typename T, int D, int R> constexpr int ctas_of() { return Shape<T, D, R>::CTAS; }

}  // namespace

int rows_per_group(const rpa_dims &d, int32_t max_q) {
  // the smallest group that holds a whole KV head's rows (its keys are then
  // read once), up to 16; fp32 rows have three times the columns: up to 8
  const int64_t rows = (int64_t)max_q * (d.num_q_heads / d.num_kv_heads);
  if (rows <= 4) return 4;
  if (rows <= 8 || d.dtype == RPA_F32) return 8;
  return 16;
}

int rows_grid(const rpa_dims &d, int32_t max_seqs, int32_t max_q, int R) {
  const int G = d.num_q_heads / d.num_kv_heads;
  const int64_t cap = (int64_t)d.max_pages_per_seq * d.page_size;
  const int64_t seqs = std::min<int64_t>(max_seqs, d.total_q_tokens);
  const int64_t groups = ((int64_t)max_q * G + R - 1) / R;
  int ctas = 1;
  const bool f32 = d.dtype == RPA_F32;
#define RPA_Q8_CTAS(DD)                                                                       \
  case DD:                                                                                    \
    ctas = f32 ? (R == 4 ? ctas_of<float, DD, 4>() : ctas_of<float, DD, 8>())                 \
               : R == 4 ? ctas_of<__nv_bfloat16, DD, 4>()                                     \
                        : R == 8 ? ctas_of<__nv_bfloat16, DD, 8>() : ctas_of<__nv_bfloat16, DD, 16>(); \
    break;
  switch (d.head_dim) {
    RPA_Q8_CTAS(64)
    RPA_Q8_CTAS(128)
    RPA_Q8_CTAS(256)
  }
#undef RPA_Q8_CTAS
  // the same number of CTAs for every head, as many as are resident on 148 SMs;
  // fewer where the lengths cannot fill them
  const double most = (double)seqs * groups * (double)((cap + BN - 1) / BN);   // (a run without a block is of no use)
  const int runs = std::max(1, 148 * ctas / d.num_kv_heads);
  return d.num_kv_heads * (int)std::max(1.0, std::min(most, (double)runs));
}

RowsLayout rows_layout(int grid, int R, int D) {
  RowsLayout w;
  auto up = [](int64_t x) { return (x + 255) / 256 * 256; };
  w.heads = 0;
  w.ml = up((int64_t)grid * sizeof(PartHead));
  w.o = up(w.ml + (int64_t)grid * 2 * R * 2 * 4);
  w.total = up(w.o + (int64_t)grid * 2 * R * D * 4);
  return w;
}

cudaError_t launch_rows(const AttendArgs &a, const rpa_dims &d, int32_t max_seqs, int32_t max_q, int32_t q_limit,
                        uint8_t *ws, bool join, cudaStream_t stream) {
  const int R = rows_per_group(d, std::min(max_q, q_limit));
  const int grid = rows_grid(d, max_seqs, std::min(max_q, q_limit), R);
#define RPA_Q8_ROWS(DD)                                                                                   \
  case DD:                                                                                                \
    if (d.dtype == RPA_F32)                                                                               \
      return R == 4 ? launch_t<float, DD, 4>(a, q_limit, grid, ws, join, stream)                                \
                    : launch_t<float, DD, 8>(a, q_limit, grid, ws, join, stream);                               \
    return R == 4   ? launch_t<__nv_bfloat16, DD, 4>(a, q_limit, grid, ws, join, stream)                        \
           : R == 8 ? launch_t<__nv_bfloat16, DD, 8>(a, q_limit, grid, ws, join, stream)                        \
                    : launch_t<__nv_bfloat16, DD, 16>(a, q_limit, grid, ws, join, stream);
  switch (d.head_dim) {
    RPA_Q8_ROWS(64)
    RPA_Q8_ROWS(128)
    RPA_Q8_ROWS(256)
    default: return cudaErrorInvalidValue;
  }
#undef RPA_Q8_ROWS
}

}  // namespace q8
}  // namespace rpa
