// q8_kernels.h -- launch interface of the attention kernels on the 8-bit cache.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "ptx.cuh"
#include "q8_common.cuh"
#include "rpa.h"

namespace rpa {
namespace q8 {

// What every attention kernel of a call reads.
struct AttendArgs {
  const void *q;
  Cache c;
  Lengths len;
  const int32_t *page_table;
  uint32_t *err;                 // may be null
  void *out;
  float *lse;                    // may be null
  int32_t hq, hkv, p, p_shift, num_pages, max_pages, causal;
  float scale;
};

__device__ __forceinline__ void store(float *p, float v) { *p = v; }
__device__ __forceinline__ void store(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

// Waits for a phase, for at most kWaitLimitNs: false, with RPA_DEV_TIMEOUT raised, when
// that runs out or another warp of the block gave up.  The clock is looked at every 64
// polls.  The poll loop is a function of its own, not part of every wait: these kernels'
// warps run long straight loops that share the instruction caches, and with it inlined the
// chunk kernel took 444 us for 8 prompts of 2048 tokens instead of 414.
inline __device__ __noinline__ bool wait_long(uint64_t *bar, uint32_t parity, volatile int *abort_flag, uint32_t *err) {
  const uint64_t t0 = ptx::globaltimer();
  for (uint32_t n = 1; !ptx::mbar_try_wait(bar, parity); ++n) {
    if ((n & 63) != 0) continue;
    if (*abort_flag || ptx::globaltimer() - t0 > ptx::kWaitLimitNs) {
      *abort_flag = 1;
      raise(err, RPA_DEV_TIMEOUT);
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ bool wait_bar(uint64_t *bar, uint32_t parity, volatile int *abort_flag, uint32_t *err) {
  return ptx::mbar_try_wait(bar, parity) || wait_long(bar, parity, abort_flag, err);
}
__device__ __forceinline__ bool wait_warp(uint64_t *bar, uint32_t parity, volatile int *abort_flag, uint32_t *err) {
  return __all_sync(0xffffffffu, wait_bar(bar, parity, abort_flag, err));
}

// A launch that may begin while the kernel queued before it on `stream` ends
// (programmatic dependent launch).  Every kernel of these files waits for what it
// reads, and at the latest before it ends, with griddepcontrol.wait.
template <typename K, typename... Args>
cudaError_t launch_behind(K kern, int grid, int threads, int smem, cudaStream_t stream, const Args &...args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3((unsigned)grid, 1, 1);
  cfg.blockDim = dim3((unsigned)threads, 1, 1);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

// Few query rows per KV head.  Sequences with q_len > q_limit are left out.  launch_rows is called
// twice: without `join` for the attention itself, and with it, behind the chunk kernel where the
// call has one, for joining the parts that several CTAs share (between the two attention
// kernels it would keep the second from beginning as the first ends).
int rows_per_group(const rpa_dims &d, int32_t max_q);
int rows_grid(const rpa_dims &d, int32_t max_seqs, int32_t max_q, int R);
struct RowsLayout {
  int64_t heads, ml, o, total;   // byte offsets into the workspace
};
RowsLayout rows_layout(int grid, int R, int D);
cudaError_t launch_rows(const AttendArgs &a, const rpa_dims &d, int32_t max_seqs, int32_t max_q, int32_t q_limit,
                        uint8_t *ws, bool join, cudaStream_t stream);

// Chunks of query rows (bf16).  Sequences with q_len <=
// q_limit are left out.
bool chunk_takes(const rpa_dims &d);
int chunk_grid(const rpa_dims &d, int32_t max_seqs, int32_t max_q);
struct ChunkLayout {
  int64_t heads, ml, o, total;
};
ChunkLayout chunk_layout(int grid, int D);
// Called twice as launch_rows; the first, the attention, is queued with launch_behind
// right behind the row-group kernel of the call.
cudaError_t launch_chunk(const AttendArgs &a, const rpa_dims &d, int32_t max_seqs, int32_t max_q, int32_t q_limit,
                         uint8_t *ws, bool join, cudaStream_t stream);

}  // namespace q8
}  // namespace rpa
