// q8_host.h -- host-side helpers of the 8-bit cache's entry points.
#pragma once
#include <stdint.h>

#include "q8_common.cuh"
#include "rpa.h"

namespace rpa {
namespace q8 {

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

inline bool aligned32(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 31) == 0; }

inline int log2_of(int32_t pow2) {
  int s = 0;
  while ((1 << s) < pow2) ++s;
  return s;
}

inline Cache cache_of(const rpa_q8_cache *c) {
  return Cache{static_cast<uint8_t *>(c->k_codes), static_cast<uint8_t *>(c->v_codes),
               static_cast<uint8_t *>(c->k_scales), static_cast<uint8_t *>(c->v_scales)};
}

inline Lengths lengths_of(const int32_t *cu, const int32_t *kv, const int32_t *num_seqs, int32_t max_seqs,
                          const rpa_dims *d, int32_t max_q, bool self) {
  const int64_t cap = (int64_t)d->max_pages_per_seq * d->page_size;
  return Lengths{cu, kv, num_seqs, max_seqs, d->total_q_tokens,
                 (int32_t)(cap > INT32_MAX - 256 ? INT32_MAX - 256 : cap), max_q, self ? 1 : 0};
}

}  // namespace q8
}  // namespace rpa
