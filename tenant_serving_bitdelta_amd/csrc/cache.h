// Internal declarations of the paged cache: what the attention and the writing and reading of the cache
// check and lay out alike, and the latter's kernels (cache.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/bitdelta.h"
#include "attend.h"

namespace bd {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Every refusal of a cache for `heads` query heads.
bitdelta_status check_kv_cache(const bitdelta_kv_cache* c, int32_t heads);
// The kernels' form of a cache that check_kv_cache passes.
PagedCache paged_cache(const bitdelta_kv_cache& c);

constexpr int64_t kCacheMaxHeads = int64_t(1) << 16;
constexpr int64_t kCacheMaxRows = int64_t(1) << 30;  // tokens x kv heads

struct CacheArgs {
  uint16_t* rows[2];                     // keys, values
  int64_t row_token[2], row_head[2];     // strides in elements
  PagedCache cache;
  const int32_t* table;                  // [batch][width]
  const int32_t* lens;                   // [batch]
  const int32_t* q_offsets;              // [batch + 1] or null: row t is the last token of sequence t
  int32_t width, batch, tokens, kv_heads;
  float scale[2];
  float inverse[2];                      // 1 / scale where that is exact, else 0
  float near[2];                         // 1 / scale rounded where a division by it may start from that, else 0
};

hipError_t launch_cache_write(const CacheArgs& a, int dim, int dtype, hipStream_t stream);
hipError_t launch_cache_read(const CacheArgs& a, int dim, int dtype, hipStream_t stream);

}  // namespace bd
