// C ABI of token sampling: argument checks before anything is enqueued.
#include <stdint.h>

#include "../../include/bitdelta.h"
#include "sample.h"

namespace bd {
bitdelta_status status_of_hip(hipError_t e);
}

extern "C" bitdelta_status bitdelta_sample(const void* logits, int32_t logits_dtype, int64_t rows,
                                           int64_t vocab, int64_t row_stride, const float* u,
                                           const float* temperature, const int32_t* top_k,
                                           const float* top_p, const float* min_p, int32_t* tokens,
                                           float* logprob, bitdelta_stream stream) {
  if (rows < 0 || vocab < 1) return BITDELTA_ERR_INVALID_ARG;
  if (logits_dtype != BITDELTA_OUT_BF16 && logits_dtype != BITDELTA_OUT_F32)
    return BITDELTA_ERR_INVALID_ARG;
  if (rows == 0) return BITDELTA_OK;
  if (!logits || !u || !tokens) return BITDELTA_ERR_INVALID_ARG;
  if (row_stride < vocab) return BITDELTA_ERR_SHAPE;
  if (rows > (int64_t(1) << 30) || vocab > (int64_t(1) << 30)) return BITDELTA_ERR_UNSUPPORTED;
  const uintptr_t size = logits_dtype == BITDELTA_OUT_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(logits) % size != 0) return BITDELTA_ERR_ALIGNMENT;
  for (const void* p : {static_cast<const void*>(u), static_cast<const void*>(temperature),
                        static_cast<const void*>(top_k), static_cast<const void*>(top_p),
                        static_cast<const void*>(min_p), static_cast<const void*>(tokens),
                        static_cast<const void*>(logprob)})
    if (reinterpret_cast<uintptr_t>(p) % 4 != 0) return BITDELTA_ERR_ALIGNMENT;
  bd::SampleArgs a{};
  a.logits = logits;
  a.row_stride = row_stride;
  a.rows = (int32_t)rows;
  a.vocab = (int32_t)vocab;
  a.u = u;
  a.temperature = temperature;
  a.top_k = top_k;
  a.top_p = top_p;
  a.min_p = min_p;
  a.tokens = tokens;
  a.logprob = logprob;
  return bd::status_of_hip(bd::launch_sample(a, logits_dtype == BITDELTA_OUT_F32,
                                             static_cast<hipStream_t>(stream)));
}
