// Internal declarations of the token sampling kernel.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace bd {

struct SampleArgs {
  const void* logits;        // [rows] rows of vocab values, row_stride elements apart
  int64_t row_stride;
  int32_t rows, vocab;
  const float* u;            // [rows]
  const float* temperature;  // [rows] or null: 1
  const int32_t* top_k;      // [rows] or null: off
  const float* top_p;        // [rows] or null: off
  const float* min_p;        // [rows] or null: off
  int32_t* tokens;           // [rows]
  float* logprob;            // [rows] or null
};

hipError_t launch_sample(const SampleArgs& a, bool f32, hipStream_t stream);

}  // namespace bd
