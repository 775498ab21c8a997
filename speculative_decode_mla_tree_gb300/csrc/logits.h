// Host-side declarations of the calls that read logits.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

namespace mt {

struct LogprobArgs {
  const void* logits;           // row r at element r * row_stride
  int64_t row_stride;
  int rows, vocab;
  const int32_t* tokens;        // [rows, per_row], row r at r * token_stride
  int64_t token_stride;
  int per_row, top_k;
  float* logprobs;              // [rows, per_row]
  float* lse;                   // [rows] or nullptr
  float* entropy;               // [rows] or nullptr
  int32_t* top_ids;             // [rows, top_k]
  float* top_logprobs;          // [rows, top_k] or nullptr
  int32_t* status;
};
cudaError_t launch_token_logprobs(const LogprobArgs& a, int logits_type, int num_sms, cudaStream_t stream);

}  // namespace mt
