// Arguments of a verification's launches.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/tim.h"

namespace tim {

// The row of sequence b, position j begins at logits + b ld_seq + j ld_pos elements.
struct VerifyMatrix {
  const void* logits;
  int64_t ld_seq, ld_pos;
};

size_t verify_bytes(int64_t B, int32_t N);
cudaError_t launch_verify(const VerifyMatrix& target, const VerifyMatrix& draft, int dtype, int64_t B,
                          int N, int V, const int32_t* ids, const float* uniform,
                          const float* uniform_draw, const tim_sample_params& target_set,
                          const tim_sample_params& draft_set, int32_t* out_ids, float* out_logprob,
                          int32_t* out_accepted, void* ws, cudaStream_t stream, int num_sms);

}  // namespace tim
