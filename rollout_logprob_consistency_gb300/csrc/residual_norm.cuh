// Arguments of the residual update's launches.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/tim.h"

namespace tim {

struct NormArgs {
  tim_block b;
  const void* residual;
  int64_t ld_residual;
  void* out_h;
  int64_t ld_h;
  void* out_y;
  int64_t ld_y;
};

struct NormGradArgs {
  tim_block b;
  const void* h;
  int64_t ld_h;
  const void* dh;  // or null: zeros
  int64_t ld_dh;
  const void* dy;  // or null: zeros
  int64_t ld_dy;
  void* out_dresidual;
  int64_t ld_dresidual;
  void* out_dblock;
  int64_t ld_dblock;
  float* out_dgamma;
  float* out_dgamma_post;
  void* out_dgate;
  int64_t ld_dgate;
  int accumulate;
  float* partial;
};

cudaError_t launch_residual_norm(const NormArgs& a, cudaStream_t stream);
size_t residual_norm_backward_bytes(int64_t T, int d);
cudaError_t launch_residual_norm_backward(const NormGradArgs& a, cudaStream_t stream, int num_sms);

}  // namespace tim
