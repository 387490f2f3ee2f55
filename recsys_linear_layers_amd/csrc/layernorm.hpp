// Layer norm and its gradients: arguments and launches (layernorm.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ll {

struct NormArgs {
  const void* x;
  const void* gamma;  // null: ones
  const void* beta;   // null: zeros
  void* y;
  float* mean;        // null: not written
  float* rstd;
  int64_t N, ldx, ldy;
  int32_t D;
  int32_t param_f32;  // gamma and beta are fp32 (else of x's type)
  float eps;
};

struct NormGradArgs {
  const void* dy;
  const void* x;
  const void* gamma;  // null: ones
  const float* mean;
  const float* rstd;
  void* dx;
  void* dgamma;       // null: not wanted (with dbeta)
  void* dbeta;
  float* partial;     // [workgroups][2][D]
  int64_t N, lddy, ldx, lddx;
  int32_t D;
  int32_t param_f32;
};

hipError_t launch_norm(const NormArgs& a, int type, int cus, hipStream_t s);
// Workgroups (partial rows) of the gradient's first kernel: two for each of 256 CUs,
// whatever the device has, so that sizes alone decide which rows are added up together.
int norm_grad_blocks(int64_t N);
hipError_t launch_norm_grad(const NormGradArgs& a, int type, int cus, hipStream_t s);

}  // namespace ll
