// Root-mean-square norm and its gradients: arguments and launches (rmsnorm.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ll {

struct RmsArgs {
  const void* x;
  const void* residual;  // null: none
  const void* gamma;     // null: ones
  void* h;               // with a residual
  void* y;
  float* scale;          // of an 8-bit y
  float* rstd;           // null: not written
  int64_t N, ldx, ldr, ldh, ldy, sn, sb;
  int32_t D;
  int32_t param_f32;     // gamma is fp32 (else of x's type)
  float eps;
};

struct RmsGradArgs {
  const void* dy;
  const void* h;
  const void* gamma;     // null: ones
  const float* rstd;
  const void* dh;        // null: none
  void* dx;
  void* dgamma;          // null: not wanted
  float* partial;        // [workgroups][D]
  int64_t N, lddy, ldh, lddh, lddx;
  int32_t D;
  int32_t param_f32;
};

hipError_t launch_rmsnorm(const RmsArgs& a, int type, int y_type, int cus, hipStream_t s);
// Workgroups (partial rows) of the gradient's first kernel: two for each of 256 CUs,
// whatever the device has, so that sizes alone decide which rows are added up together.
int rms_grad_blocks(int64_t N);
hipError_t launch_rmsnorm_grad(const RmsGradArgs& a, int type, int cus, hipStream_t s);

}  // namespace ll
