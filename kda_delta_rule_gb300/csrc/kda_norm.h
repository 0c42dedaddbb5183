// The norms around a block (kda_gated_norm, kda_residual_norm): arguments of their kernels.  Validated by kda_norm.cpp.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace kda {

struct GatedNormArgs {
  const void *x, *gate, *weight;      // rows of H heads of d values, *_stride elements apart; gate or nullptr; [d] or [H][d]
  int64_t x_stride, gate_stride;
  int weight_stride;                  // elements between the heads' weights (0: shared)
  void* y;                            // [T][H][d]
  float eps;
  int64_t T;
  int H, d, dtype, act, gate_first;
};
cudaError_t launch_gated_norm(const GatedNormArgs& a, cudaStream_t s);

struct ResidualNormArgs {
  const void *y, *gate;               // T rows of D values, *_stride elements apart; gate or nullptr
  int64_t y_stride, gate_stride;
  const void *h_in;                   // T rows of D values of h_dtype
  void* h_out;                        // same (may be h_in)
  int64_t h_stride;
  const void *post_weight, *pre_weight, *channel_scale;   // [D] or nullptr (pre_weight: given)
  void* x;                            // [T][D]
  float res_scale, eps;
  int64_t T;
  int D, dtype, h_dtype, act;
};
cudaError_t launch_residual_norm(const ResidualNormArgs& a, cudaStream_t s);

}  // namespace kda
