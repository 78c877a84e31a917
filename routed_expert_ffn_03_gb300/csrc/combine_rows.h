// combine_rows.h - arguments and launchers of the weighted sum of experts' rows (internal).
#pragma once
#include <cuda_runtime.h>

namespace moe {

struct CombineRowsArgs {
  const void* y;
  const float* weights;      // [T][k]
  const int* places;         // [T][k] or null
  const void* residual;      // of the result's type, or null
  void* out;
  long long y_rows, ldy, ld_res, ldo;
  int T, k, H, y_type, out_type;
};
cudaError_t launch_combine_rows(const CombineRowsArgs& a, cudaStream_t s);

struct CombineGradArgs {
  const void *dout, *y;
  const float* weights;
  const int* places;
  void* dy;
  float* dweights;
  long long y_rows, ld_dout, ldy, ld_dy;
  int T, k, H, dout_type, y_type, dy_type;
};
cudaError_t launch_combine_rows_grad(const CombineGradArgs& a, cudaStream_t s);

}  // namespace moe
