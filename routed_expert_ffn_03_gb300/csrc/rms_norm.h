// rms_norm.h - arguments and launchers of the norm kernels (internal).
#pragma once
#include <cuda_runtime.h>

#include "grouped.h"

#include <cstddef>
#include <cstdint>

namespace moe {

constexpr int NORM_MAX_H = 32768;

struct NormArgs {
  const void *x, *residual, *gain;   // residual and gain may be null
  void *sum, *out;                   // sum: with residual; out may be null
  uint8_t* out8;                     // or null
  float *scale, *rstd;               // scale: with out8; rstd may be null
  long long ldx, ld_res, ld_sum, ldo, ldo8;
  int T, H, x_type, res_type, gain_type, out_type;
  float eps;
  bool norm;                         // false: rows quantised as they are
};
cudaError_t launch_rms_norm(const NormArgs& a, int num_sms, cudaStream_t s);

struct NormGradArgs {
  const void *dy, *h, *gain, *dsum;  // gain and dsum may be null
  const float* rstd;
  void* dh;
  float *dgain, *partial;            // dgain may be null; partial [blocks][H]
  long long ld_dy, ld_h, ld_dsum, ld_dh;
  int T, H, dy_type, h_type, gain_type, dsum_type, dh_type;
};
// Blocks that the gain's gradient is summed over, a function of the sizes alone, so that neither the workspace nor the bits depend
// on the device.
int norm_grad_blocks(int T, int H);
cudaError_t launch_rms_norm_grad(const NormGradArgs& a, const WaitLimit& wait, cudaStream_t s);
cudaError_t rms_norm_set_attributes();

}  // namespace moe
