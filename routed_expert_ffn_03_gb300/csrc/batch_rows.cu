// batch_rows.cu - entry points of the batch operators on rows (moe_rms_norm, moe_rms_norm_backward, moe_quantize_rows,
// moe_combine_rows, moe_combine_rows_backward): argument checks, then one launcher each.
#include "batch.h"
#include "combine_rows.h"
#include "rms_norm.h"

using namespace moe;

namespace {

// [rows][len] of `type` at p, ld apart
bool matrix_ok(const void* p, int type, long long rows, long long ld, int len) {
  return is_dtype(type, true) && aligned(p, dtype_bytes(type)) && rows_fit(rows, ld, len);
}
bool length_ok(int T, int H) { return T >= 0 && H >= 1 && H <= NORM_MAX_H; }
constexpr int kMaxColumns = 1 << 24;

}  // namespace

extern "C" moe_status moe_rms_norm(const moe_rms_norm_args* a, void* stream) {
  if (!a || !length_ok(a->T, a->H) || !(a->eps >= 0.f && a->eps <= 3e38f)) return MOE_EINVAL;
  if ((!a->x && a->T) || !a->residual != !a->sum || (!a->out8 != !a->scale) || (!a->out && !a->out8 && !a->sum && !a->rstd && a->T))
    return MOE_EINVAL;
  if (!matrix_ok(a->x, a->dtype, a->T, a->ldx, a->H)) return MOE_EINVAL;
  if (a->residual && (!matrix_ok(a->residual, a->residual_dtype, a->T, a->ld_residual, a->H) ||
                      !matrix_ok(a->sum, a->residual_dtype, a->T, a->ld_sum, a->H)))
    return MOE_EINVAL;
  if (a->gain && !matrix_ok(a->gain, a->gain_dtype, 1, a->H, a->H)) return MOE_EINVAL;
  if (a->out && !matrix_ok(a->out, a->out_dtype, a->T, a->ldo, a->H)) return MOE_EINVAL;
  if (a->out8 && (!rows_fit(a->T, a->ldo8, a->H) || !aligned(a->scale, 4))) return MOE_EINVAL;
  if (!aligned(a->rstd, 4)) return MOE_EINVAL;
  if (a->T == 0) return MOE_OK;
  const NormArgs n{a->x, a->residual, a->gain, a->sum, a->out, static_cast<uint8_t*>(a->out8), a->scale, a->rstd,
                   a->ldx, a->ld_residual, a->ld_sum, a->ldo, a->ldo8, a->T, a->H, a->dtype, a->residual_dtype, a->gain_dtype,
                   a->out_dtype, a->eps, true};
  BatchDevice d;
  const moe_status st = batch_device(&d);
  if (st != MOE_OK) return st;
  return done(launch_rms_norm(n, d.num_sms, (cudaStream_t)stream));
}

extern "C" moe_status moe_quantize_rows(const void* x, long long ldx, int dtype, int T, int H, void* out8, long long ldo8, float* scale,
                                        void* stream) {
  if (!length_ok(T, H) || ((!x || !out8 || !scale) && T) || !matrix_ok(x, dtype, T, ldx, H) || !rows_fit(T, ldo8, H) || !aligned(scale, 4))
    return MOE_EINVAL;
  if (T == 0) return MOE_OK;
  NormArgs n{};
  n.x = x;
  n.ldx = ldx;
  n.x_type = dtype;
  n.out8 = static_cast<uint8_t*>(out8);
  n.ldo8 = ldo8;
  n.scale = scale;
  n.T = T;
  n.H = H;
  BatchDevice d;
  const moe_status st = batch_device(&d);
  if (st != MOE_OK) return st;
  return done(launch_rms_norm(n, d.num_sms, (cudaStream_t)stream));
}

extern "C" size_t moe_rms_norm_backward_workspace(int T, int H) {
  return T < 1 || !length_ok(T, H) ? 0 : (size_t)norm_grad_blocks(T, H) * H * sizeof(float);
}

extern "C" moe_status moe_rms_norm_backward(const moe_rms_norm_grad_args* a, void* stream) {
  if (!a || !length_ok(a->T, a->H) || ((!a->dy || !a->h || !a->rstd || !a->dh) && a->T)) return MOE_EINVAL;
  if (!matrix_ok(a->dy, a->dy_dtype, a->T, a->ld_dy, a->H) || !matrix_ok(a->h, a->h_dtype, a->T, a->ld_h, a->H) ||
      !matrix_ok(a->dh, a->dh_dtype, a->T, a->ld_dh, a->H) || !aligned(a->rstd, 4) || !aligned(a->dgain, 4))
    return MOE_EINVAL;
  if (a->gain && !matrix_ok(a->gain, a->gain_dtype, 1, a->H, a->H)) return MOE_EINVAL;
  if (a->dsum && !matrix_ok(a->dsum, a->dsum_dtype, a->T, a->ld_dsum, a->H)) return MOE_EINVAL;
  const size_t need = a->dgain ? moe_rms_norm_backward_workspace(a->T, a->H) : 0;
  if (!aligned(a->workspace, 16) || (need && (!a->workspace || a->workspace_bytes < need))) return MOE_EINVAL;
  const NormGradArgs g{a->dy, a->h, a->gain, a->dsum, a->rstd, a->dh, a->dgain, static_cast<float*>(a->workspace),
                       a->ld_dy, a->ld_h, a->ld_dsum, a->ld_dh, a->T, a->H, a->dy_dtype, a->h_dtype, a->gain_dtype, a->dsum_dtype,
                       a->dh_dtype};
  BatchDevice d;
  const moe_status st = batch_device(&d);
  if (st != MOE_OK) return st;
  if (a->T == 0) return a->dgain ? done(cudaMemsetAsync(a->dgain, 0, (size_t)a->H * sizeof(float), (cudaStream_t)stream)) : MOE_OK;
  return done(launch_rms_norm_grad(g, d.wait, (cudaStream_t)stream));
}

extern "C" moe_status moe_combine_rows(const moe_combine_args* a, void* stream) {
  if (!a || a->T < 0 || a->k < 1 || a->k > 32 || a->H < 1 || a->H > kMaxColumns || (long long)a->T * a->k > 0x7fffffffLL) return MOE_EINVAL;
  if ((!a->y && a->y_rows != 0) || ((!a->weights || !a->out) && a->T)) return MOE_EINVAL;
  if (!matrix_ok(a->y, a->dtype, a->y_rows, a->ldy, a->H) || !matrix_ok(a->out, a->out_dtype, a->T, a->ldo, a->H)) return MOE_EINVAL;
  if (a->residual && !matrix_ok(a->residual, a->out_dtype, a->T, a->ld_residual, a->H)) return MOE_EINVAL;
  if (!a->places && (long long)a->T * a->k > a->y_rows) return MOE_EINVAL;
  if (!aligned(a->weights, 4) || !aligned(a->places, 4)) return MOE_EINVAL;
  if (a->T == 0) return MOE_OK;
  const CombineRowsArgs c{a->y, a->weights, a->places, a->residual, a->out, a->y_rows, a->ldy, a->ld_residual, a->ldo,
                          a->T, a->k, a->H, a->dtype, a->out_dtype};
  BatchDevice d;
  const moe_status st = batch_device(&d);
  if (st != MOE_OK) return st;
  return done(launch_combine_rows(c, (cudaStream_t)stream));
}

extern "C" moe_status moe_combine_rows_backward(const moe_combine_grad_args* a, void* stream) {
  if (!a || a->T < 0 || a->k < 1 || a->k > 32 || a->H < 1 || a->H > kMaxColumns || (long long)a->T * a->k > 0x7fffffffLL) return MOE_EINVAL;
  if (((!a->y || !a->dy) && a->y_rows != 0) || ((!a->dout || !a->weights || !a->dweights) && a->T)) return MOE_EINVAL;
  if (!matrix_ok(a->dout, a->dout_dtype, a->T, a->ld_dout, a->H) || !matrix_ok(a->y, a->dtype, a->y_rows, a->ldy, a->H) ||
      !matrix_ok(a->dy, a->dtype, a->y_rows, a->ld_dy, a->H))
    return MOE_EINVAL;
  if (!a->places && (long long)a->T * a->k > a->y_rows) return MOE_EINVAL;
  if (!aligned(a->weights, 4) || !aligned(a->places, 4) || !aligned(a->dweights, 4)) return MOE_EINVAL;
  if (a->T == 0) return MOE_OK;
  const CombineGradArgs c{a->dout, a->y, a->weights, a->places, a->dy, a->dweights, a->y_rows, a->ld_dout, a->ldy, a->ld_dy,
                          a->T, a->k, a->H, a->dout_dtype, a->dtype, a->dtype};
  BatchDevice d;
  const moe_status st = batch_device(&d);
  if (st != MOE_OK) return st;
  return done(launch_combine_rows_grad(c, (cudaStream_t)stream));
}
