// Host-side launch descriptions of the gated recurrence and of the norms over
// a layer's width.
#pragma once
#include "ssm_internal.h"

namespace ssm {

// Gated recurrence.  Strides are elements between consecutive steps.
struct GatedScanLaunch {
  const void* x;
  const void* ga;
  const void* gx;
  const float* log_a;
  const void* z;           // nullable
  const int32_t* lengths;  // nullable
  const float* h0;         // nullable, [batch][width]
  void* y;
  float* h_last;           // nullable
  float* ckpt;             // nullable: states before every kGatedCkpt-th step; the gradient reads them
  int64_t batch, seqlen, width;
  int64_t x_stride, ga_stride, gx_stride, z_stride;
  bool bf16;
  float* workspace;
  hipStream_t stream;
  // Gradient only.
  const void* dy;
  const float* dh_last;  // nullable
  void* dx;
  void* dga;
  void* dgx;
  void* dz;       // with z
  float* dlog_a;  // nullable
  float* dh0;     // nullable
};
constexpr int kGatedCkpt = 64;  // steps between saved states, [batch][steps / kGatedCkpt, rounded up][width]
// Floats of workspace and of saved states; sizes must have been checked for overflow.
int64_t gated_scan_items(int64_t batch, int64_t seqlen, int64_t width);  // pieces of work, at most
int64_t gated_scan_ckpt_floats(int64_t batch, int64_t seqlen, int64_t width);
int64_t gated_scan_fwd_floats(int64_t batch, int64_t seqlen, int64_t width, bool bf16);
int64_t gated_scan_bwd_floats(int64_t batch, int64_t seqlen, int64_t width, bool bf16, bool ckpt_given);
hipError_t launch_gated_scan_fwd(const GatedScanLaunch& p);
hipError_t launch_gated_scan_bwd(const GatedScanLaunch& p);

struct GatedUpdateLaunch {
  float* h;
  const int32_t* slots;  // nullable
  const void* x;
  const void* ga;
  const void* gx;
  const float* log_a;
  const void* z;  // nullable
  void* y;
  int64_t batch, n_slots, width;
  int64_t x_stride, ga_stride, gx_stride, z_stride;
  bool bf16;
  hipStream_t stream;
};
int64_t gated_update_tiles(int64_t width);  // workgroups a request, at most
hipError_t launch_gated_scan_update(const GatedUpdateLaunch& p);

// Group RMS norm with a SiLU gate (gradient when dy is used: y, dz receive dx, dz).
struct GatedNormLaunch {
  const void* x;
  const void* z;   // nullable
  const float* w;  // nullable
  void* y;
  int64_t rows, width, groups;
  int64_t x_stride, z_stride;
  float eps;
  bool gate_first;
  bool bf16;
  hipStream_t stream;
  const void* dy;
  void* dz;
  float* dw;  // nullable
  float* workspace;
};
// Residual update with the norm of what is added and of the sum (gradient when dy is used).
struct ResidualNormLaunch {
  const void* x;
  const void* residual;  // nullable; the gradient reads res_out
  const float* w_pre;    // nullable
  const float* w_post;   // nullable
  void* res_out;
  void* y;
  int64_t rows, width, x_stride;
  float alpha, eps;
  bool post_norm;
  bool bf16, res_bf16;
  hipStream_t stream;
  const void* dy;
  const void* dres_out;  // nullable
  void* dx;
  void* dres;      // nullable
  float* dw_pre;   // nullable
  float* dw_post;  // nullable
  float* workspace;
};
constexpr int64_t kMaxNormWidth = 16384;  // values of one group
int64_t gated_norm_bwd_floats(int64_t rows, int64_t width, int64_t groups);
int64_t residual_norm_bwd_floats(int64_t rows, int64_t width);
hipError_t launch_gated_norm(const GatedNormLaunch& p);
hipError_t launch_gated_norm_bwd(const GatedNormLaunch& p);
hipError_t launch_residual_norm(const ResidualNormLaunch& p);
hipError_t launch_residual_norm_bwd(const ResidualNormLaunch& p);

}  // namespace ssm
