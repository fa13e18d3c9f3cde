// C ABI of the gated recurrence and of the norms over a layer's width: argument
// checks and dispatch.  Every check runs on the host before any HIP call, so a
// rejected call has no side effects.
#include "ssm_scan.h"
#include "abi_checks.h"
#include "gated_launch.h"

#include <hip/hip_runtime.h>
#include <limits.h>
#include <stdint.h>

namespace {

constexpr int64_t kMaxSteps = INT32_MAX - 256;
constexpr int64_t kMaxWidth = (int64_t)1 << 23;
constexpr int64_t kMaxStep = (int64_t)1 << 40;      // elements between rows
constexpr int64_t kMaxScanStep = (int64_t)1 << 25;  // between steps of a scan, which addresses 16 by 32-bit offsets
constexpr int64_t kMaxStates = (int64_t)1 << 31;
// Every byte count below stays far inside 64 bits when no tensor has more elements than this.
constexpr int64_t kMaxElems = (int64_t)1 << 48;
// Workgroups of 256 threads in a launch: an axis of the grid holds fewer than 2^32 threads.
constexpr int64_t kMaxGroups = ((int64_t)1 << 24) - 1;

bool dtype_ok(int32_t d) { return d == SSM_DTYPE_F32 || d == SSM_DTYPE_BF16; }

// The distance between steps (0: dense), which must keep `rows` of them in range.
int check_step(int64_t* stride, int64_t width, int64_t rows, int64_t most = kMaxStep) {
  if (*stride == 0) *stride = width;
  if (*stride < width || *stride > most) return SSM_ERR_BAD_DIM;
  int64_t n;
  if (__builtin_mul_overflow(rows, *stride, &n) || n > kMaxElems * 16) return SSM_ERR_BAD_DIM;
  return SSM_OK;
}

int check_scan_dims(int64_t batch, int64_t seqlen, int64_t width) {
  if (batch < 0 || seqlen < 0 || width < 0) return SSM_ERR_BAD_DIM;
  if (batch > kMaxElems || seqlen > kMaxSteps || width > kMaxWidth) return SSM_ERR_BAD_DIM;
  int64_t n, st;
  if (!mul3(batch, seqlen, width, &n) || !mul3(batch, width, 1, &st) || n > kMaxElems || st > kMaxStates)
    return SSM_ERR_BAD_DIM;
  int64_t tokens;
  if (!mul3(batch, seqlen, 1, &tokens) || tokens > kMaxElems) return SSM_ERR_BAD_DIM;
  if (ssm::gated_scan_items(batch, seqlen, width) > INT32_MAX) return SSM_ERR_BAD_DIM;
  return SSM_OK;
}

int check_workspace(const void* ws, size_t have, int64_t floats, const Rows* ins, int n_in, const Rows* outs,
                    int n_out) {
  if (floats <= 0) return SSM_OK;
  if (ws == nullptr || have < (size_t)floats * 4) return SSM_ERR_WORKSPACE;
  if (!aligned(ws, kWorkspaceAlign)) return SSM_ERR_MISALIGNED;
  const Rows w = dense(ws, floats * 4);
  int rc = check_alias(&w, 1, ins, n_in);
  return rc != SSM_OK ? rc : check_alias(&w, 1, outs, n_out);
}

// Forward and gradient share their checks.
int gated_scan_impl(ssm::GatedScanLaunch p, int32_t io_dtype, bool grad, size_t workspace_bytes) {
  int rc = check_scan_dims(p.batch, p.seqlen, p.width);
  if (rc != SSM_OK) return rc;
  if (!dtype_ok(io_dtype)) return SSM_ERR_UNSUPPORTED;
  p.bf16 = io_dtype == SSM_DTYPE_BF16;
  const int64_t es = p.bf16 ? 2 : 4, tokens = p.batch * p.seqlen, n = tokens * p.width, states = p.batch * p.width;
  if ((rc = check_step(&p.x_stride, p.width, tokens, kMaxScanStep)) != SSM_OK) return rc;
  if ((rc = check_step(&p.ga_stride, p.width, tokens, kMaxScanStep)) != SSM_OK) return rc;
  if ((rc = check_step(&p.gx_stride, p.width, tokens, kMaxScanStep)) != SSM_OK) return rc;
  if (p.z != nullptr && (rc = check_step(&p.z_stride, p.width, tokens, kMaxScanStep)) != SSM_OK) return rc;

  if (n > 0 && (p.x == nullptr || p.ga == nullptr || p.gx == nullptr)) return SSM_ERR_NULL_ARG;
  if (states > 0 && p.log_a == nullptr) return SSM_ERR_NULL_ARG;
  if (n > 0 && !grad && p.y == nullptr) return SSM_ERR_NULL_ARG;
  if (n > 0 && grad && (p.dy == nullptr || p.dx == nullptr || p.dga == nullptr || p.dgx == nullptr))
    return SSM_ERR_NULL_ARG;
  if (n > 0 && grad && (p.z != nullptr) != (p.dz != nullptr)) return SSM_ERR_NULL_ARG;

  const void* io[] = {p.x, p.ga, p.gx, p.z, p.y, p.dy, p.dx, p.dga, p.dgx, p.dz};
  for (const void* q : io)
    if (!aligned(q, (uintptr_t)es)) return SSM_ERR_MISALIGNED;
  const void* f32[] = {p.log_a, p.lengths, p.h0, p.h_last, p.ckpt, p.dh_last, p.dlog_a, p.dh0};
  for (const void* q : f32)
    if (!aligned(q, 4)) return SSM_ERR_MISALIGNED;

  const int64_t b_row = p.width * es, b_io = n * es, b_st = states * 4;
  const int64_t b_ck = ssm::gated_scan_ckpt_floats(p.batch, p.seqlen, p.width) * 4;
  // h_last may be h0 itself, so h0 is compared apart from the other inputs; the
  // saved states are an output of the forward call and an input of the gradient.
  const Rows ins[] = {Rows{p.x, tokens, b_row, p.x_stride * es},
                      Rows{p.ga, tokens, b_row, p.ga_stride * es},
                      Rows{p.gx, tokens, b_row, p.gx_stride * es},
                      Rows{p.z, tokens, b_row, p.z_stride * es},
                      dense(p.log_a, p.width * 4),
                      dense(p.lengths, p.batch * 4),
                      dense(p.h_last == p.h0 ? nullptr : p.h0, b_st),
                      dense(p.dy, b_io),
                      dense(p.dh_last, b_st),
                      dense(grad ? p.ckpt : nullptr, b_ck)};
  const Rows outs[] = {dense(p.y, b_io),   dense(p.h_last, b_st), dense(grad ? nullptr : p.ckpt, b_ck),
                       dense(p.dx, b_io),  dense(p.dga, b_io),    dense(p.dgx, b_io),
                       dense(p.dz, b_io),  dense(p.dlog_a, p.width * 4),
                       dense(p.dh0, b_st)};
  if ((rc = check_alias(outs, 9, ins, 10)) != SSM_OK) return rc;
  // h_last in place of h0: what else is written must leave it alone.
  const Rows h0 = dense(p.h0, b_st);
  if (p.h_last == p.h0 && (overlap(h0, outs[0]) || overlap(h0, outs[2]))) return SSM_ERR_ALIAS;
  const int64_t floats = grad ? ssm::gated_scan_bwd_floats(p.batch, p.seqlen, p.width, p.bf16, p.ckpt != nullptr)
                              : ssm::gated_scan_fwd_floats(p.batch, p.seqlen, p.width, p.bf16);
  if ((rc = check_workspace(p.workspace, workspace_bytes, floats, ins, 10, outs, 9)) != SSM_OK) return rc;
  if (floats > 0 && overlap(dense(p.workspace, floats * 4), h0)) return SSM_ERR_ALIAS;
  if (p.width == 0 || (p.batch == 0 && !grad)) return SSM_OK;
  const hipError_t err = grad ? ssm::launch_gated_scan_bwd(p) : ssm::launch_gated_scan_fwd(p);
  return err == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

int gated_update_impl(ssm::GatedUpdateLaunch p, int32_t io_dtype) {
  if (p.batch < 0 || p.n_slots < 0 || p.width < 0) return SSM_ERR_BAD_DIM;
  if (p.width > kMaxWidth || p.batch > kMaxSteps || p.n_slots > kMaxSteps) return SSM_ERR_BAD_DIM;
  if (p.slots == nullptr && p.n_slots != p.batch) return SSM_ERR_BAD_DIM;
  if (!dtype_ok(io_dtype)) return SSM_ERR_UNSUPPORTED;
  if (p.batch * ssm::gated_update_tiles(p.width) > kMaxGroups) return SSM_ERR_BAD_DIM;
  p.bf16 = io_dtype == SSM_DTYPE_BF16;
  const int64_t es = p.bf16 ? 2 : 4, n = p.batch * p.width;
  int rc;
  if ((rc = check_step(&p.x_stride, p.width, p.batch)) != SSM_OK) return rc;
  if ((rc = check_step(&p.ga_stride, p.width, p.batch)) != SSM_OK) return rc;
  if ((rc = check_step(&p.gx_stride, p.width, p.batch)) != SSM_OK) return rc;
  if (p.z != nullptr && (rc = check_step(&p.z_stride, p.width, p.batch)) != SSM_OK) return rc;
  if (n > 0 && (p.x == nullptr || p.ga == nullptr || p.gx == nullptr || p.log_a == nullptr || p.y == nullptr))
    return SSM_ERR_NULL_ARG;
  if (n > 0 && p.n_slots > 0 && p.h == nullptr) return SSM_ERR_NULL_ARG;
  const void* io[] = {p.x, p.ga, p.gx, p.z, p.y};
  for (const void* q : io)
    if (!aligned(q, (uintptr_t)es)) return SSM_ERR_MISALIGNED;
  if (!aligned(p.h, 4) || !aligned(p.slots, 4) || !aligned(p.log_a, 4)) return SSM_ERR_MISALIGNED;
  const int64_t b_row = p.width * es;
  const Rows ins[] = {Rows{p.x, p.batch, b_row, p.x_stride * es},   Rows{p.ga, p.batch, b_row, p.ga_stride * es},
                      Rows{p.gx, p.batch, b_row, p.gx_stride * es}, Rows{p.z, p.batch, b_row, p.z_stride * es},
                      dense(p.log_a, p.width * 4),                  dense(p.slots, p.batch * 4)};
  const Rows outs[] = {dense(p.h, p.n_slots * p.width * 4), dense(p.y, n * es)};
  if ((rc = check_alias(outs, 2, ins, 6)) != SSM_OK) return rc;
  if (n == 0) return SSM_OK;
  return ssm::launch_gated_scan_update(p) == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

// Rows of `width` values, `groups` norms a row.
int check_norm_dims(int64_t rows, int64_t width, int64_t groups) {
  if (rows < 0 || width < 0 || groups <= 0 || width > kMaxWidth || groups > kMaxWidth) return SSM_ERR_BAD_DIM;
  int64_t n;
  if (!mul3(rows, width, 1, &n) || n > kMaxElems || rows > kMaxElems) return SSM_ERR_BAD_DIM;
  if (width % groups != 0 || width / groups > ssm::kMaxNormWidth) return SSM_ERR_UNSUPPORTED;
  return SSM_OK;
}

int gated_norm_impl(ssm::GatedNormLaunch p, int32_t gate_first, int32_t io_dtype, bool grad, size_t workspace_bytes) {
  int rc = check_norm_dims(p.rows, p.width, p.groups);
  if (rc != SSM_OK) return rc;
  if (!dtype_ok(io_dtype) || !(p.eps >= 0.f) || (gate_first != 0 && gate_first != 1)) return SSM_ERR_UNSUPPORTED;
  p.gate_first = gate_first == 1;
  p.bf16 = io_dtype == SSM_DTYPE_BF16;
  const int64_t es = p.bf16 ? 2 : 4, n = p.rows * p.width;
  if ((rc = check_step(&p.x_stride, p.width, p.rows)) != SSM_OK) return rc;
  if (p.z != nullptr && (rc = check_step(&p.z_stride, p.width, p.rows)) != SSM_OK) return rc;
  if (n > 0 && (p.x == nullptr || p.y == nullptr || (grad && p.dy == nullptr))) return SSM_ERR_NULL_ARG;
  if (n > 0 && grad && (p.z != nullptr) != (p.dz != nullptr)) return SSM_ERR_NULL_ARG;
  const void* io[] = {p.x, p.z, p.y, p.dy, p.dz};
  for (const void* q : io)
    if (!aligned(q, (uintptr_t)es)) return SSM_ERR_MISALIGNED;
  if (!aligned(p.w, 4) || !aligned(p.dw, 4)) return SSM_ERR_MISALIGNED;
  const bool in_place = !grad && p.y == p.x && p.x_stride == p.width;
  const Rows ins[] = {Rows{in_place ? nullptr : p.x, p.rows, p.width * es, p.x_stride * es},
                      Rows{p.z, p.rows, p.width * es, p.z_stride * es}, dense(p.w, p.width * 4), dense(p.dy, n * es)};
  const Rows outs[] = {dense(p.y, n * es), dense(p.dz, n * es), dense(p.dw, p.width * 4)};
  if ((rc = check_alias(outs, 3, ins, 4)) != SSM_OK) return rc;
  if (grad && p.dw != nullptr) {
    rc = check_workspace(p.workspace, workspace_bytes, ssm::gated_norm_bwd_floats(p.rows, p.width, p.groups), ins, 4,
                         outs, 3);
    if (rc != SSM_OK) return rc;
  }
  if (p.width == 0 || (p.rows == 0 && !grad)) return SSM_OK;
  const hipError_t err = grad ? ssm::launch_gated_norm_bwd(p) : ssm::launch_gated_norm(p);
  return err == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

int residual_norm_impl(ssm::ResidualNormLaunch p, int32_t post_norm, int32_t io_dtype, int32_t res_dtype, bool grad,
                       size_t workspace_bytes) {
  int rc = check_norm_dims(p.rows, p.width, 1);
  if (rc != SSM_OK) return rc;
  if (!dtype_ok(io_dtype) || !dtype_ok(res_dtype) || !(p.eps >= 0.f) || (post_norm != 0 && post_norm != 1))
    return SSM_ERR_UNSUPPORTED;
  p.post_norm = post_norm == 1;
  p.bf16 = io_dtype == SSM_DTYPE_BF16;
  p.res_bf16 = res_dtype == SSM_DTYPE_BF16;
  if (!p.bf16 && p.res_bf16) return SSM_ERR_UNSUPPORTED;
  const int64_t es = p.bf16 ? 2 : 4, er = p.res_bf16 ? 2 : 4, n = p.rows * p.width;
  if ((rc = check_step(&p.x_stride, p.width, p.rows)) != SSM_OK) return rc;
  if (n > 0 && !grad && (p.x == nullptr || p.res_out == nullptr || p.y == nullptr)) return SSM_ERR_NULL_ARG;
  if (n > 0 && grad && (p.residual == nullptr || p.dy == nullptr || p.dx == nullptr)) return SSM_ERR_NULL_ARG;
  // Without the norm of x its gradient does not depend on x.
  if (n > 0 && grad && p.x == nullptr && (p.post_norm || p.dw_post != nullptr)) return SSM_ERR_NULL_ARG;
  const void* io[] = {p.x, p.y, p.dy, p.dx};
  for (const void* q : io)
    if (!aligned(q, (uintptr_t)es)) return SSM_ERR_MISALIGNED;
  const void* rs[] = {p.residual, p.res_out, p.dres_out, p.dres};
  for (const void* q : rs)
    if (!aligned(q, (uintptr_t)er)) return SSM_ERR_MISALIGNED;
  const void* f32[] = {p.w_pre, p.w_post, p.dw_pre, p.dw_post};
  for (const void* q : f32)
    if (!aligned(q, 4)) return SSM_ERR_MISALIGNED;
  const bool in_place = !grad && p.res_out == p.residual;
  const Rows ins[] = {Rows{p.x, p.rows, p.width * es, p.x_stride * es}, dense(in_place ? nullptr : p.residual, n * er),
                      dense(p.w_pre, p.width * 4), dense(p.w_post, p.width * 4), dense(p.dy, n * es),
                      dense(p.dres_out, n * er)};
  const Rows outs[] = {dense(p.res_out, n * er), dense(p.y, n * es),           dense(p.dx, n * es),
                       dense(p.dres, n * er),    dense(p.dw_pre, p.width * 4), dense(p.dw_post, p.width * 4)};
  if ((rc = check_alias(outs, 6, ins, 6)) != SSM_OK) return rc;
  if (grad && (p.dw_pre != nullptr || p.dw_post != nullptr)) {
    rc = check_workspace(p.workspace, workspace_bytes, ssm::residual_norm_bwd_floats(p.rows, p.width), ins, 6, outs,
                         6);
    if (rc != SSM_OK) return rc;
  }
  if (p.width == 0 || (p.rows == 0 && !grad)) return SSM_OK;
  const hipError_t err = grad ? ssm::launch_residual_norm_bwd(p) : ssm::launch_residual_norm(p);
  return err == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

}  // namespace

extern "C" {

int ssm_gated_scan_fwd(const void* x, const void* ga, const void* gx, const float* log_a, const void* z,
                       const int32_t* lengths, const float* h0, void* y, float* h_last, float* ckpt, int64_t batch,
                       int64_t seqlen, int64_t width, int64_t x_stride, int64_t ga_stride, int64_t gx_stride,
                       int64_t z_stride, int32_t io_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  ssm::GatedScanLaunch p{};
  p.x = x;
  p.ga = ga;
  p.gx = gx;
  p.log_a = log_a;
  p.z = z;
  p.lengths = lengths;
  p.h0 = h0;
  p.y = y;
  p.h_last = h_last;
  p.ckpt = ckpt;
  p.batch = batch;
  p.seqlen = seqlen;
  p.width = width;
  p.x_stride = x_stride;
  p.ga_stride = ga_stride;
  p.gx_stride = gx_stride;
  p.z_stride = z_stride;
  p.workspace = static_cast<float*>(workspace);
  p.stream = static_cast<hipStream_t>(stream);
  return gated_scan_impl(p, io_dtype, false, workspace_bytes);
}

size_t ssm_gated_scan_fwd_workspace_size(int64_t batch, int64_t seqlen, int64_t width, int32_t io_dtype) {
  if (check_scan_dims(batch, seqlen, width) != SSM_OK || !dtype_ok(io_dtype)) return (size_t)-1;
  return (size_t)ssm::gated_scan_fwd_floats(batch, seqlen, width, io_dtype == SSM_DTYPE_BF16) * 4;
}

size_t ssm_gated_scan_ckpt_bytes(int64_t batch, int64_t seqlen, int64_t width) {
  if (check_scan_dims(batch, seqlen, width) != SSM_OK) return (size_t)-1;
  return (size_t)ssm::gated_scan_ckpt_floats(batch, seqlen, width) * 4;
}

int ssm_gated_scan_bwd(const void* x, const void* ga, const void* gx, const float* log_a, const void* z,
                       const int32_t* lengths, const float* h0, const void* dy, const float* dh_last,
                       const float* ckpt, void* dx, void* dga, void* dgx, void* dz, float* dlog_a, float* dh0,
                       int64_t batch, int64_t seqlen, int64_t width, int64_t x_stride, int64_t ga_stride,
                       int64_t gx_stride, int64_t z_stride, int32_t io_dtype, void* workspace, size_t workspace_bytes,
                       void* stream) {
  ssm::GatedScanLaunch p{};
  p.x = x;
  p.ga = ga;
  p.gx = gx;
  p.log_a = log_a;
  p.z = z;
  p.lengths = lengths;
  p.h0 = h0;
  p.dy = dy;
  p.dh_last = dh_last;
  p.ckpt = const_cast<float*>(ckpt);
  p.dx = dx;
  p.dga = dga;
  p.dgx = dgx;
  p.dz = dz;
  p.dlog_a = dlog_a;
  p.dh0 = dh0;
  p.batch = batch;
  p.seqlen = seqlen;
  p.width = width;
  p.x_stride = x_stride;
  p.ga_stride = ga_stride;
  p.gx_stride = gx_stride;
  p.z_stride = z_stride;
  p.workspace = static_cast<float*>(workspace);
  p.stream = static_cast<hipStream_t>(stream);
  return gated_scan_impl(p, io_dtype, true, workspace_bytes);
}

size_t ssm_gated_scan_bwd_workspace_size(int64_t batch, int64_t seqlen, int64_t width, int32_t io_dtype,
                                         int32_t ckpt_given) {
  if (check_scan_dims(batch, seqlen, width) != SSM_OK || !dtype_ok(io_dtype)) return (size_t)-1;
  if (ckpt_given != 0 && ckpt_given != 1) return (size_t)-1;
  return (size_t)ssm::gated_scan_bwd_floats(batch, seqlen, width, io_dtype == SSM_DTYPE_BF16, ckpt_given == 1) * 4;
}

int ssm_gated_scan_update(float* h, const int32_t* slots, const void* x, const void* ga, const void* gx,
                          const float* log_a, const void* z, void* y, int64_t batch, int64_t n_slots, int64_t width,
                          int64_t x_stride, int64_t ga_stride, int64_t gx_stride, int64_t z_stride, int32_t io_dtype,
                          void* stream) {
  ssm::GatedUpdateLaunch p{h,       slots,    x,         ga,        gx,       log_a, z,
                           y,       batch,    n_slots,   width,     x_stride, ga_stride, gx_stride,
                           z_stride, false,   static_cast<hipStream_t>(stream)};
  return gated_update_impl(p, io_dtype);
}

int ssm_gated_norm_fwd(const void* x, const void* z, const float* w, void* y, int64_t rows, int64_t width,
                       int64_t groups, int64_t x_stride, int64_t z_stride, float eps, int32_t gate_first,
                       int32_t io_dtype, void* stream) {
  ssm::GatedNormLaunch p{};
  p.x = x;
  p.z = z;
  p.w = w;
  p.y = y;
  p.rows = rows;
  p.width = width;
  p.groups = groups;
  p.x_stride = x_stride;
  p.z_stride = z_stride;
  p.eps = eps;
  p.stream = static_cast<hipStream_t>(stream);
  return gated_norm_impl(p, gate_first, io_dtype, false, 0);
}

int ssm_gated_norm_bwd(const void* x, const void* z, const float* w, const void* dy, void* dx, void* dz, float* dw,
                       int64_t rows, int64_t width, int64_t groups, int64_t x_stride, int64_t z_stride, float eps,
                       int32_t gate_first, int32_t io_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  ssm::GatedNormLaunch p{};
  p.x = x;
  p.z = z;
  p.w = w;
  p.dy = dy;
  p.y = dx;
  p.dz = dz;
  p.dw = dw;
  p.rows = rows;
  p.width = width;
  p.groups = groups;
  p.x_stride = x_stride;
  p.z_stride = z_stride;
  p.eps = eps;
  p.workspace = static_cast<float*>(workspace);
  p.stream = static_cast<hipStream_t>(stream);
  return gated_norm_impl(p, gate_first, io_dtype, true, workspace_bytes);
}

size_t ssm_gated_norm_bwd_workspace_size(int64_t rows, int64_t width, int64_t groups) {
  if (check_norm_dims(rows, width, groups) != SSM_OK) return (size_t)-1;
  return width == 0 ? 0 : (size_t)ssm::gated_norm_bwd_floats(rows, width, groups) * 4;
}

int ssm_residual_norm_fwd(const void* x, const void* residual, const float* w_pre, const float* w_post, void* res_out,
                          void* y, int64_t rows, int64_t width, int64_t x_stride, float alpha, float eps,
                          int32_t post_norm, int32_t io_dtype, int32_t res_dtype, void* stream) {
  ssm::ResidualNormLaunch p{};
  p.x = x;
  p.residual = residual;
  p.w_pre = w_pre;
  p.w_post = w_post;
  p.res_out = res_out;
  p.y = y;
  p.rows = rows;
  p.width = width;
  p.x_stride = x_stride;
  p.alpha = alpha;
  p.eps = eps;
  p.stream = static_cast<hipStream_t>(stream);
  return residual_norm_impl(p, post_norm, io_dtype, res_dtype, false, 0);
}

int ssm_residual_norm_bwd(const void* x, const void* res_out, const float* w_pre, const float* w_post, const void* dy,
                          const void* dres_out, void* dx, void* dres, float* dw_pre, float* dw_post, int64_t rows,
                          int64_t width, int64_t x_stride, float alpha, float eps, int32_t post_norm, int32_t io_dtype,
                          int32_t res_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  ssm::ResidualNormLaunch p{};
  p.x = x;
  p.residual = res_out;
  p.w_pre = w_pre;
  p.w_post = w_post;
  p.dy = dy;
  p.dres_out = dres_out;
  p.dx = dx;
  p.dres = dres;
  p.dw_pre = dw_pre;
  p.dw_post = dw_post;
  p.rows = rows;
  p.width = width;
  p.x_stride = x_stride;
  p.alpha = alpha;
  p.eps = eps;
  p.workspace = static_cast<float*>(workspace);
  p.stream = static_cast<hipStream_t>(stream);
  return residual_norm_impl(p, post_norm, io_dtype, res_dtype, true, workspace_bytes);
}

size_t ssm_residual_norm_bwd_workspace_size(int64_t rows, int64_t width) {
  if (check_norm_dims(rows, width, 1) != SSM_OK) return (size_t)-1;
  return width == 0 ? 0 : (size_t)ssm::residual_norm_bwd_floats(rows, width) * 4;
}

}  // extern "C"
