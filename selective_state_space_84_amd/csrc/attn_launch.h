// Host-side launch descriptions of the linear attention and of the query/key
// norm with rotation.
#pragma once
#include "ssm_internal.h"

namespace ssm {

// Linear attention with a constant decay per head.  Strides are elements
// between consecutive steps.
struct LinAttnLaunch {
  const void* q;
  const void* k;
  const void* v;
  const float* log_decay;
  const int32_t* lengths;  // nullable
  const float* h0;         // nullable, [batch][nheads][d_v][d_k]
  void* o;
  float* h_last;           // nullable
  int64_t batch, seqlen, nheads, nheads_kv, d_k, d_v;
  int64_t q_stride, k_stride, v_stride;
  float scale;
  bool bf16;
  float* workspace;
  hipStream_t stream;
  // Gradient only.
  const void* d_o;
  const float* dh_last;  // nullable
  void* dq;
  void* dk;
  void* dv;
  float* dh0;  // nullable
};

// The sequence is cut into n_spans spans of span_len steps when the (row,
// head) pairs alone leave the chip idle.
struct LinAttnPlan {
  int64_t span_len;
  int64_t n_spans;
};
LinAttnPlan linear_attn_plan(int64_t batch, int64_t seqlen, int64_t nheads, int64_t d_k, int64_t d_v, bool bf16,
                             bool grad);
// Workgroups of the widest launch for every span, and threads of the sum over shared heads (0: none).
int64_t linear_attn_groups(int64_t batch, int64_t nheads, int64_t d_k, int64_t d_v, bool bf16, bool grad);
int64_t linear_attn_sum_threads(int64_t batch, int64_t seqlen, int64_t nheads_kv, int64_t d_k, int64_t d_v);
// Floats of workspace; sizes must have been checked for overflow.
int64_t linear_attn_fwd_floats(int64_t batch, int64_t seqlen, int64_t nheads, int64_t d_k, int64_t d_v, bool bf16);
int64_t linear_attn_bwd_floats(int64_t batch, int64_t seqlen, int64_t nheads, int64_t nheads_kv, int64_t d_k,
                               int64_t d_v, bool bf16);
hipError_t launch_linear_attn_fwd(const LinAttnLaunch& p);
hipError_t launch_linear_attn_bwd(const LinAttnLaunch& p);

struct LinAttnUpdateLaunch {
  float* h;
  const int32_t* slots;  // nullable
  const void* q;
  const void* k;
  const void* v;
  const float* log_decay;
  void* o;
  int64_t batch, n_slots, nheads, nheads_kv, d_k, d_v;
  int64_t q_stride, k_stride, v_stride;
  float scale;
  bool bf16;
  hipStream_t stream;
};
int64_t linear_attn_update_blocks(int64_t batch, int64_t nheads, int64_t d_k, int64_t d_v);
hipError_t launch_linear_attn_update(const LinAttnUpdateLaunch& p);

// Norm and rotation of queries and keys (gradient when dq_out / dk_out are used).
struct QkNormRopeLaunch {
  const void* q;
  const void* k;
  const float* wq;  // nullable
  const float* wk;  // nullable
  const float* inv_freq;
  const int64_t* positions;  // nullable
  void* q_out;
  void* k_out;
  int64_t batch, seqlen, nheads, nheads_k, headdim, rot_dim;
  int64_t q_stride, k_stride, q_out_stride, k_out_stride;
  float eps;
  bool interleaved;
  bool bf16;
  hipStream_t stream;
  // Gradient only: q_out, k_out receive dq, dk.
  const void* dq_out;
  const void* dk_out;
  float* dwq;  // nullable
  float* dwk;  // nullable
  float* workspace;
};
int64_t qk_norm_rope_bwd_floats(int64_t tokens, int64_t headdim);
int64_t qk_norm_rope_groups(const QkNormRopeLaunch& p);  // workgroups of the forward launch
hipError_t launch_qk_norm_rope(const QkNormRopeLaunch& p);
hipError_t launch_qk_norm_rope_bwd(const QkNormRopeLaunch& p);

}  // namespace ssm
