// Shared pieces of the linear attention sweeps (gfx950 only).
//
// Linear attention with a constant decay gamma per head and its three
// gradients are one computation with the operands in different roles:
//   out_t = sum_i gamma^|t - i| (a_t . b_i) c_i   over i <= t, or i >= t in reverse
//             a    b    c
//   o         q    k    v    forward in time
//   dq        do   v    k    forward
//   dk        v    do   q    reverse
//   dv        k    q    do   reverse
// (G_t = gamma G_{t+1} + scale q_t do_t^T is the gradient of the state H_t;
// dk_t = G_t v_t and dv_t = G_t^T k_t read it as o_t = H_t q_t reads H.)
// The state of a sweep is S[n][p] = sum of decayed b_i[n] c_i[p], KD x VD.
//
// A sweep walks blocks of steps [t0, t0 + m).  With j = t - t0 and E the state
// that enters the block:
//   forward: out_t = s_pair (pairs i <= t) + s_read gamma^(j + 1) E^T a_t
//            E' = gamma^m E + s_write sum_i gamma^(m - 1 - j_i) b_i c_i^T
//   reverse: out_t = s_pair (pairs i >= t) + s_read gamma^(m - 1 - j) E^T a_t
//            E' = gamma^m E + s_write sum_i gamma^(j_i + 1) b_i c_i^T
// In reverse, E is gamma times the state gradient behind the block (dh_last at
// the end of the sequence, which no decay separates from the last step), and
// what leaves step 0 is dh0.
#pragma once

#include "ssm_device.h"
#include "attn_launch.h"

namespace ssm {

// One operand: the first step's first head, elements between steps, and how
// many of the nheads sweeps share one of its heads.
struct AttnOperand {
  const void* p;
  int64_t stride;
  int32_t rep;
};

struct AttnSweep {
  AttnOperand a, b, c;
  const float* log_decay;
  const int32_t* lengths;  // nullable
  const float* entry;      // state entering span 0 (the last span in reverse), nullable for zeros; with spans,
                           // span s of row r enters with entry[(s * rows + r) * KD * VD]
  float* exit;             // nullable: state behind the last span (span 0 in reverse); in a summary sweep,
                           // span s of row r leaves exit[(s * rows + r) * KD * VD]
  void* out;               // [batch][seqlen][nheads][VD]
  int64_t sn, sp;          // state element (n, p) at n sn + p sp
  int64_t seqlen, span_len, n_spans;
  int32_t nheads;
  int64_t rows;            // batch * nheads
  float s_pair, s_read, s_write;
};

// The sweeps for bf16 operands (linear_attn_bf16.hip): a forward sweep with bf16
// outputs; the spans' states forwards and (r not NULL) in reverse; the three
// gradient sweeps, dk and dv to fp32 buffers when out32.
hipError_t launch_attn_sweep_bf16(const AttnSweep& s, int64_t kd, int64_t vd, hipStream_t stream);
hipError_t launch_attn_span_states_bf16(const AttnSweep& f, const AttnSweep* r, int64_t kd, int64_t vd,
                                        hipStream_t stream);
hipError_t launch_attn_sweep_grad_bf16(const AttnSweep& q, const AttnSweep& k, const AttnSweep& v, int64_t d_k,
                                       int64_t d_v, bool out32, hipStream_t stream);

// Calls f with the widths (64 or 128) as constants.
template <typename F>
hipError_t by_width(int64_t a, int64_t b, F f) {
  typedef std::integral_constant<int, 64> W64;
  typedef std::integral_constant<int, 128> W128;
  if (a == 64) return b == 64 ? f(W64(), W64()) : f(W64(), W128());
  return b == 64 ? f(W128(), W64()) : f(W128(), W128());
}

// log2(gamma); -inf is kept finite so that 0 steps of decay give 1 (0 * -inf
// would be NaN) and one step or more still gives 0.
__device__ __forceinline__ float decay_log2(float log_decay) {
  const float g = log_decay * kLog2e;
  return g < -1e30f ? -1e30f : g;
}

__device__ __forceinline__ int64_t row_length(const int32_t* lengths, int64_t b, int64_t seqlen) {
  if (lengths == nullptr) return seqlen;
  const int64_t n = lengths[b];
  return n < 0 ? 0 : (n < seqlen ? n : seqlen);
}

}  // namespace ssm
