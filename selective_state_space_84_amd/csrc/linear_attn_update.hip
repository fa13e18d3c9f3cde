// One recurrent step of linear attention (decode): h <- gamma h + v k^T,
// o = scale h q, on the fp32 state h[d_v][d_k] of every (request, head).
//
// Bound by HBM: 8 bytes of state move per state element against ~3 vector
// instructions (233 requests x 32 heads of 128 x 128: 183 us, 5.3 TB/s, where a
// copy reaches 5.1 to 5.3; one request x 16 heads: 3.2 us; with fp32
// operands 196 us).  A state row (d_k floats) belongs to d_k / 8 lanes, 8
// elements (two 16-byte accesses) a lane, so that the row's dot product with q
// closes with 3 or 4 adds across lanes.  One row a lane: four,
// with k and q kept in registers over them, took 196 us there and no less at any
// size tried (1 to 256 requests).
#include "linear_attn.h"

namespace ssm {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint16_t u16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ void load8(const float* p, float* v) {
  const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[j] = a[j];
    v[4 + j] = b[j];
  }
}
__device__ __forceinline__ void load8(const uint16_t* p, float* v) {
  const u16x8 a = *reinterpret_cast<const u16x8*>(p);
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = io_to_f32(a[j]);
}

// State rows of a workgroup: those 256 lanes hold at once.
constexpr int rows_per_group(int d_k) { return 2048 / d_k; }

template <typename T, int DK>
__global__ void __launch_bounds__(256)
k_attn_update(float* __restrict__ h, const int32_t* __restrict__ slots, const T* __restrict__ q,
              const T* __restrict__ k, const T* __restrict__ v, const float* __restrict__ log_decay,
              T* __restrict__ o, int64_t n_slots, int32_t nheads, int32_t rep, int32_t d_v, int64_t qs, int64_t ks,
              int64_t vs, float scale) {
  constexpr int LPR = DK / 8;  // lanes per state row
  const int parts = d_v / rows_per_group(DK);
  const int64_t id = blockIdx.x;
  const int part = (int)(id % parts);
  const int64_t bh = id / parts;
  const int64_t b = bh / nheads;
  const int hd = (int)(bh % nheads);
  const int64_t slot = slots != nullptr ? slots[b] : b;
  const int ln = threadIdx.x % LPR;
  const int r = part * rows_per_group(DK) + threadIdx.x / LPR;
  T* const op = o + bh * d_v + r;
  if (slot < 0 || slot >= n_slots) {
    if (ln == 0) io_store(op, 0.f);
    return;
  }
  float* const hp = h + ((slot * nheads + hd) * d_v + r) * DK + 8 * ln;
  float st[8], kk[8], qq[8];
  load8(hp, st);
  load8(k + b * ks + (hd / rep) * DK + 8 * ln, kk);
  load8(q + b * qs + (int64_t)hd * DK + 8 * ln, qq);
  const float vv = io_to_f32(v[b * vs + (hd / rep) * d_v + r]);
  const float g = hw_exp2(decay_log2(log_decay[hd]));
  float dot = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    st[j] = __builtin_fmaf(g, st[j], vv * kk[j]);
    dot = __builtin_fmaf(st[j], qq[j], dot);
  }
  *reinterpret_cast<f32x4*>(hp) = f32x4{st[0], st[1], st[2], st[3]};
  *reinterpret_cast<f32x4*>(hp + 4) = f32x4{st[4], st[5], st[6], st[7]};
#pragma unroll
  for (int d = 1; d < LPR; d *= 2) dot += __shfl_xor(dot, d);
  if (ln == 0) io_store(op, dot * scale);
}

template <typename T, int DK>
hipError_t go(const LinAttnUpdateLaunch& p) {
  return launch(k_attn_update<T, DK>, dim3((unsigned)linear_attn_update_blocks(p.batch, p.nheads, p.d_k, p.d_v)),
                dim3(256), 0, p.stream, p.h, p.slots, static_cast<const T*>(p.q), static_cast<const T*>(p.k),
                static_cast<const T*>(p.v), p.log_decay, static_cast<T*>(p.o), p.n_slots, (int32_t)p.nheads,
                (int32_t)(p.nheads / p.nheads_kv), (int32_t)p.d_v, p.q_stride, p.k_stride, p.v_stride, p.scale);
}

}  // namespace

int64_t linear_attn_update_blocks(int64_t batch, int64_t nheads, int64_t d_k, int64_t d_v) {
  return batch * nheads * (d_v / rows_per_group((int)d_k));
}

hipError_t launch_linear_attn_update(const LinAttnUpdateLaunch& p) {
  if (p.bf16) return p.d_k == 64 ? go<uint16_t, 64>(p) : go<uint16_t, 128>(p);
  return p.d_k == 64 ? go<float, 64>(p) : go<float, 128>(p);
}

}  // namespace ssm
