// One recurrent step of linear attention (decode): h <- gamma h + v k^T,
// o = scale h q, on the fp32 state h[d_v][d_k] of every (request, head).
//
// Bound by HBM: 8 bytes of state move per state element against ~3 vector
// instructions (233 requests x 32 heads of 128 x 128: 196 us, 5.0 TB/s, where a
// copy reaches 5.1; one request x 16 heads: 3.3 us).  A state row (d_k floats) belongs to d_k / 8 lanes, 8
// elements (two 16-byte accesses) a lane, so that the row's dot product with q
// closes with 3 or 4 adds across lanes; a lane keeps its 8 values of k and q in
// registers over the rows it walks.
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

constexpr int kIters = 4;  // state rows a lane group has in flight

// RPB: state rows per workgroup, a multiple of the rows 256 lanes hold at once.
template <typename T, int DK, int IT>
__global__ void __launch_bounds__(256)
k_attn_update(float* __restrict__ h, const int32_t* __restrict__ slots, const T* __restrict__ q,
              const T* __restrict__ k, const T* __restrict__ v, const float* __restrict__ log_decay,
              T* __restrict__ o, int64_t n_slots, int32_t nheads, int32_t rep, int32_t d_v, int32_t parts,
              int64_t qs, int64_t ks, int64_t vs, float scale) {
  constexpr int LPR = DK / 8;      // lanes per state row
  constexpr int RPI = 256 / LPR;   // rows per pass
  const int64_t id = blockIdx.x;
  const int part = (int)(id % parts);
  const int64_t bh = id / parts;
  const int64_t b = bh / nheads;
  const int hd = (int)(bh % nheads);
  const int64_t slot = slots != nullptr ? slots[b] : b;
  const int ln = threadIdx.x % LPR;
  const int r0 = part * (RPI * IT) + threadIdx.x / LPR;
  T* const ob = o + bh * d_v;
  if (slot < 0 || slot >= n_slots) {
    if (ln == 0) {
#pragma unroll
      for (int it = 0; it < IT; ++it) io_store(ob + r0 + it * RPI, 0.f);
    }
    return;
  }
  float* const hp = h + ((slot * nheads + hd) * d_v + r0) * DK + 8 * ln;
  const T* const vp = v + b * vs + (hd / rep) * d_v + r0;
  float st[IT][8], vv[IT], kk[8], qq[8];
#pragma unroll
  for (int it = 0; it < IT; ++it) load8(hp + it * RPI * DK, st[it]);
  load8(k + b * ks + (hd / rep) * DK + 8 * ln, kk);
  load8(q + b * qs + (int64_t)hd * DK + 8 * ln, qq);
#pragma unroll
  for (int it = 0; it < IT; ++it) vv[it] = io_to_f32(vp[it * RPI]);
  const float g = hw_exp2(decay_log2(log_decay[hd]));
#pragma unroll
  for (int it = 0; it < IT; ++it) {
    float dot = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      st[it][j] = __builtin_fmaf(g, st[it][j], vv[it] * kk[j]);
      dot = __builtin_fmaf(st[it][j], qq[j], dot);
    }
    float* const sp = hp + it * RPI * DK;
    *reinterpret_cast<f32x4*>(sp) = f32x4{st[it][0], st[it][1], st[it][2], st[it][3]};
    *reinterpret_cast<f32x4*>(sp + 4) = f32x4{st[it][4], st[it][5], st[it][6], st[it][7]};
#pragma unroll
    for (int d = 1; d < LPR; d *= 2) dot += __shfl_xor(dot, d);
    if (ln == 0) io_store(ob + r0 + it * RPI, dot * scale);
  }
}

// State rows a workgroup walks in one pass per iteration: 256 / (d_k / 8).
int64_t update_parts(int64_t d_k, int64_t d_v, int it) { return d_v / (2048 / d_k * it); }

// Four rows per lane group where that still leaves every CU several
// workgroups; one row otherwise (latency).
int update_iters(int64_t batch, int64_t nheads, int64_t d_k, int64_t d_v) {
  int it = kIters;
  while (it > 1 && (d_v % (2048 / d_k * it) != 0 || batch * nheads * update_parts(d_k, d_v, it) < 1024)) it /= 2;
  return it;
}

template <typename T, int DK>
hipError_t go(const LinAttnUpdateLaunch& p) {
  const int it = update_iters(p.batch, p.nheads, p.d_k, p.d_v);
  const int64_t parts = update_parts(p.d_k, p.d_v, it);
  auto run = [&](auto kern) {
    return launch(kern, dim3((unsigned)(p.batch * p.nheads * parts)), dim3(256), 0, p.stream, p.h, p.slots,
                  static_cast<const T*>(p.q), static_cast<const T*>(p.k), static_cast<const T*>(p.v), p.log_decay,
                  static_cast<T*>(p.o), p.n_slots, (int32_t)p.nheads, (int32_t)(p.nheads / p.nheads_kv),
                  (int32_t)p.d_v, (int32_t)parts, p.q_stride, p.k_stride, p.v_stride, p.scale);
  };
  if (it == 4) return run(k_attn_update<T, DK, 4>);
  if (it == 2) return run(k_attn_update<T, DK, 2>);
  return run(k_attn_update<T, DK, 1>);
}

}  // namespace

int64_t linear_attn_update_blocks(int64_t batch, int64_t nheads, int64_t d_k, int64_t d_v) {
  return batch * nheads * update_parts(d_k, d_v, update_iters(batch, nheads, d_k, d_v));
}

hipError_t launch_linear_attn_update(const LinAttnUpdateLaunch& p) {
  if (p.bf16) return p.d_k == 64 ? go<uint16_t, 64>(p) : go<uint16_t, 128>(p);
  return p.d_k == 64 ? go<float, 64>(p) : go<float, 128>(p);
}

}  // namespace ssm
