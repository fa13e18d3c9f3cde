// RMS norm of query and key heads with the position rotation in the same
// pass, and its gradient.
//
//   n = w x r, r = 1 / sqrt(mean(x^2) + eps);  y = R(p) n
// with R(p) turning pair j of the first rot_dim values by p inv_freq[j].
// Gradient: g = R(p)^T dy,  dw = sum g x r,
//           dx = r (w g) - x r^3 mean(w g x).
//
// Bound by HBM: x is read once and y written once.  A head belongs to G lanes
// (the next power of two of headdim / 8), 8 values a lane; the mean closes with
// log2(G) adds across lanes, and the pairs of the half-split rotation come from
// the lane rot_dim / 16 away.  A workgroup takes all heads of one or a few
// steps, so that a step's angles are formed once, by one lane each, and shared
// through LDS by its heads.  Angles are products in 64 bits, reduced to a
// fraction of a turn before they are rounded to fp32 (an fp32 product at
// position 10^6 would be off by 0.06 radians).
#include "ssm_device.h"
#include "ssm_internal.h"

namespace ssm {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint16_t u16x8 __attribute__((ext_vector_type(8)));

struct QkArgs {
  const void* x[2];     // q, k
  const void* dy[2];    // gradient only
  void* y[2];           // outputs, or dq, dk
  const float* w[2];    // nullable
  const float* inv_freq;
  const int64_t* positions;  // nullable
  float* part;          // gradient only, nullable: [2][workgroups][headdim] partial sums of dw
  int64_t xs[2], ys[2];  // elements between steps
  int64_t tokens, seqlen;
  int32_t heads[2];
  int32_t dim, rot, tb;  // tb: steps per workgroup
  float eps;
};

constexpr int kMaxAngles = 1024;  // pairs of one workgroup's steps

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
__device__ __forceinline__ void store8(float* p, const float* v) {
  *reinterpret_cast<f32x4*>(p) = f32x4{v[0], v[1], v[2], v[3]};
  *reinterpret_cast<f32x4*>(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
}
__device__ __forceinline__ void store8(uint16_t* p, const float* v) {
  u16x8 r;
#pragma unroll
  for (int j = 0; j < 8; ++j) r[j] = __builtin_bit_cast(uint16_t, (__bf16)v[j]);
  *reinterpret_cast<u16x8*>(p) = r;
}

template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int d = 1; d < G; d *= 2) v += __shfl_xor(v, d);
  return v;
}

// cos and sin of position * inv_freq, the angle reduced to [-1/2, 1/2] turns in
// 64 bits.
__device__ __forceinline__ float2 turn(int64_t pos, float inv_freq) {
  const double t = (double)pos * (double)inv_freq * 0.15915494309189533577;
  const float f = (float)(t - rint(t));
  float sn, cs;
  sincospif(2.0f * f, &sn, &cs);
  return make_float2(cs, sn);
}

// Angles of steps [t0, t0 + n) into cs (one thread per pair).
__device__ __forceinline__ void fill_angles(const QkArgs& a, int64_t t0, int n, float2* cs) {
  const int half = a.rot / 2;
  for (int i = threadIdx.x; i < n * half; i += 256) {
    const int64_t t = t0 + i / half;
    const int64_t pos = a.positions != nullptr ? a.positions[t] : t % a.seqlen;
    cs[i] = turn(pos, a.inv_freq[i % half]);
  }
}

// Turns this lane's 8 values (elements 8 ln ..) by the step's angles, or back.
// Every lane of the group takes part in the exchange.
template <int G, bool INTER, bool BACK>
__device__ __forceinline__ void rotate8(float* v, const float2* cs, int ln, int rot) {
  if (INTER) {
    if (8 * ln < rot) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 c = cs[4 * ln + j];
        const float sn = BACK ? -c.y : c.y;
        const float x = v[2 * j], y = v[2 * j + 1];
        v[2 * j] = x * c.x - y * sn;
        v[2 * j + 1] = __builtin_fmaf(x, sn, y * c.x);
      }
    }
    return;
  }
  if (rot == 0) return;
  const int hl = rot / 16;  // lanes of half the rotated part
  const bool first = ln < hl, in = ln < 2 * hl;
  const int src = first ? ln + hl : (in ? ln - hl : ln);
  const int base = (threadIdx.x & 63) - ln;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float o = __shfl(v[j], base + src);
    if (in) {
      const float2 c = cs[8 * (first ? ln : ln - hl) + j];
      const float sn = (first != BACK) ? -c.y : c.y;
      v[j] = __builtin_fmaf(o, sn, v[j] * c.x);
    }
  }
}

template <typename T, int G, bool INTER>
__global__ void __launch_bounds__(256) k_qk_norm_rope(const QkArgs a) {
  __shared__ float2 cs[kMaxAngles];
  const int64_t t0 = (int64_t)blockIdx.x * a.tb;
  const int n = (int)min((int64_t)a.tb, a.tokens - t0);
  fill_angles(a, t0, n, cs);
  __syncthreads();
  const int ln = threadIdx.x % G;
  const bool live = 8 * ln < a.dim;
  const float inv_d = 1.0f / (float)a.dim;
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    const int heads = a.heads[side];
    const T* const x = static_cast<const T*>(a.x[side]);
    T* const y = static_cast<T*>(a.y[side]);
    float wv[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) wv[j] = live && a.w[side] != nullptr ? a.w[side][8 * ln + j] : 1.0f;
    // The whole wave walks the same number of rows: the exchanges need it.
    const int rows = n * heads;
    for (int r0 = 0; r0 < rows; r0 += 256 / G) {
      const int r = r0 + threadIdx.x / G;
      const bool on = live && r < rows;
      const int t = r < rows ? r / heads : 0, hd = r < rows ? r % heads : 0;
      float v[8] = {};
      if (on) load8(x + (t0 + t) * a.xs[side] + (int64_t)hd * a.dim + 8 * ln, v);
      float ss = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = __builtin_fmaf(v[j], v[j], ss);
      const float rs = __builtin_amdgcn_rsqf(__builtin_fmaf(group_sum<G>(ss), inv_d, a.eps));
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= rs * wv[j];
      rotate8<G, INTER, false>(v, cs + t * (a.rot / 2), ln, a.rot);
      if (on) store8(y + (t0 + t) * a.ys[side] + (int64_t)hd * a.dim + 8 * ln, v);
    }
  }
}

template <typename T, int G, bool INTER>
__global__ void __launch_bounds__(256) k_qk_norm_rope_bwd(const QkArgs a) {
  __shared__ float2 cs[kMaxAngles];
  __shared__ float sw[256 * 8];
  const int ln = threadIdx.x % G;
  const bool live = 8 * ln < a.dim;
  const float inv_d = 1.0f / (float)a.dim;
  float wv[2][8], dw[2][8] = {};
#pragma unroll
  for (int side = 0; side < 2; ++side)
#pragma unroll
    for (int j = 0; j < 8; ++j) wv[side][j] = live && a.w[side] != nullptr ? a.w[side][8 * ln + j] : 1.0f;
  for (int64_t t0 = (int64_t)blockIdx.x * a.tb; t0 < a.tokens; t0 += (int64_t)gridDim.x * a.tb) {
    const int n = (int)min((int64_t)a.tb, a.tokens - t0);
    __syncthreads();
    fill_angles(a, t0, n, cs);
    __syncthreads();
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      const int heads = a.heads[side];
      const T* const x = static_cast<const T*>(a.x[side]);
      const T* const dy = static_cast<const T*>(a.dy[side]);
      T* const dx = static_cast<T*>(a.y[side]);
      const int rows = n * heads;
      for (int r0 = 0; r0 < rows; r0 += 256 / G) {
        const int r = r0 + threadIdx.x / G;
        const bool on = live && r < rows;
        const int t = r < rows ? r / heads : 0, hd = r < rows ? r % heads : 0;
        float v[8] = {}, g[8] = {};
        if (on) {
          load8(x + (t0 + t) * a.xs[side] + (int64_t)hd * a.dim + 8 * ln, v);
          load8(dy + ((t0 + t) * heads + hd) * a.dim + 8 * ln, g);
        }
        rotate8<G, INTER, true>(g, cs + t * (a.rot / 2), ln, a.rot);
        float ss = 0.f, sg = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          ss = __builtin_fmaf(v[j], v[j], ss);
          sg = __builtin_fmaf(wv[side][j] * g[j], v[j], sg);
        }
        const float rs = __builtin_amdgcn_rsqf(__builtin_fmaf(group_sum<G>(ss), inv_d, a.eps));
        const float c = group_sum<G>(sg) * inv_d * rs * rs;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          // Rows that do not exist leave dw alone (with eps 0 their rs is infinite).
          if (on) dw[side][j] = __builtin_fmaf(g[j], v[j] * rs, dw[side][j]);
          g[j] = rs * (wv[side][j] * g[j] - v[j] * c);
        }
        if (on) store8(dx + ((t0 + t) * heads + hd) * a.dim + 8 * ln, g);
      }
    }
  }
  if (a.part == nullptr) return;
  // The workgroup's sums over its lane groups, in group order.
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) sw[(threadIdx.x / G) * (8 * G) + 8 * ln + j] = dw[side][j];
    __syncthreads();
    if ((int)threadIdx.x < a.dim) {
      float s = 0.f;
      for (int k = 0; k < 256 / G; ++k) s += sw[k * (8 * G) + threadIdx.x];
      a.part[((int64_t)side * gridDim.x + blockIdx.x) * a.dim + threadIdx.x] = s;
    }
  }
}

// dw[side][c] = sum over workgroups: 16 columns per workgroup, 16 interleaved
// partial sums per column, joined in order.
__global__ void __launch_bounds__(256) k_qk_reduce_dw(const float* part, float* dwq, float* dwk, int32_t groups,
                                                      int32_t dim) {
  __shared__ float s[16][17];
  const int side = blockIdx.y;
  float* const dw = side == 0 ? dwq : dwk;
  if (dw == nullptr) return;
  const int c = threadIdx.x & 15, k0 = threadIdx.x >> 4;
  const int col = blockIdx.x * 16 + c;  // dim is a multiple of 16
  const float* p = part + (int64_t)side * groups * dim + col;
  float v = 0.f;
  for (int k = k0; k < groups; k += 16) v += p[(int64_t)k * dim];
  s[k0][c] = v;
  __syncthreads();
  if (k0 == 0) {
    for (int k = 1; k < 16; ++k) v += s[k][c];
    dw[col] = v;
  }
}

// Steps per workgroup: at least ~32 heads of work, as many angles as LDS holds.
int32_t steps_per_group(int64_t heads, int64_t rot) {
  int64_t tb = heads > 0 ? (32 + heads - 1) / heads : 1;
  const int64_t cap = rot > 0 ? kMaxAngles / (rot / 2) : 32;
  if (tb > cap) tb = cap;
  return (int32_t)(tb < 1 ? 1 : tb);
}

constexpr int64_t kBwdGroups = 1024;  // workgroups (and partial sums) of the gradient

QkArgs args(const QkNormRopeLaunch& p) {
  QkArgs a{};
  a.x[0] = p.q;
  a.x[1] = p.k;
  a.y[0] = p.q_out;
  a.y[1] = p.k_out;
  a.w[0] = p.wq;
  a.w[1] = p.wk;
  a.inv_freq = p.inv_freq;
  a.positions = p.positions;
  a.xs[0] = p.q_stride;
  a.xs[1] = p.k_stride;
  a.ys[0] = p.q_out_stride;
  a.ys[1] = p.k_out_stride;
  a.tokens = p.batch * p.seqlen;
  a.seqlen = p.seqlen;
  a.heads[0] = (int32_t)p.nheads;
  a.heads[1] = (int32_t)p.nheads_k;
  a.dim = (int32_t)p.headdim;
  a.rot = (int32_t)p.rot_dim;
  a.tb = steps_per_group(p.nheads + p.nheads_k, p.rot_dim);
  a.eps = p.eps;
  a.dy[0] = p.dq_out;
  a.dy[1] = p.dk_out;
  return a;
}

// Calls f with the kernel's lane group size as a constant.
template <typename F>
hipError_t by_group(int64_t dim, F f) {
  if (dim <= 16) return f(std::integral_constant<int, 2>());
  if (dim <= 32) return f(std::integral_constant<int, 4>());
  if (dim <= 64) return f(std::integral_constant<int, 8>());
  if (dim <= 128) return f(std::integral_constant<int, 16>());
  return f(std::integral_constant<int, 32>());
}

}  // namespace

int64_t qk_norm_rope_blocks(int64_t tokens, int64_t nheads, int64_t nheads_k, int64_t rot_dim) {
  const int64_t tb = steps_per_group(nheads + nheads_k, rot_dim);
  return (tokens + tb - 1) / tb;
}

int64_t qk_norm_rope_bwd_floats(int64_t tokens, int64_t nheads, int64_t nheads_k, int64_t headdim) {
  // The number of workgroups for one step each is the largest.
  const int64_t groups = tokens < kBwdGroups ? tokens : kBwdGroups;
  (void)nheads;
  (void)nheads_k;
  return 2 * groups * headdim;
}

hipError_t launch_qk_norm_rope(const QkNormRopeLaunch& p) {
  const QkArgs a = args(p);
  const unsigned grid = (unsigned)qk_norm_rope_blocks(a.tokens, p.nheads, p.nheads_k, p.rot_dim);
  return by_group(p.headdim, [&](auto g) {
    constexpr int G = decltype(g)::value;
    auto go = [&](auto kern) { return launch(kern, dim3(grid), dim3(256), 0, p.stream, a); };
    if (p.bf16) return p.interleaved ? go(k_qk_norm_rope<uint16_t, G, true>) : go(k_qk_norm_rope<uint16_t, G, false>);
    return p.interleaved ? go(k_qk_norm_rope<float, G, true>) : go(k_qk_norm_rope<float, G, false>);
  });
}

hipError_t launch_qk_norm_rope_bwd(const QkNormRopeLaunch& p) {
  QkArgs a = args(p);
  int64_t groups = qk_norm_rope_blocks(a.tokens, p.nheads, p.nheads_k, p.rot_dim);
  if (groups > kBwdGroups) groups = kBwdGroups;
  const bool want = p.dwq != nullptr || p.dwk != nullptr;
  a.part = want ? p.workspace : nullptr;
  if (groups > 0) {
    const hipError_t rc = by_group(p.headdim, [&](auto g) {
      constexpr int G = decltype(g)::value;
      auto go = [&](auto kern) { return launch(kern, dim3((unsigned)groups), dim3(256), 0, p.stream, a); };
      if (p.bf16)
        return p.interleaved ? go(k_qk_norm_rope_bwd<uint16_t, G, true>) : go(k_qk_norm_rope_bwd<uint16_t, G, false>);
      return p.interleaved ? go(k_qk_norm_rope_bwd<float, G, true>) : go(k_qk_norm_rope_bwd<float, G, false>);
    });
    if (rc != hipSuccess) return rc;
  }
  if (!want) return hipSuccess;
  return launch(k_qk_reduce_dw, dim3((unsigned)(p.headdim / 16), 2), dim3(256), 0, p.stream, p.workspace, p.dwq,
                p.dwk, (int32_t)groups, (int32_t)p.headdim);
}

}  // namespace ssm
