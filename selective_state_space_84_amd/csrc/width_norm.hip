// Norms over a layer's width: the gated norm behind a mixer, the residual update
// with the norms before and after a block, and their gradients.
//
//   gated norm:    t = x s(z), y = w t r;  or t = x, y = w t r s(z)
//   residual norm: n = w_post x r_x (or w_post x), R = residual + alpha n, y = w_pre R r_R
// with s(z) = z / (1 + e^-z) and r = 1 / sqrt(mean(t^2) + eps) over a group.
// Gradient of n = w t r:  dt = r (w g) - t r^3 mean(w g t),  dw = sum g t r.
//
// A group of values belongs to a team of lanes that holds it in registers, 8 or 16 values a lane: 8, 16, 32 or 64
// lanes of a wave, or a whole workgroup whose size follows the group.  Every value is read once, all
// sums over a row close together (one barrier where the team is a workgroup), and a gradient's team adds up
// its rows' weight gradients in registers.
//
// Bound by HBM (a copy reaches 5.1 to 5.3 TB/s): the gated norm of 32768 rows of 5120 in bf16 takes 174 us, 5.8
// TB/s; its gradient over 8 groups of 512 in 16384 rows 122 us, 5.5 TB/s; the residual norm of 32768 x 2560 with
// an fp32 stream 181 us, 5.6 TB/s (bf16: 120, 5.6); its gradient of 16384 x 2560 143 us, 5.3 TB/s (bf16: 95, 5.3).
// Groups that are not whole 16-byte pieces are read value by value (gradient of 8192 x 2501: 93 us, 4.0 TB/s).  All
// figures of this file with outputs that go to other memory from pass to pass: written over the same 250 MB, which the
// last-level cache partly holds, that gradient takes 130 us.
#include "col_sum.h"
#include "gated_launch.h"
#include "ssm_device.h"

namespace ssm {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// With bf16 values the gated norm and both gradients take the rows that they read, and bf16 rows that they write, as
// data used once, which the caches need not keep: gated norm of 32768 x 5120 185 -> 174 us, its gradient over 8 groups
// of 512 in 16384 rows 128 -> 125, the residual norm's of 16384 x 2560 with an fp32 stream 147 -> 143.  Not so
// weights, fp32 values (gated gradient of 8192 x 4096 130 -> 149) and the residual update (32768 x 2560 with an fp32
// stream 181 -> 189).
template <typename T>
constexpr bool kOnce = sizeof(T) == 2;
template <bool ONCE, typename P>
__device__ __forceinline__ P fetch(const P* p) {
  return ONCE ? __builtin_nontemporal_load(p) : *p;
}
template <bool ONCE, typename P>
__device__ __forceinline__ void leave(P* p, P v) {
  if constexpr (ONCE)
    __builtin_nontemporal_store(v, p);
  else
    *p = v;
}

// Eight values of one lane.  VEC: neighbours, in 16-byte accesses.  Else: one by one,
// `step` apart, so that the lanes of a team read neighbours; those from `left`
// on do not exist.
template <typename T, bool VEC>
struct Eight;
template <>
struct Eight<float, true> {
  u32x4 a[2];
  __device__ __forceinline__ void zero() { a[0] = a[1] = u32x4{0, 0, 0, 0}; }
  template <bool ONCE>
  __device__ __forceinline__ void load(const float* p, int, int) {
    a[0] = fetch<ONCE>(reinterpret_cast<const u32x4*>(p));
    a[1] = fetch<ONCE>(reinterpret_cast<const u32x4*>(p + 4));
  }
  __device__ __forceinline__ float get(int j) const {
    const uint32_t v = a[j / 4][j % 4];
    return __builtin_bit_cast(float, v);
  }
  __device__ __forceinline__ void forget() {}
};
template <>
struct Eight<uint16_t, true> {
  u32x4 a;
  __device__ __forceinline__ void zero() { a = u32x4{0, 0, 0, 0}; }
  template <bool ONCE>
  __device__ __forceinline__ void load(const uint16_t* p, int, int) {
    a = fetch<ONCE>(reinterpret_cast<const u32x4*>(p));
  }
  __device__ __forceinline__ float get(int j) const {
    const uint32_t v = a[j / 2];
    return __builtin_bit_cast(float, j % 2 ? v & 0xffff0000u : v << 16);
  }
  // What was derived from the values so far is formed again, not held.
  __device__ __forceinline__ void forget() { asm volatile("" : "+v"(a)); }
};
template <typename T>
struct Eight<T, false> {
  T a[8];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int j = 0; j < 8; ++j) a[j] = T(0);
  }
  template <bool ONCE>
  __device__ __forceinline__ void load(const T* p, int step, int left) {
#pragma unroll
    for (int j = 0; j < 8; ++j) a[j] = j * step < left ? p[j * step] : T(0);
  }
  __device__ __forceinline__ float get(int j) const { return io_to_f32(a[j]); }
  __device__ __forceinline__ void forget() {}
};

template <bool VEC, bool ONCE>
__device__ __forceinline__ void put8(float* p, const float* v, int step, int left) {
  if constexpr (VEC) {
    leave<ONCE>(reinterpret_cast<f32x4*>(p), f32x4{v[0], v[1], v[2], v[3]});
    leave<ONCE>(reinterpret_cast<f32x4*>(p + 4), f32x4{v[4], v[5], v[6], v[7]});
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j * step < left) p[j * step] = v[j];
  }
}
template <bool VEC, bool ONCE>
__device__ __forceinline__ void put8(uint16_t* p, const float* v, int step, int left) {
  if constexpr (VEC) {
    u32x4 r;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      r[k] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{v[2 * k], v[2 * k + 1]}, bf16x2));
    leave<ONCE>(reinterpret_cast<u32x4*>(p), r);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j * step < left) io_store(p + j * step, v[j]);
  }
}

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}

// Sum over aligned groups of G lanes (8 at least), in every lane.
template <int G>
__device__ __forceinline__ float lane_sum(float v) {
  v += dpp<0xB1>(v);              // quad_perm 1 0 3 2
  v += dpp<0x4E>(v);              // quad_perm 2 3 0 1
  v += dpp<0x141>(v);             // row_half_mirror
  if (G > 8) v += dpp<0x140>(v);  // row_mirror
  if (G > 16) v += __shfl_xor(v, 16);
  if (G > 32) v += __shfl_xor(v, 32);
  return v;
}

// Sums of squares, and of products of two values, go over the team as 1/64 of what a lane's 8 or 16 values add up to:
// those of 16384 values up to 10^18 stay in fp32's range, and a power of two rounds nothing, put back with the
// mean (one product a lane and row).
constexpr float kShare = 1.0f / 64, kWhole = 64.0f;

// A lane's place: TEAM lanes a group (0: the whole workgroup), NV pieces of 8
// values a lane.  Team q of all takes group q % groups of rows q / groups,
// q / groups + dr, ...
constexpr int kMaxWaves = 16, kMaxSums = 8;
template <int TEAM, int NV, bool VEC>
struct Place {
  int lanes, ln, dim;  // lanes of the team, this one, values of a group
  int64_t team, row, dr, col;  // col: the group's first value in its row
  int phase = 0;
  float (*red)[kMaxWaves][kMaxSums];
  __device__ __forceinline__ Place(int dim_, int64_t groups, float (*red_)[kMaxWaves][kMaxSums])
      : dim(dim_), red(red_) {
    lanes = TEAM > 0 ? TEAM : (int)blockDim.x;
    ln = TEAM > 0 ? (int)threadIdx.x % (TEAM > 0 ? TEAM : 1) : (int)threadIdx.x;
    const int per = TEAM > 0 ? (int)blockDim.x / (TEAM > 0 ? TEAM : 1) : 1;
    team = (int64_t)blockIdx.x * per + (TEAM > 0 ? (int)threadIdx.x / (TEAM > 0 ? TEAM : 1) : 0);
    row = team / groups;
    col = (team % groups) * dim;
    dr = (int64_t)gridDim.x * per / groups;
  }
  // Piece v: its first value within the group, the values' distance, and how many of the group are left from there.
  __device__ __forceinline__ int at(int v) const { return VEC ? (v * lanes + ln) * 8 : v * 8 * lanes + ln; }
  __device__ __forceinline__ int step() const { return VEC ? 1 : lanes; }
  __device__ __forceinline__ int left(int v) const { return dim - at(v); }
  template <bool ONCE, typename E, typename T>
  __device__ __forceinline__ void load(E& e, const T* p, int v) const {
    if (left(v) > 0)
      e.template load<ONCE>(p + at(v), step(), left(v));
    else
      e.zero();
  }
  template <bool ONCE, typename T>
  __device__ __forceinline__ void store(T* p, const float* x, int v) const {
    if (left(v) > 0) put8<VEC, ONCE>(p + at(v), x, step(), left(v));
  }
  __device__ __forceinline__ void weight(float (&w)[8], const float* p, int v) const {
    Eight<float, VEC> e;
    if (p != nullptr) load<false>(e, p + col, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = p != nullptr ? e.get(j) : 1.0f;
  }
  __device__ __forceinline__ void weights(float (&w)[NV][8], const float* p) const {
#pragma unroll
    for (int v = 0; v < NV; ++v) weight(w[v], p, v);
  }
  // The first N sums over the team, in every lane of it.  The waves' sums change places between
  // two halves, so that one barrier a call is enough.
  template <int N, int M>
  __device__ __forceinline__ void sums(float (&x)[M]) {
    constexpr int W = TEAM > 0 ? TEAM : 64;
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = lane_sum<W>(x[i]);
    if constexpr (TEAM == 0) {
      float(*const r)[kMaxSums] = red[phase];
      phase ^= 1;
      if (threadIdx.x % 64 == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) r[threadIdx.x / 64][i] = x[i];
      __syncthreads();
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] = 0.0f;
      for (int w = 0; w < (int)blockDim.x / 64; ++w)
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] += r[w][i];
    }
  }
  __device__ __forceinline__ float sum(float v) {
    float x[1] = {v};
    sums<1>(x);
    return x[0];
  }
};

struct NormArgs {
  const void* x;
  const void* z;
  const float* w;
  void* y;
  int64_t rows, width, groups, xs, zs;
  float eps;
  const void* dy;
  void* dz;
  float* part;
};

template <typename T, bool VEC, int TEAM, int NV, bool Z, bool FIRST>
__global__ void __launch_bounds__(TEAM > 0 ? 256 : 1024) k_gated_norm(const NormArgs a) {
  __shared__ __align__(16) float red[2][kMaxWaves][kMaxSums];
  Place<TEAM, NV, VEC> at((int)(a.width / a.groups), a.groups, red);
  const float inv = 1.0f / (float)at.dim;
  float w[NV][8];
  at.weights(w, a.w);
  for (int64_t r = at.row; r < a.rows; r += at.dr) {
    const T* const xp = static_cast<const T*>(a.x) + r * a.xs + at.col;
    const T* const zp = static_cast<const T*>(a.z) + r * a.zs + at.col;
    Eight<T, VEC> x[NV], z[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      at.template load<kOnce<T>>(x[v], xp, v);
      if (Z) at.template load<kOnce<T>>(z[v], zp, v);
    }
    float t[NV][8], ss = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        t[v][j] = x[v].get(j);
        if (Z && FIRST) t[v][j] *= silu(z[v].get(j));
        ss = __builtin_fmaf(t[v][j], t[v][j], ss);
      }
    const float rs = __builtin_amdgcn_rsqf(__builtin_fmaf(at.sum(kShare * ss), kWhole * inv, a.eps));
    T* const yp = static_cast<T*>(a.y) + r * a.width + at.col;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        t[v][j] *= rs * w[v][j];
        if (Z && !FIRST) t[v][j] *= silu(z[v].get(j));
      }
      at.template store<kOnce<T>>(yp, t[v], v);
    }
  }
}

// rs, and what turns w g into the gradient of t.  ss: kShare of the sum of squares.
struct NormGrad {
  float rs, c;
  __device__ __forceinline__ void take(float ss, float sg, float inv, float eps) {
    rs = __builtin_amdgcn_rsqf(__builtin_fmaf(ss, kWhole * inv, eps));
    c = sg * inv * rs * rs;
  }
  __device__ __forceinline__ float operator()(float t, float wg) const { return rs * __builtin_fmaf(-t, c, wg); }
};

// This lane's weights in the gradients, whose registers go to the sums and to the next row's values: in LDS
// (32 bytes a lane and weight), or, with two pieces a lane, read again for every row.
template <int NV, typename P>
struct Kept {
  const P& at;
  const float* w;
  float* lds;
  __device__ __forceinline__ Kept(const P& at_, const float* w_, float* lds_)
      : at(at_), w(w_), lds(lds_ + 4 * threadIdx.x) {
    if (NV > 1) return;
    float v[NV][8];
    at.weights(v, w);
    *reinterpret_cast<f32x4*>(lds) = f32x4{v[0][0], v[0][1], v[0][2], v[0][3]};
    *reinterpret_cast<f32x4*>(lds + 4 * blockDim.x) = f32x4{v[0][4], v[0][5], v[0][6], v[0][7]};
  }
  __device__ __forceinline__ void get(float (&v)[8], int k) const {
    if (NV > 1) {
      at.weight(v, w, k);
      return;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const f32x4 q = *reinterpret_cast<const f32x4*>(lds + 4 * i * blockDim.x);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[4 * i + j] = q[j];
    }
  }
};
constexpr int kKeptBytes = 32;

// What the gated norm's gradient reads of a row.
template <typename T, bool VEC, int NV, bool Z>
struct GatedRow {
  Eight<T, VEC> x[NV], z[NV], dy[NV];
  template <typename P>
  __device__ __forceinline__ void load(const NormArgs& a, const P& at, int64_t r) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      at.template load<kOnce<T>>(x[v], static_cast<const T*>(a.x) + r * a.xs + at.col, v);
      if (Z) at.template load<kOnce<T>>(z[v], static_cast<const T*>(a.z) + r * a.zs + at.col, v);
      at.template load<kOnce<T>>(dy[v], static_cast<const T*>(a.dy) + r * a.width + at.col, v);
    }
  }
};

template <typename T, bool VEC, int TEAM, int NV, bool Z, bool FIRST>
__global__ void __launch_bounds__(TEAM > 0 ? 256 : 1024) k_gated_norm_bwd(const NormArgs a) {
  __shared__ __align__(16) float red[2][kMaxWaves][kMaxSums];
  extern __shared__ __align__(16) float lds[];
  Place<TEAM, NV, VEC> at((int)(a.width / a.groups), a.groups, red);
  const float inv = 1.0f / (float)at.dim;
  const Kept<NV, Place<TEAM, NV, VEC>> kept(at, a.w, lds);
  float dw[NV][8] = {};
  for (int64_t r = at.row; r < a.rows; r += at.dr) {
    GatedRow<T, VEC, NV, Z> now;
    now.load(a, at, r);
    float s[2] = {};
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float w[8];
      kept.get(w, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float t = now.x[v].get(j), g = now.dy[v].get(j);
        if (Z) (FIRST ? t : g) *= silu(now.z[v].get(j));
        s[0] = __builtin_fmaf(t, t, s[0]);
        s[1] = __builtin_fmaf(w[j] * g, t, s[1]);
      }
    }
    s[0] *= kShare;
    at.template sums<2>(s);
    NormGrad n;
    n.take(s[0], s[1], inv, a.eps);
    T* const dx = static_cast<T*>(a.y) + r * a.width + at.col;
    T* const dz = static_cast<T*>(a.dz) + r * a.width + at.col;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float w[8], ox[8], oz[8];
      kept.get(w, v);
      now.x[v].forget();
      now.z[v].forget();
      now.dy[v].forget();
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float xv = now.x[v].get(j), dv = now.dy[v].get(j);
        if (Z) {
          const float zv = now.z[v].get(j), q = hw_rcp(1.0f + hw_exp2(-zv * kLog2e));
          const float s = zv * q, slope = q * __builtin_fmaf(zv, 1.0f - q, 1.0f);
          const float t = FIRST ? xv * s : xv, g = FIRST ? dv : dv * s;
          const float dt = n(t, w[j] * g);
          dw[v][j] = __builtin_fmaf(g * t, n.rs, dw[v][j]);
          ox[j] = FIRST ? dt * s : dt;
          oz[j] = (FIRST ? dt * xv : dv * (w[j] * (t * n.rs))) * slope;
        } else {
          dw[v][j] = __builtin_fmaf(dv * xv, n.rs, dw[v][j]);
          ox[j] = n(xv, w[j] * dv);
        }
      }
      at.template store<kOnce<T>>(dx, ox, v);
      if (Z) at.template store<kOnce<T>>(dz, oz, v);
    }
  }
  if (a.part == nullptr || at.row >= a.rows) return;
#pragma unroll
  for (int v = 0; v < NV; ++v) at.template store<false>(a.part + at.team * at.dim, dw[v], v);
}

struct ResArgs {
  const void* x;
  const void* res;
  const float* w_pre;
  const float* w_post;
  void* res_out;
  void* y;
  int64_t rows, width, xs;
  float alpha, eps;
  const void* dy;
  const void* dres_out;
  void* dx;
  void* dres;
  float* part;
  int64_t part_post;  // floats before the sums of dw_post
};

template <typename T, typename R, bool VEC, int TEAM, int NV, bool POST>
__global__ void __launch_bounds__(TEAM > 0 ? 256 : 1024) k_residual_norm(const ResArgs a) {
  __shared__ __align__(16) float red[2][kMaxWaves][kMaxSums];
  Place<TEAM, NV, VEC> at((int)a.width, 1, red);
  const float inv = 1.0f / (float)at.dim;
  float wo[NV][8], wp[NV][8];
  at.weights(wo, a.w_post);
  at.weights(wp, a.w_pre);
  for (int64_t r = at.row; r < a.rows; r += at.dr) {
    Eight<T, VEC> x[NV];
    Eight<R, VEC> e[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      at.template load<false>(x[v], static_cast<const T*>(a.x) + r * a.xs, v);
      if (a.res != nullptr)
        at.template load<false>(e[v], static_cast<const R*>(a.res) + r * a.width, v);
      else
        e[v].zero();
    }
    float c = a.alpha;
    if (POST) {
      float ss = 0.0f;
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = __builtin_fmaf(x[v].get(j), x[v].get(j), ss);
      c *= __builtin_amdgcn_rsqf(__builtin_fmaf(at.sum(kShare * ss), kWhole * inv, a.eps));
    }
    float t[NV][8], ss = 0.0f;
    R* const rp = static_cast<R*>(a.res_out) + r * a.width;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        t[v][j] = __builtin_fmaf(c * x[v].get(j), wo[v][j], e[v].get(j));
        // Behind the group there are only zeros (with weights of 1): they add nothing.
        ss = __builtin_fmaf(t[v][j], t[v][j], ss);
      }
      at.template store<false>(rp, t[v], v);
    }
    const float rs = __builtin_amdgcn_rsqf(__builtin_fmaf(at.sum(kShare * ss), kWhole * inv, a.eps));
#pragma unroll
    for (int v = 0; v < NV; ++v) {
#pragma unroll
      for (int j = 0; j < 8; ++j) t[v][j] *= rs * wp[v][j];
      at.template store<false>(static_cast<T*>(a.y) + r * a.width, t[v], v);
    }
  }
}

// What the residual norm's gradient reads of a row.
template <typename T, typename R, bool VEC, int NV>
struct ResRow {
  Eight<T, VEC> x[NV], dy[NV];
  Eight<R, VEC> e[NV], de[NV];
  template <typename P>
  __device__ __forceinline__ void load(const ResArgs& a, const P& at, int64_t r) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      x[v].zero();
      de[v].zero();
      if (a.x != nullptr) at.template load<kOnce<T>>(x[v], static_cast<const T*>(a.x) + r * a.xs, v);
      at.template load<kOnce<T>>(dy[v], static_cast<const T*>(a.dy) + r * a.width, v);
      at.template load<kOnce<T>>(e[v], static_cast<const R*>(a.res) + r * a.width, v);
      if (a.dres_out != nullptr) at.template load<kOnce<T>>(de[v], static_cast<const R*>(a.dres_out) + r * a.width, v);
    }
  }
};

template <typename T, typename R, bool VEC, int TEAM, int NV, bool POST>
__global__ void __launch_bounds__(TEAM > 0 ? 256 : 1024) k_residual_norm_bwd(const ResArgs a) {
  __shared__ __align__(16) float red[2][kMaxWaves][kMaxSums];
  extern __shared__ __align__(16) float lds[];
  Place<TEAM, NV, VEC> at((int)a.width, 1, red);
  const float inv = 1.0f / (float)at.dim;
  const Kept<NV, Place<TEAM, NV, VEC>> pre(at, a.w_pre, lds), post(at, a.w_post, lds + 8 * blockDim.x);
  float dwo[NV][8] = {}, dwp[NV][8] = {};
  for (int64_t r = at.row; r < a.rows; r += at.dr) {
    ResRow<T, R, VEC, NV> now;
    now.load(a, at, r);
    // With g the gradient of the sum R: g = rs (w_pre dy - R c) + dres_out, and for x's own norm sum(w_post alpha g x),
    // which falls into three sums that need neither rs nor c: all sums close at once.
    float s[6] = {};
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float wp[8], wo[8];
      pre.get(wp, v);
      if (POST) post.get(wo, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float t = now.e[v].get(j), wd = wp[j] * now.dy[v].get(j);
        s[0] = __builtin_fmaf(t, t, s[0]);
        s[1] = __builtin_fmaf(wd, t, s[1]);
        if (POST) {
          const float x = now.x[v].get(j), wx = wo[j] * x;
          s[2] = __builtin_fmaf(x, x, s[2]);
          s[3] = __builtin_fmaf(wx, wd, s[3]);
          s[4] = __builtin_fmaf(wx, t, s[4]);
          s[5] = __builtin_fmaf(wx, now.de[v].get(j), s[5]);
        }
      }
    }
    s[0] *= kShare;
    s[2] *= kShare;
    s[4] *= kShare;
    at.template sums<POST ? 6 : 2>(s);
    NormGrad n, m;
    n.take(s[0], s[1], inv, a.eps);
    m.rs = 1.0f;
    m.c = 0.0f;
    if (POST)
      m.take(s[2], a.alpha * __builtin_fmaf(n.rs, __builtin_fmaf(-(kWhole * n.c), s[4], s[3]), s[5]), inv, a.eps);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float wp[8], wo[8], g[8], gx[8];
      pre.get(wp, v);
      post.get(wo, v);
      now.e[v].forget();
      now.dy[v].forget();
      now.x[v].forget();
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float t = now.e[v].get(j), d = now.dy[v].get(j), x = now.x[v].get(j);
        dwp[v][j] = __builtin_fmaf(d * t, n.rs, dwp[v][j]);
        g[j] = n(t, wp[j] * d) + now.de[v].get(j);
        const float ag = a.alpha * g[j];
        dwo[v][j] = __builtin_fmaf(ag * x, m.rs, dwo[v][j]);
        gx[j] = POST ? m(x, wo[j] * ag) : wo[j] * ag;
      }
      if (a.dres != nullptr) at.template store<false>(static_cast<R*>(a.dres) + r * a.width, g, v);
      at.template store<kOnce<T>>(static_cast<T*>(a.dx) + r * a.width, gx, v);
    }
  }
  if (a.part == nullptr || at.row >= a.rows) return;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    at.template store<false>(a.part + at.team * at.dim, dwp[v], v);
    at.template store<false>(a.part + a.part_post + at.team * at.dim, dwo[v], v);
  }
}

// The shape of a launch: lanes a team (0: the workgroup), pieces a lane, threads and
// workgroups.
struct Shape {
  int team, nv, threads;
  int64_t teams;  // a multiple of the groups
  unsigned grid;
};

// Workgroups of w waves a CU is given, each of which walks every so-many-th row.
// Forward: eight times what a CU holds at once (32 waves of one piece a lane, 16 of two), so that CUs that
// get ahead take more (32768 rows of 5120, gate first: 174 us; four times and 16 times 179; twice 187; 32768 x 2560
// with residual: 181, 187, 180, 194, in bf16 120, 124, 123, 129; 32768 x 1024 with residual: 74, 75, 74, 77; against
// that the gated norm of 32768 x 1024: 37.3, 34.2, 37.2, 35.7).
// Gradients: eight waves, in whole workgroups: more only add sums of weights to write and to join, and
// rows in between (16384 x 2560 with residual: 143 us, with 16 waves 174, with 24 165, in bf16 95, 127, 116; 32768 x
// 1024 with residual: 116, 125, 133; 32768 x 768: 94, 99, 106; 16384 x 8 x 512: 125, 128, 139; 16384 x 5120: 181, 186,
// 190; against that the gated norm of 32768 x 1024: 73.9, 69.9, 79.6).
int64_t groups_per_cu(int w, int nv, bool grad) {
  if (grad) return w < 8 ? (7 + w) / w : 1;
  return 8 * (nv == 1 ? 32 / w : 1);
}

// rows x groups teams of work.
Shape shape_of(int64_t rows, int64_t dim, int64_t groups, bool grad) {
  Shape s{};
  const int64_t pieces = (dim + 7) / 8;
  if (pieces <= 64) {
    s.team = pieces <= 8 ? 8 : pieces <= 16 ? 16 : pieces <= 32 ? 32 : 64;
    s.nv = 1;
    s.threads = 256;
  } else {
    s.team = 0;
    s.nv = pieces <= 1024 ? 1 : 2;
    s.threads = (int)((pieces + 64 * s.nv - 1) / (64 * s.nv) * 64);
  }
  const int per = s.team > 0 ? s.threads / s.team : 1;
  // Teams: no more than there is work, whole workgroups and whole rows of groups.
  int64_t rows_at_once = 256 * groups_per_cu(s.threads / 64, s.nv, grad) * per / groups;
  if (rows_at_once > rows) rows_at_once = rows;
  if (rows_at_once < 1) rows_at_once = 1;
  while (rows_at_once * groups % per != 0) ++rows_at_once;
  s.teams = rows_at_once * groups;
  s.grid = (unsigned)(s.teams / per);
  return s;
}

// f(team, pieces) with both as constants.
template <typename F>
hipError_t by_shape(const Shape& s, F f) {
  using std::integral_constant;
  switch (s.team) {
    case 8: return f(integral_constant<int, 8>(), integral_constant<int, 1>());
    case 16: return f(integral_constant<int, 16>(), integral_constant<int, 1>());
    case 32: return f(integral_constant<int, 32>(), integral_constant<int, 1>());
    case 64: return f(integral_constant<int, 64>(), integral_constant<int, 1>());
    default:
      return s.nv == 1 ? f(integral_constant<int, 0>(), integral_constant<int, 1>())
                       : f(integral_constant<int, 0>(), integral_constant<int, 2>());
  }
}

bool at16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

bool whole(const GatedNormLaunch& p) {
  const int64_t es = p.bf16 ? 2 : 4;
  return p.width / p.groups % 8 == 0 && p.x_stride * es % 16 == 0 && (p.z == nullptr || p.z_stride * es % 16 == 0) &&
         at16(p.x) && at16(p.z) && at16(p.w) && at16(p.y) && at16(p.dy) && at16(p.dz);
}
bool whole(const ResidualNormLaunch& p) {
  const int64_t es = p.bf16 ? 2 : 4;
  return p.width % 8 == 0 && p.x_stride * es % 16 == 0 && at16(p.x) && at16(p.residual) && at16(p.w_pre) &&
         at16(p.w_post) && at16(p.res_out) && at16(p.y) && at16(p.dy) && at16(p.dres_out) && at16(p.dx) &&
         at16(p.dres);
}

template <typename F>
hipError_t by_bool(bool v, F f) {
  return v ? f(std::true_type()) : f(std::false_type());
}

NormArgs args(const GatedNormLaunch& p) {
  NormArgs a{};
  a.x = p.x;
  a.z = p.z;
  a.w = p.w;
  a.y = p.y;
  a.rows = p.rows;
  a.width = p.width;
  a.groups = p.groups;
  a.xs = p.x_stride;
  a.zs = p.z_stride;
  a.eps = p.eps;
  a.dy = p.dy;
  a.dz = p.dz;
  return a;
}
ResArgs args(const ResidualNormLaunch& p) {
  ResArgs a{};
  a.x = p.x;
  a.res = p.residual;
  a.w_pre = p.w_pre;
  a.w_post = p.w_post;
  a.res_out = p.res_out;
  a.y = p.y;
  a.rows = p.rows;
  a.width = p.width;
  a.xs = p.x_stride;
  a.alpha = p.alpha;
  a.eps = p.eps;
  a.dy = p.dy;
  a.dres_out = p.dres_out;
  a.dx = p.dx;
  a.dres = p.dres;
  return a;
}

template <bool GRAD, typename T>
hipError_t go_gated(const GatedNormLaunch& p, const NormArgs& a, const Shape& s) {
  return by_shape(s, [&](auto team, auto nv) {
    return by_bool(whole(p), [&](auto vec) {
      return by_bool(p.z != nullptr, [&](auto z) {
        return by_bool(p.gate_first, [&](auto first) {
          constexpr int TEAM = decltype(team)::value, NV = decltype(nv)::value;
          constexpr bool VEC = decltype(vec)::value, Z = decltype(z)::value, FIRST = decltype(first)::value || !Z;
          if constexpr (GRAD)
            return launch(k_gated_norm_bwd<T, VEC, TEAM, NV, Z, FIRST>, dim3(s.grid), dim3(s.threads),
                          NV == 1 ? s.threads * kKeptBytes : 0, p.stream, a);
          else
            return launch(k_gated_norm<T, VEC, TEAM, NV, Z, FIRST>, dim3(s.grid), dim3(s.threads), 0, p.stream, a);
        });
      });
    });
  });
}

template <bool GRAD, typename T, typename R>
hipError_t go_residual(const ResidualNormLaunch& p, const ResArgs& a, const Shape& s) {
  return by_shape(s, [&](auto team, auto nv) {
    return by_bool(whole(p), [&](auto vec) {
      return by_bool(p.post_norm, [&](auto post) {
        constexpr int TEAM = decltype(team)::value, NV = decltype(nv)::value;
        constexpr bool VEC = decltype(vec)::value, POST = decltype(post)::value;
        if constexpr (GRAD)
          return launch(k_residual_norm_bwd<T, R, VEC, TEAM, NV, POST>, dim3(s.grid), dim3(s.threads),
                        NV == 1 ? 2 * s.threads * kKeptBytes : 0, p.stream, a);
        else
          return launch(k_residual_norm<T, R, VEC, TEAM, NV, POST>, dim3(s.grid), dim3(s.threads), 0, p.stream, a);
      });
    });
  });
}

// Rows of sums: the teams of one group, those without a row left out.
int64_t parts_of(const Shape& s, int64_t rows, int64_t groups) {
  const int64_t n = s.teams / groups;
  return n < rows ? n : rows;
}

}  // namespace

int64_t gated_norm_bwd_floats(int64_t rows, int64_t width, int64_t groups) {
  return rows == 0 ? 0 : parts_of(shape_of(rows, width / groups, groups, true), rows, groups) * width;
}
int64_t residual_norm_bwd_floats(int64_t rows, int64_t width) {
  return rows == 0 ? 0 : 2 * parts_of(shape_of(rows, width, 1, true), rows, 1) * width;
}

hipError_t launch_gated_norm(const GatedNormLaunch& p) {
  const Shape s = shape_of(p.rows, p.width / p.groups, p.groups, false);
  const NormArgs a = args(p);
  return p.bf16 ? go_gated<false, uint16_t>(p, a, s) : go_gated<false, float>(p, a, s);
}

hipError_t launch_gated_norm_bwd(const GatedNormLaunch& p) {
  int64_t n = 0;
  if (p.rows > 0) {
    const Shape s = shape_of(p.rows, p.width / p.groups, p.groups, true);
    NormArgs a = args(p);
    a.part = p.dw != nullptr ? p.workspace : nullptr;
    n = parts_of(s, p.rows, p.groups);
    const hipError_t rc = p.bf16 ? go_gated<true, uint16_t>(p, a, s) : go_gated<true, float>(p, a, s);
    if (rc != hipSuccess) return rc;
  }
  return p.dw == nullptr ? hipSuccess : col_sum(p.workspace, p.dw, nullptr, 0, n, p.width, p.stream);
}

hipError_t launch_residual_norm(const ResidualNormLaunch& p) {
  const Shape s = shape_of(p.rows, p.width, 1, false);
  const ResArgs a = args(p);
  if (!p.bf16) return go_residual<false, float, float>(p, a, s);
  return p.res_bf16 ? go_residual<false, uint16_t, uint16_t>(p, a, s) : go_residual<false, uint16_t, float>(p, a, s);
}

hipError_t launch_residual_norm_bwd(const ResidualNormLaunch& p) {
  const bool want = p.dw_pre != nullptr || p.dw_post != nullptr;
  int64_t n = 0, second = 0;
  if (p.rows > 0) {
    const Shape s = shape_of(p.rows, p.width, 1, true);
    ResArgs a = args(p);
    a.part = want ? p.workspace : nullptr;
    n = parts_of(s, p.rows, 1);
    a.part_post = second = n * p.width;
    const hipError_t rc = !p.bf16 ? go_residual<true, float, float>(p, a, s)
                          : p.res_bf16 ? go_residual<true, uint16_t, uint16_t>(p, a, s)
                                       : go_residual<true, uint16_t, float>(p, a, s);
    if (rc != hipSuccess) return rc;
  }
  return want ? col_sum(p.workspace, p.dw_pre, p.dw_post, second, n, p.width, p.stream) : hipSuccess;
}

}  // namespace ssm
