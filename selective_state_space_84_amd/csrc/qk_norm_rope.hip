// RMS norm of query and key heads with the position rotation in the same
// pass, and its gradient.
//
//   n = w x r, r = 1 / sqrt(mean(x^2) + eps);  y = R(p) n
// with R(p) turning pair j of the first rot_dim values by p inv_freq[j].
// Gradient: g = R(p)^T dy,  dw = sum g x r,
//           dx = r (w g) - x r^3 mean(w g x).
//
// Bound by HBM: x is read once and y written once (8192 steps x 64 heads of 128
// in bf16: 54-58 us, 4.7-5.0 TB/s, in fp32 106 us, 5.1 TB/s; gradient of 16384
// steps x 32 heads: 91 us, 4.4 TB/s, two workgroups a CU by its registers; a copy
// reaches 5.1 TB/s).  A head belongs to G lanes (the next power of two of headdim
// / 8), 8 values a lane; the mean closes with log2(G) adds across lanes, and the pairs of the half-split rotation come from
// the lane rot_dim / 16 away.  A workgroup takes all heads of one or a few
// steps, so that a step's angles are formed once, by one lane each, and shared
// through LDS by its heads; the first heads' loads are on their way
// meanwhile.  Angles are products in 64 bits, reduced to a
// fraction of a turn before they are rounded to fp32 (an fp32 product at
// position 10^6 would be off by 0.06 radians).
#include "ssm_device.h"
#include "attn_launch.h"

namespace ssm {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

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
  int32_t dim, rot, tb, rounds;  // steps per workgroup: tb (a power of two) at a time, rounds times
  float eps;
};

constexpr int kMaxAngles = 1024;  // pairs of one workgroup's steps

// A lane's 8 values as loaded (W words), and widened.
template <typename T>
struct Raw;
template <>
struct Raw<float> {
  static constexpr int W = 8;
  u32x4 a[2];
  __device__ __forceinline__ void load(const float* p) {
    a[0] = *reinterpret_cast<const u32x4*>(p);
    a[1] = *reinterpret_cast<const u32x4*>(p + 4);
  }
  __device__ __forceinline__ float get(int j) const {
    const uint32_t v = a[j / 4][j % 4];  // bit_cast of a vector's element in place reads its first one
    return __builtin_bit_cast(float, v);
  }
};
template <>
struct Raw<uint16_t> {
  static constexpr int W = 4;
  u32x4 a[1];
  __device__ __forceinline__ void load(const uint16_t* p) { a[0] = *reinterpret_cast<const u32x4*>(p); }
  __device__ __forceinline__ float get(int j) const {
    const uint32_t v = a[0][j / 2];
    return __builtin_bit_cast(float, j % 2 ? v & 0xffff0000u : v << 16);
  }
};
template <typename T>
__device__ __forceinline__ void zero(Raw<T>& x) {
#pragma unroll
  for (int k = 0; k < Raw<T>::W / 4; ++k) x.a[k] = u32x4{0, 0, 0, 0};
}
// The same 8 values of another lane, before they are widened.
template <typename T>
__device__ __forceinline__ Raw<T> from_lane(const Raw<T>& x, int src) {
  Raw<T> r;
#pragma unroll
  for (int k = 0; k < Raw<T>::W; ++k) r.a[k / 4][k % 4] = (uint32_t)__shfl((int)x.a[k / 4][k % 4], src);
  return r;
}
__device__ __forceinline__ void store8(float* p, const float* v) {
  *reinterpret_cast<f32x4*>(p) = f32x4{v[0], v[1], v[2], v[3]};
  *reinterpret_cast<f32x4*>(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
}
__device__ __forceinline__ void store8(uint16_t* p, const float* v) {
  u32x4 r;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    r[k] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{v[2 * k], v[2 * k + 1]}, bf16x2));
  *reinterpret_cast<u32x4*>(p) = r;
}

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}

// Sum over the G lanes of a head, in every lane of it: neighbours, pairs, then
// mirrored halves and rows (whose quads, halves hold one value by then).
template <int G>
__device__ __forceinline__ float group_sum(float v) {
  v += dpp<0xB1>(v);                 // quad_perm 1 0 3 2
  if (G > 2) v += dpp<0x4E>(v);      // quad_perm 2 3 0 1
  if (G > 4) v += dpp<0x141>(v);     // row_half_mirror
  if (G > 8) v += dpp<0x140>(v);     // row_mirror
  if (G > 16) v += __shfl_xor(v, 16);
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

// This lane's part in the rotation of its step: value j becomes
//   c[j] v[j] + s[j] (the pair's other value),
// with 1 and 0 where nothing turns.  The other value is the lane's own
// neighbour (INTER) or value j of lane src.
template <bool INTER, bool BACK>
struct Rotation {
  int src;
  float c[8], s[8];
  // cs: the step's angles; ln: the lane's place in its head.
  __device__ __forceinline__ void take(const float2* cs, int ln, int rot) {
    const int hl = rot / 16;  // lanes of half the rotated part
    const bool in = 8 * ln < rot, first = ln < hl;
    src = (threadIdx.x & 63) + (in && !INTER ? (first ? hl : -hl) : 0);
    const int base = INTER ? 4 * ln : 8 * (first ? ln : ln - hl);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 v = in ? cs[base + (INTER ? j / 2 : j)] : make_float2(1.f, 0.f);
      const bool minus = (INTER ? j % 2 == 0 : first) != BACK;
      c[j] = v.x;
      s[j] = minus ? -v.y : v.y;
    }
  }
};

// The pair's other value of each of a lane's 8, from `other` (from_lane of src).
template <bool INTER, typename T>
__device__ __forceinline__ float pair_of(const Raw<T>& x, const Raw<T>& other, int j) {
  return INTER ? x.get(j ^ 1) : other.get(j);
}

// Where a lane works: G lanes a head, 256 / G heads at a time, of which tb (a
// power of two) belong to different steps, so that a lane keeps its step and
// its angles while it walks the heads h0, h0 + dh, ... of a step.
template <int G>
struct Place {
  int ln, t, h0, dh;
  bool live;
  __device__ __forceinline__ explicit Place(const QkArgs& a) {
    const int grp = threadIdx.x / G;
    ln = threadIdx.x % G;
    t = grp & (a.tb - 1);
    h0 = grp / a.tb;
    dh = 256 / G / a.tb;
    live = 8 * ln < a.dim;
  }
};

// N heads of a lane group from head b on, zero where there is none.
template <typename T, int N, int G>
__device__ __forceinline__ void load_heads(Raw<T> (&x)[N], const T* p, const Place<G>& at, int b, int heads, int dim,
                                           bool live) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int h = b + i * at.dh + at.h0;
    zero(x[i]);
    if (live && h < heads) x[i].load(p + h * dim);
  }
}

// Weights of both sides, ones where there are none (also behind the head).
__device__ __forceinline__ void fill_weights(const QkArgs& a, float (&w)[2][256]) {
  for (int side = 0; side < 2; ++side)
    w[side][threadIdx.x] = a.w[side] != nullptr && (int)threadIdx.x < a.dim ? a.w[side][threadIdx.x] : 1.0f;
}

template <typename T, int G, bool INTER>
__global__ void __launch_bounds__(256) k_qk_norm_rope(const QkArgs a) {
  __shared__ float2 cs[kMaxAngles];
  __shared__ __align__(16) float w[2][256];
  constexpr int N = 4;  // heads a lane has on their way
  const int64_t t0 = (int64_t)blockIdx.x * a.tb * a.rounds;
  const int n = (int)min((int64_t)a.tb * a.rounds, a.tokens - t0);
  const float inv_d = 1.0f / (float)a.dim;
  const Place<G> at(a);
  fill_weights(a, w);
  // A side's first heads are requested while the side before is worked on.
  Raw<T> xx[2][N];
  auto ask = [&](int r, int side) {
    load_heads(xx[side], static_cast<const T*>(a.x[side]) + (t0 + r + at.t) * a.xs[side] + 8 * at.ln, at, 0,
               a.heads[side], a.dim, at.live && r + at.t < n);
  };
  ask(0, 0);
  fill_angles(a, t0, n, cs);
  __syncthreads();
  for (int r = 0; r < n; r += a.tb) {
    const bool live = at.live && r + at.t < n;
    const int64_t t = t0 + r + at.t;
    Rotation<INTER, false> rot;
    rot.take(cs + (live ? r + at.t : 0) * (a.rot / 2), at.ln, a.rot);
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      const int heads = a.heads[side];
      Raw<T>(&x)[N] = xx[side];
      ask(side == 0 ? r : r + a.tb, side ^ 1);
      const T* const xp = static_cast<const T*>(a.x[side]) + t * a.xs[side] + 8 * at.ln;
      T* const yp = static_cast<T*>(a.y[side]) + t * a.ys[side] + 8 * at.ln;
      // The weights go into the coefficients: the other value of a pair has its own.
      float ca[8], cb[8];
      const int other = 8 * (at.ln + (rot.src - (int)(threadIdx.x & 63)));
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        ca[j] = rot.c[j] * w[side][8 * at.ln + j];
        cb[j] = rot.s[j] * w[side][INTER ? 8 * at.ln + (j ^ 1) : other + j];
      }
      // Every lane walks the same number of rounds: the exchanges need whole groups.
      for (int b = 0; b < heads; b += at.dh * N) {
        if (b > 0) load_heads(x, xp, at, b, heads, a.dim, live);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const Raw<T> o = INTER ? x[i] : from_lane(x[i], rot.src);
          float v[8], ss = 0.f;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            v[j] = x[i].get(j);
            ss = __builtin_fmaf(v[j], v[j], ss);
          }
          const float rs = __builtin_amdgcn_rsqf(__builtin_fmaf(group_sum<G>(ss), inv_d, a.eps));
          float y[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) y[j] = rs * __builtin_fmaf(pair_of<INTER>(x[i], o, j), cb[j], v[j] * ca[j]);
          const int h = b + i * at.dh + at.h0;
          if (live && h < heads) store8(yp + h * a.dim, y);
        }
      }
    }
  }
}

template <typename T, int G, bool INTER>
__global__ void __launch_bounds__(256) k_qk_norm_rope_bwd(const QkArgs a) {
  __shared__ float2 cs[kMaxAngles];
  __shared__ float sw[256 * 8];
  constexpr int N = sizeof(T) == 2 ? 4 : 2;
  const float inv_d = 1.0f / (float)a.dim;
  const Place<G> at(a);
  float w[2][8], dw[2][8] = {};
#pragma unroll
  for (int side = 0; side < 2; ++side)
#pragma unroll
    for (int j = 0; j < 8; ++j) w[side][j] = at.live && a.w[side] != nullptr ? a.w[side][8 * at.ln + j] : 1.0f;
  const int64_t step = (int64_t)a.tb * a.rounds;
  for (int64_t t0 = (int64_t)blockIdx.x * step; t0 < a.tokens; t0 += (int64_t)gridDim.x * step) {
    const int n = (int)min(step, a.tokens - t0);
    __syncthreads();
    Raw<T> xx[2][N], gg[2][N];
    auto ask = [&](int r, int side) {
      const bool live = at.live && r + at.t < n;
      const int64_t t = t0 + r + at.t;
      load_heads(xx[side], static_cast<const T*>(a.x[side]) + t * a.xs[side] + 8 * at.ln, at, 0, a.heads[side], a.dim,
                 live);
      load_heads(gg[side], static_cast<const T*>(a.dy[side]) + t * a.heads[side] * a.dim + 8 * at.ln, at, 0,
                 a.heads[side], a.dim, live);
    };
    ask(0, 0);
    fill_angles(a, t0, n, cs);
    __syncthreads();
    for (int r = 0; r < n; r += a.tb) {
      const bool live = at.live && r + at.t < n;
      const int64_t t = t0 + r + at.t;
      Rotation<INTER, true> rot;
      rot.take(cs + (live ? r + at.t : 0) * (a.rot / 2), at.ln, a.rot);
#pragma unroll
      for (int side = 0; side < 2; ++side) {
        const int heads = a.heads[side];
        const T* const xp = static_cast<const T*>(a.x[side]) + t * a.xs[side] + 8 * at.ln;
        const T* const gp = static_cast<const T*>(a.dy[side]) + t * heads * a.dim + 8 * at.ln;
        T* const out = static_cast<T*>(a.y[side]) + t * heads * a.dim + 8 * at.ln;
        Raw<T>(&x)[N] = xx[side], (&dy)[N] = gg[side];
        ask(side == 0 ? r : r + a.tb, side ^ 1);
        for (int b = 0; b < heads; b += at.dh * N) {
          if (b > 0) {
            load_heads(x, xp, at, b, heads, a.dim, live);
            load_heads(dy, gp, at, b, heads, a.dim, live);
          }
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const int h = b + i * at.dh + at.h0;
            const bool on = live && h < heads;
            const Raw<T> o = INTER ? dy[i] : from_lane(dy[i], rot.src);
            float v[8], g[8], wg[8], ss = 0.f, sg = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              v[j] = x[i].get(j);
              g[j] = __builtin_fmaf(pair_of<INTER>(dy[i], o, j), rot.s[j], dy[i].get(j) * rot.c[j]);
              wg[j] = w[side][j] * g[j];
              ss = __builtin_fmaf(v[j], v[j], ss);
              sg = __builtin_fmaf(wg[j], v[j], sg);
            }
            const float rs = __builtin_amdgcn_rsqf(__builtin_fmaf(group_sum<G>(ss), inv_d, a.eps));
            const float c = group_sum<G>(sg) * inv_d * rs * rs;
            if (on) {  // heads that do not exist leave dw alone (with eps 0 their rs is infinite)
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                dw[side][j] = __builtin_fmaf(g[j] * v[j], rs, dw[side][j]);
                g[j] = rs * __builtin_fmaf(-v[j], c, wg[j]);
              }
              store8(out + h * a.dim, g);
            }
          }
        }
      }
    }
  }
  if (a.part == nullptr) return;
  // The workgroup's sums over its lane groups, in group order.
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) sw[threadIdx.x / G * (8 * G) + 8 * at.ln + j] = dw[side][j];
    __syncthreads();
    if ((int)threadIdx.x < a.dim) {
      float s = 0.f;
#pragma unroll 4
      for (int k = 0; k < 256 / G; ++k) s += sw[k * (8 * G) + threadIdx.x];
      a.part[((int64_t)side * gridDim.x + blockIdx.x) * a.dim + threadIdx.x] = s;
    }
  }
}

// dw[side][c] = sum over workgroups: 16 columns per workgroup, 64 interleaved
// partial sums per column (eight loads of each on their way), joined pairwise.
__global__ void __launch_bounds__(1024) k_qk_reduce_dw(const float* part, float* dwq, float* dwk, int32_t groups,
                                                       int32_t dim) {
  __shared__ float s[64][17];
  const int side = blockIdx.y;
  float* const dw = side == 0 ? dwq : dwk;
  if (dw == nullptr) return;
  const int c = threadIdx.x & 15, k0 = threadIdx.x >> 4;
  const int col = blockIdx.x * 16 + c;  // dim is a multiple of 16
  const float* p = part + (int64_t)side * groups * dim + col;
  float v = 0.f;
  for (int k = k0; k < groups; k += 8 * 64) {
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = k + 64 * i < groups ? p[(int64_t)(k + 64 * i) * dim] : 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) v += q[i];
  }
  for (int d = 32; d > 0; d /= 2) {
    s[k0][c] = v;
    __syncthreads();
    if (k0 < d) v += s[k0 + d][c];
    __syncthreads();
  }
  if (k0 == 0) dw[col] = v;
}

// Next power of two of the 8-value pieces of a head (2 lanes at least).
int lanes_per_head(int64_t dim) { return dim <= 16 ? 2 : dim <= 32 ? 4 : dim <= 64 ? 8 : dim <= 128 ? 16 : 32; }

// Steps a workgroup takes at a time (tb, a power of two) and how often (rounds)
// on one set of angles: at a time, as many as give every lane group four heads;
// together, as many as LDS holds the angles of, while `left` workgroups are left
// (8192 steps x 64 heads of 128 in bf16: 51.6 us with 2048, 60 us with 1024, 72 us
// with one step each).
void set_steps(QkArgs& a, int64_t left) {
  const int64_t groups = 256 / lanes_per_head(a.dim), heads = a.heads[0] + a.heads[1];
  const int64_t cap = a.rot > 0 ? kMaxAngles / (a.rot / 2) : 64;
  int64_t tb = 1, all = 1;
  while (2 * tb <= groups && 2 * tb <= cap && 2 * tb * heads <= 4 * groups && 2 * tb * left <= a.tokens) tb *= 2;
  all = tb;
  while (2 * all <= cap && 2 * all <= 16 && 2 * all * left <= a.tokens) all *= 2;
  a.tb = (int32_t)tb;
  a.rounds = (int32_t)(all / tb);
}

constexpr int64_t kFwdGroups = 2048;
// Workgroups (and partial sums) of the gradient: the two a CU that its registers
// allow (16384 steps x 32 heads of 128 in bf16: 91.5 us; 95 us with 1024, 103 us
// with 2048).  Their turns, of a power of two of steps, come out even where it
// divides the steps; else the longest workgroup walks up to twice what others do (40
// heads of 128: 6000 steps in 750 turns take 69 us, 8192 in 512 take 77).
constexpr int64_t kBwdGroups = 512;

QkArgs args(const QkNormRopeLaunch& p, bool grad) {
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
  a.eps = p.eps;
  a.dy[0] = p.dq_out;
  a.dy[1] = p.dk_out;
  set_steps(a, grad ? kBwdGroups : kFwdGroups);
  return a;
}

// Calls f with the kernel's lane group size as a constant.
template <typename F>
hipError_t by_group(int64_t dim, F f) {
  switch (lanes_per_head(dim)) {
    case 2: return f(std::integral_constant<int, 2>());
    case 4: return f(std::integral_constant<int, 4>());
    case 8: return f(std::integral_constant<int, 8>());
    case 16: return f(std::integral_constant<int, 16>());
    default: return f(std::integral_constant<int, 32>());
  }
}

int64_t groups_of(const QkArgs& a) {
  const int64_t n = (int64_t)a.tb * a.rounds;
  return (a.tokens + n - 1) / n;
}

}  // namespace

int64_t qk_norm_rope_bwd_floats(int64_t tokens, int64_t headdim) {
  // Every workgroup takes one step at least.
  return 2 * (tokens < kBwdGroups ? tokens : kBwdGroups) * headdim;
}

int64_t qk_norm_rope_groups(const QkNormRopeLaunch& p) { return groups_of(args(p, false)); }

hipError_t launch_qk_norm_rope(const QkNormRopeLaunch& p) {
  const QkArgs a = args(p, false);
  const unsigned grid = (unsigned)groups_of(a);
  return by_group(p.headdim, [&](auto g) {
    constexpr int G = decltype(g)::value;
    auto go = [&](auto kern) { return launch(kern, dim3(grid), dim3(256), 0, p.stream, a); };
    if (p.bf16) return p.interleaved ? go(k_qk_norm_rope<uint16_t, G, true>) : go(k_qk_norm_rope<uint16_t, G, false>);
    return p.interleaved ? go(k_qk_norm_rope<float, G, true>) : go(k_qk_norm_rope<float, G, false>);
  });
}

hipError_t launch_qk_norm_rope_bwd(const QkNormRopeLaunch& p) {
  QkArgs a = args(p, true);
  // Without heads there is no gradient to form (inv_freq may be NULL then): dw alone, a sum over nothing.
  int64_t groups = p.nheads + p.nheads_k > 0 ? groups_of(a) : 0;
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
  return launch(k_qk_reduce_dw, dim3((unsigned)(p.headdim / 16), 2), dim3(1024), 0, p.stream, p.workspace, p.dwq,
                p.dwk, (int32_t)groups, (int32_t)p.headdim);
}

}  // namespace ssm
