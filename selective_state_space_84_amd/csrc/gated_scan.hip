// Gated linear recurrence over whole sequences and its gradient.
#include "gated_launch.h"
#include "gated_math.h"

namespace ssm {
namespace {

struct GatedArgs {
  const void* x;
  const void* ga;
  const void* gx;
  const void* z;
  const float* log_a;
  const int32_t* lengths;
  const float* h0;
  void* y;
  float* h_last;
  float* ckpt;
  int64_t batch, seqlen, width;
  int64_t xs, as, is, zs;
  const void* dy;
  const float* dh_last;
  void* dx;
  void* dga;
  void* dgx;
  void* dz;
  float* part;
  float* dh0;
};

__device__ __forceinline__ int64_t steps_of(const GatedArgs& a, int64_t b) {
  if (a.lengths == nullptr) return a.seqlen;
  const int64_t n = a.lengths[b];
  return n < 0 ? 0 : n > a.seqlen ? a.seqlen : n;
}

template <typename T>
__device__ __forceinline__ float get(const void* p, int64_t i) {
  return io_to_f32(static_cast<const T*>(p)[i]);
}
template <typename T>
__device__ __forceinline__ void put(void* p, int64_t i, float v) {
  io_store(static_cast<T*>(p) + i, v);
}

// One channel of one row a lane.
template <typename T>
__global__ void __launch_bounds__(256) k_gated_fwd(const GatedArgs a) {
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (id >= a.batch * a.width) return;
  const int64_t b = id / a.width, d = id % a.width;
  const int64_t n = steps_of(a, b), nck = (a.seqlen + kGatedCkpt - 1) / kGatedCkpt;
  const float c2 = a.log_a[d] * kLog2e;
  float h = a.h0 != nullptr ? a.h0[id] : 0.0f;
  for (int64_t t = 0; t < a.seqlen; ++t) {
    const int64_t r = b * a.seqlen + t;
    if (a.ckpt != nullptr && t % kGatedCkpt == 0) a.ckpt[(b * nck + t / kGatedCkpt) * a.width + d] = h;
    if (t < n) {
      const GatedStep s = gated_step(get<T>(a.ga, r * a.as + d), get<T>(a.gx, r * a.is + d), c2);
      h = __builtin_fmaf(s.a, h, s.m * s.sx * get<T>(a.x, r * a.xs + d));
      const float gate = a.z != nullptr ? silu(get<T>(a.z, r * a.zs + d)) : 1.0f;
      if (a.y != nullptr) put<T>(a.y, r * a.width + d, h * gate);
    } else if (a.y != nullptr) {
      put<T>(a.y, r * a.width + d, 0.0f);
    }
  }
  if (a.h_last != nullptr) a.h_last[id] = h;
}

template <typename T>
__global__ void __launch_bounds__(256) k_gated_bwd(const GatedArgs a) {
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (id >= a.batch * a.width) return;
  const int64_t b = id / a.width, d = id % a.width;
  const int64_t n = steps_of(a, b), nck = (a.seqlen + kGatedCkpt - 1) / kGatedCkpt;
  const float la = a.log_a[d], c2 = la * kLog2e;
  float p = a.dh_last != nullptr ? a.dh_last[id] : 0.0f, sum = 0.0f;
  for (int64_t c = nck - 1; c >= 0; --c) {
    const int64_t t0 = c * kGatedCkpt, t1 = min(t0 + kGatedCkpt, a.seqlen);
    float before[kGatedCkpt];
    float h = a.ckpt[(b * nck + c) * a.width + d];
    for (int64_t t = t0; t < min(t1, n); ++t) {
      const int64_t r = b * a.seqlen + t;
      before[t - t0] = h;
      const GatedStep s = gated_step(get<T>(a.ga, r * a.as + d), get<T>(a.gx, r * a.is + d), c2);
      h = __builtin_fmaf(s.a, h, s.m * s.sx * get<T>(a.x, r * a.xs + d));
    }
    for (int64_t t = t1 - 1; t >= t0; --t) {
      const int64_t r = b * a.seqlen + t, o = r * a.width + d;
      float dx = 0.0f, dga = 0.0f, dgx = 0.0f, dz = 0.0f;
      if (t < n) {
        const GatedStep s = gated_step(get<T>(a.ga, r * a.as + d), get<T>(a.gx, r * a.is + d), c2);
        const float x = get<T>(a.x, r * a.xs + d), w = s.sx * x;
        float e = get<T>(a.dy, o);
        if (a.z != nullptr) {
          const float z = get<T>(a.z, r * a.zs + d), q = sigmoid(z);
          const float after = __builtin_fmaf(s.a, before[t - t0], s.m * w);
          dz = e * after * q * __builtin_fmaf(z, 1.0f - q, 1.0f);
          e *= z * q;
        }
        const float g = e + p;
        const float gm = g * s.m;
        const float dla = g * __builtin_fmaf(s.a, before[t - t0], -(s.a * s.a * s.inv_m) * w);
        dx = gm * s.sx;
        dgx = dx * x * (1.0f - s.sx);
        dga = dla * la * s.sa * (1.0f - s.sa);
        sum = __builtin_fmaf(dla, s.sa, sum);
        p = s.a * g;
      }
      put<T>(a.dx, o, dx);
      put<T>(a.dga, o, dga);
      put<T>(a.dgx, o, dgx);
      if (a.dz != nullptr) put<T>(a.dz, o, dz);
    }
  }
  if (a.dh0 != nullptr) a.dh0[id] = p;
  if (a.part != nullptr) a.part[id] = sum;
}

__global__ void __launch_bounds__(256) k_gated_sum(const float* part, float* out, int64_t rows, int64_t width) {
  const int64_t d = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (d >= width) return;
  float s = 0.0f;
  for (int64_t r = 0; r < rows; ++r) s += part[r * width + d];
  out[d] = s;
}

GatedArgs args(const GatedScanLaunch& p) {
  GatedArgs a{};
  a.x = p.x;
  a.ga = p.ga;
  a.gx = p.gx;
  a.z = p.z;
  a.log_a = p.log_a;
  a.lengths = p.lengths;
  a.h0 = p.h0;
  a.y = p.y;
  a.h_last = p.h_last;
  a.ckpt = p.ckpt;
  a.batch = p.batch;
  a.seqlen = p.seqlen;
  a.width = p.width;
  a.xs = p.x_stride;
  a.as = p.ga_stride;
  a.is = p.gx_stride;
  a.zs = p.z_stride;
  a.dy = p.dy;
  a.dh_last = p.dh_last;
  a.dx = p.dx;
  a.dga = p.dga;
  a.dgx = p.dgx;
  a.dz = p.dz;
  a.dh0 = p.dh0;
  return a;
}

unsigned groups(int64_t n) { return (unsigned)((n + 255) / 256); }

}  // namespace

int64_t gated_scan_ckpt_floats(int64_t batch, int64_t seqlen, int64_t width) {
  return batch * ((seqlen + kGatedCkpt - 1) / kGatedCkpt) * width;
}
int64_t gated_scan_fwd_floats(int64_t, int64_t, int64_t, bool) { return 0; }
int64_t gated_scan_bwd_floats(int64_t batch, int64_t seqlen, int64_t width, bool, bool ckpt_given) {
  return batch * width + (ckpt_given ? 0 : gated_scan_ckpt_floats(batch, seqlen, width));
}

hipError_t launch_gated_scan_fwd(const GatedScanLaunch& p) {
  const GatedArgs a = args(p);
  return launch(p.bf16 ? k_gated_fwd<uint16_t> : k_gated_fwd<float>, dim3(groups(p.batch * p.width)), dim3(256), 0,
                p.stream, a);
}

hipError_t launch_gated_scan_bwd(const GatedScanLaunch& p) {
  GatedArgs a = args(p);
  a.part = p.dlog_a != nullptr ? p.workspace : nullptr;
  hipError_t rc;
  const dim3 grid(groups(p.batch * p.width));
  if (p.batch > 0) {
    if (a.ckpt == nullptr) {
      a.ckpt = p.workspace + p.batch * p.width;
      GatedArgs f = a;
      f.y = nullptr;
      f.h_last = nullptr;
      rc = launch(p.bf16 ? k_gated_fwd<uint16_t> : k_gated_fwd<float>, grid, dim3(256), 0, p.stream, f);
      if (rc != hipSuccess) return rc;
    }
    rc = launch(p.bf16 ? k_gated_bwd<uint16_t> : k_gated_bwd<float>, grid, dim3(256), 0, p.stream, a);
    if (rc != hipSuccess) return rc;
  }
  if (p.dlog_a == nullptr) return hipSuccess;
  return launch(k_gated_sum, dim3(groups(p.width)), dim3(256), 0, p.stream, p.workspace, p.dlog_a, p.batch, p.width);
}

}  // namespace ssm
