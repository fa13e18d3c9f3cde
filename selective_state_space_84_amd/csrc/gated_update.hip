// One step of the gated recurrence (decode), in place on the states of a
// batch of requests.
#include "gated_launch.h"
#include "gated_math.h"

namespace ssm {
namespace {

struct UpdateArgs {
  float* h;
  const int32_t* slots;
  const void* x;
  const void* ga;
  const void* gx;
  const void* z;
  const float* log_a;
  void* y;
  int64_t n_slots, width;
  int64_t xs, as, is, zs;
  uint32_t tiles;  // workgroups a row
};

// V channels a lane.
template <typename T, int V>
__global__ void __launch_bounds__(256) k_gated_update(const UpdateArgs a) {
  typedef T in_t __attribute__((ext_vector_type(V)));
  typedef float st_t __attribute__((ext_vector_type(V)));
  const int64_t b = blockIdx.x / a.tiles;
  const int64_t d = ((int64_t)(blockIdx.x % a.tiles) * 256 + threadIdx.x) * V;
  if (d >= a.width) return;
  auto in = [&](const void* p, int64_t stride) {
    return *reinterpret_cast<const in_t*>(static_cast<const T*>(p) + b * stride + d);
  };
  T* const y = static_cast<T*>(a.y) + b * a.width + d;
  const int64_t slot = a.slots != nullptr ? a.slots[b] : b;
  if (slot < 0 || slot >= a.n_slots) {
#pragma unroll
    for (int j = 0; j < V; ++j) io_store(y + j, 0.0f);
    return;
  }
  st_t* const hp = reinterpret_cast<st_t*>(a.h + slot * a.width + d);
  const in_t x = in(a.x, a.xs), ga = in(a.ga, a.as), gx = in(a.gx, a.is);
  in_t z{};
  if (a.z != nullptr) z = in(a.z, a.zs);
  const st_t c = *reinterpret_cast<const st_t*>(a.log_a + d);
  st_t h = *hp;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const GatedStep s = gated_step(io_to_f32(ga[j]), io_to_f32(gx[j]), c[j] * kLog2e);
    h[j] = __builtin_fmaf(s.a, h[j], s.m() * s.sx * io_to_f32(x[j]));
    io_store(y + j, a.z != nullptr ? h[j] * silu(io_to_f32(z[j])) : h[j]);
  }
  *hp = h;
}

}  // namespace

int64_t gated_update_tiles(int64_t width) { return (width + 255) / 256; }

hipError_t launch_gated_scan_update(const GatedUpdateLaunch& p) {
  const UpdateArgs a{p.h, p.slots,   p.x,     p.ga,       p.gx,        p.z,         p.log_a,
                     p.y, p.n_slots, p.width, p.x_stride, p.ga_stride, p.gx_stride, p.z_stride,
                     (uint32_t)gated_update_tiles(p.width)};
  const dim3 grid((unsigned)(p.batch * gated_update_tiles(p.width)));
  if (p.bf16) return launch(k_gated_update<uint16_t, 1>, grid, dim3(256), 0, p.stream, a);
  return launch(k_gated_update<float, 1>, grid, dim3(256), 0, p.stream, a);
}

}  // namespace ssm
