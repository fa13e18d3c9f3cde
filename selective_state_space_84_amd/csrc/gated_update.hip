// One step of the gated recurrence (decode), in place on the states of a
// batch of requests: every lane forms the gates of its channels and moves their
// state.  Bound by HBM for large batches (8 bytes of state and 8 to 10 of bf16
// operands a channel) and by the launch for small ones.
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
  in_t out;
  in_t* const y = reinterpret_cast<in_t*>(static_cast<T*>(a.y) + b * a.width + d);
  const int64_t slot = a.slots != nullptr ? a.slots[b] : b;
  if (slot < 0 || slot >= a.n_slots) {
    *y = in_t(T(0));
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
    T o;
    io_store(&o, a.z != nullptr ? h[j] * silu(io_to_f32(z[j])) : h[j]);
    out[j] = o;
  }
  *hp = h;
  *y = out;
}

// Four channels a lane where every row allows accesses of four.
bool fours(const GatedUpdateLaunch& p) {
  const int64_t n = p.width | p.x_stride | p.ga_stride | p.gx_stride | (p.z != nullptr ? p.z_stride : 0);
  uintptr_t io = 0;
  for (const void* q : {p.x, p.ga, p.gx, p.z, (const void*)p.y}) io |= reinterpret_cast<uintptr_t>(q);
  const uintptr_t f32 = reinterpret_cast<uintptr_t>(p.h) | reinterpret_cast<uintptr_t>(p.log_a);
  return n % 4 == 0 && io % (p.bf16 ? 8 : 16) == 0 && f32 % 16 == 0;
}

template <typename T, int V>
hipError_t go(const GatedUpdateLaunch& p, UpdateArgs a) {
  a.tiles = (uint32_t)((p.width + 256 * V - 1) / (256 * V));
  return launch(k_gated_update<T, V>, dim3((unsigned)(p.batch * a.tiles)), dim3(256), 0, p.stream, a);
}

}  // namespace

int64_t gated_update_tiles(int64_t width) { return (width + 255) / 256; }

hipError_t launch_gated_scan_update(const GatedUpdateLaunch& p) {
  const UpdateArgs a{p.h, p.slots,   p.x,     p.ga,       p.gx,        p.z,         p.log_a,
                     p.y, p.n_slots, p.width, p.x_stride, p.ga_stride, p.gx_stride, p.z_stride, 0};
  if (fours(p)) return p.bf16 ? go<uint16_t, 4>(p, a) : go<float, 4>(p, a);
  return p.bf16 ? go<uint16_t, 1>(p, a) : go<float, 1>(p, a);
}

}  // namespace ssm
