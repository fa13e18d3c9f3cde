// Gated linear recurrence over whole sequences and its gradient.
//
// One pass over the data.  A workgroup takes a piece of the sequence, W waves of TS steps each, for 64 V channels
// (V a lane).  A wave loads its steps at once, forms decays and inputs and folds them to h_out = A h_in + S; the
// waves' folds meet in LDS, and the piece's fold is published.  The state that enters the piece comes from the
// pieces before it: these are grouped in blocks of 8 or 32, a block's last piece publishes the state behind the
// block, and the others fold the (A, S) of the pieces before them in the block onto the state in front of it.  So
// a sequence's chain is one hop a block long, its sums have a fixed order (the block's length does not show in
// them), and every input is read once.
//
// Published words carry their own validity: a word is all ones until it is written, and no (A, S) or state is
// stored as that pattern.  Relaxed 64- and 32-bit atomics at agent scope are therefore enough.  The pieces of a
// chain are handed out by a counter of its own, earlier ones first: who waits for a piece waits for a workgroup
// that is running, whatever else the device runs.  A workspace that two calls share by mistake gives wrong
// results, but no access out of range (a piece beyond the last is left) and no endless wait (kPolls).
//
// The gradient runs the same way from the last piece to the first, on P_t = a_t (e_t + P_{t+1}), e = dy silu(z):
// what reaches the state before step t.  The states inside a piece are formed again from the state at its start,
// saved by the forward call or by a forward pass without outputs.  While a piece waits, it forms what its
// gradients are in multiples of g, the gradient of a step's state, so that six products a step are left then.  What is
// left of a gate, 1 - s, is formed without a difference and waits in LDS (gx) or comes from e^-ga once more: against
// products of s alone, which lose it for open gates, 8 x 2048 x 4096 with the forward call takes the same, 1 x 16384 x
// 2560 218 us for 215.
//
// Bound by HBM, and nearly as much by the vector units (33 instructions an element forward, six of them
// transcendental, busy 60% of the time).  Measured in bf16 (a copy reaches 5.1 to 5.3 TB/s): 4 x 8192 x 5120 with
// output gate 312 us, 5.4 TB/s; 1 x 32768 x 2560 146 us, 4.6 TB/s; 8 x 2048 x 4096 forward and gradient 325 us, 4.6
// TB/s.
// Shapes, before the last steps: 16 steps a wave and 8 waves forward, 1 x 32768 x 2560: 166 us; 8 steps 16 waves 195,
// 16 steps 4 waves 203, 8 steps 8 waves 202, 16 steps 16 waves 177; four channels a lane 222 against 153.  Gradient
// of 8 steps and 8 waves, 8 x 2048 x 4096 with the forward call: 369 us; 4 steps and 16 waves 475.
#include "col_sum.h"
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
  int64_t xs, as, is, zs;  // bytes between steps
  const void* dy;
  const float* dh_last;
  void* dx;
  void* dga;
  void* dgx;
  void* dz;
  float* part;  // [batch][pieces][width] sums of dlog_a
  float* dh0;
  uint32_t* tickets;  // [batch][tiles], all ones at first
  uint64_t* folds;   // [batch][pieces][width] (A, S)
  uint32_t* states;  // [batch][blocks][width]
  int32_t pieces, tiles, block;
  int32_t first;  // of all pieces of work, this launch's
};

constexpr int kMaxBlock = 32;      // pieces
constexpr int kPolls = 1 << 18;    // reads of a word before its wait is given up, 0.1 s at least
constexpr int kWavesPerSimd = 4;   // two workgroups a CU: one loads while the other computes or waits

__device__ __forceinline__ int steps_of(const GatedArgs& a, int64_t b) {
  if (a.lengths == nullptr) return (int)a.seqlen;
  const int n = a.lengths[b];
  return n < 0 ? 0 : n > (int)a.seqlen ? (int)a.seqlen : n;
}

// Rows go through buffer instructions: a resource (4 SGPRs) a tensor over this wave's steps, the
// lane's offset in one VGPR, the step's in an SGPR, so that an access costs no vector
// instruction.  Raw buffers (word 3 is the gfx9 data format, which must not be 0); what lies at or
// past `bytes` is not written.
typedef __amdgpu_buffer_rsrc_t rsrc_t;
__device__ __forceinline__ rsrc_t rows_of(const void* p, int64_t bytes_before, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(static_cast<const char*>(p)) + bytes_before, 0, (int)bytes,
                                           0x00020000);
}
constexpr uint32_t kNowhere = 0x80000000u;  // a lane's offset behind every resource

// How the caches take an access: in the usual way, or as data that passes through once.
constexpr int kUsual = 0, kOnce = 2;

// V values of one lane as loaded.
template <typename T, int V>
struct Io;
template <>
struct Io<float, 1> {
  uint32_t r;
  template <int HINT>
  __device__ __forceinline__ void load(rsrc_t b, uint32_t lane, uint32_t row) {
    r = __builtin_amdgcn_raw_buffer_load_b32(b, lane, row, HINT);
  }
  __device__ __forceinline__ float get(int) const { return __builtin_bit_cast(float, r); }
  __device__ __forceinline__ void forget() {}
};
template <>
struct Io<uint16_t, 1> {
  uint16_t r;
  template <int HINT>
  __device__ __forceinline__ void load(rsrc_t b, uint32_t lane, uint32_t row) {
    r = __builtin_amdgcn_raw_buffer_load_b16(b, lane, row, HINT);
  }
  __device__ __forceinline__ float get(int) const { return io_to_f32(r); }
  __device__ __forceinline__ void forget() {}
};
template <>
struct Io<uint16_t, 2> {
  uint32_t r;
  template <int HINT>
  __device__ __forceinline__ void load(rsrc_t b, uint32_t lane, uint32_t row) {
    r = __builtin_amdgcn_raw_buffer_load_b32(b, lane, row, HINT);
  }
  __device__ __forceinline__ float get(int v) const {
    return __builtin_bit_cast(float, v ? r & 0xffff0000u : r << 16);
  }
  // Makes the compiler forget what it has derived from the register: what is unpacked from it is
  // unpacked again where it is next used, instead of held in two more.
  __device__ __forceinline__ void forget() { asm volatile("" : "+v"(r)); }
};
template <int HINT>
__device__ __forceinline__ void put(rsrc_t b, uint32_t lane, uint32_t row, const float (&v)[1], const float*) {
  __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, v[0]), b, lane, row, HINT);
}
template <int HINT>
__device__ __forceinline__ void put(rsrc_t b, uint32_t lane, uint32_t row, const float (&v)[1], const uint16_t*) {
  __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, (__bf16)v[0]), b, lane, row, HINT);
}
template <int HINT>
__device__ __forceinline__ void put(rsrc_t b, uint32_t lane, uint32_t row, const float (&v)[2], const uint16_t*) {
  typedef float f2 __attribute__((ext_vector_type(2)));
  typedef __bf16 b2 __attribute__((ext_vector_type(2)));
  __builtin_amdgcn_raw_buffer_store_b32(
      __builtin_bit_cast(uint32_t, __builtin_convertvector(f2{v[0], v[1]}, b2)), b, lane, row, HINT);
}

// Fold of a piece, or of what lies behind it: h_out = a h + s.
struct Fold {
  float a, s;
  __device__ __forceinline__ float operator()(float h) const { return __builtin_fmaf(a, h, s); }
  __device__ __forceinline__ Fold then(Fold b) const { return Fold{a * b.a, b(s)}; }
};

__device__ __forceinline__ float quiet(float v) { return v != v ? __builtin_nanf("") : v; }
__device__ __forceinline__ void publish(uint64_t* p, Fold f) {
  const uint64_t w = ((uint64_t)__builtin_bit_cast(uint32_t, quiet(f.s)) << 32) | __builtin_bit_cast(uint32_t, f.a);
  __hip_atomic_store(p, w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void publish(uint32_t* p, float h) {
  __hip_atomic_store(p, __builtin_bit_cast(uint32_t, quiet(h)), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <typename W>
__device__ __forceinline__ W read_word(const W* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// The word when it is there (`first`: what was read before).  Given up, it is all ones, which reads as NaN.
template <typename W>
__device__ __forceinline__ W wait_word(const W* p, W first) {
  W w = first;
  for (int k = 0; w == (W)~(W)0 && k < kPolls; ++k) {
    __builtin_amdgcn_s_sleep(1);
    w = read_word(p);
  }
  return w;
}

// The chain of pieces, seen from piece q (counted in the chain's direction; its first piece is q0, its last `last`).
struct Link {
  int q, j0, blk, before;  // j0: the first piece of q's block, `before`: how many pieces of it come before q
  bool heads, closes, ends;  // nothing comes before the block; q is the block's last piece; nothing comes behind q
  __device__ __forceinline__ Link(int q_, int q0, int last, int block) : q(q_) {
    blk = q / block;
    heads = blk == q0 / block;
    j0 = heads ? q0 : blk * block;
    before = q - j0;
    closes = q % block == block - 1;
    ends = q == last;
  }
};

// What the pieces before hand on, word by word over the waves into LDS: the folds of the block's pieces before q,
// and the state in front of the block.  folds, states: of piece 0 and block 0 for this lane's channels,
// `stride` words from one to the next.
template <int V, int W>
__device__ __forceinline__ void collect(const Link& l, int wave, int lane, const uint64_t* folds,
                                        const uint32_t* states, int64_t stride, Fold (*pre)[64 * V], float* front) {
  for (int k = wave; k < l.before; k += W) {
    const uint64_t* const p = folds + (l.j0 + k) * stride;
    uint64_t w[V];
#pragma unroll
    for (int v = 0; v < V; ++v) w[v] = read_word(p + v);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const uint64_t f = wait_word(p + v, w[v]);
      pre[k][lane * V + v] =
          Fold{__builtin_bit_cast(float, (uint32_t)f), __builtin_bit_cast(float, (uint32_t)(f >> 32))};
    }
  }
  if (wave == W - 1 && !l.heads)
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const uint32_t* const p = states + (l.blk - 1) * stride + v;
      front[lane * V + v] = __builtin_bit_cast(float, wait_word(p, read_word(p)));
    }
}

// Workgroup i of a round over all chains takes this one.  Workgroups go to the 8 XCDs in turn, so that neighbours in i
// share no L2, while neighbouring tiles share the cache lines at their border where rows are not whole lines, and pages
// of memory always.  Eight neighbouring tiles therefore go to one XCD (forward and gradient of 8 x 2048 x 2049: 204
// us, else 248; 4 x 8192 x 5120 with output gate, before such rows passed the caches by: 333, else 346); not more, so
// that every XCD has a share of every row, which may end early (padded batch 8 x 2048 x 4096: 101 us, with 16 tiles
// 116, with an eighth of all 129).
__device__ __forceinline__ int neighbours(int i, int chains) {
  constexpr int kXcd = 8, kGroup = 8;
  const int whole = chains / (kXcd * kGroup) * (kXcd * kGroup);
  if (i >= whole) return whole + xcd_remap(i - whole, chains - whole);
  const int k = i / kXcd;
  return (k / kGroup * kXcd + i % kXcd) * kGroup + k % kGroup;
}

// Where a lane works: channels d .. d + V - 1 of row b, piece q of that chain.  Lanes behind the row's width do
// the last channels' work once more, and write the same values to the same places.
template <int V>
struct Spot {
  int64_t b, d;
  int q;
  // Work goes to the chains in turn.  Within one, the piece is the next that no workgroup has
  // started.  shared: read and written by the whole workgroup.
  __device__ __forceinline__ Spot(const GatedArgs& a, int* shared) {
    const int chains = a.tiles * (int)a.batch;
    const int chain = neighbours(((int)blockIdx.x + a.first) % chains, chains);
    b = chain / a.tiles;
    d = min(((int64_t)(chain % a.tiles) * 64 + (threadIdx.x & 63)) * V, a.width - V);
    q = 0;
    if (a.pieces > 1) {
      if (threadIdx.x == 0)
        *shared = (int)(__hip_atomic_fetch_add(a.tickets + chain, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) + 1u);
      __syncthreads();
      q = __builtin_amdgcn_readfirstlane(*shared);
    }
  }
};

// Steps row .. row + m - 1 (1 <= m <= TS) of one input; what lies behind them repeats the last.  (TS
// steps lie within 2^31 bytes.)
template <int HINT, typename T, int V, int TS>
__device__ __forceinline__ void load_steps(Io<T, V> (&r)[TS], const void* base, int64_t row, int64_t stride,
                                           uint32_t lane, int m) {
  const rsrc_t b = rows_of(base, row * stride, (uint32_t)TS * (uint32_t)stride);
#pragma unroll
  for (int i = 0; i < TS; ++i) r[i].template load<HINT>(b, lane, (uint32_t)min(i, m - 1) * (uint32_t)stride);
}

// Values that are formed here and now: the compiler would put many of them off to where they are used, and hold what
// they come from instead.
__device__ __forceinline__ void settle(float& a) { asm volatile("" : "+v"(a)); }
template <typename... F>
__device__ __forceinline__ void settle(float& a, F&... more) {
  settle(a);
  settle(more...);
}

template <typename T, int V, int TS, int W, bool Z, bool OUT, int GET, int PUT>
__global__ void __launch_bounds__(64 * W, kWavesPerSimd) k_gated_fwd(const GatedArgs a) {
  __shared__ Fold folds[W][64 * V], pre[kMaxBlock - 1][64 * V];
  __shared__ float front[64 * V];
  __shared__ int shared;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const Spot<V> at(a, &shared);
  if ((uint32_t)at.q >= (uint32_t)a.pieces) return;  // a counter that another call moves too
  const int n = steps_of(a, at.b), seqlen = (int)a.seqlen;
  const int c0 = at.q * (W * TS), t0 = c0 + wave * TS;
  const int m = min(max(n - t0, 0), TS);
  const int64_t row = at.b * a.seqlen + t0, st = at.b * a.width + at.d;
  const uint32_t off = (uint32_t)(at.d * sizeof(T)), ws = (uint32_t)(a.width * sizeof(T));
  const rsrc_t py = rows_of(a.y, row * ws, TS * ws);
  const T* const tag = nullptr;
  if (c0 >= n && at.q > 0) {  // behind the row's end
    const float o[V] = {};
    for (int i = 0; OUT && i < TS && t0 + i < seqlen; ++i)
      put<PUT>(py, off, i * ws, o, tag);
    return;
  }
  float dec[TS][V], u[TS][V], start[V];
#pragma unroll
  for (int v = 0; v < V; ++v) start[v] = a.h0 != nullptr && at.q < a.block ? a.h0[st + v] : 0.0f;
  Io<T, V> z[TS];
  if (m > 0) {
    Io<T, V> x[TS], ga[TS], gx[TS];
    load_steps<GET>(ga, a.ga, row, a.as, off, m);
    load_steps<GET>(gx, a.gx, row, a.is, off, m);
    load_steps<GET>(x, a.x, row, a.xs, off, m);
    float c2[V];
#pragma unroll
    for (int v = 0; v < V; ++v) c2[v] = a.log_a[at.d + v] * kLog2e;
#pragma unroll
    for (int i = 0; i < TS; ++i) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const GatedStep s = gated_step(ga[i].get(v), gx[i].get(v), c2[v]);
        dec[i][v] = s.a;
        u[i][v] = s.m() * s.sx * x[i].get(v);
      }
#pragma unroll
      for (int v = 0; v < V; ++v) settle(dec[i][v], u[i][v]);
    }
    if (Z && OUT) load_steps<GET>(z, a.z, row, a.zs, off, m);
  }
  if (m < TS)
#pragma unroll
    for (int i = 0; i < TS; ++i)
      if (i >= m)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          dec[i][v] = 1.0f;
          u[i][v] = 0.0f;
        }
  // h_last may be h0 itself, and is written only when every fold of the first block has been published (or behind a
  // barrier, by a piece that is alone): h0 is in registers before that.
#pragma unroll
  for (int v = 0; v < V; ++v) asm volatile("" : "+v"(start[v]));
  Fold f[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    f[v] = Fold{dec[0][v], u[0][v]};
#pragma unroll
    for (int i = 1; i < TS; ++i) f[v] = f[v].then(Fold{dec[i][v], u[i][v]});
    folds[wave][lane * V + v] = f[v];
  }
  __syncthreads();
  const Link l(at.q, 0, n > 0 ? (n - 1) / (W * TS) : 0, a.block);
  uint64_t* const fp = a.folds + at.b * a.pieces * a.width + at.d;
  uint32_t* const sp = a.states + at.b * ((a.pieces + a.block - 1) / a.block) * a.width + at.d;
  if (wave == 0 && !l.ends)
#pragma unroll
    for (int v = 0; v < V; ++v) {
      for (int k = 1; k < W; ++k) f[v] = f[v].then(folds[k][lane * V + v]);
      if (!l.closes) publish(fp + at.q * a.width + v, f[v]);
    }
  if (a.pieces > 1) {
    collect<V, W>(l, wave, lane, fp, sp, a.width, pre, front);
    __syncthreads();
  }
  float h[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    h[v] = l.heads ? start[v] : front[lane * V + v];
    for (int k = 0; k < l.before; ++k) h[v] = pre[k][lane * V + v](h[v]);
    if (wave == 0 && l.closes && !l.ends) publish(sp + l.blk * a.width + v, f[v](h[v]));
    for (int k = 0; k < wave; ++k) h[v] = folds[k][lane * V + v](h[v]);
  }
  if (a.ckpt != nullptr && t0 % kGatedCkpt == 0 && t0 < seqlen) {
    float* const ck = a.ckpt + (at.b * ((a.seqlen + kGatedCkpt - 1) / kGatedCkpt) + t0 / kGatedCkpt) * a.width + at.d;
#pragma unroll
    for (int v = 0; v < V; ++v) ck[v] = h[v];
  }
  // all: no step of these is behind the row's end (most waves need no checks).
  auto walk = [&](auto all) {
    constexpr bool ALL = decltype(all)::value;
#pragma unroll
    for (int i = 0; i < TS; ++i) {
      float o[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        h[v] = Fold{dec[i][v], u[i][v]}(h[v]);
        o[v] = Z && OUT ? h[v] * silu(z[i].get(v)) : h[v];
        if (!ALL && i >= m) o[v] = 0.0f;
      }
      if (OUT && (ALL || t0 + i < seqlen)) put<PUT>(py, off, i * ws, o, tag);
    }
  };
  if (m == TS)
    walk(std::true_type());
  else
    walk(std::false_type());
  // The last wave carries the state behind the row's last step to the end of its piece.
  if (a.h_last != nullptr && wave == W - 1 && l.ends)
#pragma unroll
    for (int v = 0; v < V; ++v) a.h_last[st + v] = h[v];
}

template <typename T, int V, int TS, int W, bool Z, int HINT>
__global__ void __launch_bounds__(64 * W, kWavesPerSimd) k_gated_bwd(const GatedArgs a) {
  __shared__ Fold fwd[W - 1][64 * V], rev[W][64 * V], pre[kMaxBlock - 1][64 * V];
  __shared__ float front[64 * V];
  // 1 - sx, which no register has room for; two workgroups (80 KB each with two channels a lane) still fit a CU.
  __shared__ __align__(8) float left[W][TS][64 * V];
  __shared__ int shared;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const Spot<V> at(a, &shared);  // q counts from the sequence's end
  if ((uint32_t)at.q >= (uint32_t)a.pieces) return;
  const int n = steps_of(a, at.b), seqlen = (int)a.seqlen;
  const int c = a.pieces - 1 - at.q, c0 = c * (W * TS), t0 = c0 + wave * TS;
  const int m = min(max(n - t0, 0), TS);
  const int64_t row = at.b * a.seqlen + t0, st = at.b * a.width + at.d;
  const int64_t step = a.width * (int64_t)sizeof(T);
  const uint32_t off = (uint32_t)(at.d * sizeof(T)), ws = (uint32_t)step;
  const rsrc_t px = rows_of(a.dx, row * step, TS * ws);
  const rsrc_t pa = rows_of(a.dga, row * step, TS * ws);
  const rsrc_t pi = rows_of(a.dgx, row * step, TS * ws);
  const rsrc_t pz = rows_of(a.dz, row * step, TS * ws);
  const T* const tag = nullptr;
  float* const part = a.part + (at.b * a.pieces + c) * a.width + at.d;
  if (c0 >= n) {  // behind the row's end
    const float o[V] = {};
    for (int i = 0; i < TS && t0 + i < seqlen; ++i) {
        put<HINT>(px, off, i * ws, o, tag);
        put<HINT>(pa, off, i * ws, o, tag);
        put<HINT>(pi, off, i * ws, o, tag);
        if (Z) put<HINT>(pz, off, i * ws, o, tag);
      }
    if (wave == 0)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (a.part != nullptr) part[v] = 0.0f;
        if (a.dh0 != nullptr && c == 0) a.dh0[st + v] = a.dh_last != nullptr ? a.dh_last[st + v] : 0.0f;
      }
    return;
  }
  Io<T, V> x[TS], dy[TS], z[TS];
  float dec[TS][V], ea[TS][V], kx[TS][V], i2[TS][V];  // ea = e^-ga, kx = m sx, i2 = 1 / m^2
  if (m > 0) {
    Io<T, V> ga[TS], gx[TS];
    load_steps<HINT>(ga, a.ga, row, a.as, off, m);
    load_steps<HINT>(gx, a.gx, row, a.is, off, m);
    load_steps<HINT>(x, a.x, row, a.xs, off, m);
    load_steps<HINT>(dy, a.dy, row, step, off, m);
    if (Z) load_steps<HINT>(z, a.z, row, a.zs, off, m);
    float c2[V];
#pragma unroll
    for (int v = 0; v < V; ++v) c2[v] = a.log_a[at.d + v] * kLog2e;
#pragma unroll
    for (int i = 0; i < TS; ++i) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const GatedStep s = gated_step(ga[i].get(v), gx[i].get(v), c2[v]);
        const float inv = s.inv_m();
        dec[i][v] = s.a;
        ea[i][v] = s.ea;
        i2[i][v] = inv * inv;
        kx[i][v] = s.m2 * inv * s.sx;
        left[wave][i][lane * V + v] = left_of(s.ex, s.sx);
      }
#pragma unroll
      for (int v = 0; v < V; ++v) settle(dec[i][v], ea[i][v], i2[i][v], kx[i][v]);
    }
  }
  if (m < TS)  // steps that do not exist hand everything on
#pragma unroll
    for (int i = 0; i < TS; ++i)
      if (i >= m) {
        x[i].r = 0;
        dy[i].r = 0;
        if (Z) z[i].r = 0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          dec[i][v] = 1.0f;
          ea[i][v] = __builtin_inff();  // a gate that is shut
          kx[i][v] = i2[i][v] = 0.0f;
          left[wave][i][lane * V + v] = 0.0f;
        }
      }
  Fold f[V], r[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    f[v] = Fold{dec[0][v], kx[0][v] * x[0].get(v)};
    r[v].s = 0.0f;
#pragma unroll
    for (int i = 1; i < TS; ++i) f[v] = f[v].then(Fold{dec[i][v], kx[i][v] * x[i].get(v)});
#pragma unroll
    for (int i = TS - 1; i >= 0; --i) {
      const float e = Z ? dy[i].get(v) * silu(z[i].get(v)) : dy[i].get(v);
      r[v].s = dec[i][v] * (e + r[v].s);
    }
    r[v].a = f[v].a;
    if (wave < W - 1) fwd[wave][lane * V + v] = f[v];
    rev[wave][lane * V + v] = r[v];
  }
  __syncthreads();
  const Link l(at.q, a.pieces - 1 - (n - 1) / (W * TS), a.pieces - 1, a.block);
  uint64_t* const fp = a.folds + at.b * a.pieces * a.width + at.d;
  uint32_t* const sp = a.states + at.b * ((a.pieces + a.block - 1) / a.block) * a.width + at.d;
  if (wave == W - 1 && !l.ends)
#pragma unroll
    for (int v = 0; v < V; ++v) {
      // The piece's fold from its last wave to its first.
      for (int k = W - 2; k >= 0; --k) r[v] = r[v].then(rev[k][lane * V + v]);
      if (!l.closes) publish(fp + at.q * a.width + v, r[v]);
    }
  // The states before each step, and what a step's gradients are in multiples of that of its state:
  //   dx = g kx, dgx = g ki, d(log a) sa = g gs, dga = g gs log_a ka.
  float gs[TS][V], ka[TS][V], ki[TS][V], e[TS][V];
  const int64_t saved = (a.seqlen + kGatedCkpt - 1) / kGatedCkpt;
  const float* const ck = a.ckpt + (at.b * saved + c0 / kGatedCkpt) * a.width + at.d;
  float h[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    h[v] = ck[v];
    for (int k = 0; k < wave; ++k) h[v] = fwd[k][lane * V + v](h[v]);
  }
#pragma unroll
  for (int i = 0; i < TS; ++i) {
    x[i].forget();
    dy[i].forget();
    if (Z) z[i].forget();
    float dz[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float ac = dec[i][v], u = kx[i][v] * x[i].get(v), s = sigmoid_of(ea[i][v]);
      gs[i][v] = ac * s * __builtin_fmaf(-(ac * i2[i][v]), u, h[v]);
      ka[i][v] = left_of(ea[i][v], s);
      ki[i][v] = u * left[wave][i][lane * V + v];
      h[v] = __builtin_fmaf(ac, h[v], u);
      if (Z) {
        const float zv = z[i].get(v), q = sigmoid(zv), d = dy[i].get(v);
        e[i][v] = d * (zv * q);
        dz[v] = i < m ? d * h[v] * q * __builtin_fmaf(zv, 1.0f - q, 1.0f) : 0.0f;
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      settle(gs[i][v], ka[i][v], ki[i][v], h[v]);
      if (Z) settle(e[i][v]);
    }
    if (Z) put<HINT>(pz, t0 + i < seqlen ? off : kNowhere, i * ws, dz, tag);
  }
  if (a.pieces > 1) {
    collect<V, W>(l, wave, lane, fp, sp, a.width, pre, front);
    __syncthreads();
  }
  float p[V], sum[V] = {}, la[V];
#pragma unroll
  for (int v = 0; v < V; ++v) la[v] = a.log_a[at.d + v];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    p[v] = !l.heads ? front[lane * V + v] : a.dh_last != nullptr ? a.dh_last[st + v] : 0.0f;
    for (int k = 0; k < l.before; ++k) p[v] = pre[k][lane * V + v](p[v]);
    if (wave == W - 1 && l.closes && !l.ends) publish(sp + l.blk * a.width + v, r[v](p[v]));
    for (int k = W - 1; k > wave; --k) p[v] = rev[k][lane * V + v](p[v]);
  }
  // all: no step of these is behind the row's end (most waves need no checks).
  auto walk = [&](auto all) {
    constexpr bool ALL = decltype(all)::value;
#pragma unroll
    for (int i = TS - 1; i >= 0; --i) {
      float dx[V], da[V], di[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float g = (Z ? e[i][v] : dy[i].get(v)) + p[v], t = g * gs[i][v];
        dx[v] = g * kx[i][v];
        di[v] = g * ki[i][v];
        da[v] = t * la[v] * ka[i][v];
        if (!ALL && i >= m) dx[v] = di[v] = da[v] = 0.0f;  // even where what comes from behind is not finite
        if (ALL || i < m) sum[v] += t;
        p[v] = dec[i][v] * g;
      }
      if (ALL || t0 + i < seqlen) {
        put<HINT>(px, off, i * ws, dx, tag);
        put<HINT>(pa, off, i * ws, da, tag);
        put<HINT>(pi, off, i * ws, di, tag);
      }
    }
  };
  if (m == TS)
    walk(std::true_type());
  else
    walk(std::false_type());
  if (a.dh0 != nullptr && c == 0 && wave == 0)
#pragma unroll
    for (int v = 0; v < V; ++v) a.dh0[st + v] = p[v];
  if (a.part == nullptr) return;
  // The waves' sums in their order.
  __syncthreads();
#pragma unroll
  for (int v = 0; v < V; ++v) rev[wave][lane * V + v].a = sum[v];
  __syncthreads();
  if (wave == 0)
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float t = 0.0f;
      for (int k = 0; k < W; ++k) t += rev[k][lane * V + v].a;
      part[v] = t;
    }
}

// All ones into n 16-byte words.
__global__ void __launch_bounds__(256) k_gated_clear(uint4* p, int64_t n) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i < n) p[i] = make_uint4(~0u, ~0u, ~0u, ~0u);
}

constexpr int kFwdSteps = 16, kFwdWaves = 8;  // 128 steps a piece
constexpr int kBwdSteps = 8, kBwdWaves = 8;   // 64: every piece starts at a saved state
static_assert(kBwdSteps * kBwdWaves % kGatedCkpt == 0 && kGatedCkpt % kFwdSteps == 0, "pieces start at saved states");
constexpr int64_t kMaxGrid = 1 << 22;  // workgroups of a launch

int64_t pieces_of(int64_t seqlen, int64_t len) { return seqlen <= len ? 1 : (seqlen + len - 1) / len; }
// Pieces of a block.  A wide block has fewer hops, but every piece reads half a block of folds: worth it
// where few chains leave the chip waiting for the hops (bf16, 32768 x 512: 64 us with 8, 51 with 32; 32768 x
// 1024, 8 chains, 82 and 80; 32768 x 1536, 12 chains, 103 and 104; gradient and forward of 16384 x 256: 98 and 69).
int64_t block_of(int64_t chains) { return chains <= 8 ? kMaxBlock : 8; }
int64_t blocks_of(int64_t pieces) { return (pieces + 7) / 8; }  // room for the narrow ones
// Words of 4 bytes that the chains use: the counters, the folds, the states.
int64_t ticket_words(int64_t batch, int64_t width) { return (batch * ((width + 63) / 64) + 63) / 64 * 64; }
int64_t chain_words(int64_t batch, int64_t width, int64_t pieces) {
  if (pieces <= 1) return 0;
  const int64_t n = ticket_words(batch, width) + batch * width * (2 * pieces + blocks_of(pieces));
  return (n + 63) / 64 * 64;
}

// Every address that the rows begin at, and every distance between rows, as one union of bits.
uint64_t places(const GatedScanLaunch& p) {
  uint64_t at = (uint64_t)(p.x_stride | p.ga_stride | p.gx_stride | p.width | (p.z != nullptr ? p.z_stride : 0));
  at *= p.bf16 ? 2 : 4;
  for (const void* q : {p.x, p.ga, p.gx, p.z, (const void*)p.y, p.dy, (const void*)p.dx, (const void*)p.dga,
                        (const void*)p.dgx, (const void*)p.dz})
    at |= reinterpret_cast<uintptr_t>(q);
  return at;
}
// Two bf16 channels a lane where every row allows 4-byte accesses.
bool pairs(const GatedScanLaunch& p) { return p.bf16 && places(p) % 4 == 0; }
// Rows of whole cache lines, 128 bytes: no two waves touch the same one (a wave's access is 128 or 256 bytes).
// Such calls let the caches take what they write, and what they read, as data used once: 4 x 8192 x 5120 with
// output gate 332 -> 312 us, 1 x 32768 x 2560 152 -> 146, forward and gradient of 8 x 2048 x 4096 347 -> 325 (fp32, 2 x
// 4096 x 2560: 186 -> 166), of 4 x 1024 x 2048 58 -> 53 (fp32, 2 x 1024 x 2048: 49 -> 46); 1 x 512 x 1024 the same,
// alone or with a norm or a product that reads y next.  A forward call that saves states reads in the usual way, since
// a gradient that may read the same again follows.  With lines that two waves share it is the other way round: 8 x
// 2048 x 2049 forward and gradient 204 -> 228 with such writes, 310 with both.
bool lines(const GatedScanLaunch& p) { return places(p) % 128 == 0; }

GatedArgs args(const GatedScanLaunch& p, int64_t pieces, uint32_t* chain) {
  const int64_t es = p.bf16 ? 2 : 4;
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
  a.xs = p.x_stride * es;
  a.as = p.ga_stride * es;
  a.is = p.gx_stride * es;
  a.zs = p.z_stride * es;
  a.dy = p.dy;
  a.dh_last = p.dh_last;
  a.dx = p.dx;
  a.dga = p.dga;
  a.dgx = p.dgx;
  a.dz = p.dz;
  a.dh0 = p.dh0;
  a.pieces = (int32_t)pieces;
  const int64_t lanes = pairs(p) ? 128 : 64;
  a.tiles = (int32_t)((p.width + lanes - 1) / lanes);
  a.block = (int32_t)block_of(p.batch * a.tiles);
  if (pieces > 1) {
    a.tickets = chain;
    a.folds = reinterpret_cast<uint64_t*>(chain + ticket_words(p.batch, p.width));
    a.states = chain + ticket_words(p.batch, p.width) + 2 * p.batch * p.width * pieces;
  }
  return a;
}

hipError_t clear(uint32_t* p, int64_t words, hipStream_t stream) {
  if (words == 0) return hipSuccess;
  const int64_t n = words / 4;
  return launch(k_gated_clear, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, stream, reinterpret_cast<uint4*>(p), n);
}

// All pieces of all chains, in as many launches as it takes.
template <typename K>
hipError_t go(K kern, GatedArgs a, int threads, hipStream_t stream) {
  const int64_t items = a.batch * a.tiles * a.pieces;
  for (int64_t i = 0; i < items; i += kMaxGrid) {
    a.first = (int32_t)i;
    const int64_t n = items - i < kMaxGrid ? items - i : kMaxGrid;
    const hipError_t rc = launch(kern, dim3((unsigned)n), dim3(threads), 0, stream, a);
    if (rc != hipSuccess) return rc;
  }
  return hipSuccess;
}

template <typename T, int V, bool OUT, int GET, int PUT>
hipError_t go_fwd(const GatedArgs& a, hipStream_t stream) {
  return OUT && a.z != nullptr
             ? go(k_gated_fwd<T, V, kFwdSteps, kFwdWaves, OUT, OUT, GET, PUT>, a, 64 * kFwdWaves, stream)
             : go(k_gated_fwd<T, V, kFwdSteps, kFwdWaves, false, OUT, GET, PUT>, a, 64 * kFwdWaves, stream);
}
template <typename T, int V, int HINT>
hipError_t go_bwd(const GatedArgs& a, hipStream_t stream) {
  return a.z != nullptr ? go(k_gated_bwd<T, V, kBwdSteps, kBwdWaves, true, HINT>, a, 64 * kBwdWaves, stream)
                        : go(k_gated_bwd<T, V, kBwdSteps, kBwdWaves, false, HINT>, a, 64 * kBwdWaves, stream);
}
template <typename T, int V, bool OUT>
hipError_t fwd_lines(const GatedScanLaunch& p, const GatedArgs& a) {
  if (!OUT || !lines(p)) return go_fwd<T, V, OUT, kUsual, kUsual>(a, p.stream);
  return a.ckpt != nullptr ? go_fwd<T, V, OUT, kUsual, OUT ? kOnce : kUsual>(a, p.stream)
                           : go_fwd<T, V, OUT, OUT ? kOnce : kUsual, OUT ? kOnce : kUsual>(a, p.stream);
}
template <bool OUT>
hipError_t fwd(const GatedScanLaunch& p, const GatedArgs& a) {
  return !p.bf16    ? fwd_lines<float, 1, OUT>(p, a)
         : pairs(p) ? fwd_lines<uint16_t, 2, OUT>(p, a)
                    : go_fwd<uint16_t, 1, OUT, kUsual, kUsual>(a, p.stream);
}
hipError_t bwd(const GatedScanLaunch& p, const GatedArgs& a) {
  if (lines(p)) return p.bf16 ? go_bwd<uint16_t, 2, kOnce>(a, p.stream) : go_bwd<float, 1, kOnce>(a, p.stream);
  return !p.bf16    ? go_bwd<float, 1, kUsual>(a, p.stream)
         : pairs(p) ? go_bwd<uint16_t, 2, kUsual>(a, p.stream)
                    : go_bwd<uint16_t, 1, kUsual>(a, p.stream);
}

constexpr int64_t kFwdLen = kFwdSteps * kFwdWaves, kBwdLen = kBwdSteps * kBwdWaves;

}  // namespace

int64_t gated_scan_items(int64_t batch, int64_t seqlen, int64_t width) {
  return batch * ((width + 63) / 64) * pieces_of(seqlen, kBwdLen);
}
int64_t gated_scan_ckpt_floats(int64_t batch, int64_t seqlen, int64_t width) {
  return batch * ((seqlen + kGatedCkpt - 1) / kGatedCkpt) * width;
}
int64_t gated_scan_fwd_floats(int64_t batch, int64_t seqlen, int64_t width, bool) {
  return chain_words(batch, width, pieces_of(seqlen, kFwdLen));
}
int64_t gated_scan_bwd_floats(int64_t batch, int64_t seqlen, int64_t width, bool, bool ckpt_given) {
  const int64_t pieces = pieces_of(seqlen, kBwdLen);
  int64_t n = chain_words(batch, width, pieces) + (batch * pieces * width + 63) / 64 * 64;
  if (!ckpt_given)
    n += gated_scan_fwd_floats(batch, seqlen, width, true) + gated_scan_ckpt_floats(batch, seqlen, width);
  return n;
}

hipError_t launch_gated_scan_fwd(const GatedScanLaunch& p) {
  const int64_t pieces = pieces_of(p.seqlen, kFwdLen);
  uint32_t* const words = reinterpret_cast<uint32_t*>(p.workspace);
  const hipError_t rc = clear(words, chain_words(p.batch, p.width, pieces), p.stream);
  return rc != hipSuccess ? rc : fwd<true>(p, args(p, pieces, words));
}

// The workspace: the gradient's chain, the forward pass's chain when there is one, the sums of
// dlog_a, the states.
hipError_t launch_gated_scan_bwd(const GatedScanLaunch& p) {
  const int64_t pieces = pieces_of(p.seqlen, kBwdLen), fpieces = pieces_of(p.seqlen, kFwdLen);
  uint32_t* const words = reinterpret_cast<uint32_t*>(p.workspace);
  const bool again = p.ckpt == nullptr;
  const int64_t back = chain_words(p.batch, p.width, pieces);
  const int64_t fore = again ? chain_words(p.batch, p.width, fpieces) : 0;
  float* const part = p.workspace + back + fore;
  if (p.batch > 0) {
    hipError_t rc = clear(words, back + fore, p.stream);
    if (rc != hipSuccess) return rc;
    GatedArgs a = args(p, pieces, words);
    a.part = p.dlog_a != nullptr ? part : nullptr;
    if (again) {
      a.ckpt = part + (p.batch * pieces * p.width + 63) / 64 * 64;
      GatedArgs f = args(p, fpieces, words + back);
      f.ckpt = a.ckpt;
      if (p.seqlen > 0 && (rc = fwd<false>(p, f)) != hipSuccess) return rc;
    }
    if ((rc = bwd(p, a)) != hipSuccess) return rc;
  }
  if (p.dlog_a == nullptr) return hipSuccess;
  return col_sum(part, p.dlog_a, nullptr, 0, p.batch * pieces, p.width, p.stream);
}

}  // namespace ssm
