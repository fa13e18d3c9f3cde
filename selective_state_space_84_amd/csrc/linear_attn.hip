// Linear attention with a constant decay per head: the sweep on the fp32
// matrix instructions, the carries between spans, the sums over shared heads,
// and the launch sequences of the forward and gradient calls.
#include "linear_attn.h"

namespace ssm {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint16_t u16x4 __attribute__((ext_vector_type(4)));

// ---- the sweep, fp32 products -------------------------------------------
//
// One workgroup (4 waves) per (row, head), span and slice of 64 output
// columns; wave w owns 16 of them, for the outputs and for the state, which
// stays in the accumulators.  Blocks of 32 steps: a, b and c are staged in LDS
// as fp32 while the next block's rows are on their way in registers.  All
// products run on v_mfma_f32_16x16x4_f32: S^T = B A^T (shared through LDS),
// out^T = C^T P^T + E^T A^T, E += B^T (w o C).  The contraction index is
// taken in the order the accumulators hold rows (4 (lane / 16) + j), so the
// state and the 16-byte LDS reads feed the products without moving.
//
// Bound by the fp32 matrix rate (153 TFLOP/s in a large product on this
// card), an eighth of the bf16 one; 32 steps keep the pair products (which
// grow with the block) below a fifth of the state products.  1 x 4096 steps x 16
// heads of 128: 114 us with the spans' states, 38 TFLOP/s counting only the two
// products of a step with the state: with one workgroup a CU a SIMD has one wave,
// whose LDS reads and three barriers a block nothing covers.
constexpr int kT = 32;        // steps per block
constexpr int kCols = 64;     // output columns per workgroup
constexpr int kSc = kCols + 4;  // LDS row strides (floats) with rows 4 apart on different banks
constexpr int kSp = kT + 4;

__device__ __forceinline__ f32x4 load4(const float* p) { return *reinterpret_cast<const f32x4*>(p); }
__device__ __forceinline__ void store4(float* p, const f32x4& v) { *reinterpret_cast<f32x4*>(p) = v; }
__device__ __forceinline__ void store4(uint16_t* p, const f32x4& v) {
  u16x4 r;
#pragma unroll
  for (int j = 0; j < 4; ++j) r[j] = __builtin_bit_cast(uint16_t, (__bf16)v[j]);
  *reinterpret_cast<u16x4*>(p) = r;
}

// LDS of a sweep with operands of KD columns (floats).
constexpr int sum_lds(int kd) { return kT * (kd + 4 + kSc); }
constexpr int sweep_lds(int kd) { return sum_lds(kd) + kT * (kd + 4 + kSp); }
constexpr int larger(int a, int b) { return a > b ? a : b; }

// One slice of one span of one row.  VD: all output columns.  SUM: only the state
// of the span from a zero entry (a and out unused).
template <int KD, int VD, bool REV, bool SUM>
__device__ __forceinline__ void sweep_span_f32(const AttnSweep& s, float* lds, int64_t row, int64_t span, int slice) {
  constexpr int kSa = KD + 4;
  constexpr int NT = KD / 16;          // state tiles
  constexpr int PA = kT * KD / 4 / 256;  // 4-element pieces of a and b per thread
  constexpr int PC = kT * kCols / 4 / 256;
  float* const sB = lds;
  float* const sC = sB + kT * kSa;
  float* const sA = sC + kT * kSc;
  float* const sP = sA + kT * kSa;  // decayed pairs [t][i]

  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r16 = lane & 15, q4 = lane >> 4;
  const int64_t b = row / s.nheads;
  const int h = (int)(row % s.nheads);
  const int col0 = slice * kCols;
  const int64_t len = row_length(s.lengths, b, s.seqlen);
  const int64_t s0 = span * s.span_len;
  const int64_t s1 = min(s0 + s.span_len, s.seqlen);
  const int64_t e = min(s1, len) > s0 ? min(s1, len) : s0;  // steps [s0, e) are computed
  const float g = decay_log2(s.log_decay[h]);

  const float* const A = SUM ? nullptr : static_cast<const float*>(s.a.p) + b * s.seqlen * s.a.stride + (h / s.a.rep) * KD;
  const float* const B = static_cast<const float*>(s.b.p) + b * s.seqlen * s.b.stride + (h / s.b.rep) * KD;
  const float* const C = static_cast<const float*>(s.c.p) + b * s.seqlen * s.c.stride + (h / s.c.rep) * VD + col0;
  float* const out = SUM ? nullptr : static_cast<float*>(s.out) + (b * s.seqlen * s.nheads + h) * VD + col0;

  // State S[n][p], p = 16 w + r16 of the slice: acc[nt][j] = S[16 nt + 4 q4 + j][p].
  f32x4 acc[NT];
  const int64_t soff = (int64_t)(col0 + 16 * w + r16) * s.sp;
  {
    const float* ep = nullptr;
    if (!SUM && s.entry != nullptr) ep = s.entry + ((s.n_spans > 1 ? span * s.rows : 0) + row) * KD * VD + soff;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[nt][j] = ep != nullptr ? ep[(16 * nt + 4 * q4 + j) * s.sn] : 0.f;
  }

  f32x4 ra[SUM ? 1 : PA], rb[PA], rc[PC];
  auto fetch = [&](int64_t t0) {
    const int m = (int)min((int64_t)kT, e - t0);
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int r = 0; r < PA; ++r) {
      const int piece = tid + 256 * r, t = piece / (KD / 4), n = piece % (KD / 4) * 4;
      if (!SUM) ra[r] = t < m ? load4(A + (t0 + t) * s.a.stride + n) : zero;
      rb[r] = t < m ? load4(B + (t0 + t) * s.b.stride + n) : zero;
    }
#pragma unroll
    for (int r = 0; r < PC; ++r) {
      const int piece = tid + 256 * r, t = piece / (kCols / 4), p = piece % (kCols / 4) * 4;
      rc[r] = t < m ? load4(C + (t0 + t) * s.c.stride + p) : zero;
    }
  };

  const int64_t nblk = (e - s0 + kT - 1) / kT;
  if (nblk > 0) fetch(s0 + (REV ? nblk - 1 : 0) * kT);
  for (int64_t k = 0; k < nblk; ++k) {
    const int64_t t0 = s0 + (REV ? nblk - 1 - k : k) * kT;
    const int m = (int)min((int64_t)kT, e - t0);
    __syncthreads();  // the previous block is done with the tiles
#pragma unroll
    for (int r = 0; r < PA; ++r) {
      const int piece = tid + 256 * r, t = piece / (KD / 4), n = piece % (KD / 4) * 4;
      if (!SUM) *reinterpret_cast<f32x4*>(&sA[t * kSa + n]) = ra[r];
      *reinterpret_cast<f32x4*>(&sB[t * kSa + n]) = rb[r];
    }
#pragma unroll
    for (int r = 0; r < PC; ++r) {
      const int piece = tid + 256 * r, t = piece / (kCols / 4), p = piece % (kCols / 4) * 4;
      *reinterpret_cast<f32x4*>(&sC[t * kSc + p]) = rc[r];
    }
    __syncthreads();
    if (k + 1 < nblk) fetch(s0 + (REV ? nblk - 2 - k : k + 1) * kT);

    if (!SUM) {
      // Pairs: tile (it, tt) of wave w, rows i, columns t; the masked one is zero.
      const int it = w >> 1, tt = w & 1;
      f32x4 sc = {0.f, 0.f, 0.f, 0.f};
      if (REV ? it >= tt : it <= tt) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const f32x4 bv = *reinterpret_cast<const f32x4*>(&sB[(16 * it + r16) * kSa + 16 * nt + 4 * q4]);
          const f32x4 av = *reinterpret_cast<const f32x4*>(&sA[(16 * tt + r16) * kSa + 16 * nt + 4 * q4]);
#pragma unroll
          for (int j = 0; j < 4; ++j) sc = __builtin_amdgcn_mfma_f32_16x16x4f32(bv[j], av[j], sc, 0, 0, 0);
        }
      }
      const int t = 16 * tt + r16;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = 16 * it + 4 * q4 + j;
        const int d = REV ? i - t : t - i;
        // In reverse rows without a step come last: their zeros would meet powers beyond the block's steps
        // (infinite where gamma is above 1).
        sc[j] = d >= 0 && (!REV || i < m) ? sc[j] * (hw_exp2(g * (float)d) * s.s_pair) : 0.f;
      }
      *reinterpret_cast<f32x4*>(&sP[t * kSp + 16 * it + 4 * q4]) = sc;
      __syncthreads();
    }

    // This wave's columns of c over the block: cv[it][j] = c[16 it + 4 q4 + j][p].
    f32x4 cv[2];
#pragma unroll
    for (int it = 0; it < 2; ++it)
#pragma unroll
      for (int j = 0; j < 4; ++j) cv[it][j] = sC[(16 * it + 4 * q4 + j) * kSc + 16 * w + r16];

    if (!SUM) {
#pragma unroll
      for (int tt = 0; tt < 2; ++tt) {
        const int t = 16 * tt + r16;
        f32x4 op = {0.f, 0.f, 0.f, 0.f}, oe = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int it = 0; it < 2; ++it) {
          const f32x4 pv = *reinterpret_cast<const f32x4*>(&sP[t * kSp + 16 * it + 4 * q4]);
#pragma unroll
          for (int j = 0; j < 4; ++j) op = __builtin_amdgcn_mfma_f32_16x16x4f32(cv[it][j], pv[j], op, 0, 0, 0);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const f32x4 av = *reinterpret_cast<const f32x4*>(&sA[t * kSa + 16 * nt + 4 * q4]);
#pragma unroll
          for (int j = 0; j < 4; ++j) oe = __builtin_amdgcn_mfma_f32_16x16x4f32(acc[nt][j], av[j], oe, 0, 0, 0);
        }
        if (t < m) {
          const float rf = hw_exp2(g * (float)(REV ? m - 1 - t : t + 1)) * s.s_read;
          f32x4 v;
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] = __builtin_fmaf(rf, oe[j], op[j]);
          store4(out + (t0 + t) * s.nheads * VD + 16 * w + 4 * q4, v);
        }
      }
    }

    // E <- gamma^m E + B^T (w o C).
    const float fac = hw_exp2(g * (float)m);
#pragma unroll
    for (int it = 0; it < 2; ++it)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = 16 * it + 4 * q4 + j;
        const float wt = i < m ? hw_exp2(g * (float)(REV ? i + 1 : m - 1 - i)) * s.s_write : 0.f;
        cv[it][j] *= wt;
      }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      acc[nt] *= fac;
#pragma unroll
      for (int it = 0; it < 2; ++it)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float bv = sB[(16 * it + 4 * q4 + j) * kSa + 16 * nt + r16];
          acc[nt] = __builtin_amdgcn_mfma_f32_16x16x4f32(bv, cv[it][j], acc[nt], 0, 0, 0);
        }
    }
  }

  if (!SUM) {
    // Rows behind the sequence's end.
    for (int64_t t = e + (tid >> 4); t < s1; t += 16)
      store4(out + t * s.nheads * VD + 4 * (tid & 15), f32x4{0.f, 0.f, 0.f, 0.f});
  }
  if (s.exit != nullptr && (SUM || span == (REV ? 0 : s.n_spans - 1))) {
    float* xp = s.exit + ((SUM ? span * s.rows : 0) + row) * KD * VD + soff;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 4; ++j) xp[(16 * nt + 4 * q4 + j) * s.sn] = acc[nt][j];
  }
}

// The forward sweep; the spans' own states (role 0: of H, role 1: of G); and the
// three gradient sweeps in one launch.  Slices and roles of one row and span are
// neighbours, and find each other's operands in their XCD's L2.
template <int KD, int VD>
__global__ void __launch_bounds__(256) k_attn_sweep_f32(const AttnSweep s) {
  __shared__ __align__(16) float lds[sweep_lds(KD)];
  constexpr int N = VD / kCols;
  const int64_t id = xcd_remap(blockIdx.x, gridDim.x);
  sweep_span_f32<KD, VD, false, false>(s, lds, id / N % s.rows, id / N / s.rows, (int)(id % N));
}

template <int KD, int VD>
__global__ void __launch_bounds__(256) k_attn_span_states_f32(const AttnSweep f, const AttnSweep r, int roles) {
  __shared__ __align__(16) float lds[sum_lds(KD)];
  const int n = VD / kCols * roles;
  const int64_t id = xcd_remap(blockIdx.x, gridDim.x);
  const int64_t row = id / n % f.rows, span = id / n / f.rows;
  const int part = (int)(id % n), slice = part % (VD / kCols);
  if (part < VD / kCols) {
    sweep_span_f32<KD, VD, false, true>(f, lds, row, span, slice);
  } else {
    sweep_span_f32<KD, VD, true, true>(r, lds, row, span + 1, slice);
  }
}

template <int DK, int DV>
__global__ void __launch_bounds__(256) k_attn_sweep_grad_f32(const AttnSweep q, const AttnSweep k, const AttnSweep v) {
  __shared__ __align__(16) float lds[larger(sweep_lds(DK), sweep_lds(DV))];
  constexpr int NK = DK / kCols, N = 2 * NK + DV / kCols;
  const int64_t id = xcd_remap(blockIdx.x, gridDim.x);
  const int64_t row = id / N % q.rows, span = id / N / q.rows;
  const int part = (int)(id % N);
  if (part < NK) {
    sweep_span_f32<DV, DK, false, false>(q, lds, row, span, part);
  } else if (part < 2 * NK) {
    sweep_span_f32<DV, DK, true, false>(k, lds, row, span, part - NK);
  } else {
    sweep_span_f32<DK, DV, true, false>(v, lds, row, span, part - 2 * NK);
  }
}

// ---- carries between spans ----------------------------------------------
// In place: st[span][row][...] holds every span's state from a zero entry (but
// the last one's) and receives the state that enters the span: E_0 = start,
// E_{s+1} = gamma^len_s E_s + S_s (from the last span downwards in reverse).
// Four elements a thread, sums in span order.  Bound by HBM: 67 MB in 13 us (16
// spans of 32 states of 128 x 128).
struct AttnCarry {
  float* st;
  const float* start;  // nullable for zeros
};
template <bool REV>
__device__ __forceinline__ void carry_spans(const AttnCarry& c, const AttnSweep& s, int64_t state4) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= s.rows * state4) return;
  const int64_t row = i / state4, n = s.n_spans;
  const float g = decay_log2(s.log_decay[row % s.nheads]);
  const int64_t len = row_length(s.lengths, row / s.nheads, s.seqlen);
  f32x4* const p = reinterpret_cast<f32x4*>(c.st) + i;
  f32x4 e = c.start != nullptr ? reinterpret_cast<const f32x4*>(c.start)[i] : f32x4{0.f, 0.f, 0.f, 0.f};
  constexpr int kAhead = 8;  // spans on their way
  for (int64_t k0 = 0; k0 < n; k0 += kAhead) {
    f32x4 own[kAhead];
#pragma unroll
    for (int x = 0; x < kAhead; ++x) {
      const int64_t k = k0 + x < n - 1 ? k0 + x : n - 2;
      own[x] = p[(REV ? n - 1 - k : k) * s.rows * state4];
    }
#pragma unroll
    for (int x = 0; x < kAhead; ++x) {
      const int64_t k = k0 + x;
      if (k >= n) break;
      const int64_t sp = REV ? n - 1 - k : k;
      p[sp * s.rows * state4] = e;
      const int64_t s0 = sp * s.span_len, s1 = min(s0 + s.span_len, s.seqlen);
      const int64_t m = min(s1, len) > s0 ? min(s1, len) - s0 : 0;
      const float f = hw_exp2(g * (float)m);
#pragma unroll
      for (int j = 0; j < 4; ++j) e[j] = __builtin_fmaf(f, e[j], own[x][j]);
    }
  }
}
// blockIdx.y 1: in reverse.
__global__ void __launch_bounds__(256) k_attn_carry(const AttnCarry f, const AttnCarry r, const AttnSweep s,
                                                    int64_t state4) {
  if (blockIdx.y == 0) {
    carry_spans<false>(f, s, state4);
  } else {
    carry_spans<true>(r, s, state4);
  }
}

// ---- sums over the heads that share a key/value head --------------------
// blockIdx.y: dk or dv; part holds [step][nheads][4 d4] fp32 (and is not read without query heads: rep 0, zeros).
struct HeadSum {
  const float* part;
  void* out;
  int64_t n4;  // steps x kv heads x d4
  int32_t d4;
};
template <typename T>
__global__ void __launch_bounds__(256) k_attn_sum_heads(const HeadSum k, const HeadSum v, int32_t rep) {
  const HeadSum& s = blockIdx.y == 0 ? k : v;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;  // (step, kv head, 4 columns)
  if (i >= s.n4) return;
  const int64_t head = i / s.d4;
  const f32x4* p = reinterpret_cast<const f32x4*>(s.part) + head * rep * s.d4 + i % s.d4;
  f32x4 x = rep > 0 ? p[0] : f32x4{0.f, 0.f, 0.f, 0.f};
  for (int r = 1; r < rep; ++r) x += p[(int64_t)r * s.d4];
  store4(static_cast<T*>(s.out) + i * 4, x);
}

int64_t up64(int64_t n) { return (n + 63) / 64 * 64; }

hipError_t launch_attn_sweep_f32(const AttnSweep& s, int64_t kd, int64_t vd, hipStream_t stream) {
  const unsigned grid = (unsigned)(s.rows * s.n_spans * (vd / kCols));
  return by_width(kd, vd, [&](auto k, auto v) {
    return launch(k_attn_sweep_f32<decltype(k)::value, decltype(v)::value>, dim3(grid), dim3(256), 0, stream, s);
  });
}

hipError_t launch_attn_span_states_f32(const AttnSweep& f, const AttnSweep* r, int64_t kd, int64_t vd,
                                       hipStream_t stream) {
  const int roles = r != nullptr ? 2 : 1;
  const unsigned grid = (unsigned)(f.rows * (f.n_spans - 1) * (vd / kCols) * roles);
  return by_width(kd, vd, [&](auto k, auto v) {
    return launch(k_attn_span_states_f32<decltype(k)::value, decltype(v)::value>, dim3(grid), dim3(256), 0, stream, f,
                  r != nullptr ? *r : f, roles);
  });
}

hipError_t launch_attn_sweep_grad_f32(const AttnSweep& q, const AttnSweep& k, const AttnSweep& v, int64_t d_k,
                                      int64_t d_v, hipStream_t stream) {
  const unsigned grid = (unsigned)(q.rows * q.n_spans * ((2 * d_k + d_v) / kCols));
  return by_width(d_k, d_v, [&](auto a, auto b) {
    return launch(k_attn_sweep_grad_f32<decltype(a)::value, decltype(b)::value>, dim3(grid), dim3(256), 0, stream, q,
                  k, v);
  });
}

// The states that enter the spans, of H from h0 into hs and (gs not NULL) of G
// from dh_last into gs; f and r are the sweeps that add to them.
hipError_t span_entries(const LinAttnLaunch& p, AttnSweep f, AttnSweep r, float* hs, float* gs) {
  f.sn = r.sn = 1;
  f.sp = r.sp = p.d_k;
  f.exit = hs;
  r.exit = gs;
  const AttnSweep* const rev = gs != nullptr ? &r : nullptr;
  const hipError_t rc = p.bf16 ? launch_attn_span_states_bf16(f, rev, p.d_k, p.d_v, p.stream)
                               : launch_attn_span_states_f32(f, rev, p.d_k, p.d_v, p.stream);
  if (rc != hipSuccess) return rc;
  const int64_t state4 = p.d_k * p.d_v / 4;
  const unsigned grid = (unsigned)((f.rows * state4 + 255) / 256);
  return launch(k_attn_carry, dim3(grid, gs != nullptr ? 2 : 1), dim3(256), 0, p.stream, AttnCarry{hs, p.h0},
                AttnCarry{gs, p.dh_last}, f, state4);
}

AttnSweep base(const LinAttnLaunch& p, const LinAttnPlan& pl) {
  AttnSweep s{};
  s.log_decay = p.log_decay;
  s.lengths = p.lengths;
  s.seqlen = p.seqlen;
  s.span_len = pl.span_len;
  s.n_spans = pl.n_spans;
  s.nheads = (int32_t)p.nheads;
  s.rows = p.batch * p.nheads;
  return s;
}

}  // namespace

// When the (row, head) pairs are few, the sequence is cut into spans, at the
// price of a pass over b and c for the spans' states: as many spans as make two
// workgroups a CU (512 in all), or one a CU where they would be shorter than
// kShortSpan steps; kMaxSpans at most (the carry walks them one after the other),
// of whole steps of kSpanStep, rounded up.  Two spans do not pay: a CU takes
// two blocks of different workgroups together in ~1.6 times the time of one, and
// the states cost 0.4 of a sweep.  Measured (bf16, heads of 128): 8 x 2048 steps x
// 32 heads 157 us whole, 202 us in two spans; 1 x 32768 x 32 402 us in 16 spans,
// 433 us in 8, 440 us in 32; 1 x 4096 x 16 50 us in 16 spans, 58 us in 32; 1 x 8000
// x 1 38 us in 63 spans, 50 us in 125.
// In bf16 spans of one block (64 steps) pay against two where they and their states
// (of both directions in the gradient), which the carry moves, are few, and again
// where they give nearly every CU a workgroup: 1 x 1000 x 4 24.1 and 26.5 us, 1500 x 4
// (96 states) 27.5 and 28.5, 2000 x 1 (32 spans) 25.0 and 26.9; 896 x 16 (224 states)
// 31.5 and 32.2, 1000 x 16 30.2 and 33.4, 2000 x 8 (256) 32.1 and 34.1; not between:
// 1700 x 4 (108) 29.8 and 27.8, 1500 x 8 (192) 33.7 and 31.9, gradient of 1300 x 4 (168)
// 32.0 and 31.1; nor in more than 32 spans: 2500 x 4 35.9 and 32.1, 3500 x 1 31.1 and
// 28.7 (2500 x 1 27.1 and 28.1).  In fp32, whose blocks take longer, they pay
// throughout: 1000 x 4 36.9 and 45.6, 4000 x 1 42.3 and 46.7.
// Short sequences stay whole, since three launches cost more than the blocks they
// save: 1 x 256 steps x 4 heads whole 19.9 us, cut 22.8, 1 x 320 x 4 23.6 and 22.9
// (gradient of 256 x 2 20.5 and 28.4, 512 x 2 35.2 and 28.3); fp32 192 x 4 31.0 and
// 32.3, 256 x 4 38.9 and 32.5.
constexpr int64_t kTargetGroups = 512;
constexpr int64_t kShortSpan = 256;
constexpr int64_t kMaxSpans = 64;
constexpr int64_t kSpanStep = 64;  // spans start on block boundaries of both sweeps
constexpr int64_t kMinCutBf16 = 320, kMinCutF32 = 256;
constexpr int64_t kOneBlockSpans = 32, kOneBlockFew = 96, kOneBlockMany = 200;

// states: of one span, in both directions for the gradient.
static LinAttnPlan make_plan(int64_t groups, int64_t states, int64_t seqlen, bool bf16) {
  const int64_t steps = seqlen > 0 ? (seqlen + kSpanStep - 1) / kSpanStep : 1;  // of kSpanStep, the last one not whole
  int64_t n = groups > 0 ? kTargetGroups / groups : 1;
  if (groups > 0 && n > seqlen / kShortSpan) n = kTargetGroups / 2 / groups;
  if (n > kMaxSpans) n = kMaxSpans;
  if (n < 1 || seqlen < (bf16 ? kMinCutBf16 : kMinCutF32)) n = 1;
  int64_t each = (steps + n - 1) / n;
  const bool between = steps * states > kOneBlockFew && steps * states < kOneBlockMany;
  if (bf16 && each == 1 && (steps > kOneBlockSpans || between)) each = 2;
  if ((steps + each - 1) / each < 3) each = steps;
  return LinAttnPlan{each * kSpanStep, (steps + each - 1) / each};
}

// The three gradient sweeps share a launch, and the fp32 sweep has a workgroup for
// every 64 columns.
int64_t linear_attn_groups(int64_t batch, int64_t nheads, int64_t d_k, int64_t d_v, bool bf16, bool grad) {
  return batch * nheads * (bf16 ? (grad ? 3 : 1) : (grad ? 2 * d_k + d_v : d_v) / kCols);
}

int64_t linear_attn_sum_threads(int64_t batch, int64_t seqlen, int64_t nheads_kv, int64_t d_k, int64_t d_v) {
  return (batch * seqlen * nheads_kv * (d_k > d_v ? d_k : d_v) / 4 + 255) / 256 * 256;
}

LinAttnPlan linear_attn_plan(int64_t batch, int64_t seqlen, int64_t nheads, int64_t d_k, int64_t d_v, bool bf16,
                             bool grad) {
  return make_plan(linear_attn_groups(batch, nheads, d_k, d_v, bf16, grad), batch * nheads * (grad ? 2 : 1), seqlen,
                   bf16);
}

static int64_t span_floats(int64_t batch, int64_t nheads, int64_t d_k, int64_t d_v, const LinAttnPlan& pl) {
  return pl.n_spans > 1 ? pl.n_spans * batch * nheads * d_k * d_v : 0;
}

int64_t linear_attn_fwd_floats(int64_t batch, int64_t seqlen, int64_t nheads, int64_t d_k, int64_t d_v, bool bf16) {
  return span_floats(batch, nheads, d_k, d_v, linear_attn_plan(batch, seqlen, nheads, d_k, d_v, bf16, false));
}

int64_t linear_attn_bwd_floats(int64_t batch, int64_t seqlen, int64_t nheads, int64_t nheads_kv, int64_t d_k,
                               int64_t d_v, bool bf16) {
  int64_t n = 2 * span_floats(batch, nheads, d_k, d_v, linear_attn_plan(batch, seqlen, nheads, d_k, d_v, bf16, true));
  if (nheads != nheads_kv) n += up64(batch * seqlen * nheads * d_k) + up64(batch * seqlen * nheads * d_v);
  return n;
}

hipError_t launch_linear_attn_fwd(const LinAttnLaunch& p) {
  const LinAttnPlan pl = linear_attn_plan(p.batch, p.seqlen, p.nheads, p.d_k, p.d_v, p.bf16, false);
  const int32_t rep = (int32_t)(p.nheads / p.nheads_kv);
  AttnSweep s = base(p, pl);
  s.a = AttnOperand{p.q, p.q_stride, 1};
  s.b = AttnOperand{p.k, p.k_stride, rep};
  s.c = AttnOperand{p.v, p.v_stride, rep};
  s.sn = 1;
  s.sp = p.d_k;
  s.s_pair = s.s_read = p.scale;
  s.s_write = 1.f;
  s.entry = p.h0;
  if (pl.n_spans > 1) {
    const hipError_t rc = span_entries(p, s, s, p.workspace, nullptr);
    if (rc != hipSuccess) return rc;
    s.entry = p.workspace;
  }
  s.exit = p.h_last;
  s.out = p.o;
  return p.bf16 ? launch_attn_sweep_bf16(s, p.d_k, p.d_v, p.stream)
                : launch_attn_sweep_f32(s, p.d_k, p.d_v, p.stream);
}

hipError_t launch_linear_attn_bwd(const LinAttnLaunch& p) {
  const LinAttnPlan pl = linear_attn_plan(p.batch, p.seqlen, p.nheads, p.d_k, p.d_v, p.bf16, true);
  const int32_t rep = (int32_t)(p.nheads / p.nheads_kv);
  const AttnOperand q{p.q, p.q_stride, 1}, k{p.k, p.k_stride, rep}, v{p.v, p.v_stride, rep},
      d{p.d_o, p.nheads * p.d_v, 1};
  const int64_t states = span_floats(p.batch, p.nheads, p.d_k, p.d_v, pl);
  const bool shared = p.nheads != p.nheads_kv;
  float* const pk = p.workspace + 2 * states;
  float* const pv = pk + up64(p.batch * p.seqlen * p.nheads * p.d_k);

  AttnSweep sq = base(p, pl);  // dq: the state is H^T
  sq.a = d;
  sq.b = v;
  sq.c = k;
  sq.sn = p.d_k;
  sq.sp = 1;
  sq.s_pair = sq.s_read = p.scale;
  sq.s_write = 1.f;
  sq.entry = p.h0;
  sq.out = p.dq;
  AttnSweep sk = sq;  // dk: the state is G^T
  sk.a = v;
  sk.b = d;
  sk.c = q;
  sk.s_read = 1.f;
  sk.s_write = p.scale;
  sk.entry = p.dh_last;
  sk.out = shared ? pk : p.dk;
  AttnSweep sv = sk;  // dv: the state is G
  sv.a = k;
  sv.b = q;
  sv.c = d;
  sv.sn = 1;
  sv.sp = p.d_k;
  sv.exit = p.dh0;
  sv.out = shared ? pv : p.dv;
  hipError_t rc;
  if (pl.n_spans > 1) {
    AttnSweep f = sq, r = sv;
    f.b = k;
    f.c = v;
    rc = span_entries(p, f, r, p.workspace, p.workspace + states);
    if (rc != hipSuccess) return rc;
    sq.entry = p.workspace;
    sk.entry = sv.entry = p.workspace + states;
  }
  rc = hipSuccess;
  if (p.nheads > 0)
    rc = p.bf16 ? launch_attn_sweep_grad_bf16(sq, sk, sv, p.d_k, p.d_v, shared, p.stream)
                : launch_attn_sweep_grad_f32(sq, sk, sv, p.d_k, p.d_v, p.stream);
  const int64_t heads = p.batch * p.seqlen * p.nheads_kv;
  if (rc != hipSuccess || !shared || heads == 0) return rc;
  const HeadSum hk{pk, p.dk, heads * p.d_k / 4, (int32_t)(p.d_k / 4)}, hv{pv, p.dv, heads * p.d_v / 4,
                                                                          (int32_t)(p.d_v / 4)};
  const int64_t threads = linear_attn_sum_threads(p.batch, p.seqlen, p.nheads_kv, p.d_k, p.d_v);
  const dim3 grid((unsigned)(threads / 256), 2);
  if (p.bf16) return launch(k_attn_sum_heads<uint16_t>, grid, dim3(256), 0, p.stream, hk, hv, rep);
  return launch(k_attn_sum_heads<float>, grid, dim3(256), 0, p.stream, hk, hv, rep);
}

}  // namespace ssm
