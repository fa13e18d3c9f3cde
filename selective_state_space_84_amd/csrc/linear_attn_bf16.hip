// The linear attention sweep for bf16 operands, on the bf16 matrix
// instructions (roles, formulas and the state's recurrence: linear_attn.h).
//
// One workgroup (4 waves, or 8) per (row, head) and span; wave w owns R = 16 or 32
// of the VD output columns, for the outputs and for the state S[n][p], which
// stays in fp32 accumulators.  Per block of 64 steps:
//   pairs   P[t][i] = decay (a_t . b_i), shared between the waves through LDS
//   read    out^T = (S^T A^T) diag(s_read decay)      then the state moves on:
//   update  S = gamma^m S + B^T (w o C)
//   join    out^T += C^T P^T
// on R x R tiles (v_mfma_f32_32x32x16_bf16 or 16x16x32_bf16).
//
// Precision.  a, b and c meet the matrix cores exactly.  What is formed in
// between is split: P and the state of `read` into two bf16 values (about 16
// significant bits, so that the rounding of a bf16 output stays the largest
// error), w o C into three (24 bits: the state keeps fp32's precision over any
// number of blocks, since each block adds to it at that precision).  Three parts
// everywhere leave the error of o, dq, dk and dv against 64 bits as it is (0.00166
// of their norm, what rounding alone costs) and take the difference from products
// in 32 bits, which round a few outputs the other way, from 1e-4 to 2e-5..4e-5:
// long prompt 412 -> 447 us, padded batch 130 -> 155, gradient of 4 x 4096 x 16 x
// 128 259 -> 301.  Not taken.
//
// Mapping.
//   * The accumulators' layout (lane = column p, four rows n per register
//     quad) is the A operand of S^T A^T when the contraction takes n in the
//     order the registers hold it; a is read from its rows in the same order
//     (two 8-byte reads), so the state never moves.
//   * c is needed with the steps along the contraction for both join and
//     update: ds_read_b64_tr_b16 transposes this wave's columns once per block.
//     b^T for the update comes out of b's rows the same way.
//   * read and update do not need P: they run between the writing of P and the
//     barrier that completes it, so the barrier finds the waves together.  After
//     it only P and registers are read, so the next block's rows are staged
//     without another barrier: two barriers a block.
//   * The next block's rows are requested into registers after the first barrier
//     (a) and after the pairs (b, c), and are on their way while this one is
//     worked on.
//
// Measured, one MI355X (a copy reaches 5.1 TB/s): 1 x 32768 steps x 32 heads of
// 128 in 16 spans: 407-422 us (1.07 GB, 2.6 TB/s), a third of it the spans'
// states; gradient of 4 x 4096 x 16 heads of 128: 258-260 us.  In units of a 64 x
// 128 x 128 product a block takes 0.31 (pairs) + 2 (read) + 3 (update) + 0.75
// (join), and 3 more for its span's state: the splits and the second update make
// 305 GFLOP of the long prompt, 251 us at the rate of a large product.  The rest is
// not one resource: over the long sweep the matrix units are busy 38% of the time,
// a SIMD issues 54k vector instructions in its 523k cycles (4 to 5 cycles each,
// measured alone), 37% of the LDS cycles (13% of a CU's) are bank conflicts of rows
// that lie 8 dwords (modulo 64) apart, and waves wait a third of their cycles; a
// block is a chain of load, stage, pairs, barrier, join.  Against 427 us at the
// time: rows loaded straight
// to LDS, four waves a SIMD 447 us; the splits interleaved with the products by
// hand 447 us; 32-step blocks 418 us, taken as the noise between runs and
// not pursued; the update in two parts (16 bits) 398 us, but
// with h_last 2e-6 instead of 3e-7 off.
#include "linear_attn.h"

namespace ssm {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint16_t u16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

constexpr int kQ = 64;  // steps per block

// R x R result tile: A holds row lane % R, B column lane % R, both 8 contraction
// positions 8 (lane / R) + j; register f of the result is row
// (256 / R) (f / 4) + 4 (lane / R) + f % 4 of column lane % R.
template <int R>
struct Tile;
template <>
struct Tile<32> {
  typedef f32x16 acc;
  static __device__ __forceinline__ acc mma(u32x4 a, u32x4 b, acc c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                    0, 0);
  }
};
template <>
struct Tile<16> {
  typedef f32x4 acc;
  static __device__ __forceinline__ acc mma(u32x4 a, u32x4 b, acc c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                    0, 0);
  }
};

__device__ __forceinline__ uint32_t pack(float v0, float v1) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{v0, v1}, bf16x2));
}
__device__ __forceinline__ float lo_f32(uint32_t v) { return __builtin_bit_cast(float, v << 16); }
__device__ __forceinline__ float hi_f32(uint32_t v) { return __builtin_bit_cast(float, v & 0xffff0000u); }
// A pair of values as a sum of bf16 pairs: takes the leading one off v0, v1.
__device__ __forceinline__ uint32_t peel(float& v0, float& v1) {
  const uint32_t p = pack(v0, v1);
  v0 -= lo_f32(p);
  v1 -= hi_f32(p);
  return p;
}

__device__ __forceinline__ float uniform_f32(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, v)));
}

// Rows of a block without a step hold zeros, but may meet powers of gamma beyond the block's steps.  These are kept
// finite, and multiplied to the row's value one after the other, so that they leave zeros.
__device__ __forceinline__ float finite(float w) { return __builtin_amdgcn_fmed3f(w, -__FLT_MAX__, __FLT_MAX__); }

__device__ __forceinline__ u32x2 lds_tr4(const uint16_t* p) {
  return __builtin_bit_cast(u32x2,
                            __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(s16x4*)const_cast<uint16_t*>(p)));
}
__device__ __forceinline__ u32x4 cat(u32x2 a, u32x2 b) { return u32x4{a[0], a[1], b[0], b[1]}; }
__device__ __forceinline__ u32x4 lds16(const uint16_t* p) { return *reinterpret_cast<const u32x4*>(p); }

// Lanes in halves (R = 32) or 16s (R = 16), even ones 2i and odd ones 2i + 1:
// {a of lane 2i, a of 2i + 1} in even lanes, {b of 2i, b of 2i + 1} in odd ones.
template <int R>
__device__ __forceinline__ u32x2 swap_lanes(uint32_t a, uint32_t b) {
  if constexpr (R == 32) {
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(a, b, false, false));
  } else {
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(a, b, false, false));
  }
}

// Rows of one operand on their way from memory to LDS: 16-byte pieces, NT
// threads, W columns, LDS row stride S.  Rows outside [lo, hi) are zero: the
// loads take the nearest row inside instead (no branch, so that nothing waits
// for a load before the rows are put).
template <int W, int S, int NT>
struct Stage {
  static constexpr int kPerRow = W / 8, kRows = NT / kPerRow, N = kQ / kRows;
  static_assert(N >= 1 && kQ % kRows == 0, "every thread takes whole pieces");
  u32x4 r[N];
  __device__ __forceinline__ void load(const uint16_t* base, int64_t stride, int lo, int hi) {
    const uint32_t sb = (uint32_t)stride * 2;
    const uint32_t first = (uint32_t)lo * sb, last = (uint32_t)(hi - 1) * sb;
    uint32_t row = threadIdx.x / kPerRow * sb;
    asm volatile("" : "+v"(row));  // keeps the clamped offsets from being held in registers between blocks
    const uint32_t c = threadIdx.x % kPerRow * 16;
    const gchar* p = uniform_ptr(base);
#pragma unroll
    for (int k = 0; k < N; ++k)
      r[k] = gldr<u32x4>(p, max(min(row + (uint32_t)(k * kRows) * sb, last), first) + c);
  }
  __device__ __forceinline__ void put(uint16_t* lds, int lo, int hi) {
    const int t = threadIdx.x / kPerRow, c = threadIdx.x % kPerRow * 8;
    if (hi - lo != kQ) {
#pragma unroll
      for (int k = 0; k < N; ++k)
        if (t + k * kRows < lo || t + k * kRows >= hi) r[k] = u32x4{0, 0, 0, 0};
    }
#pragma unroll
    for (int k = 0; k < N; ++k) *reinterpret_cast<u32x4*>(&lds[(t + k * kRows) * S + c]) = r[k];
  }
};

// LDS of a sweep with operands of KD and VD columns (elements).
constexpr int kSP = kQ + 8;  // row strides: rows read along the contraction 4 (mod 64) dwords apart,
constexpr int row_stride_a(int kd) { return kd + 8; }
constexpr int row_stride_t(int w) { return w + 16; }  // rows read through the transpose 8 apart
constexpr int sum_lds(int kd, int vd) { return kQ * (row_stride_t(kd) + row_stride_t(vd)); }
constexpr int sweep_lds(int kd, int vd) { return sum_lds(kd, vd) + kQ * (row_stride_a(kd) + 2 * kSP); }
constexpr int larger(int a, int b) { return a > b ? a : b; }

// One span of one row by NW waves of R columns each.  SUM: only the state of the
// span from a zero entry (a and out unused).
template <typename O, int KD, int R, int NW, bool REV, bool SUM>
__device__ __forceinline__ void sweep_span(const AttnSweep& s, uint16_t* lds, int64_t row, int64_t span) {
  constexpr int VD = NW * R;
  constexpr int TH = 64 * NW;
  constexpr int NG = 64 / R;       // lane groups
  constexpr int KC = 8 * NG;       // contraction of one instruction
  constexpr int AR = R * R / 64;   // accumulator registers of a tile
  constexpr int NS = KD * R / 64;  // state registers
  constexpr int TT = kQ / R;       // tiles of steps
  constexpr int KT = kQ / KC;      // contraction slices over the steps
  constexpr int SA = row_stride_a(KD), SB = row_stride_t(KD), SC = row_stride_t(VD), SP = kSP;
  typedef Tile<R> M;
  typedef typename M::acc Acc;
  uint16_t* const sB = lds;
  uint16_t* const sC = sB + kQ * SB;
  uint16_t* const sA = sC + kQ * SC;
  uint16_t* const sP = sA + kQ * SA;  // pairs [t][i], leading and second part
  constexpr int kP2 = kQ * SP;

  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane % R, g = lane / R;
  const int r16 = lane & 15, q4 = lane >> 4;
  const int64_t b = row / s.nheads;
  const int h = (int)(row % s.nheads);
  const int64_t len = row_length(s.lengths, b, s.seqlen);
  const int64_t s0 = span * s.span_len;
  const int64_t s1 = min(s0 + s.span_len, s.seqlen);
  const int64_t e = min(s1, len) > s0 ? min(s1, len) : s0;  // steps [s0, e) are computed
  const float gl = decay_log2(s.log_decay[h]);

  const uint16_t* const A =
      SUM ? nullptr : static_cast<const uint16_t*>(s.a.p) + b * s.seqlen * s.a.stride + (h / s.a.rep) * KD;
  const uint16_t* const B = static_cast<const uint16_t*>(s.b.p) + b * s.seqlen * s.b.stride + (h / s.b.rep) * KD;
  const uint16_t* const C = static_cast<const uint16_t*>(s.c.p) + b * s.seqlen * s.c.stride + (h / s.c.rep) * VD;
  O* const out = SUM ? nullptr : static_cast<O*>(s.out) + (b * s.seqlen * s.nheads + h) * VD;

  // State register f: S[4 NG (f / 4) + 4 g + f % 4][R w + r].
  Acc st[NS / AR];
  const int64_t soff = (int64_t)(R * w + r) * s.sp;
  {
    const float* ep = nullptr;
    if (!SUM && s.entry != nullptr) ep = s.entry + ((s.n_spans > 1 ? span * s.rows : 0) + row) * KD * VD + soff;
#pragma unroll
    for (int f = 0; f < NS; f += 4) {
      const int n0 = NG * f + 4 * g;
      f32x4 v = {0.f, 0.f, 0.f, 0.f};
      if (ep != nullptr) {
        if (s.sn == 1) {
          v = *reinterpret_cast<const f32x4*>(ep + n0);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] = ep[(n0 + j) * s.sn];
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) st[(f + j) / AR][(f + j) % AR] = v[j];
    }
  }

  // The masked 16 x 16 tiles of P inside the tiles that join reads are never
  // written: zero once.
  if (!SUM && tid < 2 * kQ) {
    const int t = (REV ? 16 : 0) + 32 * (tid >> 6) + (lane >> 2), i = (REV ? 0 : 16) + 32 * (tid >> 6) + 4 * (lane & 3);
    *reinterpret_cast<u32x2*>(&sP[t * SP + i]) = u32x2{0, 0};
    *reinterpret_cast<u32x2*>(&sP[kP2 + t * SP + i]) = u32x2{0, 0};
  }

  // Decays that are the same in every block.  A step's weight in the update is
  // gamma^(63 - i) (gamma^(i + 1) in reverse) for row i = KC kt + 8 g + j of the
  // block: a power of the lane group times one of (kt, j), the latter uniform.
  // So that this also holds for a block of fewer than 64 steps, forward blocks
  // keep their steps in the last rows (in reverse: the first), the others zero.
  const float wg = hw_exp2(gl * (float)(REV ? 8 * g : 8 * (NG - 1 - g))) * s.s_write;
  float wj[8], wk[KT];
#pragma unroll
  for (int j = 0; j < 8; ++j) wj[j] = uniform_f32(finite(hw_exp2(gl * (float)(REV ? j + 1 : 7 - j))));
#pragma unroll
  for (int kt = 0; kt < KT; ++kt) wk[kt] = uniform_f32(hw_exp2(gl * (float)(REV ? KC * kt : KC * (KT - 1 - kt))));
  // Pairs of neighbouring 16 x 16 tiles: gamma^|t - i| at j = 3 (j = 0 in
  // reverse), the smallest power of the lane's four (at least 1).
  const float po = hw_exp2(gl * (float)(16 + (REV ? 4 * q4 - r16 : r16 - 4 * q4 - 3))) * s.s_pair;
  const float g16 = hw_exp2(gl * 16.f);

  Stage<KD, SA, TH> ga;
  Stage<KD, SB, TH> gb;
  Stage<VD, SC, TH> gc;
  const int64_t nblk = (e - s0 + kQ - 1) / kQ;
  // Block k: m steps, of which row x is step tb + x.
  auto block = [&](int64_t k, int64_t& tb, int& m) {
    const int64_t t0 = s0 + (REV ? nblk - 1 - k : k) * kQ;
    m = (int)min((int64_t)kQ, e - t0);
    tb = REV ? t0 : t0 - (kQ - m);
  };
  // Requests rows of block k: a, b or c.
  auto fetch = [&](int64_t k, int which) {
    int64_t tb;
    int m;
    block(k, tb, m);
    const int lo = REV ? 0 : kQ - m, hi = REV ? m : kQ;
    if (!SUM && which == 0) ga.load(A + tb * s.a.stride, s.a.stride, lo, hi);
    if (which == 1) gb.load(B + tb * s.b.stride, s.b.stride, lo, hi);
    if (which == 2) gc.load(C + tb * s.c.stride, s.c.stride, lo, hi);
  };
  if (nblk > 0) {
    fetch(0, 0);
    fetch(0, 1);
    fetch(0, 2);
  }
  for (int64_t k = 0; k < nblk; ++k) {
    int64_t tb;
    int m;
    block(k, tb, m);
    const int lo = REV ? 0 : kQ - m, hi = REV ? m : kQ;
    if (!SUM) ga.put(sA, lo, hi);
    gb.put(sB, lo, hi);
    gc.put(sC, lo, hi);
    __syncthreads();
    // The next block's rows are requested in two parts, so that the waves do not
    // stand in line for the memory pipeline (48 KB take it 768 cycles).
    const bool more = k + 1 < nblk;
    if (more) fetch(k + 1, 0);
    if (SUM && more) fetch(k + 1, 1);
    if (SUM && more) fetch(k + 1, 2);

    Acc o[SUM ? 1 : TT];
    if (!SUM) {
      // pairs: the ten tiles (rows i of tile it, steps t of tile tt) on or beside
      // the diagonal, dealt to the waves; with four waves two at a time, for their
      // products' sake (with eight the waves of one tile would wait: 256 -> 267 us
      // on the gradient of 4 x 4096 x 16 x 128).
      constexpr int kTiles = kQ / 16 * (kQ / 16 + 1) / 2;
      auto product = [&](int x) {
        const int big = x < 1 ? 0 : x < 3 ? 1 : x < 6 ? 2 : 3, small = x - big * (big + 1) / 2;
        const int it = REV ? big : small, tt = REV ? small : big;
        f32x4 p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int kk = 0; kk < KD / 32; ++kk)
          p = Tile<16>::mma(lds16(&sB[(16 * it + r16) * SB + 32 * kk + 8 * q4]),
                            lds16(&sA[(16 * tt + r16) * SA + 32 * kk + 8 * q4]), p);
        return p;
      };
      auto decayed = [&](int x, const f32x4& p) {
        const int big = x < 1 ? 0 : x < 3 ? 1 : x < 6 ? 2 : 3, small = x - big * (big + 1) / 2;
        const int it = REV ? big : small, tt = REV ? small : big;
        float v[4];
        if (big == small) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int d = REV ? 4 * q4 + j - r16 : r16 - 4 * q4 - j;
            v[j] = d >= 0 ? p[j] * finite(hw_exp2(gl * (float)d)) * s.s_pair : 0.f;
          }
        } else {
          const float f = finite(po * (big - small == 1 ? 1.f : (big - small == 2 ? g16 : g16 * g16)));
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] = p[j] * f * (REV ? (j == 0 ? 1.f : wj[j - 1]) : wj[4 + j]);
        }
        const int at = (16 * tt + r16) * SP + 16 * it + 4 * q4;
        const uint32_t h0 = peel(v[0], v[1]), h1 = peel(v[2], v[3]);
        *reinterpret_cast<u32x2*>(&sP[at]) = u32x2{h0, h1};
        *reinterpret_cast<u32x2*>(&sP[kP2 + at]) = u32x2{pack(v[0], v[1]), pack(v[2], v[3])};
      };
      if constexpr (NW == 4) {
        const f32x4 p0 = product(w), p1 = product(w + 4);
        decayed(w, p0);
        decayed(w + 4, p1);
        if (w < kTiles - 8) decayed(w + 8, product(w + 8));
      } else {
        for (int x = w; x < kTiles; x += NW) decayed(x, product(x));
      }

      if (more) fetch(k + 1, 1);
      if (more) fetch(k + 1, 2);
      __builtin_amdgcn_sched_barrier(0);
      // read
#pragma unroll
      for (int tt = 0; tt < TT; ++tt)
#pragma unroll
        for (int j = 0; j < AR; ++j) o[tt][j] = 0.f;
#pragma unroll
      for (int ks = 0; ks < KD / KC; ++ks) {
        u32x4 hi, lo;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int f = 8 * ks + 2 * q;
          float v0 = st[f / AR][f % AR], v1 = st[(f + 1) / AR][(f + 1) % AR];
          hi[q] = peel(v0, v1);
          lo[q] = pack(v0, v1);
        }
        u32x4 a[TT];
#pragma unroll
        for (int tt = 0; tt < TT; ++tt) {
          const uint16_t* p = &sA[(R * tt + r) * SA + KC * ks + 4 * g];
          a[tt] = cat(*reinterpret_cast<const u32x2*>(p), *reinterpret_cast<const u32x2*>(p + 4 * NG));
        }
#pragma unroll
        for (int tt = 0; tt < TT; ++tt) o[tt] = M::mma(hi, a[tt], o[tt]);
#pragma unroll
        for (int tt = 0; tt < TT; ++tt) o[tt] = M::mma(lo, a[tt], o[tt]);
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int tt = 0; tt < TT; ++tt) {
        // Rows without a step (exponent below the first's) are not stored.
        const int x = R * tt + r;
        const float rf = hw_exp2(gl * (float)max(REV ? m - 1 - x : x + 1 - (kQ - m), 0)) * s.s_read;
        o[tt] *= rf;
      }
    }

    // This wave's columns of c, steps along the contraction: lane (r, g) of slice
    // kt holds c[KC kt + 8 g + j][R w + r].
    u32x4 cv[KT];
    {
      const int sub = lane & 15;
      const uint16_t* p = &sC[(8 * g + (sub >> 2)) * SC + R * w + (r & 16) + 4 * (sub & 3)];
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) cv[kt] = cat(lds_tr4(p + KC * kt * SC), lds_tr4(p + (KC * kt + 4) * SC));
    }

    __builtin_amdgcn_sched_barrier(0);
    // update
    const float fac = hw_exp2(gl * (float)m);
#pragma unroll
    for (int i = 0; i < NS / AR; ++i) st[i] *= fac;
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) {
      u32x4 w0, w1, w2;
      const float wl = finite(wg * wk[kt]);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float v0 = lo_f32(cv[kt][q]) * wl * wj[2 * q];
        float v1 = hi_f32(cv[kt][q]) * wl * wj[2 * q + 1];
        w0[q] = peel(v0, v1);
        w1[q] = peel(v0, v1);
        w2[q] = pack(v0, v1);
      }
      const int sub = lane & 15;
      const uint16_t* p = &sB[(KC * kt + 8 * g + (sub >> 2)) * SB + (r & 16) + 4 * (sub & 3)];
#pragma unroll
      for (int nt = 0; nt < KD / R; ++nt) {
        const u32x4 bv = cat(lds_tr4(p + R * nt), lds_tr4(p + 4 * SB + R * nt));
        st[nt] = M::mma(bv, w0, st[nt]);
        st[nt] = M::mma(bv, w1, st[nt]);
        st[nt] = M::mma(bv, w2, st[nt]);
      }
        __builtin_amdgcn_sched_barrier(0);
    }
    __syncthreads();  // P complete; a, b and c no longer read

    if (!SUM) {
      // join
#pragma unroll
      for (int tt = 0; tt < TT; ++tt) {
        const uint16_t* p = &sP[(R * tt + r) * SP + 8 * g];
        const int first = REV ? R * tt / KC : 0, last = REV ? KT : (R * tt + R + KC - 1) / KC;
#pragma unroll
        for (int kt = first; kt < last; ++kt) {
          o[tt] = M::mma(cv[kt], lds16(p + KC * kt), o[tt]);
          o[tt] = M::mma(cv[kt], lds16(p + kP2 + KC * kt), o[tt]);
        }
      }
      // out.  bf16 outputs change lanes first, so that each stores 16 bytes of a row:
      // with R = 32 between the halves of the wave (one takes the first, the other
      // the second of two runs of 8 columns), with R = 16 between neighbouring 16
      // lanes (one takes the first, the other the second of two tiles).
      gchar* const ob = uniform_ptr(out + tb * s.nheads * VD);
      const uint32_t orow = (uint32_t)(s.nheads * VD) * sizeof(O), ocol = R * w * sizeof(O);
      if constexpr (sizeof(O) == 2) {
        constexpr int NP = TT * AR / 8;  // 16-byte pieces of a lane
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          const int t0 = R == 32 ? i / 2 : 2 * i, t1 = R == 32 ? t0 : t0 + 1;  // tiles and registers
          const int f0 = R == 32 ? 8 * (i % 2) : 0, f1 = R == 32 ? f0 + 4 : 0;
          const u32x2 a = swap_lanes<R>(pack(o[t0][f0], o[t0][f0 + 1]), pack(o[t1][f1], o[t1][f1 + 1]));
          const u32x2 c = swap_lanes<R>(pack(o[t0][f0 + 2], o[t0][f0 + 3]), pack(o[t1][f1 + 2], o[t1][f1 + 3]));
          const int x = R * (R == 32 ? t0 : t0 + (g & 1)) + r;
          const int col = R == 32 ? 8 * (2 * (i % 2) + g) : 8 * (g >> 1);
          if (x >= lo && x < hi) gstr<u32x4>(ob, (uint32_t)x * orow + ocol + 2 * col, u32x4{a[0], c[0], a[1], c[1]});
        }
      } else {
#pragma unroll
        for (int tt = 0; tt < TT; ++tt) {
          const int x = R * tt + r;
          if (x >= lo && x < hi) {
#pragma unroll
            for (int q = 0; q < AR / 4; ++q)
              gstr<f32x4>(ob, (uint32_t)x * orow + ocol + (4 * NG * q + 4 * g) * 4,
                          f32x4{o[tt][4 * q], o[tt][4 * q + 1], o[tt][4 * q + 2], o[tt][4 * q + 3]});
          }
        }
      }
    }
  }

  if (!SUM) {
    // Rows behind the sequence's end.
    for (int64_t t = e + tid / (VD / 4); t < s1; t += TH / (VD / 4)) {
      O* op = out + t * s.nheads * VD + 4 * (tid % (VD / 4));
#pragma unroll
      for (int j = 0; j < 4; ++j) io_store(op + j, 0.f);
    }
  }
  if (s.exit != nullptr && (SUM || span == (REV ? 0 : s.n_spans - 1))) {
    float* xp = s.exit + ((SUM ? span * s.rows : 0) + row) * KD * VD + soff;
#pragma unroll
    for (int f = 0; f < NS; f += 4) {
      const int n0 = NG * f + 4 * g;
      f32x4 v;
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = st[(f + j) / AR][(f + j) % AR];
      if (s.sn == 1) {
        *reinterpret_cast<f32x4*>(xp + n0) = v;
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) xp[(n0 + j) * s.sn] = v[j];
      }
    }
  }
}

// A workgroup's part of a launch of `roles` sweeps over the same rows and
// spans: the sweeps of one row and span are neighbours, so that they find each
// other's operands in their XCD's L2.
struct Part {
  int role;
  int64_t row, span;
};
__device__ __forceinline__ Part part_of(const AttnSweep& s, int roles) {
  const int64_t id = xcd_remap(blockIdx.x, gridDim.x);
  return Part{(int)(id % roles), id / roles % s.rows, id / roles / s.rows};
}

template <int KD, int VD, int NW>
__global__ void __launch_bounds__(64 * NW) __attribute__((amdgpu_waves_per_eu(2)))
k_attn_sweep(const AttnSweep s) {
  __shared__ __align__(16) uint16_t lds[sweep_lds(KD, VD)];
  const Part p = part_of(s, 1);
  sweep_span<uint16_t, KD, VD / NW, NW, false, false>(s, lds, p.row, p.span);
}

// The spans' own states: of H (role 0) and, in the gradient, of G (role 1).  The
// last span of a direction has no use for its own.
template <int KD, int VD>
__global__ void __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2)))
k_attn_span_states(const AttnSweep f, const AttnSweep r, int roles) {
  __shared__ __align__(16) uint16_t lds[sum_lds(KD, VD)];
  const Part p = part_of(f, roles);
  if (p.role == 0) {
    sweep_span<float, KD, VD / 4, 4, false, true>(f, lds, p.row, p.span);
  } else {
    sweep_span<float, KD, VD / 4, 4, true, true>(r, lds, p.row, p.span + 1);
  }
}

// dq, dk and dv: three sweeps in one launch.  The three inlined roles hold three
// launch descriptions: 77 to 93 of their scalars lie in lanes of vector registers
// (8 at most in a sweep alone).
template <typename O, int DK, int DV, int NW>
__global__ void __launch_bounds__(64 * NW) __attribute__((amdgpu_waves_per_eu(2)))
k_attn_sweep_grad(const AttnSweep q, const AttnSweep k, const AttnSweep v) {
  __shared__ __align__(16) uint16_t lds[larger(sweep_lds(DV, DK), sweep_lds(DK, DV))];
  const Part p = part_of(q, 3);
  if (p.role == 0) {
    sweep_span<uint16_t, DV, DK / NW, NW, false, false>(q, lds, p.row, p.span);
  } else if (p.role == 1) {
    sweep_span<O, DV, DK / NW, NW, true, false>(k, lds, p.row, p.span);
  } else {
    sweep_span<O, DK, DV / NW, NW, true, false>(v, lds, p.row, p.span);
  }
}

// Up to this many workgroups, one a CU: then eight waves of 16 columns each,
// two a SIMD, instead of four of 32 (operands of 128 columns).  Measured, eight
// against four waves, 1000 steps, heads of 128: 64 (row, head) pairs (256
// workgroups) 47 against 49 us, 256 pairs 75 against 81, 320 pairs 137 against
// 116, 512 pairs 159 against 141; gradient of 4 x 4096 x 16 257 against 289, of 7
// x 1000 x 16 heads (336 workgroups) 129 against 101.  Heads of 64 by 128 have the
// four-wave form alone: eight waves of 16 columns would take 5% off 8 x 1000 steps x
// 32 of them (54 against 57 us).
constexpr int64_t kOneEach = 256;

}  // namespace

hipError_t launch_attn_sweep_bf16(const AttnSweep& s, int64_t kd, int64_t vd, hipStream_t stream) {
  const int64_t grid = s.rows * s.n_spans;
  return by_width(kd, vd, [&](auto k, auto v) {
    constexpr int KD = decltype(k)::value, VD = decltype(v)::value;
    if constexpr (KD == 128 && VD == 128) {
      if (grid <= kOneEach)
        return launch(k_attn_sweep<KD, VD, 8>, dim3((unsigned)grid), dim3(512), 0, stream, s);
    }
    return launch(k_attn_sweep<KD, VD, 4>, dim3((unsigned)grid), dim3(256), 0, stream, s);
  });
}

hipError_t launch_attn_span_states_bf16(const AttnSweep& f, const AttnSweep* r, int64_t kd, int64_t vd,
                                        hipStream_t stream) {
  const int roles = r != nullptr ? 2 : 1;
  const int64_t grid = f.rows * (f.n_spans - 1) * roles;
  return by_width(kd, vd, [&](auto k, auto v) {
    constexpr int KD = decltype(k)::value, VD = decltype(v)::value;
    return launch(k_attn_span_states<KD, VD>, dim3((unsigned)grid), dim3(256), 0, stream, f, r != nullptr ? *r : f,
                  roles);
  });
}

hipError_t launch_attn_sweep_grad_bf16(const AttnSweep& q, const AttnSweep& k, const AttnSweep& v, int64_t d_k,
                                       int64_t d_v, bool out32, hipStream_t stream) {
  const int64_t grid = 3 * q.rows * q.n_spans;
  return by_width(d_k, d_v, [&](auto a, auto b) {
    constexpr int DK = decltype(a)::value, DV = decltype(b)::value;
    auto go = [&](auto kern, int waves) {
      return launch(kern, dim3((unsigned)grid), dim3(64 * waves), 0, stream, q, k, v);
    };
    if constexpr (DK == 128 && DV == 128) {
      if (grid <= kOneEach)
        return out32 ? go(k_attn_sweep_grad<float, DK, DV, 8>, 8) : go(k_attn_sweep_grad<uint16_t, DK, DV, 8>, 8);
    }
    return out32 ? go(k_attn_sweep_grad<float, DK, DV, 4>, 4) : go(k_attn_sweep_grad<uint16_t, DK, DV, 4>, 4);
  });
}

}  // namespace ssm
