// Host-side argument checks shared by the C ABI's translation units.
#pragma once

#include "ssm_scan.h"

#include <stdint.h>

namespace {

// Workspace alignment the library asks for.
constexpr uintptr_t kWorkspaceAlign = 256;

bool mul3(int64_t a, int64_t b, int64_t c, int64_t* out) {
  int64_t t;
  if (__builtin_mul_overflow(a, b, &t)) return false;
  if (__builtin_mul_overflow(t, c, out)) return false;
  return true;
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Byte ranges [p, p+n) and [q, q+m) overlap (empty ranges never overlap).
bool overlap(const void* p, int64_t n, const void* q, int64_t m) {
  if (p == nullptr || q == nullptr || n <= 0 || m <= 0) return false;
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return a < b + (uintptr_t)m && b < a + (uintptr_t)n;
}

// Rows of a tensor read in place from a wider one: `rows` rows of `width`
// bytes, `stride` bytes apart.
struct Rows {
  const void* p;
  int64_t rows, width, stride;
};

// Some byte of x is also one of y.  Two tensors of the same stride may be
// column ranges of one buffer, whose extents overlap although their rows do not.
bool overlap(const Rows& x, const Rows& y) {
  if (x.p == nullptr || y.p == nullptr || x.rows <= 0 || y.rows <= 0 || x.width <= 0 || y.width <= 0) return false;
  if (!overlap(x.p, (x.rows - 1) * x.stride + x.width, y.p, (y.rows - 1) * y.stride + y.width)) return false;
  if (x.stride != y.stride || x.rows == 1 || y.rows == 1) return true;
  const int64_t s = x.stride;
  const int64_t d = (int64_t)(reinterpret_cast<uintptr_t>(y.p) - reinterpret_cast<uintptr_t>(x.p)) % s;
  const int64_t off = d < 0 ? d + s : d;  // y's first byte within x's rows
  return off < x.width || off + y.width > s;
}

Rows dense(const void* p, int64_t bytes) { return Rows{p, 1, bytes, bytes}; }

// Outputs against the inputs, each other and the workspace.
int check_alias(const Rows* outs, int n_out, const Rows* ins, int n_in) {
  for (int o = 0; o < n_out; ++o) {
    for (int k = 0; k < n_in; ++k)
      if (overlap(outs[o], ins[k])) return SSM_ERR_ALIAS;
    for (int k = o + 1; k < n_out; ++k)
      if (overlap(outs[o], outs[k])) return SSM_ERR_ALIAS;
  }
  return SSM_OK;
}

}  // namespace
