// Argument checks shared by the C ABI of the block operators: layout and
// alignment of views, extents, and which views share memory.
#pragma once

#include "internal.h"
#include "linattn.h"

#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <utility>

namespace la {

constexpr int64_t kMaxDim = (int64_t)1 << 30;     // tokens, features
constexpr int64_t kMaxBatch = (int64_t)1 << 24;
constexpr int64_t kMaxChannels = (int64_t)1 << 20;

inline bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

inline int64_t size_of(la_dtype t) { return t == LA_BF16 ? 2 : t == LA_E4M3 ? 1 : 4; }

// Data, row width and strides (of extents above 1) at multiples of `align` bytes.
inline bool valid_layout(const la_rows* r, int64_t align) {
  if (r->B < 0 || r->n < 0 || r->d < 1) return false;
  const int64_t e = size_of(r->dtype);
  if ((r->d * e) % align) return false;
  if (r->B > 1 && (r->stride_b < 0 || (r->stride_b * e) % align)) return false;
  if (r->n > 1 && (r->stride_n < 0 || (r->stride_n * e) % align)) return false;
  if (r->B > 0 && r->n > 0 && (!r->data || !aligned(r->data, align))) return false;
  return true;
}

// The rules shared by every la_rows argument: layout and alignment.
inline bool valid_rows(const la_rows* r, la_dtype dtype) {
  if (!r || (r->dtype != LA_BF16 && r->dtype != LA_F32) || r->dtype != dtype) return false;
  return valid_layout(r, 16);
}

// The same for 8-bit operands.
inline bool valid_e4m3(const la_rows* r, int64_t align) {
  return r && r->dtype == LA_E4M3 && valid_layout(r, align);
}

// No two elements of a view coincide (outputs).
inline bool disjoint_rows(const la_rows* r) {
  const bool many_b = r->B > 1, many_n = r->n > 1;
  if (many_b && r->stride_b < r->d) return false;
  if (many_n && r->stride_n < r->d) return false;
  if (!many_b || !many_n) return true;
  // products of 64-bit sizes: compared by division, so that none overflows
  const bool by_batch = r->stride_n <= (r->stride_b - r->d) / (r->n - 1);
  const bool by_token = r->stride_b <= (r->stride_n - r->d) / (r->B - 1);
  return by_batch || by_token;
}

// The extents are within what the kernels index, the strides within 2^40.
inline bool supported_rows(const la_rows* r) {
  return r->B <= kMaxBatch && r->n <= kMaxDim && r->d <= kMaxDim &&
         (r->B <= 1 || r->stride_b <= ((int64_t)1 << 40)) &&
         (r->n <= 1 || r->stride_n <= ((int64_t)1 << 36));
}

inline bool same_extent(const la_rows* a, const la_rows* b) {
  return a->B == b->B && a->n == b->n && a->d == b->d;
}

inline bool valid_param(const void* p) { return aligned(p, 16); }

inline bool valid_activation(la_activation a) { return a >= LA_ACT_NONE && a <= LA_ACT_SOFTPLUS; }

// Strides of extents 1 are not looked at by the rules: the kernels see 0.
inline Rows rows_of(const la_rows* r) {
  return Rows{r->data, r->B > 1 ? r->stride_b : 0, r->n > 1 ? r->stride_n : 0};
}

// Memory that a call reads or writes: a view, or a dense array; its first byte and
// the one after its last (which passes 64 bits only where no memory can).
struct Span {
  const la_rows* view;
  int64_t lo, hi;
};

inline Span span_of(const void* p, int64_t bytes) {
  const int64_t lo = (int64_t)reinterpret_cast<uintptr_t>(p);
  return Span{nullptr, lo, p ? lo + bytes : lo};
}

inline Span span_of(const la_rows* r) {
  const int64_t e = size_of(r->dtype), lo = (int64_t)reinterpret_cast<uintptr_t>(r->data);
  int64_t b = 0, t = 0, hi = 0;
  if (r->B == 0 || r->n == 0) return Span{r, lo, lo};
  if (__builtin_mul_overflow(r->B - 1, r->B > 1 ? r->stride_b * e : 0, &b) ||
      __builtin_mul_overflow(r->n - 1, r->n > 1 ? r->stride_n * e : 0, &t) ||
      __builtin_add_overflow(b, t, &hi) || __builtin_add_overflow(hi, lo + r->d * e, &hi))
    hi = INT64_MAX;
  return Span{r, lo, hi};
}

// The same memory as B × n rows of `row` bytes, strides in bytes (0 for extents of
// 1).  Extents times strides pass 64 bits.
using Wide = __int128;
struct Region {
  Wide at, B, n, sb, sn, row;
};

inline Region region_of(const Span& s) {
  const la_rows* r = s.view;
  if (!r) return Region{s.lo, 1, 1, 0, 0, s.hi - s.lo};
  const int64_t e = size_of(r->dtype);
  Region g{s.lo, r->B, r->n, r->B > 1 ? (Wide)r->stride_b * e : 0, r->n > 1 ? (Wide)r->stride_n * e : 0,
           (Wide)r->d * e};
  if (g.B > 1 && (g.n == 1 || g.sb == g.n * g.sn)) {   // one level of rows
    g.sn = g.n == 1 ? g.sb : g.sn;
    g.n *= g.B, g.B = 1, g.sb = 0;
  }
  if (g.n > 1 && g.sn == g.row) g.row *= g.n, g.n = 1, g.sn = 0;   // dense
  return g;
}

inline Wide floor_div(Wide a, Wide b) { return a / b - (a % b < 0); }

// Whether an element of one lies on an element of the other.  Answered exactly
// where the two have the same strides, or one is dense (the parts of a
// projection's output among them); otherwise they are taken to be apart.
inline bool coincide(const Span& p, const Span& q) {
  if (p.hi <= q.lo || q.hi <= p.lo || p.lo == p.hi || q.lo == q.hi) return false;
  const Region a = region_of(p), b = region_of(q);
  if ((a.sb && b.sb && a.sb != b.sb) || (a.sn && b.sn && a.sn != b.sn)) return false;
  // a's row meets b's where lo < Σ (difference of their indices)·stride < hi;
  // the larger stride outside, where few differences are left to try
  Wide so = a.sb ? a.sb : b.sb, si = a.sn ? a.sn : b.sn;
  Wide o0 = b.sb ? 1 - b.B : 0, o1 = a.sb ? a.B - 1 : 0;
  Wide i0 = b.sn ? 1 - b.n : 0, i1 = a.sn ? a.n - 1 : 0;
  if (si > so) std::swap(so, si), std::swap(o0, i0), std::swap(o1, i1);
  const Wide lo = b.at - a.at - a.row, hi = b.at - a.at + b.row;
  if (so > 0) {
    o0 = std::max(o0, floor_div(lo - i1 * si, so) + 1);
    o1 = std::min(o1, floor_div(hi - 1 - i0 * si, so));
  }
  if (o1 - o0 > 64) return false;   // rows that are not nested: undecided
  for (Wide o = o0; o <= o1; ++o) {
    const Wide l = lo - o * so, h = hi - o * so;
    if (si == 0 ? l < 0 && h > 0
                : std::max(i0, floor_div(l, si) + 1) <= std::min(i1, floor_div(h - 1, si)))
      return true;
  }
  return false;
}

inline bool same_view(const la_rows* a, const la_rows* b) {
  const Rows p = rows_of(a), q = rows_of(b);
  return p.data == q.data && p.sb == q.sb && p.sn == q.sn;
}

// A grid beyond what a launch takes is a request outside the kernels' range.
inline la_status launch_status(cudaError_t e) {
  return e == cudaErrorInvalidConfiguration ? LA_ERR_UNSUPPORTED : to_status(e);
}

// An empty prompt: the state after it is the one before it.
inline cudaError_t copy_state(void* to, const void* from, size_t bytes, cudaStream_t stream) {
  if (!to || !bytes) return cudaSuccess;
  return from ? cudaMemcpyAsync(to, from, bytes, cudaMemcpyDeviceToDevice, stream)
              : cudaMemsetAsync(to, 0, bytes, stream);
}

}  // namespace la
