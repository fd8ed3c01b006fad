// C ABI of the state-space block's operators (declared in include/linattn.h):
// argument validation and hand-over to the launchers.
#include "linattn.h"

#include "internal.h"

#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <utility>

namespace la {
namespace {

constexpr int64_t kMaxDim = (int64_t)1 << 30;     // tokens, features
constexpr int64_t kMaxBatch = (int64_t)1 << 24;
constexpr int64_t kMaxChannels = (int64_t)1 << 20;

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

int64_t size_of(la_dtype t) { return t == LA_BF16 ? 2 : 4; }

// The rules shared by every la_rows argument: layout and alignment.
bool valid_rows(const la_rows* r, la_dtype dtype) {
  if (!r || (r->dtype != LA_BF16 && r->dtype != LA_F32) || r->dtype != dtype) return false;
  if (r->B < 0 || r->n < 0 || r->d < 1) return false;
  const int64_t e = size_of(r->dtype);
  if ((r->d * e) % 16) return false;
  if (r->B > 1 && (r->stride_b < 0 || (r->stride_b * e) % 16)) return false;
  if (r->n > 1 && (r->stride_n < 0 || (r->stride_n * e) % 16)) return false;
  if (r->B > 0 && r->n > 0 && (!r->data || !aligned(r->data, 16))) return false;
  return true;
}

// No two elements of a view coincide (outputs).
bool disjoint_rows(const la_rows* r) {
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
bool supported_rows(const la_rows* r) {
  return r->B <= kMaxBatch && r->n <= kMaxDim && r->d <= kMaxDim &&
         (r->B <= 1 || r->stride_b <= ((int64_t)1 << 40)) &&
         (r->n <= 1 || r->stride_n <= ((int64_t)1 << 36));
}

bool same_extent(const la_rows* a, const la_rows* b) {
  return a->B == b->B && a->n == b->n && a->d == b->d;
}

bool valid_param(const void* p) { return aligned(p, 16); }

bool valid_activation(la_activation a) { return a >= LA_ACT_NONE && a <= LA_ACT_SOFTPLUS; }

// Strides of extents 1 are not looked at by the rules: the kernels see 0.
Rows rows_of(const la_rows* r) {
  return Rows{r->data, r->B > 1 ? r->stride_b : 0, r->n > 1 ? r->stride_n : 0};
}

// Memory that a call reads or writes: a view, or a dense array; its first byte and
// the one after its last (which passes 64 bits only where no memory can).
struct Span {
  const la_rows* view;
  int64_t lo, hi;
};

Span span_of(const void* p, int64_t bytes) {
  const int64_t lo = (int64_t)reinterpret_cast<uintptr_t>(p);
  return Span{nullptr, lo, p ? lo + bytes : lo};
}

Span span_of(const la_rows* r) {
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

Region region_of(const Span& s) {
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

Wide floor_div(Wide a, Wide b) { return a / b - (a % b < 0); }

// Whether an element of one lies on an element of the other.  Answered exactly
// where the two have the same strides, or one is dense (the parts of a
// projection's output among them); otherwise they are taken to be apart.
bool coincide(const Span& p, const Span& q) {
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

bool same_view(const la_rows* a, const la_rows* b) {
  const Rows p = rows_of(a), q = rows_of(b);
  return p.data == q.data && p.sb == q.sb && p.sn == q.sn;
}

la_status check_conv(const la_rows* x, const void* weight, int width, const void* bias,
                     la_activation act, la_rows* out, ConvArgs* a) {
  if (!x || !out || !weight) return LA_ERR_INVALID_ARG;
  if (!valid_rows(x, x->dtype) || !valid_rows(out, x->dtype) || !same_extent(x, out) ||
      !disjoint_rows(out))
    return LA_ERR_INVALID_ARG;
  if (!valid_param(weight) || !valid_param(bias) || !valid_activation(act))
    return LA_ERR_INVALID_ARG;
  if (width < 2 || width > 4 || (act != LA_ACT_NONE && act != LA_ACT_SILU))
    return LA_ERR_UNSUPPORTED;
  if (!supported_rows(x) || !supported_rows(out) || x->d > kMaxChannels) return LA_ERR_UNSUPPORTED;
  const Span o_at = span_of(out);
  const int64_t e = size_of(x->dtype);
  if (coincide(o_at, span_of(weight, x->d * width * e)) || coincide(o_at, span_of(bias, x->d * e)))
    return LA_ERR_INVALID_ARG;
  *a = ConvArgs{};
  a->x = rows_of(x);
  const Rows o = rows_of(out);
  a->out = out->data;
  a->out_sb = o.sb;
  a->out_sn = o.sn;
  a->weight = weight;
  a->bias = bias;
  a->B = x->B;
  a->n = x->n;
  a->D = x->d;
  a->W = width;
  a->silu = act == LA_ACT_SILU;
  a->bf16 = x->dtype == LA_BF16;
  return LA_OK;
}

la_status check_scan(const la_rows* x, const la_rows* dt, const float* a, int states,
                     const la_rows* bm, const la_rows* cm, const float* skip, const la_rows* gate,
                     const float* dt_bias, int softplus, la_rows* out, ScanArgs* s) {
  if (!x || !dt || !a || !bm || !cm || !out) return LA_ERR_INVALID_ARG;
  if (!valid_rows(x, x->dtype) || !valid_rows(dt, x->dtype) || !valid_rows(out, x->dtype) ||
      !valid_rows(bm, x->dtype) || !valid_rows(cm, x->dtype) ||
      (gate && !valid_rows(gate, x->dtype)))
    return LA_ERR_INVALID_ARG;
  if (!same_extent(x, dt) || !same_extent(x, out) || (gate && !same_extent(x, gate)) ||
      !same_extent(bm, cm) || bm->B != x->B || bm->n != x->n || bm->d != states ||
      !disjoint_rows(out))
    return LA_ERR_INVALID_ARG;
  if (!valid_param(a) || !valid_param(skip) || !valid_param(dt_bias)) return LA_ERR_INVALID_ARG;
  if (states != 8 && states != 16 && states != 32 && states != 64) return LA_ERR_UNSUPPORTED;
  for (const la_rows* r : {x, dt, bm, cm, (const la_rows*)out})
    if (!supported_rows(r)) return LA_ERR_UNSUPPORTED;
  if ((gate && !supported_rows(gate)) || x->d > kMaxChannels) return LA_ERR_UNSUPPORTED;
  const Span o_at = span_of(out);
  for (const la_rows* r : {x, dt, gate})
    if (r && !same_view(out, r) && coincide(o_at, span_of(r))) return LA_ERR_INVALID_ARG;
  if (coincide(o_at, span_of(bm)) || coincide(o_at, span_of(cm)) ||
      coincide(o_at, span_of(a, x->d * states * 4)) || coincide(o_at, span_of(skip, x->d * 4)) ||
      coincide(o_at, span_of(dt_bias, x->d * 4)))
    return LA_ERR_INVALID_ARG;
  *s = ScanArgs{};
  s->x = rows_of(x);
  s->dt = rows_of(dt);
  s->b = rows_of(bm);
  s->c = rows_of(cm);
  s->gate = gate ? rows_of(gate) : Rows{nullptr, 0, 0};
  const Rows o = rows_of(out);
  s->out = out->data;
  s->out_sb = o.sb;
  s->out_sn = o.sn;
  s->a = a;
  s->skip = skip;
  s->dt_bias = dt_bias;
  s->B = x->B;
  s->n = x->n;
  s->D = x->d;
  s->S = states;
  s->softplus = softplus != 0;
  s->bf16 = x->dtype == LA_BF16;
  return LA_OK;
}

// Whether a state that is written lies on an input of the scan or its step.
bool state_meets(const float* state, int64_t bytes, const la_rows* x, const la_rows* dt, const float* a,
                 int states, const la_rows* bm, const la_rows* cm, const float* skip,
                 const la_rows* gate, const float* dt_bias) {
  const Span at = span_of(state, bytes);
  for (const la_rows* r : {x, dt, bm, cm, gate})
    if (r && coincide(at, span_of(r))) return true;
  return coincide(at, span_of(a, x->d * states * 4)) || coincide(at, span_of(skip, x->d * 4)) ||
         coincide(at, span_of(dt_bias, x->d * 4));
}

// A grid beyond what a launch takes is a request outside the kernels' range.
la_status launch_status(cudaError_t e) {
  return e == cudaErrorInvalidConfiguration ? LA_ERR_UNSUPPORTED : to_status(e);
}

// An empty prompt: the state after it is the one before it.
cudaError_t copy_state(void* to, const void* from, size_t bytes, cudaStream_t stream) {
  if (!to || !bytes) return cudaSuccess;
  return from ? cudaMemcpyAsync(to, from, bytes, cudaMemcpyDeviceToDevice, stream)
              : cudaMemsetAsync(to, 0, bytes, stream);
}

}  // namespace

cudaError_t allow_smem(const void* kernel, int bytes, std::atomic<uint64_t>* done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = (uint64_t)1 << (dev & 63);
  if (done->load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done->fetch_or(bit, std::memory_order_relaxed);
  return e;
}

}  // namespace la

using namespace la;

extern "C" {

la_status la_linear(const la_rows* x, const la_rows* weight, const void* bias,
                    la_activation activation, const la_rows* residual, la_rows* out,
                    la_stream stream) {
  ApiRange range("la_linear");
  if (!x || !weight || !out) return LA_ERR_INVALID_ARG;
  if (!valid_rows(x, x->dtype) || !valid_rows(weight, x->dtype) || !valid_rows(out, x->dtype) ||
      (residual && !valid_rows(residual, x->dtype)))
    return LA_ERR_INVALID_ARG;
  if (x->B != 1 || weight->B != 1 || out->B != 1 || weight->d != x->d || out->n != x->n ||
      out->d != weight->n || weight->n < 1 || (residual && !same_extent(residual, out)) ||
      !disjoint_rows(out) || !disjoint_rows(x) || !disjoint_rows(weight))
    return LA_ERR_INVALID_ARG;
  if (!valid_param(bias) || !valid_activation(activation)) return LA_ERR_INVALID_ARG;
  for (const la_rows* r : {x, weight, (const la_rows*)out})
    if (!supported_rows(r)) return LA_ERR_UNSUPPORTED;
  if (residual && !supported_rows(residual)) return LA_ERR_UNSUPPORTED;
  const Span o_at = span_of(out);
  if (coincide(o_at, span_of(x)) || coincide(o_at, span_of(weight)) ||
      coincide(o_at, span_of(bias, weight->n * size_of(x->dtype))) ||
      (residual && !same_view(out, residual) && coincide(o_at, span_of(residual))))
    return LA_ERR_INVALID_ARG;
  if (x->n == 0) return LA_OK;
  DeviceInfo di;
  const la_status st = device_info(&di);
  if (st != LA_OK) return st;
  LinearArgs a{};
  a.x = rows_of(x);
  a.w = rows_of(weight);
  a.residual = residual ? rows_of(residual) : Rows{nullptr, 0, 0};
  a.out = out->data;
  a.out_sn = rows_of(out).sn;
  a.bias = bias;
  a.M = x->n;
  a.N = weight->n;
  a.K = x->d;
  a.act = activation;
  a.bf16 = x->dtype == LA_BF16;
  a.status = di.status;
  a.num_sms = di.num_sms;
  return launch_status(linear(a, (cudaStream_t)stream));
}

la_status la_causal_conv(const la_rows* x, const void* weight, int width, const void* bias,
                         la_activation activation, const void* state_in, const int32_t* lengths,
                         la_rows* out, void* state_out, la_stream stream) {
  ApiRange range("la_causal_conv");
  ConvArgs a;
  la_status st = check_conv(x, weight, width, bias, activation, out, &a);
  if (st != LA_OK) return st;
  if (!valid_param(state_in) || !valid_param(state_out) || !aligned(lengths, 4))
    return LA_ERR_INVALID_ARG;
  const int64_t bytes = a.B * (width - 1) * a.D * size_of(x->dtype);
  const Span o_at = span_of(out), in = span_of(state_in, bytes), after = span_of(state_out, bytes),
               lens = span_of(lengths, a.B * 4);
  if (coincide(o_at, span_of(x)) || coincide(o_at, in) || coincide(o_at, after) ||
      coincide(o_at, lens) || coincide(after, in) || coincide(after, span_of(x)) ||
      coincide(after, lens) || coincide(after, span_of(weight, a.D * width * size_of(x->dtype))) ||
      coincide(after, span_of(bias, a.D * size_of(x->dtype))))
    return LA_ERR_INVALID_ARG;
  a.state_in = state_in;
  a.state_out = state_out;
  a.lengths = lengths;
  if (a.B == 0) return LA_OK;
  if (a.n == 0) return to_status(copy_state(state_out, state_in, bytes, (cudaStream_t)stream));
  DeviceInfo di;
  st = device_info(&di);
  if (st != LA_OK) return st;
  a.num_sms = di.num_sms;
  return launch_status(causal_conv(a, (cudaStream_t)stream));
}

la_status la_causal_conv_step(void* state, const la_rows* x, const void* weight, int width,
                              const void* bias, la_activation activation, la_rows* out,
                              la_stream stream) {
  ApiRange range("la_causal_conv_step");
  ConvArgs a;
  la_status st = check_conv(x, weight, width, bias, activation, out, &a);
  if (st != LA_OK) return st;
  if (x->n != 1 || !valid_param(state)) return LA_ERR_INVALID_ARG;
  if (a.B == 0) return LA_OK;
  if (!state) return LA_ERR_INVALID_ARG;
  const int64_t e = size_of(x->dtype);
  const Span at = span_of(state, a.B * (width - 1) * a.D * e);
  if ((!same_view(out, x) && coincide(span_of(out), span_of(x))) || coincide(at, span_of(out)) ||
      coincide(at, span_of(x)) || coincide(at, span_of(weight, a.D * width * e)) ||
      coincide(at, span_of(bias, a.D * e)))
    return LA_ERR_INVALID_ARG;
  a.state_in = state;
  a.state_out = state;
  DeviceInfo di;
  st = device_info(&di);
  if (st != LA_OK) return st;
  a.num_sms = di.num_sms;
  return launch_status(causal_conv_step(a, (cudaStream_t)stream));
}

la_status la_selective_scan(const la_rows* x, const la_rows* dt, const float* a, int states,
                            const la_rows* bm, const la_rows* cm, const float* skip,
                            const la_rows* gate, const float* dt_bias, int softplus,
                            const float* state_in, const int32_t* lengths, la_rows* out,
                            float* state_out, la_stream stream) {
  ApiRange range("la_selective_scan");
  ScanArgs s;
  la_status st = check_scan(x, dt, a, states, bm, cm, skip, gate, dt_bias, softplus, out, &s);
  if (st != LA_OK) return st;
  if (!valid_param(state_in) || !valid_param(state_out) || !aligned(lengths, 4))
    return LA_ERR_INVALID_ARG;
  const int64_t bytes = s.B * s.D * s.S * (int64_t)sizeof(float);
  const Span o_at = span_of(out), in = span_of(state_in, bytes), lens = span_of(lengths, s.B * 4);
  if (coincide(o_at, in) || coincide(o_at, span_of(state_out, bytes)) || coincide(o_at, lens) ||
      state_meets(state_out, bytes, x, dt, a, states, bm, cm, skip, gate, dt_bias) ||
      coincide(span_of(state_out, bytes), in) || coincide(span_of(state_out, bytes), lens))
    return LA_ERR_INVALID_ARG;
  s.state_in = state_in;
  s.state_out = state_out;
  s.lengths = lengths;
  if (s.B == 0) return LA_OK;
  if (s.n == 0) return to_status(copy_state(state_out, state_in, bytes, (cudaStream_t)stream));
  DeviceInfo di;
  st = device_info(&di);
  if (st != LA_OK) return st;
  s.num_sms = di.num_sms;
  return launch_status(selective_scan(s, (cudaStream_t)stream));
}

la_status la_selective_step(float* state, const la_rows* x, const la_rows* dt, const float* a,
                            int states, const la_rows* bm, const la_rows* cm, const float* skip,
                            const la_rows* gate, const float* dt_bias, int softplus,
                            la_rows* out, la_stream stream) {
  ApiRange range("la_selective_step");
  ScanArgs s;
  la_status st = check_scan(x, dt, a, states, bm, cm, skip, gate, dt_bias, softplus, out, &s);
  if (st != LA_OK) return st;
  if (x->n != 1 || !valid_param(state)) return LA_ERR_INVALID_ARG;
  if (s.B == 0) return LA_OK;
  if (!state) return LA_ERR_INVALID_ARG;
  const int64_t bytes = s.B * s.D * s.S * (int64_t)sizeof(float);
  if (coincide(span_of(state, bytes), span_of(out)) ||
      state_meets(state, bytes, x, dt, a, states, bm, cm, skip, gate, dt_bias))
    return LA_ERR_INVALID_ARG;
  s.state_in = state;
  s.state_out = state;
  DeviceInfo di;
  st = device_info(&di);
  if (st != LA_OK) return st;
  s.num_sms = di.num_sms;
  return launch_status(selective_step(s, (cudaStream_t)stream));
}

const char* la_selftest_linear_kernel(la_dtype dtype, int64_t M, int64_t N, int64_t K, int num_sms) {
  if ((dtype != LA_BF16 && dtype != LA_F32) || M < 1 || N < 1 || K < 1 || M > kMaxDim || N > kMaxDim ||
      K > kMaxDim || num_sms < 1)
    return nullptr;
  LinearArgs a{};
  a.M = M;
  a.N = N;
  a.K = K;
  a.bf16 = dtype == LA_BF16;
  a.num_sms = num_sms;
  return linear_kernel(a);
}

const char* la_selftest_step_kernel(int64_t B, int64_t D, int states, int num_sms) {
  if (B < 1 || D < 1 || B > kMaxBatch || D > kMaxChannels || num_sms < 1 ||
      (states != 8 && states != 16 && states != 32 && states != 64))
    return nullptr;
  ScanArgs s{};
  s.B = B;
  s.D = D;
  s.S = states;
  s.num_sms = num_sms;
  return selective_step_kernel(s);
}

}  // extern "C"
