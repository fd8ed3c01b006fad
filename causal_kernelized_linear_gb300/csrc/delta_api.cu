// C ABI of the gated delta block's operators (declared in include/linattn.h):
// argument validation and hand-over to the launchers.
#include "linattn.h"

#include "block_check.h"
#include "internal.h"

#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

namespace la {
namespace {

constexpr int64_t kMaxHeads = (int64_t)1 << 16;
constexpr int64_t kMaxKeys = 256, kMaxValues = 512;

bool valid_heads(const la_heads* r, la_dtype dtype) {
  if (!r || (r->dtype != LA_BF16 && r->dtype != LA_F32) || r->dtype != dtype) return false;
  if (r->B < 0 || r->n < 0 || r->H < 1 || r->d < 1) return false;
  const int64_t e = size_of(r->dtype);
  if ((r->d * e) % 16) return false;
  const int64_t extents[3] = {r->B, r->n, r->H}, strides[3] = {r->stride_b, r->stride_n, r->stride_h};
  for (int i = 0; i < 3; ++i)
    if (extents[i] > 1 && (strides[i] < 0 || (strides[i] * e) % 16)) return false;
  return r->B == 0 || r->n == 0 || (r->data && aligned(r->data, 16));
}

bool supported_heads(const la_heads* r) {
  return r->B <= kMaxBatch && r->n <= kMaxDim && r->H <= kMaxHeads &&
         (r->B <= 1 || r->stride_b <= ((int64_t)1 << 40)) &&
         (r->n <= 1 || r->stride_n <= ((int64_t)1 << 36)) &&
         (r->H <= 1 || r->stride_h <= ((int64_t)1 << 40));
}

// An axis of a view: its extent and its stride in elements.
struct Axis {
  int64_t extent, stride;
};

// The axes with an extent above 1, the smallest stride first.
int axes_of(const la_heads* r, Axis (&x)[3]) {
  int c = 0;
  for (const Axis& a : {Axis{r->B, r->stride_b}, Axis{r->n, r->stride_n}, Axis{r->H, r->stride_h}})
    if (a.extent > 1) x[c++] = a;
  std::sort(x, x + c, [](const Axis& p, const Axis& q) { return p.stride < q.stride; });
  return c;
}

// No two elements of a view coincide: each axis steps over all within it.
bool disjoint_heads(const la_heads* r) {
  Axis x[3];
  const int c = axes_of(r, x);
  Wide within = r->d;
  for (int i = 0; i < c; ++i) {
    if (x[i].stride < within) return false;
    within += (Wide)(x[i].extent - 1) * x[i].stride;
  }
  return true;
}

// A view as [B, n, d] views that together are the same memory: axes that follow
// one another without a gap are one.  Returns how many, 0 for more than `most`.
int rows_of_heads(const la_heads* r, la_rows* to, int most) {
  Axis x[3];
  const int c = axes_of(r, x);
  int64_t width = r->d;
  Axis y[3] = {{1, 0}, {1, 0}, {1, 0}};
  int m = 0;
  for (int i = 0; i < c; ++i) {
    if (m == 0 && x[i].stride == width)
      width *= x[i].extent;
    else if (m > 0 && (Wide)y[m - 1].extent * y[m - 1].stride == x[i].stride)
      y[m - 1].extent *= x[i].extent;
    else
      y[m++] = x[i];
  }
  if (y[2].extent > most) return 0;
  for (int64_t i = 0; i < y[2].extent; ++i)
    to[i] = la_rows{static_cast<char*>(r->data) + i * y[2].stride * size_of(r->dtype), r->dtype,
                    y[1].extent, y[0].extent, width, y[1].stride, y[0].stride};
  return (int)y[2].extent;
}

// Whether an output meets an input, by coincide() on their parts; views that are
// no few [B, n, d] views are taken to be apart.
struct Parts {
  la_rows rows[64];
  int n = 0;
  explicit Parts(const la_heads* r) : n(r->B && r->n ? rows_of_heads(r, rows, 64) : 0) {}
  bool meets(const Span& s) const {
    for (int i = 0; i < n; ++i)
      if (coincide(span_of(rows + i), s)) return true;
    return false;
  }
  bool meets(const Parts& o) const {
    for (int i = 0; i < o.n; ++i)
      if (meets(span_of(o.rows + i))) return true;
    return false;
  }
};

Heads heads_of(const la_heads* r) {
  return Heads{r->data, r->B > 1 ? r->stride_b : 0, r->n > 1 ? r->stride_n : 0,
               r->H > 1 ? r->stride_h : 0};
}

bool valid_gate(const la_rows* g, const la_heads* v) {
  return g && (g->dtype == LA_BF16 || g->dtype == LA_F32) && valid_layout(g, size_of(g->dtype)) &&
         g->B == v->B && g->n == v->n && g->d == v->H;
}

la_status check_delta(const la_heads* q, const la_heads* k, const la_heads* v, const la_rows* dt,
                      const float* a, const la_rows* beta, const float* dt_bias, float scale,
                      la_heads* out, DeltaArgs* s) {
  if (!q || !k || !v || !dt || !a || !beta || !out) return LA_ERR_INVALID_ARG;
  if (!valid_heads(q, q->dtype) || !valid_heads(k, q->dtype) || !valid_heads(v, q->dtype) ||
      !valid_heads(out, q->dtype))
    return LA_ERR_INVALID_ARG;
  if (k->B != q->B || k->n != q->n || k->H != q->H || k->d != q->d || v->B != q->B ||
      v->n != q->n || out->B != v->B || out->n != v->n || out->H != v->H || out->d != v->d ||
      v->H % q->H || !disjoint_heads(out))
    return LA_ERR_INVALID_ARG;
  if (!valid_gate(dt, v) || !valid_gate(beta, v) || dt->dtype != beta->dtype ||
      (dt->dtype != LA_F32 && dt->dtype != q->dtype))
    return LA_ERR_INVALID_ARG;
  if (!valid_param(a) || !valid_param(dt_bias) || !std::isfinite(scale)) return LA_ERR_INVALID_ARG;
  for (const la_heads* r : {q, k, v, (const la_heads*)out})
    if (!supported_heads(r)) return LA_ERR_UNSUPPORTED;
  if (!supported_rows(dt) || !supported_rows(beta)) return LA_ERR_UNSUPPORTED;
  if (q->d % 8 || v->d % 8 || q->d > kMaxKeys || v->d > kMaxValues) return LA_ERR_UNSUPPORTED;
  *s = DeltaArgs{};
  s->q = heads_of(q);
  s->k = heads_of(k);
  s->v = heads_of(v);
  s->out = heads_of(out);
  s->dt = rows_of(dt);
  s->beta = rows_of(beta);
  s->gates_f32 = dt->dtype == LA_F32;
  s->a = a;
  s->dt_bias = dt_bias;
  s->B = q->B;
  s->n = q->n;
  s->Hk = q->H;
  s->Hv = v->H;
  s->dk = (int)q->d;
  s->dv = (int)v->d;
  s->scale = scale;
  s->bf16 = q->dtype == LA_BF16;
  return LA_OK;
}

// Whether memory that the rule writes (Parts or a Span) lies on one of its inputs.
inline bool meet(const Parts& w, const Span& s) { return w.meets(s); }
inline bool meet(const Span& w, const Span& s) { return coincide(w, s); }

template <typename W>
bool meets_inputs(const W& w, const la_heads* q, const la_heads* k, const la_heads* v,
                  const la_rows* dt, const float* a, const la_rows* beta, const float* dt_bias) {
  for (const la_heads* r : {q, k, v})
    if (Parts(r).meets(w)) return true;
  return meet(w, span_of(dt)) || meet(w, span_of(beta)) || meet(w, span_of(a, v->H * 4)) ||
         meet(w, span_of(dt_bias, v->H * 4));
}

}  // namespace
}  // namespace la

using namespace la;

extern "C" {

la_status la_gated_delta(const la_heads* q, const la_heads* k, const la_heads* v,
                         const la_rows* dt, const float* a, const la_rows* beta,
                         const float* dt_bias, int softplus, int sigmoid, int normalize,
                         float scale, const float* state_in, const int32_t* lengths,
                         la_heads* out, float* state_out, la_stream stream) {
  ApiRange range("la_gated_delta");
  DeltaArgs s;
  la_status st = check_delta(q, k, v, dt, a, beta, dt_bias, scale, out, &s);
  if (st != LA_OK) return st;
  if (!valid_param(state_in) || !valid_param(state_out) || !aligned(lengths, 4))
    return LA_ERR_INVALID_ARG;
  const int64_t bytes = s.B * s.Hv * s.dk * s.dv * (int64_t)sizeof(float);
  const Span in = span_of(state_in, bytes), after = span_of(state_out, bytes),
             lens = span_of(lengths, s.B * 4);
  const Parts o(out);
  if (o.meets(in) || o.meets(after) || o.meets(lens) || coincide(after, in) || coincide(after, lens) ||
      meets_inputs(o, q, k, v, dt, a, beta, dt_bias) ||
      (state_out && meets_inputs(after, q, k, v, dt, a, beta, dt_bias)))
    return LA_ERR_INVALID_ARG;
  s.softplus = softplus != 0;
  s.sigmoid = sigmoid != 0;
  s.normalize = normalize != 0;
  s.state_in = state_in;
  s.state_out = state_out;
  s.lengths = lengths;
  if (s.B == 0) return LA_OK;
  if (s.n == 0) return to_status(copy_state(state_out, state_in, bytes, (cudaStream_t)stream));
  DeviceInfo di;
  st = device_info(&di);
  if (st != LA_OK) return st;
  s.status = di.status;
  s.num_sms = di.num_sms;
  return launch_status(gated_delta(s, (cudaStream_t)stream));
}

la_status la_gated_delta_step(float* state, const la_heads* q, const la_heads* k,
                              const la_heads* v, const la_rows* dt, const float* a,
                              const la_rows* beta, const float* dt_bias, int softplus,
                              int sigmoid, int normalize, float scale, la_heads* out,
                              la_stream stream) {
  ApiRange range("la_gated_delta_step");
  DeltaArgs s;
  la_status st = check_delta(q, k, v, dt, a, beta, dt_bias, scale, out, &s);
  if (st != LA_OK) return st;
  if (q->n != 1 || !valid_param(state)) return LA_ERR_INVALID_ARG;
  if (s.B == 0) return LA_OK;
  if (!state) return LA_ERR_INVALID_ARG;
  const Span at = span_of(state, s.B * s.Hv * s.dk * s.dv * (int64_t)sizeof(float));
  const Parts o(out);
  if (o.meets(at) || meets_inputs(o, q, k, v, dt, a, beta, dt_bias) ||
      meets_inputs(at, q, k, v, dt, a, beta, dt_bias))
    return LA_ERR_INVALID_ARG;
  s.softplus = softplus != 0;
  s.sigmoid = sigmoid != 0;
  s.normalize = normalize != 0;
  s.state_in = state;
  s.state_out = state;
  DeviceInfo di;
  st = device_info(&di);
  if (st != LA_OK) return st;
  s.status = di.status;
  s.num_sms = di.num_sms;
  return launch_status(gated_delta(s, (cudaStream_t)stream));
}

la_status la_rms_norm(const la_rows* x, const void* weight, int64_t group, float eps,
                      const la_rows* residual, const la_rows* gate, la_rows* out, float* scale,
                      la_rows* sum, la_stream stream) {
  ApiRange range("la_rms_norm");
  if (!x || !out) return LA_ERR_INVALID_ARG;
  const bool quantize = out->dtype == LA_E4M3;
  if (!valid_rows(x, x->dtype) || (residual && !valid_rows(residual, x->dtype)) ||
      (gate && !valid_rows(gate, x->dtype)) || (sum && !valid_rows(sum, x->dtype)) ||
      !(quantize ? valid_e4m3(out, 8) : valid_rows(out, x->dtype)))
    return LA_ERR_INVALID_ARG;
  if (x->B != 1 || !same_extent(x, out) || (residual && !same_extent(x, residual)) ||
      (gate && !same_extent(x, gate)) || (sum && !same_extent(x, sum)) || !disjoint_rows(out) ||
      (sum && !disjoint_rows(sum)))
    return LA_ERR_INVALID_ARG;
  const int64_t e = size_of(x->dtype);
  if (group < 1 || x->d % group || (group * e) % 16 || (quantize && group % 8) ||
      !valid_param(weight) || !(eps >= 0.f) || !std::isfinite(eps) || !aligned(scale, 4) ||
      (sum && !residual))
    return LA_ERR_INVALID_ARG;
  if (x->n > 0 && quantize != (scale != nullptr)) return LA_ERR_INVALID_ARG;
  for (const la_rows* r : {x, residual, gate, (const la_rows*)sum, (const la_rows*)out})
    if (r && !supported_rows(r)) return LA_ERR_UNSUPPORTED;
  if (!rms_norm_supported(x->d, x->dtype == LA_BF16)) return LA_ERR_UNSUPPORTED;
  const Span o = span_of(out), w = span_of(weight, group * e), sc = span_of(scale, x->n * 4);
  if (coincide(o, w) || coincide(o, sc) || coincide(sc, w)) return LA_ERR_INVALID_ARG;
  for (const la_rows* r : {x, residual, gate}) {
    if (!r) continue;
    if (coincide(sc, span_of(r))) return LA_ERR_INVALID_ARG;
    // a CTA or warp reads its row in full before it writes any of it
    if ((quantize || !same_view(out, r)) && coincide(o, span_of(r))) return LA_ERR_INVALID_ARG;
    if (sum && (r == gate || !same_view(sum, r)) && coincide(span_of(sum), span_of(r)))
      return LA_ERR_INVALID_ARG;
  }
  if (sum && (coincide(span_of(sum), o) || coincide(span_of(sum), w) || coincide(span_of(sum), sc)))
    return LA_ERR_INVALID_ARG;
  if (x->n == 0) return LA_OK;
  NormArgs a{};
  a.x = rows_of(x);
  a.residual = residual ? rows_of(residual) : Rows{nullptr, 0, 0};
  a.gate = gate ? rows_of(gate) : Rows{nullptr, 0, 0};
  a.out = out->data;
  a.out_sn = rows_of(out).sn;
  a.sum = sum ? sum->data : nullptr;
  a.sum_sn = sum ? rows_of(sum).sn : 0;
  a.scale = scale;
  a.weight = weight;
  a.M = x->n;
  a.D = (int)x->d;
  a.group = (int)group;
  a.eps = eps;
  a.bf16 = x->dtype == LA_BF16;
  a.quantize = quantize;
  return launch_status(rms_norm(a, (cudaStream_t)stream));
}

la_status la_linear_e4m3(const la_rows* x, const float* x_scale, const la_rows* weight,
                         const float* weight_scale, const void* bias, la_activation activation,
                         const la_rows* residual, la_rows* out, la_stream stream) {
  ApiRange range("la_linear_e4m3");
  if (!x || !weight || !out || !weight_scale) return LA_ERR_INVALID_ARG;
  if (!valid_e4m3(x, 16) || !valid_e4m3(weight, 16) || !valid_rows(out, LA_BF16) ||
      (residual && !valid_rows(residual, LA_BF16)))
    return LA_ERR_INVALID_ARG;
  if (x->B != 1 || weight->B != 1 || out->B != 1 || weight->d != x->d || out->n != x->n ||
      out->d != weight->n || weight->n < 1 || (residual && !same_extent(residual, out)) ||
      !disjoint_rows(out) || !disjoint_rows(x) || !disjoint_rows(weight))
    return LA_ERR_INVALID_ARG;
  if (!valid_param(bias) || !valid_param(weight_scale) || !aligned(x_scale, 4) ||
      (!x_scale && x->n > 0) || !valid_activation(activation))
    return LA_ERR_INVALID_ARG;
  for (const la_rows* r : {x, weight, residual, (const la_rows*)out})
    if (r && !supported_rows(r)) return LA_ERR_UNSUPPORTED;
  const Span o_at = span_of(out);
  if (coincide(o_at, span_of(x)) || coincide(o_at, span_of(weight)) ||
      coincide(o_at, span_of(bias, weight->n * 2)) || coincide(o_at, span_of(x_scale, x->n * 4)) ||
      coincide(o_at, span_of(weight_scale, weight->n * 4)) ||
      (residual && !same_view(out, residual) && coincide(o_at, span_of(residual))))
    return LA_ERR_INVALID_ARG;
  if (x->n == 0) return LA_OK;
  DeviceInfo di;
  const la_status st = device_info(&di);
  if (st != LA_OK) return st;
  LinearE4m3Args a{};
  a.base.x = rows_of(x);
  a.base.w = rows_of(weight);
  a.base.residual = residual ? rows_of(residual) : Rows{nullptr, 0, 0};
  a.base.out = out->data;
  a.base.out_sn = rows_of(out).sn;
  a.base.bias = bias;
  a.base.M = x->n;
  a.base.N = weight->n;
  a.base.K = x->d;
  a.base.act = activation;
  a.base.status = di.status;
  a.base.num_sms = di.num_sms;
  a.x_scale = x_scale;
  a.w_scale = weight_scale;
  return launch_status(tc_linear_e4m3(a, (cudaStream_t)stream));
}

}  // extern "C"
