// The gated delta rule token by token on the CUDA cores:
//   w_t = β_t(v_t − k_t(α_t S_{t−1})),  S_t = α_t S_{t−1} + k_tᵀ w_t,  o_t = scale·q_t S_t.
//
// recurrent_kernel (several tokens).  The columns of S do not meet: a warp has a few of
// them (16 or 8 for dk = 128) with all their rows, 16 or 8 rows by 4 columns to a lane, and
// walks the tokens with S in registers, two tokens' q, k and v under way (4×2048 tokens of
// 32 heads of 128 in fp32: 1.61 ms).  Bound by the latency of a token's
// chain, 0.49 to 0.58 µs, while warps are few, and then by issue.  k·S and q·S of the
// state before the token are summed together over the P lanes that share a column; o_t = scale·(α q·S_{t−1} + (q·k) w_t)
// needs no second pass over S, so the next token's sums wait for w_t alone.
//
// step_kernel (one token) is bound by reading and writing S, 128 KB for a head of
// 128×128.  A CTA has 128 columns (or 64) of one head's S with all rows, in the
// registers of 256 threads: warps read whole rows of 512 bytes, all loads of a thread
// are issued before anything waits for one, and the sums over rows go through shared
// memory once.  256×32 heads of 128×128: 160 µs = 6.7 TB/s, a copy's bandwidth.
//
// Everything is fp32.
#include "block.cuh"
#include "internal.h"

#include <algorithm>
#include <atomic>
#include <type_traits>

namespace la {
namespace {

using namespace block;
using bf16 = __nv_bfloat16;

constexpr int kThreads = 128;
constexpr unsigned kAll = 0xffffffffu;

struct DeltaParams {
  Heads q, k, v, out;
  Rows dt, beta;
  const float* a;
  const float* dt_bias;
  const float* state_in;
  float* state_out;
  const int32_t* lengths;
  int64_t warps;
  // sequences in `parts` parts of part_tokens (see delta_parts in internal.h)
  int parts, part_tokens;
  float *added, *transition;
  const float* entering;
  int n, Hk, Hv, dk, dv, slices;
  float scale;
  bool gates_f32, softplus, sigmoid, normalize;
};

// Four neighbouring elements as they are in memory, and as two pairs of fp32.
template <typename T> struct Raw4;
template <> struct Raw4<bf16> {
  uint2 v = {0u, 0u};
  __device__ __forceinline__ void load(const bf16* p) { v = *reinterpret_cast<const uint2*>(p); }
  __device__ __forceinline__ f32x2 lo() const { return pack2(tc::bf16lo_to_f32(v.x), tc::bf16hi_to_f32(v.x)); }
  __device__ __forceinline__ f32x2 hi() const { return pack2(tc::bf16lo_to_f32(v.y), tc::bf16hi_to_f32(v.y)); }
};
template <> struct Raw4<float> {
  float4 v = {0.f, 0.f, 0.f, 0.f};
  __device__ __forceinline__ void load(const float* p) { v = *reinterpret_cast<const float4*>(p); }
  __device__ __forceinline__ f32x2 lo() const { return pack2(v.x, v.y); }
  __device__ __forceinline__ f32x2 hi() const { return pack2(v.z, v.w); }
};

__device__ __forceinline__ float gate_value(const Rows& r, bool f32, int64_t at) {
  return f32 ? static_cast<const float*>(r.data)[at] : to_f32(static_cast<const bf16*>(r.data)[at]);
}

// α and β of a token.  A step of zero leaves the state alone whatever the rate.
struct Gates {
  Decay alpha;
  float beta;
};
__device__ __forceinline__ Gates gates(const DeltaParams& p, int64_t b, int64_t t, int h) {
  float d = gate_value(p.dt, p.gates_f32, b * p.dt.sb + t * p.dt.sn + h);
  if (p.dt_bias) d += p.dt_bias[h];
  if (p.softplus) d = softplus(d);
  float be = gate_value(p.beta, p.gates_f32, b * p.beta.sb + t * p.beta.sn + h);
  if (p.sigmoid) be = 1.f / (1.f + expf(-be));
  return {decay_of(d == 0.f ? 0.f : d * p.a[h]), be};
}

// Sums over a column's P lanes, of four columns: lane i gets column
// 2·(i & 1) + (i >> 1 & 1).
template <int P>
__device__ __forceinline__ float sum_columns(const float (&c)[4], int lane) {
  const bool b0 = lane & 1, b1 = lane & 2;
  const float k0 = b0 ? c[2] : c[0], k1 = b0 ? c[3] : c[1];
  const float s0 = b0 ? c[0] : c[2], s1 = b0 ? c[1] : c[3];
  const float x0 = k0 + __shfl_xor_sync(kAll, s0, 1), x1 = k1 + __shfl_xor_sync(kAll, s1, 1);
  float r = (b1 ? x1 : x0) + __shfl_xor_sync(kAll, b1 ? x0 : x1, 2);
#pragma unroll
  for (int m = 4; m < P; m *= 2) r += __shfl_xor_sync(kAll, r, m);
  return r;
}

// The way back: every lane gets the four columns' values.
__device__ __forceinline__ void spread_columns(float w, int lane, float (&c)[4]) {
  const bool b0 = lane & 1, b1 = lane & 2;
  const float o = __shfl_xor_sync(kAll, w, 2);
  const float x0 = b1 ? o : w, x1 = b1 ? w : o;
  const float y0 = __shfl_xor_sync(kAll, x0, 1), y1 = __shfl_xor_sync(kAll, x1, 1);
  c[0] = b0 ? y0 : x0, c[1] = b0 ? y1 : x1, c[2] = b0 ? x0 : y0, c[3] = b0 ? x1 : y1;
}

template <int P>
__device__ __forceinline__ float sum_lanes(float v) {
#pragma unroll
  for (int m = 1; m < P; m *= 2) v += __shfl_xor_sync(kAll, v, m);
  return v;
}

__device__ __forceinline__ float both(f32x2 v) {
  float lo, hi;
  unpack2(v, lo, hi);
  return lo + hi;
}

// One warp: 128/P columns of one (b, head), 4R rows to a lane, all tokens or a part of them.  SUMMARY:
// without outputs, from zero, and (dk columns more) from the identity without v.
template <typename T, int P, int R, bool SUMMARY>
__global__ void __launch_bounds__(kThreads) recurrent_kernel(const DeltaParams p) {
  entry();
  const int64_t wid = (int64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
  if (wid >= p.warps) return;
  const int lane = threadIdx.x % 32, part = lane % P;
  const int slices = SUMMARY ? p.slices + (p.dk + 128 / P - 1) / (128 / P) : p.slices, parts = p.parts - SUMMARY;
  const int which = (int)(wid % slices);
  const bool identity = SUMMARY && which >= p.slices;
  const int slice = identity ? which - p.slices : which, seg = (int)(wid / slices % parts);
  const int64_t bh = wid / slices / parts;
  const int h = (int)(bh % p.Hv);
  const int64_t b = bh / p.Hv;
  const int hk = h / (p.Hv / p.Hk);
  const int col0 = slice * (128 / P) + lane / P * 4;           // this lane's columns
  const int mine = col0 + 2 * (lane & 1) + (lane >> 1 & 1);    // the one it sums
  const int cols = identity ? p.dk : p.dv;                     // multiples of 8
  const bool in = col0 < cols;
  const int64_t t0 = (int64_t)seg * p.part_tokens;
  const int n = min((int)(p.n - t0), p.part_tokens);
  const int live = max(0, min((int)(live_tokens(p.lengths, b, p.n) - t0), n));
  const float* state_in = nullptr;
  float* state_out;
  if (SUMMARY) {
    state_out = identity ? p.transition + (bh * parts + seg) * p.dk * p.dk : p.added + (bh * parts + seg) * p.dk * p.dv;
  } else {
    state_in = seg ? p.entering + (bh * (parts - 1) + seg - 1) * p.dk * p.dv
                   : p.state_in ? p.state_in + bh * p.dk * p.dv : nullptr;
    state_out = seg == parts - 1 && p.state_out ? p.state_out + bh * p.dk * p.dv : nullptr;
  }

  // rows 4(iP + part) + j of S, in pairs of rows
  f32x2 S[4][2 * R];
  bool row_in[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int r = 4 * (i * P + part);
    row_in[i] = r < p.dk;
    float4 m[4] = {};
    if (state_in && in && row_in[i]) {
      const float* at = state_in + (int64_t)r * p.dv + col0;
#pragma unroll
      for (int j = 0; j < 4; ++j) m[j] = *reinterpret_cast<const float4*>(at + (int64_t)j * p.dv);
    }
    if (identity && r == col0) m[0].x = m[1].y = m[2].z = m[3].w = 1.f;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      S[0][2 * i + j] = pack2(m[2 * j].x, m[2 * j + 1].x);
      S[1][2 * i + j] = pack2(m[2 * j].y, m[2 * j + 1].y);
      S[2][2 * i + j] = pack2(m[2 * j].z, m[2 * j + 1].z);
      S[3][2 * i + j] = pack2(m[2 * j].w, m[2 * j + 1].w);
    }
  }

  const T* qp = static_cast<const T*>(p.q.data) + b * p.q.sb + t0 * p.q.sn + (int64_t)hk * p.q.sh;
  const T* kp = static_cast<const T*>(p.k.data) + b * p.k.sb + t0 * p.k.sn + (int64_t)hk * p.k.sh;
  const T* vp = static_cast<const T*>(p.v.data) + b * p.v.sb + t0 * p.v.sn + (int64_t)h * p.v.sh + mine;
  T* op = static_cast<T*>(const_cast<void*>(p.out.data)) + b * p.out.sb + t0 * p.out.sn + (int64_t)h * p.out.sh + mine;
  struct Token {
    Raw4<T> q[R], k[R];
    T v = from_f32<T>(0.f);
  };
  Token even, odd;   // tokens under way
  auto load = [&](Token& to, int t) {   // token t's share of this lane
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (row_in[i]) {
        const int r = 4 * (i * P + part);
        if (!SUMMARY) to.q[i].load(qp + t * p.q.sn + r);
        to.k[i].load(kp + t * p.k.sn + r);
      }
    if (in && !identity) to.v = vp[t * p.v.sn];
  };
  if (live > 0) load(even, 0);
  if (live > 1) load(odd, 1);
  Gates g = {{1.f, 0.f}, 0.f};   // of 32 tokens, one to a lane
  uint32_t near = 0;             // those whose α is near 1
  auto walk = [&](Token& at, int t) {
    if (t % 32 == 0) {
      if (t + lane < live) g = gates(p, b, t0 + t + lane, h);
      near = __ballot_sync(kAll, g.alpha.keep != 0.f);
    }
    const bool keep = near >> t % 32 & 1;
    const Decay alpha{keep ? 1.f : 0.f, __shfl_sync(kAll, g.alpha.more, t % 32)};
    const float beta = __shfl_sync(kAll, g.beta, t % 32);
    f32x2 q[2 * R], k[2 * R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      q[2 * i] = at.q[i].lo(), q[2 * i + 1] = at.q[i].hi();
      k[2 * i] = at.k[i].lo(), k[2 * i + 1] = at.k[i].hi();
    }
    const float v = to_f32(at.v);
    if (t + 2 < live) load(at, t + 2);
    f32x2 qk2 = 0, qq2 = 0, kk2 = 0, ks2[4] = {}, qs2[4] = {};
#pragma unroll
    for (int i = 0; i < 2 * R; ++i) {
      qk2 = fma2(q[i], k[i], qk2);
      qq2 = fma2(q[i], q[i], qq2);
      kk2 = fma2(k[i], k[i], kk2);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        ks2[c] = fma2(k[i], S[c][i], ks2[c]);
        qs2[c] = fma2(q[i], S[c][i], qs2[c]);
      }
    }
    float ks[4], qs[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) ks[c] = both(ks2[c]), qs[c] = both(qs2[c]);
    float rk = 1.f, rq = p.scale;
    if (p.normalize) {
      rk = rsqrtf(sum_lanes<P>(both(kk2)) + 1e-6f);
      rq *= rsqrtf(sum_lanes<P>(both(qq2)) + 1e-6f);
    }
    const float qk = sum_lanes<P>(both(qk2));
    const float ksum = sum_columns<P>(ks, lane), qsum = sum_columns<P>(qs, lane);
    const float w = rk * (beta * (v - decayed(alpha, rk * ksum)));
    float wc[4];
    spread_columns(w, lane, wc);
    const f32x2 more = pack2(alpha.more, alpha.more);
    auto update = [&](auto near_one) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const f32x2 w2 = pack2(wc[c], wc[c]);
#pragma unroll
        for (int i = 0; i < 2 * R; ++i)
          S[c][i] = fma2(k[i], w2, decltype(near_one)::value ? fma2(more, S[c][i], S[c][i]) : mul2(more, S[c][i]));
      }
    };
    if (keep) update(std::true_type()); else update(std::false_type());   // (the same for the whole warp)
    if (!SUMMARY && in && part < 4) op[t * p.out.sn] = from_f32<T>(rq * decayed(alpha, qsum, qk * w));
  };
#pragma unroll 1
  for (int t = 0; t < live; t += 2) {
    walk(even, t);
    if (t + 1 < live) walk(odd, t + 1);
  }
  if (!SUMMARY && in && part < 4)
    for (int t = live; t < n; ++t) op[t * p.out.sn] = from_f32<T>(0.f);
  if (!state_out || !in) return;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    if (!row_in[i]) continue;
    float* at = state_out + (int64_t)(4 * (i * P + part)) * cols + col0;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float4 lo, hi;
      unpack2(S[0][2 * i + j], lo.x, hi.x);
      unpack2(S[1][2 * i + j], lo.y, hi.y);
      unpack2(S[2][2 * i + j], lo.z, hi.z);
      unpack2(S[3][2 * i + j], lo.w, hi.w);
      *reinterpret_cast<float4*>(at + (int64_t)(2 * j) * cols) = lo;
      *reinterpret_cast<float4*>(at + (int64_t)(2 * j + 1) * cols) = hi;
    }
  }
}

// ------------------------------------------------------------------ one token

constexpr int kStepThreads = 256;

// CG groups of four columns, RPT rows per thread.
template <typename T, int CG, int RPT>
__global__ void __launch_bounds__(kStepThreads, RPT > 16 ? 1 : 2) step_kernel(const DeltaParams p) {
  constexpr int RG = kStepThreads / CG, kRows = RG * RPT;
  __shared__ float4 part[2][RG][CG];
  __shared__ float ks[kRows], qs[kRows];
  __shared__ float red[3][kStepThreads / 32];
  entry();
  const int slice = (int)(blockIdx.x % p.slices);
  const int64_t bh = blockIdx.x / p.slices, b = bh / p.Hv;
  const int h = (int)(bh % p.Hv), hk = h / (p.Hv / p.Hk);
  const int t = threadIdx.x, cg = t % CG, rg = t / CG;
  const int col = (slice * CG + cg) * 4;
  const bool in = col < p.dv;
  const float* from = p.state_in + bh * p.dk * p.dv + col;
  float* to = p.state_out + bh * p.dk * p.dv + col;
  float4 S[RPT];
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    const int r = i * RG + rg;
    S[i] = in && r < p.dk ? __ldcs(reinterpret_cast<const float4*>(from + (int64_t)r * p.dv)) : make_float4(0, 0, 0, 0);
  }
  // k and q, their lengths and product; one element of each per thread
  const T* kp = static_cast<const T*>(p.k.data) + b * p.k.sb + (int64_t)hk * p.k.sh;
  const T* qp = static_cast<const T*>(p.q.data) + b * p.q.sb + (int64_t)hk * p.q.sh;
  const float ke = t < p.dk ? to_f32(kp[t]) : 0.f, qe = t < p.dk ? to_f32(qp[t]) : 0.f;
  const Gates g = gates(p, b, 0, h);
  Raw4<T> vr;
  if (in) vr.load(static_cast<const T*>(p.v.data) + b * p.v.sb + (int64_t)h * p.v.sh + col);
  if (t < kRows) ks[t] = ke, qs[t] = qe;
  const float kk = sum_lanes<32>(ke * ke), qq = sum_lanes<32>(qe * qe), qk = sum_lanes<32>(qe * ke);
  if (t % 32 == 0) red[0][t / 32] = kk, red[1][t / 32] = qq, red[2][t / 32] = qk;
  __syncthreads();
  float4 a = make_float4(0, 0, 0, 0), c = a;   // k·S and q·S
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    const float k = ks[i * RG + rg], q = qs[i * RG + rg];
    a.x = fmaf(k, S[i].x, a.x), a.y = fmaf(k, S[i].y, a.y), a.z = fmaf(k, S[i].z, a.z), a.w = fmaf(k, S[i].w, a.w);
    c.x = fmaf(q, S[i].x, c.x), c.y = fmaf(q, S[i].y, c.y), c.z = fmaf(q, S[i].z, c.z), c.w = fmaf(q, S[i].w, c.w);
  }
  part[0][rg][cg] = a;
  part[1][rg][cg] = c;
  float s[3] = {};
#pragma unroll
  for (int i = 0; i < kStepThreads / 32; ++i) s[0] += red[0][i], s[1] += red[1][i], s[2] += red[2][i];
  const float rk = p.normalize ? rsqrtf(s[0] + 1e-6f) : 1.f;
  const float rq = p.scale * (p.normalize ? rsqrtf(s[1] + 1e-6f) : 1.f);
  __syncthreads();
  float ksum[4] = {}, qsum[4] = {};
#pragma unroll
  for (int r = 0; r < RG; ++r) {
    const float4 x = part[0][r][cg];
    ksum[0] += x.x, ksum[1] += x.y, ksum[2] += x.z, ksum[3] += x.w;
  }
  if (rg == 0)
#pragma unroll
    for (int r = 0; r < RG; ++r) {
      const float4 x = part[1][r][cg];
      qsum[0] += x.x, qsum[1] += x.y, qsum[2] += x.z, qsum[3] += x.w;
    }
  float v[4], w[4];
  unpack2(vr.lo(), v[0], v[1]);
  unpack2(vr.hi(), v[2], v[3]);
#pragma unroll
  for (int j = 0; j < 4; ++j) w[j] = rk * (g.beta * (v[j] - decayed(g.alpha, rk * ksum[j])));
  auto update = [&](auto near_one) {
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      const int r = i * RG + rg;
      const float k = ks[r], m = g.alpha.more;
      auto next = [&](float s, float wj) { return fmaf(k, wj, near_one ? fmaf(m, s, s) : m * s); };
      const float4 n = make_float4(next(S[i].x, w[0]), next(S[i].y, w[1]), next(S[i].z, w[2]), next(S[i].w, w[3]));
      if (in && r < p.dk) __stcs(reinterpret_cast<float4*>(to + (int64_t)r * p.dv), n);
    }
  };
  if (g.alpha.keep != 0.f) update(std::true_type()); else update(std::false_type());   // (the same for the CTA)
  if (rg == 0 && in) {
    T* op = static_cast<T*>(const_cast<void*>(p.out.data)) + b * p.out.sb + (int64_t)h * p.out.sh + col;
#pragma unroll
    for (int j = 0; j < 4; ++j) op[j] = from_f32<T>(rq * decayed(g.alpha, qsum[j], s[2] * w[j]));
  }
}

template <typename T, int CG, int RPT>
cudaError_t launch_step(const DeltaArgs& a, DeltaParams p, cudaStream_t s) {
  p.slices = (a.dv + 4 * CG - 1) / (4 * CG);
  const int64_t ctas = a.B * a.Hv * p.slices;
  if (ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
  return launch(step_kernel<T, CG, RPT>, (unsigned)ctas, kStepThreads, 0, s, 1, p);
}

template <typename T>
cudaError_t step(const DeltaArgs& a, const DeltaParams& p, cudaStream_t s) {
  // 128 columns at a time, 64 where that leaves fewer of them without work
  const int rest = a.dv % 128;
  if (rest && rest <= 64) {
    if (a.dk <= 64) return launch_step<T, 16, 4>(a, p, s);
    if (a.dk <= 128) return launch_step<T, 16, 8>(a, p, s);
    return launch_step<T, 16, 16>(a, p, s);
  }
  if (a.dk <= 64) return launch_step<T, 32, 8>(a, p, s);
  if (a.dk <= 128) return launch_step<T, 32, 16>(a, p, s);
  return launch_step<T, 32, 32>(a, p, s);
}

// ------------------------------------------------------------------ several tokens

// Parts of the sequences, and the µs that they are taken to need, with P lanes to a
// column: a warp takes `token` µs for a token while no more than two share a scheduler,
// and then as much longer as they are more.  Parts measured a seventh above that sum, or
// more (333 tokens of 8 heads of 128 with 16 lanes: 93 µs in 8 parts, 166 undivided; 2×512 of
// 16 heads with 8: 314 in 5 parts, 249 in 4, 297 undivided).
struct Plan {
  int parts;
  double us;
};
Plan plan_for(const DeltaArgs& a, int P, double token) {
  const int64_t cols = 128 / P, slices = (a.dv + cols - 1) / cols, more = (a.dk + cols - 1) / cols;
  auto share = [&](int64_t warps) { return std::max(1.0, (double)warps / (8.0 * a.num_sms)); };
  const int64_t heads = a.B * a.Hv;
  Plan best{1, a.n * token * share(heads * slices)};
  if (a.dk > 128) return best;   // what delta_join holds
  for (int g = 2; g <= 64 && g * 32 <= a.n; g += g < 8 ? 1 : 4) {
    const int64_t part = (a.n + g - 1) / g;
    const double sum = part * token * (share(heads * (g - 1) * (slices + more)) + share(heads * g * slices)) + 20.0 +
                       3.0 * (g - 1);
    const double t = 1.15 * sum;
    if (t < best.us) best = {g, t};
  }
  return best;
}

template <typename T, int P, int R>
cudaError_t launch_recurrent(const DeltaArgs& a, DeltaParams p, int parts, cudaStream_t s) {
  constexpr int kCols = 128 / P;
  const int64_t more = (a.dk + kCols - 1) / kCols, heads = a.B * a.Hv;
  p.slices = (a.dv + kCols - 1) / kCols;
  p.parts = parts;
  p.part_tokens = (int)((a.n + p.parts - 1) / p.parts);
  p.parts = (int)((a.n + p.part_tokens - 1) / p.part_tokens);
  auto ctas = [](int64_t warps) { return (warps + kThreads / 32 - 1) / (kThreads / 32); };
  const int64_t first = heads * (p.parts - 1) * (p.slices + more), warps = heads * p.parts * p.slices;
  if (ctas(warps) > INT32_MAX || ctas(first) > INT32_MAX) return cudaErrorInvalidConfiguration;
  DeltaParts w{};
  cudaError_t e = cudaSuccess;
  if (p.parts > 1) {
    if ((e = delta_parts(a, p.parts, &w, s)) != cudaSuccess) return e;
    p.added = w.added, p.transition = w.transition, p.entering = w.entering;
    p.warps = first;
    e = launch(recurrent_kernel<T, P, R, true>, (unsigned)ctas(first), kThreads, 0, s, 1, p);
    if (e == cudaSuccess) e = delta_join(a, p.parts, w, s);
  }
  p.warps = warps;
  if (e == cudaSuccess) e = launch(recurrent_kernel<T, P, R, false>, (unsigned)ctas(warps), kThreads, 0, s, 1, p);
  if (w.added) {
    const cudaError_t f = cudaFreeAsync(w.added, s);
    if (e == cudaSuccess) e = f;
  }
  return e;
}

template <typename T>
cudaError_t by_keys(const DeltaArgs& a, const DeltaParams& p, cudaStream_t s) {
  // Sixteen rows to a lane; or eight, with twice the warps, where each of them has a
  // scheduler to itself: 2×512 tokens of 16 heads of 128 (512 warps) in 252 µs undivided
  // against 297 (4×512, while a decay was one factor, in 337 against 272).
  const int lanes = a.dk <= 64 ? 4 : a.dk <= 128 ? 8 : 16;
  const Plan wide = plan_for(a, lanes, 0.6);
  if (a.dk <= 128 && a.B * a.Hv * ((a.dv * 2 * lanes + 127) / 128) <= 4 * (int64_t)a.num_sms) {
    const Plan fine = plan_for(a, 2 * lanes, 0.45);
    if (fine.us < wide.us)
      return a.dk <= 64 ? launch_recurrent<T, 8, 2>(a, p, fine.parts, s) : launch_recurrent<T, 16, 2>(a, p, fine.parts, s);
  }
  if (a.dk <= 64) return launch_recurrent<T, 4, 4>(a, p, wide.parts, s);
  if (a.dk <= 128) return launch_recurrent<T, 8, 4>(a, p, wide.parts, s);
  return launch_recurrent<T, 16, 4>(a, p, wide.parts, s);
}

}  // namespace

cudaError_t gated_delta(const DeltaArgs& a, cudaStream_t s) {
  // A chunk takes the same whatever its tokens, by 32 heads of 128 in 1, 4, 32 and 256
  // sequences 13.8, 14.8, 96 and 733 µs.  The kernels here take for 12 tokens 10.2, 16.5, 113
  // and 834, for 16 tokens 12.1, 19.9, 136 and 1001 µs.
  if (a.n >= 16 && tc_gated_delta_supported(a)) return tc_gated_delta(a, s);
  DeltaParams p{};
  p.q = a.q, p.k = a.k, p.v = a.v, p.out = a.out;
  p.dt = a.dt, p.beta = a.beta;
  p.a = a.a, p.dt_bias = a.dt_bias;
  p.state_in = a.state_in, p.state_out = a.state_out, p.lengths = a.lengths;
  p.n = (int)a.n, p.Hk = (int)a.Hk, p.Hv = (int)a.Hv, p.dk = a.dk, p.dv = a.dv;
  p.scale = a.scale;
  p.gates_f32 = a.gates_f32, p.softplus = a.softplus, p.sigmoid = a.sigmoid;
  p.normalize = a.normalize;
  if (a.n == 1 && a.state_in && a.state_out && !a.lengths) return a.bf16 ? step<bf16>(a, p, s) : step<float>(a, p, s);
  return a.bf16 ? by_keys<bf16>(a, p, s) : by_keys<float>(a, p, s);
}

}  // namespace la
