// The selective state-space recurrence over a prompt and for one token:
//   Δ = softplus(dt + dt_bias);  h_s ← exp(Δ·a_s)·h_s + Δ·x·B_s;
//   y = (Σ_s C_s·h_s + skip·x)·silu(gate),
// for every channel (a row of a) with S states.
//
// Per (token, channel, state): one 2^x and four fp32 multiply-adds.  A group
// of G = S/K lanes owns two neighbouring channels, K states of each per lane
// (in registers over the whole prompt, packed in pairs).  Tokens go in
// batches of G: each lane of a group loads and prepares one token's Δ and
// Δ·x, the group shares them through shared memory, and the G partial
// readouts are summed so that lane i ends with token i and writes it.
#include "block.cuh"
#include "internal.h"

namespace la {
namespace {

using namespace block;

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kTile = 32;   // tokens of B and C converted at a time

template <int S> struct Cfg {
  static constexpr int K = S <= 16 ? 4 : 8;        // states per lane and channel
  static constexpr int G = S / K;                  // lanes per channel pair, tokens per batch
  static constexpr int kPairs = 32 / G;            // channel pairs per warp
  static constexpr int kChannels = 2 * kPairs * kWarps;   // channels per CTA
};

template <typename T>
__device__ __forceinline__ float2 load2(const T* p) {
  if constexpr (sizeof(T) == 2) {
    const uint32_t r = __ldg(reinterpret_cast<const uint32_t*>(p));
    return make_float2(tc::bf16lo_to_f32(r), tc::bf16hi_to_f32(r));
  } else {
    return __ldg(reinterpret_cast<const float2*>(p));
  }
}

template <typename T>
__device__ __forceinline__ void store2(T* p, float a, float b) {
  if constexpr (sizeof(T) == 2)
    *reinterpret_cast<uint32_t*>(p) = tc::pack_bf16x2(a, b);
  else
    *reinterpret_cast<float2*>(p) = make_float2(a, b);
}

template <typename T, int S>
__global__ void __launch_bounds__(kThreads) scan_kernel(const ScanArgs a, int cblocks) {
  using C = Cfg<S>;
  constexpr int K = C::K, G = C::G;
  __shared__ float4 bt[kTile][S / 4], ct[kTile][S / 4];
  __shared__ float4 du[kWarps][32];
  const int64_t b = blockIdx.x / cblocks;
  const int cb = blockIdx.x % cblocks;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int lg = lane % G, pair = lane / G;
  const int D = (int)a.D, n = (int)a.n;
  const int cw = cb * C::kChannels + (warp * C::kPairs + pair) * 2;
  const bool on = cw < D;         // D is even: both channels or none
  const int c = on ? cw : 0;
  const int len = live_tokens(a.lengths, b, n);

  f32x2 A[2][K / 2], h[2][K / 2];
#pragma unroll
  for (int ch = 0; ch < 2; ++ch) {
    const int64_t at = (int64_t)(c + ch) * S + lg * K;
#pragma unroll
    for (int k = 0; k < K / 4; ++k) {
      const float4 v = *reinterpret_cast<const float4*>(a.a + at + 4 * k);
      A[ch][2 * k] = pack2(v.x * kLog2e, v.y * kLog2e);
      A[ch][2 * k + 1] = pack2(v.z * kLog2e, v.w * kLog2e);
      float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
      if (a.state_in) s = *reinterpret_cast<const float4*>(a.state_in + b * D * S + at + 4 * k);
      h[ch][2 * k] = pack2(s.x, s.y);
      h[ch][2 * k + 1] = pack2(s.z, s.w);
    }
  }
  float bias[2] = {0.f, 0.f}, skip[2] = {0.f, 0.f};
#pragma unroll
  for (int ch = 0; ch < 2; ++ch) {
    if (a.dt_bias) bias[ch] = a.dt_bias[c + ch];
    if (a.skip) skip[ch] = a.skip[c + ch];
  }
  const T* xp = static_cast<const T*>(a.x.data) + b * a.x.sb + c;
  const T* dp = static_cast<const T*>(a.dt.data) + b * a.dt.sb + c;
  const T* zp = a.gate.data ? static_cast<const T*>(a.gate.data) + b * a.gate.sb + c : nullptr;
  const T* bp = static_cast<const T*>(a.b.data) + b * a.b.sb;
  const T* cp = static_cast<const T*>(a.c.data) + b * a.c.sb;
  T* op = static_cast<T*>(a.out) + b * a.out_sb + c;

  for (int t0 = 0; t0 < len; t0 += kTile) {
    __syncthreads();
    for (int e = threadIdx.x; e < kTile * S / 2; e += kThreads) {
      const int t = e / (S / 2), s = (e % (S / 2)) * 2;
      float2 bv = make_float2(0.f, 0.f), cv = bv;
      if (t0 + t < len) {
        bv = load2(bp + (t0 + t) * a.b.sn + s);
        cv = load2(cp + (t0 + t) * a.c.sn + s);
      }
      reinterpret_cast<float2*>(&bt[t][0])[s / 2] = bv;
      reinterpret_cast<float2*>(&ct[t][0])[s / 2] = cv;
    }
    __syncthreads();
    const int tn = min(kTile, len - t0);
    for (int tb = 0; tb < tn; tb += G) {
      const int t = t0 + tb + lg;
      float2 x = make_float2(0.f, 0.f), dt = x;
      if (t < len) {
        x = load2(xp + t * a.x.sn);
        dt = load2(dp + t * a.dt.sn);
        dt.x += bias[0];
        dt.y += bias[1];
        if (a.softplus) {
          dt.x = softplus(dt.x);
          dt.y = softplus(dt.y);
        }
      }
      __syncwarp();
      du[warp][lane] = make_float4(dt.x, dt.y, dt.x * x.x, dt.y * x.y);
      __syncwarp();
      float y[2][G];
#pragma unroll
      for (int i = 0; i < G; ++i) {
        const float4 v = du[warp][pair * G + i];
        const f32x2 d2[2] = {pack2(v.x, v.x), pack2(v.y, v.y)};
        const f32x2 u2[2] = {pack2(v.z, v.z), pack2(v.w, v.w)};
        f32x2 acc[2] = {0ull, 0ull};
#pragma unroll
        for (int k = 0; k < K / 4; ++k) {
          const float4 B4 = bt[tb + i][lg * (K / 4) + k], C4 = ct[tb + i][lg * (K / 4) + k];
          const f32x2 B2[2] = {pack2(B4.x, B4.y), pack2(B4.z, B4.w)};
          const f32x2 C2[2] = {pack2(C4.x, C4.y), pack2(C4.z, C4.w)};
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int ch = 0; ch < 2; ++ch) {
              float e0, e1;
              unpack2(mul2(d2[ch], A[ch][2 * k + j]), e0, e1);
              const f32x2 dec = pack2(tc::ex2_f32(e0), tc::ex2_f32(e1));
              f32x2& hh = h[ch][2 * k + j];
              hh = fma2(dec, hh, mul2(u2[ch], B2[j]));
              acc[ch] = fma2(C2[j], hh, acc[ch]);
            }
        }
#pragma unroll
        for (int ch = 0; ch < 2; ++ch) {
          float lo, hi;
          unpack2(acc[ch], lo, hi);
          y[ch][i] = lo + hi;
        }
      }
      // lane i of the group keeps token i: halve the tokens per exchange
#pragma unroll
      for (int m = G / 2; m >= 1; m /= 2) {
        const bool up = (lg & m) != 0;
#pragma unroll
        for (int i = 0; i < m; ++i)
#pragma unroll
          for (int ch = 0; ch < 2; ++ch) {
            const float give = up ? y[ch][i] : y[ch][i + m];
            const float keep = up ? y[ch][i + m] : y[ch][i];
            y[ch][i] = keep + __shfl_xor_sync(0xffffffffu, give, m);
          }
      }
      if (on && t < len) {
        float o0 = fmaf(skip[0], x.x, y[0][0]), o1 = fmaf(skip[1], x.y, y[1][0]);
        if (zp) {
          const float2 z = load2(zp + t * a.gate.sn);
          o0 *= silu(z.x);
          o1 *= silu(z.y);
        }
        store2(op + t * a.out_sn, o0, o1);
      }
    }
  }
  // tokens past the length
  if (on)
    for (int t = len + lg; t < n; t += G) store2(op + t * a.out_sn, 0.f, 0.f);
  if (on && a.state_out) {
#pragma unroll
    for (int ch = 0; ch < 2; ++ch)
#pragma unroll
      for (int k = 0; k < K / 4; ++k) {
        float4 v;
        unpack2(h[ch][2 * k], v.x, v.y);
        unpack2(h[ch][2 * k + 1], v.z, v.w);
        *reinterpret_cast<float4*>(a.state_out + b * D * S + (int64_t)(c + ch) * S + lg * K +
                                   4 * k) = v;
      }
  }
}

// One token: a lane owns four states of a channel, S/4 lanes a channel.  The
// state's read and write are nearly all of the traffic (8 bytes per state
// element); a warp touches 512 contiguous bytes of it.
constexpr int kStepThreads = 256;

template <typename T, int S>
__global__ void __launch_bounds__(kStepThreads) step_kernel(const ScanArgs a) {
  constexpr int G = S / 4;
  const int64_t item = (int64_t)blockIdx.x * kStepThreads + threadIdx.x;
  const bool on = item < a.B * a.D * G;
  const int64_t it = on ? item : 0;
  const int q = (int)(it % G);
  const int64_t bc = it / G;
  const int c = (int)(bc % a.D);
  const int64_t b = bc / a.D;
  float* hp = a.state_out + bc * S + 4 * q;
  const float4 h = *reinterpret_cast<const float4*>(hp);
  const float4 A = *reinterpret_cast<const float4*>(a.a + (int64_t)c * S + 4 * q);
  const float x = to_f32(static_cast<const T*>(a.x.data)[b * a.x.sb + c]);
  float dt = to_f32(static_cast<const T*>(a.dt.data)[b * a.dt.sb + c]);
  const float2 B0 = load2(static_cast<const T*>(a.b.data) + b * a.b.sb + 4 * q);
  const float2 B1 = load2(static_cast<const T*>(a.b.data) + b * a.b.sb + 4 * q + 2);
  const float2 C0 = load2(static_cast<const T*>(a.c.data) + b * a.c.sb + 4 * q);
  const float2 C1 = load2(static_cast<const T*>(a.c.data) + b * a.c.sb + 4 * q + 2);
  float z = 0.f;
  if (a.gate.data) z = to_f32(static_cast<const T*>(a.gate.data)[b * a.gate.sb + c]);
  if (a.dt_bias) dt += a.dt_bias[c];
  if (a.softplus) dt = softplus(dt);
  const float u = dt * x, d2 = dt * kLog2e;
  float4 r;
  r.x = fmaf(tc::ex2_f32(d2 * A.x), h.x, u * B0.x);
  r.y = fmaf(tc::ex2_f32(d2 * A.y), h.y, u * B0.y);
  r.z = fmaf(tc::ex2_f32(d2 * A.z), h.z, u * B1.x);
  r.w = fmaf(tc::ex2_f32(d2 * A.w), h.w, u * B1.y);
  if (on) *reinterpret_cast<float4*>(hp) = r;
  float y = fmaf(r.x, C0.x, fmaf(r.y, C0.y, fmaf(r.z, C1.x, r.w * C1.y)));
#pragma unroll
  for (int m = G / 2; m >= 1; m /= 2) y += __shfl_xor_sync(0xffffffffu, y, m);
  if (on && q == 0) {
    if (a.skip) y = fmaf(a.skip[c], x, y);
    if (a.gate.data) y *= silu(z);
    static_cast<T*>(a.out)[b * a.out_sb + c] = from_f32<T>(y);
  }
}

template <typename T, int S>
cudaError_t launch_scan(const ScanArgs& a, cudaStream_t s) {
  const int64_t cblocks = (a.D + Cfg<S>::kChannels - 1) / Cfg<S>::kChannels;
  if (cblocks * a.B > INT32_MAX) return cudaErrorInvalidConfiguration;
  scan_kernel<T, S><<<(unsigned)(cblocks * a.B), kThreads, 0, s>>>(a, (int)cblocks);
  count_launches(1);
  return cudaGetLastError();
}

template <typename T, int S>
cudaError_t launch_step(const ScanArgs& a, cudaStream_t s) {
  const int64_t blocks = (a.B * a.D * (S / 4) + kStepThreads - 1) / kStepThreads;
  if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
  step_kernel<T, S><<<(unsigned)blocks, kStepThreads, 0, s>>>(a);
  count_launches(1);
  return cudaGetLastError();
}

template <typename T>
cudaError_t by_states(const ScanArgs& a, bool step, cudaStream_t s) {
  switch (a.S) {
    case 8: return step ? launch_step<T, 8>(a, s) : launch_scan<T, 8>(a, s);
    case 16: return step ? launch_step<T, 16>(a, s) : launch_scan<T, 16>(a, s);
    case 32: return step ? launch_step<T, 32>(a, s) : launch_scan<T, 32>(a, s);
    default: return step ? launch_step<T, 64>(a, s) : launch_scan<T, 64>(a, s);
  }
}

}  // namespace

cudaError_t selective_scan(const ScanArgs& a, cudaStream_t s) {
  return a.bf16 ? by_states<__nv_bfloat16>(a, false, s) : by_states<float>(a, false, s);
}

cudaError_t selective_step(const ScanArgs& a, cudaStream_t s) {
  return a.bf16 ? by_states<__nv_bfloat16>(a, true, s) : by_states<float>(a, true, s);
}

}  // namespace la
