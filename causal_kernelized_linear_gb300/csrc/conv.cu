// The short depthwise causal convolution of a state-space block:
//   out_t,c = act(bias_c + Σ_{j<W} w_c,j · X_{t+j,c}),  X = [state | x],
// over a prompt, and for one token with the state shifted in place.
//
// W multiply-adds per value against 2 values moved: bound by HBM; the
// instructions take 47 % of the issue slots (73 % before the channels were
// handled in pairs).  A thread owns the channels of one 16-byte vector and
// walks a run of tokens with the last W − 1 inputs in registers, so every input
// is read once per run (plus W − 1 rows where runs meet, which the neighbouring
// run has just read into L2) and written once; a warp's accesses are 512
// contiguous bytes.  Rows arrive through a ring in shared memory (cp.async),
// sixteen ahead of the one in use: held in registers they cost the occupancy
// that hides HBM (115 µs against 100 µs for 4×8192×4096 bf16).
//
// Measured: 4×8192×4096 bf16, four taps, silu: 87 µs = 6.2 TB/s, 0.92 of the
// copy bandwidth; 3×1501×1000 fp32 with lengths: 6.5 µs.  The step is a
// launch: 256×4096 in 4.9 µs with the call.
#include "block.cuh"
#include "internal.h"

namespace la {
namespace {

using namespace block;

constexpr int kThreads = 128;
// Runs are halved from 64 tokens down to 16 until an SM has this many threads.
// 4×8192×4096 (enough at 64): 87 µs at 64, 95 at 32, 89 at 128.  3×1501×1000
// fp32: 6.5 µs at 16, 7.8 at 32, 9.4 at 64.
constexpr int kThreadsWanted = 512;
constexpr int kGroup = 4;  // tokens per step of its ring
constexpr int kRing = 20;  // rows of the ring (12 cost 4 µs at 4×8192×4096)

// A thread's channels, run and batch entry.
struct Item {
  uint32_t vec, run;
  int64_t b;
};
__device__ __forceinline__ Item item_of(int64_t item, uint32_t vecs, uint32_t runs, int64_t B) {
  if ((int64_t)vecs * runs * B <= UINT32_MAX) {   // 32-bit divisions
    uint32_t i = (uint32_t)item;
    const uint32_t v = i % vecs;
    i /= vecs;
    return Item{v, i % runs, (int64_t)(i / runs)};
  }
  return Item{(uint32_t)(item % vecs), (uint32_t)(item / vecs % runs), item / vecs / runs};
}

// A thread's weights and bias: its channels in pairs.
template <typename T, int W>
__device__ __forceinline__ void load_taps(const ConvArgs& a, int64_t c, f32x2 (&w)[W][kVec<T> / 2],
                                          f32x2 (&bias)[kVec<T> / 2]) {
  constexpr int V = kVec<T>;
  const T* wp = static_cast<const T*>(a.weight) + c * W;   // V·W consecutive values
  float f[W * V];
#pragma unroll
  for (int v = 0; v < W; ++v) {
    float g[V];
    unpack<T>(reinterpret_cast<const uint4*>(wp)[v], g);
#pragma unroll
    for (int i = 0; i < V; ++i) f[v * V + i] = g[i];
  }
#pragma unroll
  for (int j = 0; j < W; ++j)
#pragma unroll
    for (int i = 0; i < V / 2; ++i) w[j][i] = pack2(f[2 * i * W + j], f[(2 * i + 1) * W + j]);
#pragma unroll
  for (int i = 0; i < V / 2; ++i) bias[i] = 0ull;
  if (a.bias)
    unpack_pairs<T>(*reinterpret_cast<const uint4*>(static_cast<const T*>(a.bias) + c), bias);
}

// Row r of X of batch entry b, r counted from the prompt's first token.
template <typename T, int W>
__device__ __forceinline__ uint4 row_of(const ConvArgs& a, int64_t b, int64_t r, int64_t c) {
  if (r >= 0)
    return __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(a.x.data) + b * a.x.sb +
                                                r * a.x.sn + c));
  if (!a.state_in) return make_uint4(0, 0, 0, 0);
  return *reinterpret_cast<const uint4*>(static_cast<const T*>(a.state_in) +
                                         (b * (W - 1) + (W - 1) + r) * a.D + c);
}

template <typename T, int W, bool SILU>
__device__ __forceinline__ uint4 taps(const f32x2 (&win)[W][kVec<T> / 2],
                                      const f32x2 (&w)[W][kVec<T> / 2],
                                      const f32x2 (&bias)[kVec<T> / 2]) {
  constexpr int P = kVec<T> / 2;
  f32x2 y[P];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    y[i] = bias[i];
#pragma unroll
    for (int j = 0; j < W; ++j) y[i] = fma2(w[j][i], win[j][i], y[i]);
    if constexpr (SILU) y[i] = silu2(y[i]);
  }
  return pack_pairs<T>(y);
}

// The window moves on by one token.
template <int W, int P>
__device__ __forceinline__ void shift(f32x2 (&win)[W][P]) {
#pragma unroll
  for (int j = 0; j < W - 1; ++j)
#pragma unroll
    for (int i = 0; i < P; ++i) win[j][i] = win[j + 1][i];
}

template <typename T, int W, bool SILU>
__global__ void __launch_bounds__(kThreads) conv_kernel(const ConvArgs a, uint32_t vecs,
                                                        uint32_t runs, int len_run) {
  constexpr int V = kVec<T>;
  __shared__ uint4 ring[kRing][kThreads];   // a thread reads only what it copied itself
  const int64_t item = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (item >= (int64_t)vecs * runs * a.B) return;
  entry();
  const Item at = item_of(item, vecs, runs, a.B);
  const int64_t c = (int64_t)at.vec * V, b = at.b;
  const int n = (int)a.n;
  const int len = live_tokens(a.lengths, b, n);
  const int t0 = (int)at.run * len_run;
  const int t1 = min(t0 + len_run, n), live = min(t1, len);
  const T* next = static_cast<const T*>(a.x.data) + b * a.x.sb + t0 * a.x.sn + c;   // row to copy
  const uint32_t mine = tc::smem_u32(&ring[0][threadIdx.x]);
  auto fetch = [&](int t, int slot) {   // kGroup rows from token t
    if (t + kGroup <= live) {
#pragma unroll
      for (int i = 0; i < kGroup; ++i, next += a.x.sn)
        cp_async16(mine + (slot + i) * kThreads * 16, next);
    } else {
#pragma unroll
      for (int i = 0; i < kGroup; ++i, next += a.x.sn)
        if (t + i < live) cp_async16(mine + (slot + i) * kThreads * 16, next);
    }
    cp_commit();
  };
#pragma unroll
  for (int g = 0; g < kRing / kGroup - 1; ++g) fetch(t0 + g * kGroup, g * kGroup);
  f32x2 w[W][V / 2], bias[V / 2], win[W][V / 2];
  load_taps<T, W>(a, c, w, bias);
#pragma unroll
  for (int j = 0; j < W - 1; ++j)
    unpack_pairs<T>(t0 < len ? row_of<T, W>(a, b, t0 - (W - 1) + j, c) : make_uint4(0, 0, 0, 0),
                    win[j]);
  T* out = static_cast<T*>(a.out) + b * a.out_sb + t0 * a.out_sn + c;
  int slot = 0;
  for (int t = t0; t < t1; t += kGroup) {
    fetch(t + kRing - kGroup, slot ? slot - kGroup : kRing - kGroup);
    cp_wait<kRing / kGroup - 1>();
    if (t + kGroup <= live) {
#pragma unroll
      for (int i = 0; i < kGroup; ++i, out += a.out_sn) {
        unpack_pairs<T>(ring[slot + i][threadIdx.x], win[W - 1]);
        *reinterpret_cast<uint4*>(out) = taps<T, W, SILU>(win, w, bias);
        shift(win);
      }
    } else {
      for (int i = 0; i < kGroup; ++i, out += a.out_sn) {
        uint4 y = make_uint4(0, 0, 0, 0);   // tokens past the length
        if (t + i < live) {
          unpack_pairs<T>(ring[slot + i][threadIdx.x], win[W - 1]);
          y = taps<T, W, SILU>(win, w, bias);
          shift(win);
        }
        if (t + i < t1) *reinterpret_cast<uint4*>(out) = y;
      }
    }
    slot = slot + kGroup == kRing ? 0 : slot + kGroup;
  }
  cp_wait<0>();
  if (at.run == 0 && a.state_out) {
    T* so = static_cast<T*>(a.state_out) + b * (W - 1) * a.D + c;
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
      *reinterpret_cast<uint4*>(so + j * a.D) = row_of<T, W>(a, b, (int64_t)len - (W - 1) + j, c);
  }
}

template <typename T, int W, bool SILU>
__global__ void __launch_bounds__(kThreads) conv_step_kernel(const ConvArgs a, uint32_t vecs) {
  constexpr int V = kVec<T>;
  const int64_t item = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (item >= vecs * a.B) return;
  entry();
  const Item at = item_of(item, vecs, 1, a.B);
  const int64_t c = (int64_t)at.vec * V, b = at.b;
  T* st = static_cast<T*>(a.state_out) + b * (W - 1) * a.D + c;
  uint4 raw[W];
#pragma unroll
  for (int j = 0; j < W - 1; ++j) raw[j] = *reinterpret_cast<const uint4*>(st + j * a.D);
  raw[W - 1] = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.x.data) + b * a.x.sb + c);
  f32x2 w[W][V / 2], bias[V / 2], win[W][V / 2];
  load_taps<T, W>(a, c, w, bias);
#pragma unroll
  for (int j = 0; j < W; ++j) unpack_pairs<T>(raw[j], win[j]);
#pragma unroll
  for (int j = 0; j < W - 1; ++j) *reinterpret_cast<uint4*>(st + j * a.D) = raw[j + 1];
  *reinterpret_cast<uint4*>(static_cast<T*>(a.out) + b * a.out_sb + c) =
      taps<T, W, SILU>(win, w, bias);
}

template <typename T, int W, bool SILU>
cudaError_t launch_conv(const ConvArgs& a, bool step, cudaStream_t s) {
  const uint32_t vecs = (uint32_t)(a.D / kVec<T>);
  // tokens a thread walks: as many as leave kThreadsWanted threads per SM
  int64_t run = step ? 1 : 64;
  while (run > 16 && vecs * a.B * ((a.n + run - 1) / run) < (int64_t)kThreadsWanted * a.num_sms) run /= 2;
  const uint32_t runs = step ? 1 : (uint32_t)((a.n + run - 1) / run);
  const int64_t blocks = ((int64_t)vecs * runs * a.B + kThreads - 1) / kThreads;
  if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
  return step ? launch(conv_step_kernel<T, W, SILU>, (unsigned)blocks, kThreads, 0, s, 1, a, vecs)
              : launch(conv_kernel<T, W, SILU>, (unsigned)blocks, kThreads, 0, s, 1, a, vecs, runs,
                       (int)run);
}

template <typename T, int W>
cudaError_t by_act(const ConvArgs& a, bool step, cudaStream_t s) {
  return a.silu ? launch_conv<T, W, true>(a, step, s) : launch_conv<T, W, false>(a, step, s);
}

template <typename T>
cudaError_t by_width(const ConvArgs& a, bool step, cudaStream_t s) {
  switch (a.W) {
    case 2: return by_act<T, 2>(a, step, s);
    case 3: return by_act<T, 3>(a, step, s);
    default: return by_act<T, 4>(a, step, s);
  }
}

}  // namespace

cudaError_t causal_conv(const ConvArgs& a, cudaStream_t s) {
  return a.bf16 ? by_width<__nv_bfloat16>(a, false, s) : by_width<float>(a, false, s);
}

cudaError_t causal_conv_step(const ConvArgs& a, cudaStream_t s) {
  return a.bf16 ? by_width<__nv_bfloat16>(a, true, s) : by_width<float>(a, true, s);
}

}  // namespace la
