// Device helpers of the state-space block's kernels: activations, vector
// loads of 16 bytes as fp32, packed fp32 pairs.
#pragma once

#include "common.cuh"
#include "internal.h"
#include "linattn.h"
#include "tc.cuh"

namespace la {
namespace block {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float rcp_f32(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// x/(1 + e^{−x}) with the hardware's 2^x and 1/x (2 and 1 ulp).  The exponent
// −log2(e)·x rounds by 2^-24 of itself, and log2(e) by a quarter of that, so the
// relative error grows below zero: (1.25·|x| + 9)·2^-24, 4e-6 measured at −80, against
// a rounding of 2^-24 (fp32) or 2^-8 (bf16) of the result.  Below −87.3, where the
// value is under 1.1e-36, the result is 0.
__device__ __forceinline__ float silu(float x) {
  return x * rcp_f32(1.f + tc::ex2_f32(-kLog2e * x));
}

// log(1 + e^x) = max(x, 0) + log1p(e), e = e^{−|x|} ∈ (0, 1].  With
// s = e/(2 + e) ≤ 1/3, log1p(e) = 2·atanh(s) = 2s·p(s²); p is fitted on
// [0, 1/9] (weighted least squares towards the least largest relative error,
// 8e-9 with fp32 coefficients).  Relative accuracy matters where x is far
// below zero (steps of 1e-3): log2(1 + e) would round 1 + e first.  In all
// (1.25·|x| + 12)·2^-24 relative, by the rounding of e's exponent as in silu.
constexpr float kAtanh1 = 0.3333315849304199f, kAtanh2 = 0.20012454688549042f,
                kAtanh3 = 0.13980302214622498f, kAtanh4 = 0.1408916711807251f;

__device__ __forceinline__ float softplus(float x) {
  const float e = tc::ex2_f32(-kLog2e * fabsf(x));
  const float s = e * rcp_f32(2.f + e);
  const float q = s * s;
  const float p = fmaf(fmaf(fmaf(fmaf(kAtanh4, q, kAtanh3), q, kAtanh2), q, kAtanh1), q, 1.f);
  return fmaf(2.f * s, p, fmaxf(x, 0.f));
}

// The activations of one value (gelu goes by pairs, below).
template <int ACT>
__device__ __forceinline__ float activate(float x) {
  static_assert(ACT != LA_ACT_GELU, "gelu2");
  if constexpr (ACT == LA_ACT_RELU) return x < 0.f ? 0.f : x;   // keeps NaN
  if constexpr (ACT == LA_ACT_SILU) return silu(x);
  if constexpr (ACT == LA_ACT_SOFTPLUS) return softplus(x);
  return x;
}

// Every kernel of these operators is launched with programmatic stream
// serialization: its CTAs may start while the kernel before it drains, and
// nothing of global memory is touched before entry() has returned, which waits
// until that kernel has completed with its memory visible.  The prologue of a
// short kernel (launch, barriers, TMEM) overlaps its predecessor's tail.
__device__ __forceinline__ void entry() {
  tc::grid_dependency_wait();
  tc::grid_dependents_launch();
}

template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), unsigned grid, unsigned block, size_t smem,
                   cudaStream_t s, unsigned cluster, A&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
  if (e == cudaSuccess)
    count_launches(1);
  else
    cudaGetLastError();   // the caller gets the status; nothing is left behind
  return e;
}

// Dynamic shared memory for a grid whose CTAs all fit on the GPU at once and stay to
// the end: at least `need`, and just so much that one more than an SM's share of
// them does not fit on it (228 KB per SM, 1 KB of them per CTA, in units of 128
// bytes).  Started in the predecessor's tail they would otherwise fill the SMs that
// have room first, and stay there.
constexpr size_t kSmemMax = 227 * 1024;   // of a CTA; even_smem stays below
inline size_t even_smem(size_t need, int64_t ctas, int num_sms) {
  const int64_t per = (ctas + num_sms - 1) / num_sms;
  const int64_t least = (228 * 1024 / (per + 1) - 1024 + 128) & ~(int64_t)127;
  return least > (int64_t)need ? (size_t)least : need;
}

// Elements of a 16-byte vector.
template <typename T> constexpr int kVec = 16 / (int)sizeof(T);

template <typename T>
__device__ __forceinline__ void unpack(const uint4& v, float (&f)[kVec<T>]) {
  const uint32_t r[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 2) {
      f[2 * i] = tc::bf16lo_to_f32(r[i]);
      f[2 * i + 1] = tc::bf16hi_to_f32(r[i]);
    } else {
      f[i] = __uint_as_float(r[i]);
    }
  }
}

template <typename T>
__device__ __forceinline__ uint4 pack(const float (&f)[kVec<T>]) {
  if constexpr (sizeof(T) == 2)
    return tc::pack8(f);
  else
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                      __float_as_uint(f[3]));
}

// 16 bytes from global to shared memory in the background; `bytes` 0 writes
// zeros and reads nothing.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes = 16) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits until at most N of this thread's groups are in flight.
template <int N> __device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Tokens of batch entry b that count: lengths[b] taken into [0, n].
__device__ __forceinline__ int live_tokens(const int32_t* lengths, int64_t b, int n) {
  if (!lengths) return n;
  const int l = lengths[b];
  return l < 0 ? 0 : (l > n ? n : l);
}

// Two fp32 values in one 64-bit register pair: one instruction for two
// lanes' worth of multiply-adds.
using f32x2 = unsigned long long;

__device__ __forceinline__ f32x2 pack2(float lo, float hi) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(f32x2 v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// silu of two values.
__device__ __forceinline__ f32x2 silu2(f32x2 x) {
  float e0, e1;
  unpack2(mul2(x, pack2(-kLog2e, -kLog2e)), e0, e1);
  unpack2(add2(pack2(tc::ex2_f32(e0), tc::ex2_f32(e1)), pack2(1.f, 1.f)), e0, e1);
  return mul2(x, pack2(rcp_f32(e0), rcp_f32(e1)));
}

// A 16-byte vector as pairs of fp32, and back.
template <typename T>
__device__ __forceinline__ void unpack_pairs(const uint4& v, f32x2 (&p)[kVec<T> / 2]) {
  float f[kVec<T>];
  unpack<T>(v, f);
#pragma unroll
  for (int i = 0; i < kVec<T> / 2; ++i) p[i] = pack2(f[2 * i], f[2 * i + 1]);
}
template <typename T>
__device__ __forceinline__ uint4 pack_pairs(const f32x2 (&p)[kVec<T> / 2]) {
  float f[kVec<T>];
#pragma unroll
  for (int i = 0; i < kVec<T> / 2; ++i) unpack2(p[i], f[2 * i], f[2 * i + 1]);
  return pack<T>(f);
}

// softplus of two values.
__device__ __forceinline__ float2 softplus2(float2 x) {
  const float e0 = tc::ex2_f32(-kLog2e * fabsf(x.x)), e1 = tc::ex2_f32(-kLog2e * fabsf(x.y));
  const f32x2 s = mul2(pack2(e0, e1), pack2(rcp_f32(2.f + e0), rcp_f32(2.f + e1)));
  const f32x2 q = mul2(s, s);
  f32x2 p = fma2(pack2(kAtanh4, kAtanh4), q, pack2(kAtanh3, kAtanh3));
  p = fma2(p, q, pack2(kAtanh2, kAtanh2));
  p = fma2(p, q, pack2(kAtanh1, kAtanh1));
  p = fma2(p, q, pack2(1.f, 1.f));
  p = fma2(mul2(s, pack2(2.f, 2.f)), p, pack2(fmaxf(x.x, 0.f), fmaxf(x.y, 0.f)));
  float2 r;
  unpack2(p, r.x, r.y);
  return r;
}

// x·Φ(x) of two values.  Φ(−u) = e^{−u²/2}·t·P(t) for u = |x|, t = 1/(1 + 11u/32):
// e^{u²/2}·Φ(−u) falls like 1/u, so that P is smooth; it is fitted on [0, 14]
// (weighted least squares towards the least largest relative error, 6e-8 with
// fp32 coefficients).  1 + erf(x/√2) would cancel below zero: 1e-3 of the value
// at −4, all of it at −6.  Within (1.5·x² + 20)·2^-24 of the value for x < 0 (the
// rounding of u²/2 in the exponent), 20·2^-24 above.  16384×2048×8192 bf16
// takes 341 µs so, 415 with erfc, 369 with 1 + erf; 777×128×4096 9.1, 14.5 and 10.5.
__device__ __forceinline__ float2 gelu2(float2 x) {
  auto both = [](float c) { return pack2(c, c); };
  const f32x2 u = pack2(fabsf(x.x), fabsf(x.y));
  float a0, a1;
  unpack2(fma2(u, both(0.34375f), both(1.f)), a0, a1);
  const f32x2 t = pack2(rcp_f32(a0), rcp_f32(a1));
  f32x2 p = fma2(both(-0.027809331193566322f), t, both(0.14384913444519043f));
  p = fma2(p, t, both(-0.2717140316963196f));
  p = fma2(p, t, both(0.19092102348804474f));
  p = fma2(p, t, both(-0.03930721431970596f));
  p = fma2(p, t, both(0.11265801638364792f));
  p = fma2(p, t, both(0.11674045026302338f));
  p = fma2(p, t, both(0.13754227757453918f));
  p = fma2(p, t, both(0.13711966574192047f));
  unpack2(mul2(mul2(u, u), both(-0.5f * kLog2e)), a0, a1);
  const f32x2 q = mul2(mul2(pack2(tc::ex2_f32(a0), tc::ex2_f32(a1)), t), p);   // Φ(−u)
  const f32x2 h = fma2(q, both(-1.f), both(1.f));
  float q0, q1, h0, h1;
  unpack2(q, q0, q1);
  unpack2(h, h0, h1);
  return make_float2(x.x * (x.x < 0.f ? q0 : h0), x.y * (x.y < 0.f ? q1 : h1));
}

}  // namespace block
}  // namespace la
