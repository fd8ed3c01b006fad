// Root-mean-square norm of rows, in groups of neighbouring features:
//   h = x + residual,  y = h·rsqrt(mean_group h² + eps)·weight·silu(gate),
// out = y in x's type, or 8 bits e4m3 with s = max|y|/448 of the row.
//
// Bound by HBM: a row is read once and held in registers (up to eight vectors of
// 16 bytes per thread) between the sums, the row's maximum and the output.  A row
// has R threads, 32 where eight vectors each hold it, so that its sums are warp
// shuffles and a warp has 8 to 24 loads in flight.  16384×2048 bf16 with a residual, to
// e4m3: 39 µs = 6.0 TB/s, 0.9 of a copy's bandwidth; 8192×32 groups of 128 with a gate:
// 34.5 µs = 5.8 TB/s; 16 rows of 1000 are a launch.
//
// Sums over a group: shuffles within the lanes that hold it where they are 2^i
// neighbours, else over the whole row's threads (one group), else through shared
// memory, a warp to a group.  All orders are fixed.
#include "block.cuh"
#include "internal.h"

#include <algorithm>

namespace la {
namespace {

using namespace block;
using bf16 = __nv_bfloat16;

constexpr int kMaxVectors = 8;          // of a thread
constexpr int kMaxThreads = 1024, kMidThreads = 256;
constexpr int kWarpsPerCta = 4;         // rows of a CTA where a warp has one

struct NormParams {
  Rows x, residual, gate;
  void* out;
  void* sum;
  int64_t out_sn, sum_sn;
  float* scale;
  const void* weight;
  int64_t M;
  int vectors, group;                   // of a row; of a group (vectors)
  float inv_group, eps;
};

// How a group's sum is taken.
enum Sums { kLanes, kRow, kShared };
// What a row has: a warp, up to kMidThreads or up to kMaxThreads (whose registers hold
// fewer vectors each).
enum Width { kWarp, kMid, kBig };

__device__ __forceinline__ float max_nan(float a, float b) {   // NaN wins
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Two values to e4m3, rounded to nearest, beyond ±448 to that.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Over the row's threads: all of the CTA's, or a warp's.
template <bool WARP, typename F>
__device__ __forceinline__ float over_row(float v, float* part, F f) {
#pragma unroll
  for (int m = 16; m > 0; m /= 2) v = f(v, __shfl_xor_sync(0xffffffffu, v, m));
  if constexpr (!WARP) {
    const int warps = blockDim.x / 32;
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = v;
    __syncthreads();
    v = part[0];
    for (int i = 1; i < warps; ++i) v = f(v, part[i]);
  }
  return v;
}

template <typename T, int NV, int WIDTH, int SUMS, bool E4M3, bool GATE>
__global__ void __launch_bounds__(WIDTH == kWarp ? 32 * kWarpsPerCta : WIDTH == kMid ? kMidThreads : kMaxThreads)
norm_kernel(const NormParams p) {
  constexpr int V = kVec<T>;
  constexpr bool WARP = WIDTH == kWarp;
  extern __shared__ float sums[];       // kShared: a vector's sum, then a group's factor
  __shared__ float part[2][32];
  entry();
  const int64_t row = WARP ? (int64_t)blockIdx.x * kWarpsPerCta + threadIdx.x / 32 : blockIdx.x;
  if (WARP && row >= p.M) return;
  const int R = WARP ? 32 : blockDim.x, at = WARP ? threadIdx.x % 32 : threadIdx.x;

  const T* xp = static_cast<const T*>(p.x.data) + row * p.x.sn;
  const T* rp = p.residual.data ? static_cast<const T*>(p.residual.data) + row * p.residual.sn : nullptr;
  const T* gp = static_cast<const T*>(p.gate.data) + row * p.gate.sn;
  uint4 xr[NV], rr[NV], gr[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = i * R + at;
    const bool in = c < p.vectors;
    xr[i] = in ? *reinterpret_cast<const uint4*>(xp + c * V) : make_uint4(0, 0, 0, 0);
    if (rp) rr[i] = in ? *reinterpret_cast<const uint4*>(rp + c * V) : make_uint4(0, 0, 0, 0);
    // the gate is wanted after the sums, and under way before them
    if (GATE) gr[i] = in ? *reinterpret_cast<const uint4*>(gp + c * V) : make_uint4(0, 0, 0, 0);
  }
  float h[NV][V], sq[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    unpack<T>(xr[i], h[i]);
    if (rp) {
      float r[V];
      unpack<T>(rr[i], r);
#pragma unroll
      for (int j = 0; j < V; ++j) h[i][j] += r[j];
      const int c = i * R + at;
      if (p.sum && c < p.vectors)
        *reinterpret_cast<uint4*>(static_cast<T*>(p.sum) + row * p.sum_sn + c * V) = pack<T>(h[i]);
    }
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) s = fmaf(h[i][j], h[i][j], s);
    sq[i] = s;
  }

  // the group's factor of every vector, into sq
  if constexpr (SUMS == kLanes) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      for (int m = 1; m < p.group; m *= 2) sq[i] += __shfl_xor_sync(0xffffffffu, sq[i], m);
      sq[i] = rsqrtf(fmaf(sq[i], p.inv_group, p.eps));
    }
  } else if constexpr (SUMS == kRow) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) s += sq[i];
    s = over_row<WARP>(s, part[0], [](float a, float b) { return a + b; });
    s = rsqrtf(fmaf(s, p.inv_group, p.eps));
#pragma unroll
    for (int i = 0; i < NV; ++i) sq[i] = s;
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (i * R + at < p.vectors) sums[i * R + at] = sq[i];
    __syncthreads();
    const int groups = p.vectors / p.group, lane = threadIdx.x % 32;
    for (int g = threadIdx.x / 32; g < groups; g += blockDim.x / 32) {
      float s = 0.f;
      for (int j = lane; j < p.group; j += 32) s += sums[g * p.group + j];
#pragma unroll
      for (int m = 16; m > 0; m /= 2) s += __shfl_xor_sync(0xffffffffu, s, m);
      if (lane == 0) sums[p.vectors + g] = rsqrtf(fmaf(s, p.inv_group, p.eps));
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (i * R + at < p.vectors) sq[i] = sums[p.vectors + (i * R + at) / p.group];
  }

  float most = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = i * R + at;
    if (c >= p.vectors) continue;
#pragma unroll
    for (int j = 0; j < V; ++j) h[i][j] *= sq[i];
    if (p.weight) {
      float w[V];
      const int wc = SUMS == kRow ? c : c % p.group;
      unpack<T>(__ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(p.weight) + wc * V)), w);
#pragma unroll
      for (int j = 0; j < V; ++j) h[i][j] *= w[j];
    }
    if constexpr (GATE) {
      float g[V];
      unpack<T>(gr[i], g);
#pragma unroll
      for (int j = 0; j < V; ++j) h[i][j] *= silu(g[j]);
    }
    if constexpr (E4M3) {
#pragma unroll
      for (int j = 0; j < V; ++j) most = max_nan(most, fabsf(h[i][j]));
    } else {
      *reinterpret_cast<uint4*>(static_cast<T*>(p.out) + row * p.out_sn + c * V) = pack<T>(h[i]);
    }
  }
  if constexpr (E4M3) {
    most = over_row<WARP>(most, part[1], max_nan);
    // at least the smallest normal value, so that 1/s is finite
    const float s = most == 0.f ? 1.f : max_nan(most / 448.f, 1.17549435e-38f);
    const float r = 1.f / s;            // y·r is within 2^-23 of y/s
    if (at == 0) p.scale[row] = s;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = i * R + at;
      if (c >= p.vectors) continue;
      uint32_t o[V / 4];
#pragma unroll
      for (int j = 0; j < V / 4; ++j)
        o[j] = e4m3x2(h[i][4 * j] * r, h[i][4 * j + 1] * r) |
               e4m3x2(h[i][4 * j + 2] * r, h[i][4 * j + 3] * r) << 16;
      uint8_t* to = static_cast<uint8_t*>(p.out) + row * p.out_sn + c * V;
      if constexpr (V == 8)
        *reinterpret_cast<uint2*>(to) = make_uint2(o[0], o[1]);
      else
        *reinterpret_cast<uint32_t*>(to) = o[0];
    }
  }
}

template <typename T, int NV, int WIDTH, bool E4M3, bool GATE>
cudaError_t launch_norm(const NormParams& p, int threads, cudaStream_t s) {
  constexpr bool WARP = WIDTH == kWarp;
  const int64_t ctas = WARP ? (p.M + kWarpsPerCta - 1) / kWarpsPerCta : p.M;
  if (p.M > INT32_MAX) return cudaErrorInvalidConfiguration;
  const unsigned n = (unsigned)ctas, th = WARP ? 32 * kWarpsPerCta : threads;
  if (p.group == p.vectors) return launch(norm_kernel<T, NV, WIDTH, kRow, E4M3, GATE>, n, th, 0, s, 1, p);
  if (p.group <= 32 && (p.group & (p.group - 1)) == 0)
    return launch(norm_kernel<T, NV, WIDTH, kLanes, E4M3, GATE>, n, th, 0, s, 1, p);
  return launch(norm_kernel<T, NV, WARP ? kMid : WIDTH, kShared, E4M3, GATE>, (unsigned)p.M, threads,
                (p.vectors + p.vectors / p.group) * sizeof(float), s, 1, p);
}

template <typename T, bool E4M3, bool GATE>
cudaError_t by_width(const NormArgs& a, NormParams p, cudaStream_t s) {
  constexpr int V = kVec<T>;
  p.vectors = a.D / V;
  p.group = a.group / V;
  // threads of a row: a warp while eight vectors of each lane hold it (four with a
  // gate, whose vectors are held too)
  int threads = 32;
  const int most = GATE ? kMaxVectors / 2 : kMaxVectors;
  while (threads < kMaxThreads && p.vectors > most * threads) threads *= 2;
  const int nv = (p.vectors + threads - 1) / threads;
  if (nv > kMaxVectors) return cudaErrorInvalidConfiguration;
  if (threads == 32) {
    if (nv <= 2) return launch_norm<T, 2, kWarp, E4M3, GATE>(p, threads, s);
    if (nv <= 4) return launch_norm<T, 4, kWarp, E4M3, GATE>(p, threads, s);
    return launch_norm<T, 8, kWarp, E4M3, GATE>(p, threads, s);
  }
  if (threads <= kMidThreads) {
    if (nv <= 4) return launch_norm<T, 4, kMid, E4M3, GATE>(p, threads, s);
    return launch_norm<T, 8, kMid, E4M3, GATE>(p, threads, s);
  }
  if (nv <= 4) return launch_norm<T, 4, kBig, E4M3, GATE>(p, threads, s);
  return launch_norm<T, 8, kBig, E4M3, GATE>(p, threads, s);
}

template <typename T>
cudaError_t by_kind(const NormArgs& a, const NormParams& p, cudaStream_t s) {
  const bool gate = p.gate.data != nullptr;
  if (a.quantize) return gate ? by_width<T, true, true>(a, p, s) : by_width<T, true, false>(a, p, s);
  return gate ? by_width<T, false, true>(a, p, s) : by_width<T, false, false>(a, p, s);
}

}  // namespace

bool rms_norm_supported(int64_t D, bool is_bf16) {
  return D <= (int64_t)kMaxThreads * kMaxVectors * (is_bf16 ? 8 : 4);
}

cudaError_t rms_norm(const NormArgs& a, cudaStream_t s) {
  NormParams p{};
  p.x = a.x, p.residual = a.residual, p.gate = a.gate;
  p.out = a.out, p.out_sn = a.out_sn;
  p.sum = a.sum, p.sum_sn = a.sum_sn;
  p.scale = a.scale;
  p.weight = a.weight;
  p.M = a.M;
  p.inv_group = 1.f / (float)a.group;
  p.eps = a.eps;
  return a.bf16 ? by_kind<bf16>(a, p, s) : by_kind<float>(a, p, s);
}

}  // namespace la
