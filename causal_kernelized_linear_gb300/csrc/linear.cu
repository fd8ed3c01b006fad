// out = act(x·wᵀ + bias) + residual: choice of kernel, and the fp32 CUDA-core
// kernel (one thread block per 64×64 tile of the output, K in steps of 16
// through shared memory, 4×4 outputs per thread).
#include "block.cuh"
#include "internal.h"

namespace la {
namespace {

using namespace block;

constexpr int kTile = 64, kStep = 16, kThreads = 256;

template <typename T, int ACT>
__global__ void __launch_bounds__(kThreads) linear_simt_kernel(const LinearArgs a) {
  __shared__ float xs[kStep][kTile + 4], ws[kStep][kTile + 4];
  const int64_t m0 = (int64_t)blockIdx.y * kTile, n0 = (int64_t)blockIdx.x * kTile;
  const T* x = static_cast<const T*>(a.x.data);
  const T* w = static_cast<const T*>(a.w.data);
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  const int lr = threadIdx.x / 4, lk = (threadIdx.x % 4) * 4;   // one row, four of K
  float acc[4][4] = {};
  for (int64_t k0 = 0; k0 < a.K; k0 += kStep) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t k = k0 + lk + i;
      xs[lk + i][lr] = (k < a.K && m0 + lr < a.M) ? to_f32(x[(m0 + lr) * a.x.sn + k]) : 0.f;
      ws[lk + i][lr] = (k < a.K && n0 + lr < a.N) ? to_f32(w[(n0 + lr) * a.w.sn + k]) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kStep; ++k) {
      const float4 xv = *reinterpret_cast<const float4*>(&xs[k][ty * 4]);
      const float4 wv = *reinterpret_cast<const float4*>(&ws[k][tx * 4]);
      const float xr[4] = {xv.x, xv.y, xv.z, xv.w}, wr[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(xr[i], wr[j], acc[i][j]);
    }
    __syncthreads();
  }
  const T* bias = static_cast<const T*>(a.bias);
  const T* res = static_cast<const T*>(a.residual.data);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t m = m0 + ty * 4 + i;
    if (m >= a.M) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t n = n0 + tx * 4 + j;
      if (n >= a.N) continue;
      float y = acc[i][j];
      if (bias) y += to_f32(bias[n]);
      y = activate<ACT>(y);
      if (res) y += to_f32(res[m * a.residual.sn + n]);
      static_cast<T*>(a.out)[m * a.out_sn + n] = from_f32<T>(y);
    }
  }
}

template <typename T, int ACT>
cudaError_t launch_simt(const LinearArgs& a, cudaStream_t s) {
  const int64_t gx = (a.N + kTile - 1) / kTile, gy = (a.M + kTile - 1) / kTile;
  if (gx > INT32_MAX || gy > 65535) return cudaErrorInvalidConfiguration;
  linear_simt_kernel<T, ACT><<<dim3((unsigned)gx, (unsigned)gy), kThreads, 0, s>>>(a);
  count_launches(1);
  return cudaGetLastError();
}

template <typename T>
cudaError_t simt(const LinearArgs& a, cudaStream_t s) {
  switch (a.act) {
    case LA_ACT_RELU: return launch_simt<T, LA_ACT_RELU>(a, s);
    case LA_ACT_SILU: return launch_simt<T, LA_ACT_SILU>(a, s);
    case LA_ACT_GELU: return launch_simt<T, LA_ACT_GELU>(a, s);
    case LA_ACT_SOFTPLUS: return launch_simt<T, LA_ACT_SOFTPLUS>(a, s);
    default: return launch_simt<T, LA_ACT_NONE>(a, s);
  }
}

}  // namespace

cudaError_t linear(const LinearArgs& a, cudaStream_t s) {
  return a.bf16 ? tc_linear(a, s) : simt<float>(a, s);
}

}  // namespace la
