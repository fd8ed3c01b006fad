// out = act(x·wᵀ + bias) + residual: choice of kernel, and the fp32 kernels on
// the CUDA cores.  TF32 tensor products keep 11 bits of an operand; fp32 inputs
// are held to fp32's rounding here, as in the attention kernels.
//
// tile_kernel: a CTA computes 64×128 outputs, K in steps of 16 through two
// shared-memory buffers, 8×8 outputs per thread in packed pairs: 32 packed
// multiply-adds against 4 shared loads of 16 bytes per step of K, which keeps
// the fp32 pipe and the shared-memory pipe equally busy.  Where that leaves SMs
// idle, 32×64 outputs, 4×4 per thread.
// Where tiles are few, 2 or 4 groups of threads of a CTA take K's steps in
// turn and add their sums in order at the end: one group is one warp per
// scheduler, which cannot hide its own latencies.
//
// row_kernel (few tokens, or too few tiles to fill the GPU): a CTA computes
// four output features for up to eight tokens, its lanes split K, so that w is
// read once per eight tokens in 512-byte pieces; bound by reading w for eight
// tokens, by the loads of x for more.
//
// Measured: 777×128×4096 with bias and softplus in 22.9 µs = 36 TFLOP/s (three
// tiles per SM; fp32 pipe 30 %, shared-memory pipe 46 %, issue 44 %);
// 1×2048×4096 in 7.1 µs = 4.7 TB/s (in a CUDA graph).
#include "block.cuh"
#include "internal.h"

#include <atomic>

namespace la {
namespace {

using namespace block;

// Four neighbouring columns' bias (zeros without one; adding them changes nothing).
__device__ __forceinline__ float4 bias4(const LinearArgs& a, int64_t n) {
  return a.bias ? __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(a.bias) + n))
                : make_float4(0.f, 0.f, 0.f, 0.f);
}

// bias, activation and residual on four neighbouring columns, and the store.
template <int ACT>
__device__ __forceinline__ void finish4(const LinearArgs& a, int64_t m, int64_t n, const float4& b,
                                        float (&v)[4]) {
  v[0] += b.x, v[1] += b.y, v[2] += b.z, v[3] += b.w;
  if constexpr (ACT == LA_ACT_SOFTPLUS) {
    const float2 lo = softplus2(make_float2(v[0], v[1])), hi = softplus2(make_float2(v[2], v[3]));
    v[0] = lo.x, v[1] = lo.y, v[2] = hi.x, v[3] = hi.y;
  } else if constexpr (ACT == LA_ACT_GELU) {
    const float2 lo = gelu2(make_float2(v[0], v[1])), hi = gelu2(make_float2(v[2], v[3]));
    v[0] = lo.x, v[1] = lo.y, v[2] = hi.x, v[3] = hi.y;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = activate<ACT>(v[i]);
  }
  if (a.residual.data) {
    const float4 r = *reinterpret_cast<const float4*>(static_cast<const float*>(a.residual.data) +
                                                      m * a.residual.sn + n);
    v[0] += r.x, v[1] += r.y, v[2] += r.z, v[3] += r.w;
  }
  *reinterpret_cast<float4*>(static_cast<float*>(a.out) + m * a.out_sn + n) =
      make_float4(v[0], v[1], v[2], v[3]);
}

constexpr int kBK = 16, kTileThreads = 128;

// T×T outputs per thread (8 or 4).
template <int T> struct Tile {
  static constexpr int kBM = 8 * T, kBN = 16 * T;
  static constexpr int kXF = kBK * kBM, kWF = kBK * kBN;   // floats of a buffer
};

// Column `col` of row k of a buffer.  The four rows that a warp writes at once
// (k, k + 4, k + 8, k + 12) go to different banks; four neighbouring columns
// stay together for the 16-byte reads.
__device__ __forceinline__ int swizzled(int k, int col) { return col ^ ((k >> 2) << 3); }

template <int T, int GROUPS> constexpr int kTileSmem = GROUPS * 2 * (Tile<T>::kXF + Tile<T>::kWF) * 4;

template <int ACT, int T, int GROUPS>
__global__ void __launch_bounds__(GROUPS * kTileThreads) tile_kernel(const LinearArgs a, int mtiles) {
  extern __shared__ __align__(16) float tile_smem[];
  constexpr int kBM = Tile<T>::kBM, kBN = Tile<T>::kBN, kXF = Tile<T>::kXF, kWF = Tile<T>::kWF;
  constexpr int P = T / 2;                         // packed pairs per row of a thread
  static_assert((GROUPS - 1) * T * T * kTileThreads * 4 <= kTileSmem<T, GROUPS>, "room for the groups' sums");
  const int64_t m0 = (int64_t)(blockIdx.x % mtiles) * kBM, n0 = (int64_t)(blockIdx.x / mtiles) * kBN;
  const float* x = static_cast<const float*>(a.x.data);
  const float* w = static_cast<const float*>(a.w.data);
  const int group = threadIdx.x / kTileThreads, tid = threadIdx.x % kTileThreads;
  const int tx = tid % 16, ty = tid / 16;
  const int lr = tid / 4, lk = (tid % 4) * 4;      // loads: row lr (+ 32 i), four of K
  float* const mine = tile_smem + group * 2 * (kXF + kWF);
  float4 xr[T / 4], wr[T / 2];
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  auto load = [&](int64_t k) {
    const bool in = k + lk < a.K;
#pragma unroll
    for (int i = 0; i < T / 4; ++i) {
      const int64_t m = m0 + lr + 32 * i;
      xr[i] = in && m < a.M ? __ldg(reinterpret_cast<const float4*>(x + m * a.x.sn + k + lk)) : zero;
    }
#pragma unroll
    for (int i = 0; i < T / 2; ++i) {
      const int64_t n = n0 + lr + 32 * i;
      wr[i] = in && n < a.N ? __ldg(reinterpret_cast<const float4*>(w + n * a.w.sn + k + lk)) : zero;
    }
  };
  auto put = [&](int buf) {
    float* xs = mine + buf * (kXF + kWF);
    float* ws = xs + kXF;
#pragma unroll
    for (int i = 0; i < T / 4; ++i) {
      const float v[4] = {xr[i].x, xr[i].y, xr[i].z, xr[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) xs[(lk + j) * kBM + swizzled(lk, lr + 32 * i)] = v[j];
    }
#pragma unroll
    for (int i = 0; i < T / 2; ++i) {
      const float v[4] = {wr[i].x, wr[i].y, wr[i].z, wr[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) ws[(lk + j) * kBN + swizzled(lk, lr + 32 * i)] = v[j];
    }
  };
  entry();
  f32x2 acc[T][P];
#pragma unroll
  for (int i = 0; i < T; ++i)
#pragma unroll
    for (int j = 0; j < P; ++j) acc[i][j] = 0ull;
  load((int64_t)group * kBK);
  put(0);
  __syncthreads();
  int buf = 0;
  // every group makes the same number of steps; those past K add zeros
  for (int64_t k0 = 0; k0 < a.K; k0 += GROUPS * kBK, buf ^= 1) {
    const bool more = k0 + GROUPS * kBK < a.K;
    if (more) load(k0 + (GROUPS + group) * kBK);
    const float* xs = mine + buf * (kXF + kWF);
    const float* ws = xs + kXF;
#pragma unroll
    for (int k = 0; k < kBK; ++k) {
      float xv[T];
      f32x2 wv[P];
#pragma unroll
      for (int i = 0; i < T / 4; ++i) {
        const float4 v = *reinterpret_cast<const float4*>(xs + k * kBM + 32 * i + swizzled(k, ty * 4));
        xv[4 * i] = v.x, xv[4 * i + 1] = v.y, xv[4 * i + 2] = v.z, xv[4 * i + 3] = v.w;
      }
#pragma unroll
      for (int i = 0; i < T / 4; ++i) {
        const ulonglong2 u = *reinterpret_cast<const ulonglong2*>(ws + k * kBN + 64 * i + swizzled(k, tx * 4));
        wv[2 * i] = u.x, wv[2 * i + 1] = u.y;
      }
#pragma unroll
      for (int i = 0; i < T; ++i) {
        const f32x2 d = pack2(xv[i], xv[i]);
#pragma unroll
        for (int j = 0; j < P; ++j) acc[i][j] = fma2(d, wv[j], acc[i][j]);
      }
    }
    if (more) put(buf ^ 1);
    __syncthreads();
  }
  if constexpr (GROUPS > 1) {
    // the buffers are done with: the later groups' sums, one row per pair
    f32x2* sums = reinterpret_cast<f32x2*>(tile_smem);
    if (group > 0) {
#pragma unroll
      for (int i = 0; i < T * P; ++i)
        sums[((group - 1) * T * P + i) * kTileThreads + tid] = acc[i / P][i % P];
    }
    __syncthreads();
    if (group > 0) return;
#pragma unroll
    for (int g = 0; g < GROUPS - 1; ++g)
#pragma unroll
      for (int i = 0; i < T * P; ++i) {
        float s0, s1, t0, t1;
        unpack2(acc[i / P][i % P], s0, s1);
        unpack2(sums[(g * T * P + i) * kTileThreads + tid], t0, t1);
        acc[i / P][i % P] = pack2(s0 + t0, s1 + t1);
      }
  }
#pragma unroll
  for (int j = 0; j < T / 4; ++j) {
    const int64_t n = n0 + j * 64 + tx * 4;   // N is a multiple of 4
    if (n >= a.N) continue;
    const float4 b = bias4(a, n);
#pragma unroll
    for (int i = 0; i < T; ++i) {
      const int64_t m = m0 + (i / 4) * 32 + ty * 4 + i % 4;
      if (m >= a.M) continue;
      float v[4];
      unpack2(acc[i][2 * j], v[0], v[1]);
      unpack2(acc[i][2 * j + 1], v[2], v[3]);
      finish4<ACT>(a, m, n, b, v);
    }
  }
}

constexpr int kRowWarps = 4, kRowFeatures = 4;

template <int ACT, int R>
__global__ void __launch_bounds__(32 * kRowWarps) row_kernel(const LinearArgs a, int fblocks) {
  __shared__ float sums[kRowWarps][R][kRowFeatures];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int64_t n = (int64_t)(blockIdx.x % fblocks) * kRowFeatures;   // N is a multiple of 4
  const int64_t m0 = (int64_t)(blockIdx.x / fblocks) * R;
  entry();
  const float* x = static_cast<const float*>(a.x.data);
  const float* w = static_cast<const float*>(a.w.data) + n * a.w.sn;
  float acc[R][kRowFeatures] = {};
#pragma unroll 2
  for (int64_t k = (warp * 32 + lane) * 4; k < a.K; k += 128 * kRowWarps) {
    float4 wv[kRowFeatures];
#pragma unroll
    for (int j = 0; j < kRowFeatures; ++j)
      wv[j] = __ldg(reinterpret_cast<const float4*>(w + j * a.w.sn + k));
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t m = m0 + r < a.M ? m0 + r : a.M - 1;
      const float4 xv = __ldg(reinterpret_cast<const float4*>(x + m * a.x.sn + k));
#pragma unroll
      for (int j = 0; j < kRowFeatures; ++j) {
        acc[r][j] = fmaf(xv.x, wv[j].x, acc[r][j]);
        acc[r][j] = fmaf(xv.y, wv[j].y, acc[r][j]);
        acc[r][j] = fmaf(xv.z, wv[j].z, acc[r][j]);
        acc[r][j] = fmaf(xv.w, wv[j].w, acc[r][j]);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int j = 0; j < kRowFeatures; ++j) {
#pragma unroll
      for (int s = 16; s >= 1; s /= 2) acc[r][j] += __shfl_xor_sync(0xffffffffu, acc[r][j], s);
      if (lane == r * kRowFeatures + j) sums[warp][r][j] = acc[r][j];
    }
  __syncthreads();
  const int64_t m = m0 + threadIdx.x;
  if (threadIdx.x >= R || m >= a.M) return;
  float v[4] = {};
#pragma unroll
  for (int i = 0; i < kRowWarps; ++i)
#pragma unroll
    for (int j = 0; j < kRowFeatures; ++j) v[j] += sums[i][threadIdx.x][j];
  finish4<ACT>(a, m, n, bias4(a, n), v);
}

template <int ACT, int R>
cudaError_t launch_rows(const LinearArgs& a, cudaStream_t s) {
  const int64_t fb = (a.N + kRowFeatures - 1) / kRowFeatures;
  const int64_t blocks = fb * ((a.M + R - 1) / R);
  if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
  return launch(row_kernel<ACT, R>, (unsigned)blocks, 32 * kRowWarps, 0, s, 1, a, (int)fb);
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Tiles of T that follow one another on an SM.
template <int T> int64_t tile_rounds(const LinearArgs& a) {
  return ceil_div(ceil_div(a.M, Tile<T>::kBM) * ceil_div(a.N, Tile<T>::kBN), a.num_sms);
}

// An even share of the tiles per SM: in the tail of a convolution or a product two
// of a single round's tiles would share an SM (256×1024×1024: 40 µs, 29 so;
// 200×512×1024: 21 and 15; with more tiles, 1000×1024×1024, no difference).
template <int ACT, int T, int GROUPS>
cudaError_t launch_groups(const LinearArgs& a, int64_t mt, int64_t nt, cudaStream_t s) {
  constexpr int need = kTileSmem<T, GROUPS>;
  static std::atomic<uint64_t> smem_set{0};
  const cudaError_t e = allow_smem((const void*)tile_kernel<ACT, T, GROUPS>, kSmemMax, &smem_set);
  if (e != cudaSuccess) return e;
  return launch(tile_kernel<ACT, T, GROUPS>, (unsigned)(mt * nt), GROUPS * kTileThreads,
                even_smem(need, mt * nt, a.num_sms), s, 1, a, (int)mt);
}

template <int ACT, int T, int GROUPS>
cudaError_t launch_tiles(const LinearArgs& a, cudaStream_t s) {
  const int64_t mt = ceil_div(a.M, Tile<T>::kBM), nt = ceil_div(a.N, Tile<T>::kBN);
  if (mt * nt > INT32_MAX) return cudaErrorInvalidConfiguration;
  return launch_groups<ACT, T, GROUPS>(a, mt, nt, s);
}

// SM cycles: rows at kRowRate multiply-adds per SM and cycle, for at least the
// kRowK elements of K that a CTA's lanes take at once; tiles at what one
// measured per element of K, times those that follow one another on an SM.
// Either side of the borders, in a CUDA graph: 64×2048×2048 43 µs by rows, 56 by
// small tiles; 200×512×1024 29 by rows, 12 by small tiles; 777×128×4096 21 by
// large tiles; 24×80×4096 4 by small tiles, 13 by rows.
constexpr double kRowRate = 18, kTile8 = 100, kTile4 = 48;
constexpr int64_t kRowK = 128 * kRowWarps;

// The kernel for a product: row_kernel<2> or <8>, or tiles of 8×8 or 4×4 outputs per
// thread with 1, 2 or 4 groups.
enum Choice { kRows2, kRows8, kTile8x1, kTile8x2, kTile8x4, kTile4x1, kTile4x2, kTile4x4 };

// groups until an SM has about twelve warps, as long as each has steps to take
template <int T> int tile_groups(const LinearArgs& a) {
  const int64_t rounds = tile_rounds<T>(a);
  return rounds == 1 && a.K >= 8 * kBK ? 4 : (rounds <= 2 && a.K >= 4 * kBK ? 2 : 1);
}

Choice choose(const LinearArgs& a) {
  if (a.M <= 2) return kRows2;
  const double rows = (double)a.M * a.N / a.num_sms / kRowRate * (a.K > kRowK ? a.K : kRowK);
  const double large = tile_rounds<8>(a) * kTile8 * a.K, small = tile_rounds<4>(a) * kTile4 * a.K;
  if ((a.M <= 8 && a.K >= kRowK) || (rows < large && rows < small)) return kRows8;
  const int g = small < large ? tile_groups<4>(a) : tile_groups<8>(a);
  const Choice first = small < large ? kTile4x1 : kTile8x1;
  return (Choice)(first + (g == 4 ? 2 : g - 1));
}

template <int ACT>
cudaError_t launch_f32(const LinearArgs& a, cudaStream_t s) {
  switch (choose(a)) {
    case kRows2: return launch_rows<ACT, 2>(a, s);
    case kRows8: return launch_rows<ACT, 8>(a, s);
    case kTile8x1: return launch_tiles<ACT, 8, 1>(a, s);
    case kTile8x2: return launch_tiles<ACT, 8, 2>(a, s);
    case kTile8x4: return launch_tiles<ACT, 8, 4>(a, s);
    case kTile4x1: return launch_tiles<ACT, 4, 1>(a, s);
    case kTile4x2: return launch_tiles<ACT, 4, 2>(a, s);
    default: return launch_tiles<ACT, 4, 4>(a, s);
  }
}

cudaError_t f32_linear(const LinearArgs& a, cudaStream_t s) {
  switch (a.act) {
    case LA_ACT_RELU: return launch_f32<LA_ACT_RELU>(a, s);
    case LA_ACT_SILU: return launch_f32<LA_ACT_SILU>(a, s);
    case LA_ACT_GELU: return launch_f32<LA_ACT_GELU>(a, s);
    case LA_ACT_SOFTPLUS: return launch_f32<LA_ACT_SOFTPLUS>(a, s);
    default: return launch_f32<LA_ACT_NONE>(a, s);
  }
}

}  // namespace

const char* linear_kernel(const LinearArgs& a) {
  static const char* const names[] = {"rows2", "rows8", "tile8x1", "tile8x2", "tile8x4", "tile4x1",
                                      "tile4x2", "tile4x4"};
  return a.bf16 ? tc_linear_kernel(a) : names[choose(a)];
}

cudaError_t linear(const LinearArgs& a, cudaStream_t s) {
  return a.bf16 ? tc_linear(a, s) : f32_linear(a, s);
}

}  // namespace la
