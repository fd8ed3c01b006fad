// out = act(x·wᵀ + bias) + residual in bf16 on the tcgen05 tensor cores.
//
// pair_kernel (many tokens): CTA pairs, persistent, one 256×BN tile of the
// output per pair at a time (BN 256, or 128 where that leaves fewer SMs idle).
// Each CTA loads its 128 rows of x and BN/2 rows of w per 64-wide step of K
// into a ring, the even rank issues the cta_group::2 MMAs (256×BN×16) for
// both, and each CTA's TMEM receives its 128 rows × BN columns in one of two
// accumulators, so that the epilogue of a tile overlaps the next tile's
// product.  A pair moves 64 KB per step into shared memory for 2·256·256·64
// flops; one CTA on a 128×256 tile would move 48 KB for half of them.
//
// few_kernel (few tokens): the product is bound by reading w, so w's rows are
// the MMA's 128 rows and the tokens its columns (16 to 128, no work on absent
// ones).  A cluster of CTAs splits K, and adds its partial sums through
// distributed shared memory in rank order: w is read once, by enough CTAs to
// keep HBM busy, in one launch, with a fixed order of sums.
//
// Measured: 16384×2048×8192 in 330 µs = 1.67 PFLOP/s, 0.86 of the measured
// burst rate and 0.95 of the sustained one (tensor pipe 78 % at 4096 tokens);
// 1777×4096×2048 with bias and residual in 27 µs (56 tiles of 256×256 for 76
// pairs); 16×2048×8192 in 8.4 to 8.7 µs = 4 TB/s.
#include "block.cuh"
#include "internal.h"
#include "tc_pair.cuh"

#include <algorithm>
#include <atomic>

namespace la {
namespace {

using namespace block;
using namespace tc;

using bf16 = __nv_bfloat16;

constexpr int kBK = 64;                 // K per stage: one 128-byte swizzle row

struct LinParams {
  const bf16* bias;
  const bf16* residual;
  int64_t res_sn;
  bf16* out;
  int64_t out_sn;
  int M, N, kblocks;
  int mtiles, ntiles;
  int* status;
};

// bias, activation and residual on 8 neighbouring columns of a row; either
// pointer is null where there is nothing to add.
template <int ACT>
__device__ __forceinline__ void finish8(const bf16* bias, const bf16* res, float (&v)[8]) {
  if (bias) {
    float b[8];
    unpack<bf16>(__ldg(reinterpret_cast<const uint4*>(bias)), b);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += b[i];
  }
  if constexpr (ACT == LA_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const float2 y = gelu2(make_float2(v[i], v[i + 1]));
      v[i] = y.x, v[i + 1] = y.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = activate<ACT>(v[i]);
  }
  if (res) {
    float r[8];
    unpack<bf16>(*reinterpret_cast<const uint4*>(res), r);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += r[i];
  }
}

// ------------------------------------------------------------------ many tokens

constexpr int kTileB = 128 * kBK * 2;               // 16 KB: 128 rows of one operand
constexpr int kEpiWarps = 8;                        // two per quarter of the rows
constexpr int kEpiB = 32 * 64 * 2;                  // 4 KB: 32 rows × 64 columns of the output
constexpr int kPairThreads = 128 + 32 * kEpiWarps;
constexpr int kGroupM = 8;                          // row tiles walked together, for L2

template <int BN> struct PairCfg {
  static constexpr int kW = BN / 2 * kBK * 2;       // a CTA's rows of w per step
  static constexpr int kStage = kTileB + kW;
  static constexpr int kNum = BN == 256 ? 6 : 8;
  static constexpr int kSmem = 1024 + kNum * kStage + kEpiWarps * kEpiB + 256;
  // Alone on its SM beside anything that uses tensor memory (few_kernel takes the
  // least, 18 KB), so it may hold its columns while it waits for its predecessor.
  static_assert(kSmem + 18 * 1024 > 228 * 1024, "tensor memory is not shared");
};

struct PairBars {
  uint64_t full[8], empty[8], acc_full[2], acc_empty[2], done;
  uint32_t tmem;
  int abort;
};

// Tile number → (row tile, column tile): columns fastest within groups of
// kGroupM row tiles, so that the tiles in flight share rows of x and of w.
__device__ __forceinline__ void tile_at(const LinParams& p, int64_t t, int& mt, int& nt) {
  const int64_t per = (int64_t)kGroupM * p.ntiles;
  const int g = (int)(t / per);
  const int r = (int)(t % per);
  const int rows = min(kGroupM, p.mtiles - g * kGroupM);
  mt = g * kGroupM + r % rows;
  nt = r / rows;
}

template <int BN, int ACT>
__global__ void __launch_bounds__(kPairThreads, 1)
pair_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mw,
            const __grid_constant__ CUtensorMap mo, const LinParams p) {
  using C = PairCfg<BN>;
  constexpr int kStages = C::kNum, kStageB = C::kStage;
  extern __shared__ uint8_t raw[];
  uint8_t* base = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  uint8_t* epi = base + kStages * kStageB;
  PairBars* bars = reinterpret_cast<PairBars*>(epi + kEpiWarps * kEpiB);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t rank = cluster_rank();
  const int64_t tiles = (int64_t)p.mtiles * p.ntiles;
  const int64_t first = blockIdx.x / 2, stride = gridDim.x / 2;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&bars->full[i], 1);
      mbar_init(&bars->empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->acc_full[i], 1);
      mbar_init(&bars->acc_empty[i], 2 * kEpiWarps);   // of both CTAs
    }
    mbar_init(&bars->done, 1);
    bars->abort = 0;
    fence_barrier_init();
    tma_prefetch_desc(&mx);
    tma_prefetch_desc(&mw);
    tma_prefetch_desc(&mo);
  }
  if (warp == 2) {
    tmem_alloc_pair(&bars->tmem, 2 * BN);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();          // both CTAs' barriers exist before any remote arrival
  tc_fence_after();
  entry();
  const uint32_t tmem = bars->tmem;
  volatile int* abort = &bars->abort;

  uint32_t issued = 0;     // steps that this CTA's producer has loaded
  if (warp == 0 && lane == 0) {
    // producer: this CTA's rows of x and w; completion is counted by the even rank
    uint32_t it = 0;
    for (int64_t t = first; t < tiles && !*abort; t += stride) {
      int mt, nt;
      tile_at(p, t, mt, nt);
      const int m0 = mt * 256 + (int)rank * 128, n0 = nt * BN + (int)rank * (BN / 2);
      for (int kb = 0; kb < p.kblocks; ++kb, ++it) {
        const int s = it % kStages;
        if (it >= kStages &&
            !mbar_wait(&bars->empty[s], ((it / kStages) & 1) ^ 1, p.status, abort))
          break;
        if (rank == 0) mbar_arrive_expect_tx(&bars->full[s], 2 * kStageB);
        const uint32_t bar = map_to_cta(smem_u32(&bars->full[s]), 0);
        tma_load_2d_pair(base + s * kStageB, &mx, bar, kb * kBK, m0);
        tma_load_2d_pair(base + s * kStageB + kTileB, &mw, bar, kb * kBK, n0);
      }
    }
    issued = it;
  } else if (warp == 1 && lane == 0 && rank == 0) {
    // MMA issuer, for both CTAs
    constexpr uint32_t idesc = idesc_bf16_f32(256, BN, false, false);
    uint32_t it = 0, n = 0;
    for (int64_t t = first; t < tiles && !*abort; t += stride, ++n) {
      const int buf = n & 1;
      if (n >= 2 && !mbar_wait(&bars->acc_empty[buf], ((n >> 1) & 1) ^ 1, p.status, abort)) break;
      tc_fence_after();
      const uint32_t d = tmem + buf * BN;
      bool ok = true;
      for (int kb = 0; kb < p.kblocks; ++kb, ++it) {
        const int s = it % kStages;
        if (!mbar_wait(&bars->full[s], (it / kStages) & 1, p.status, abort)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint64_t da = smem_desc(smem_u32(base + s * kStageB), 16, 1024, kSwizzle128B);
        const uint64_t db = smem_desc(smem_u32(base + s * kStageB + kTileB), 16, 1024, kSwizzle128B);
#pragma unroll
        for (int k = 0; k < kBK / 16; ++k)
          mma_ss_pair(d, desc_at(da, k * 32), desc_at(db, k * 32), idesc, (kb | k) != 0);
        mma_commit_pair(&bars->empty[s]);
      }
      if (!ok) break;
      mma_commit_pair(&bars->acc_full[buf]);
    }
  } else if (warp >= 4) {
    // epilogue: a warp has the rows of its TMEM quarter and half of the
    // columns, 64 at a time through a staging tile
    const int q = warp % 4, half = (warp - 4) / 4;
    uint8_t* st = epi + (warp - 4) * kEpiB;
    const uint32_t sa = smem_u32(st);
    const uint32_t lead_empty[2] = {map_to_cta(smem_u32(&bars->acc_empty[0]), 0),
                                    map_to_cta(smem_u32(&bars->acc_empty[1]), 0)};
    uint32_t n = 0;
    for (int64_t t = first; t < tiles; t += stride, ++n) {
      const int buf = n & 1;
      if (!warp_wait(&bars->acc_full[buf], (n >> 1) & 1, p.status, abort)) break;
      tc_fence_after();
      int mt, nt;
      tile_at(p, t, mt, nt);
      const int m0 = mt * 256 + (int)rank * 128 + q * 32, m = m0 + lane;
      const int c0 = half * (BN / 2), n0 = nt * BN + c0;
      const int cols = min(BN / 2, p.N - n0);
      if (m0 < p.M) {
        const bf16* res = p.residual && m < p.M ? p.residual + m * p.res_sn + n0 : nullptr;
        for (int c = 0; c < cols; c += 64) {
          uint32_t r[64];
          tmem_ld32(tmem_addr(tmem, q * 32, buf * BN + c0 + c), r);
          tmem_ld32(tmem_addr(tmem, q * 32, buf * BN + c0 + c + 32), r + 32);
          tmem_ld_wait();
          if (lane == 0) tma_store_wait_read0();
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[8 * j + i]);
            const bool in = c + 8 * j < cols;
            finish8<ACT>(p.bias && in ? p.bias + n0 + c + 8 * j : nullptr,
                         res && in ? res + c + 8 * j : nullptr, v);
            sts128(sa + sw_chunk(32, lane, 0, j), pack8(v));
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (LA_DCHECK(p.status, m0 >= 0 && m0 < p.M && n0 + c < p.N, 51))
              tma_store_2d(&mo, st, n0 + c, m0);
            tma_store_commit();
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(lead_empty[buf]);
    }
    if (lane == 0) tma_store_wait0();
  }
  tc_fence_before();
  __syncwarp();
  __syncthreads();
  // after an abort, products and loads in flight end before either CTA does
  if (threadIdx.x == 32 && rank == 0 && *abort) {
    mma_commit_pair(&bars->done, 1);
    mbar_wait_drain(&bars->done, 0);
  }
  if (threadIdx.x == 0 && rank == 0 && *abort)
    for (uint32_t j = issued > kStages ? issued - kStages : 0; j < issued; ++j)
      mbar_wait_drain(&bars->full[j % kStages], (j / kStages) & 1);
  cluster_sync();          // no CTA leaves while its pair may still signal or read it
  tc_fence_after();
  if (warp == 2) tmem_dealloc_pair(tmem, 2 * BN);
}

// ------------------------------------------------------------------ few tokens

constexpr int kFewThreads = 256;

template <int BT> struct FewCfg {
  static constexpr int kXB = BT * kBK * 2;
  static constexpr int kStage = kTileB + kXB;
  static constexpr int kNum = BT <= 32 ? 8 : 6;           // stages of a CTA alone on its SM
  // CTAs an SM should have (32×2048×8192: 10 µs with one, 12 with two;
  // 1×2048×8192: 9.0 with one, 8.6 with two)
  static constexpr int kPerSm = BT <= 16 ? 2 : 1;
  static constexpr int kShared = BT <= 32 ? 3 : 6;        // stages where they share it
  static constexpr int kPart = BT * 128 * 4;              // partial sums, over the stages
  static constexpr int buf(int stages) { return stages * kStage > kPart ? stages * kStage : kPart; }
  static constexpr int smem(int stages) { return 1024 + buf(stages) + 256; }
  static constexpr uint32_t kCols = BT < 32 ? 32 : BT;
};

struct FewBars {
  uint64_t full[8], empty[8], done;
  uint32_t tmem;
  int abort;
};

// Blocks: cluster rank fastest, then feature tile, then token tile.
template <int BT, int ACT>
__global__ void __launch_bounds__(kFewThreads)
few_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mw,
           const LinParams p, const int split, const int ftiles, const int stages) {
  using C = FewCfg<BT>;
  extern __shared__ uint8_t raw[];
  uint8_t* base = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  FewBars* bars = reinterpret_cast<FewBars*>(raw + C::smem(stages) - 256);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int rank = (int)(blockIdx.x % split);
  const int tile = (int)(blockIdx.x / split);
  const int n0 = tile % ftiles * 128, m0 = tile / ftiles * BT;
  const int k0 = (int)((int64_t)p.kblocks * rank / split);
  const int k1 = (int)((int64_t)p.kblocks * (rank + 1) / split);

  if (threadIdx.x == 0) {
    for (int i = 0; i < stages; ++i) {
      mbar_init(&bars->full[i], 1);
      mbar_init(&bars->empty[i], 1);
    }
    mbar_init(&bars->done, 1);
    bars->abort = 0;
    fence_barrier_init();
    tma_prefetch_desc(&mx);
    tma_prefetch_desc(&mw);
  }
  // Tensor memory is taken after the wait for the predecessor and given back
  // before the wait for the cluster: a CTA that holds some waits for nothing but
  // its own loads and products.  A kernel that needs all 512 columns of an SM may
  // be this one's predecessor or run beside it, so held across either wait they
  // could make both wait for each other.
  entry();
  const int steps = k1 - k0;
  auto load = [&](int it, int s) {
    mbar_arrive_expect_tx(&bars->full[s], C::kStage);
    tma_load_2d(base + s * C::kStage, &mw, &bars->full[s], (k0 + it) * kBK, n0);
    tma_load_2d(base + s * C::kStage + kTileB, &mx, &bars->full[s], (k0 + it) * kBK, m0);
  };
  if (threadIdx.x == 0)
    for (int it = 0; it < steps && it < stages; ++it) load(it, it);   // the ring's first lap
  if (warp == 2) {
    tmem_alloc(&bars->tmem, C::kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem;
  volatile int* abort = &bars->abort;

  int issued = 0;          // loads of this CTA (its producer)
  if (warp == 0 && lane == 0) {
    int s = 0, it = stages;
    uint32_t lap = 1;      // times the ring has been filled
    for (; it < steps; ++it) {
      if (!mbar_wait(&bars->empty[s], (lap & 1) ^ 1, p.status, abort)) break;
      load(it, s);
      if (++s == stages) s = 0, ++lap;
    }
    issued = it < steps ? it : steps;
  } else if (warp == 1 && lane == 0) {
    constexpr uint32_t idesc = idesc_bf16_f32(128, BT, false, false);
    int s = 0;
    uint32_t lap = 0;
    for (int it = 0; it < steps; ++it) {
      if (!mbar_wait(&bars->full[s], lap & 1, p.status, abort)) break;
      tc_fence_after();
      const uint64_t dw = smem_desc(smem_u32(base + s * C::kStage), 16, 1024, kSwizzle128B);
      const uint64_t dx = smem_desc(smem_u32(base + s * C::kStage + kTileB), 16, 1024, kSwizzle128B);
#pragma unroll
      for (int k = 0; k < kBK / 16; ++k)
        mma_ss(tmem, desc_at(dw, k * 32), desc_at(dx, k * 32), idesc, it > 0 || k > 0);
      mma_commit(&bars->empty[s]);
      if (++s == stages) s = 0, ++lap;
    }
    mma_commit(&bars->done);
  }
  __syncwarp();
  // every load has been consumed once `done` completes: the stages become the
  // partial sums [token][feature]
  const bool ok = warp_wait(&bars->done, 0, p.status, abort);
  tc_fence_after();
  float* part = reinterpret_cast<float*>(base);
  if (ok) {
#pragma unroll
    for (int c = warp / 4 * 16; c < BT; c += 32) {
      uint32_t r[16];
      tmem_ld16(tmem_addr(tmem, warp % 4 * 32, c), r);
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 16; ++i)
        part[(c + i) * 128 + warp % 4 * 32 + lane] = k0 < k1 ? __uint_as_float(r[i]) : 0.f;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (*abort) {
    // loads and products in flight end before the CTA does
    if (threadIdx.x == 0)
      for (int j = issued > stages ? issued - stages : 0; j < issued; ++j)
        mbar_wait_drain(&bars->full[j % stages], (j / stages) & 1);
    if (threadIdx.x == 32) mbar_wait_drain(&bars->done, 0);
    __syncthreads();
  }
  if (split > 1) cluster_arrive();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kCols);
  }
  if (split > 1) cluster_wait();
  // rank r finishes its share of the tokens: 16 lanes of 8 features per token
  const int per = (BT + split - 1) / split;
  const int tlim = min(min(BT, (rank + 1) * per), p.M - m0);
  const int f = (threadIdx.x % 16) * 8, n = n0 + f;
  if (!*abort && n < p.N) {
    for (int t = rank * per + threadIdx.x / 16; t < tlim; t += kFewThreads / 16) {
      const uint32_t at = smem_u32(part) + (t * 128 + f) * 4;
      float v[8] = {};
      for (int r0 = 0; r0 < split; r0 += 4) {   // four ranks' reads in flight
        float4 lo[4], hi[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (r0 + i < split) {
            const uint32_t pa = split > 1 ? map_to_cta(at, r0 + i) : at;
            lo[i] = split > 1 ? ld_cluster_f4(pa) : lds128f(pa);
            hi[i] = split > 1 ? ld_cluster_f4(pa + 16) : lds128f(pa + 16);
          }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (r0 + i < split) {
            v[0] += lo[i].x, v[1] += lo[i].y, v[2] += lo[i].z, v[3] += lo[i].w;
            v[4] += hi[i].x, v[5] += hi[i].y, v[6] += hi[i].z, v[7] += hi[i].w;
          }
      }
      const int64_t m = m0 + t;
      finish8<ACT>(p.bias ? p.bias + n : nullptr,
                   p.residual ? p.residual + m * p.res_sn + n : nullptr, v);
      if (LA_DCHECK(p.status, m < p.M && n + 8 <= p.N, 52))
        *reinterpret_cast<uint4*>(p.out + m * p.out_sn + n) = pack8(v);
    }
  }
  if (split > 1) cluster_sync();   // no CTA leaves while another reads its partial sums
}

// ------------------------------------------------------------------ launch

template <int BN, int ACT>
cudaError_t launch_pair(const LinearArgs& a, LinParams p, cudaStream_t s) {
  CUtensorMap mx, mw, mo;
  cudaError_t e;
  if ((e = tmap_view(&mx, a.x.data, a.M, a.K, a.x.sn ? a.x.sn : a.K, 128)) != cudaSuccess ||
      (e = tmap_view(&mw, a.w.data, a.N, a.K, a.w.sn ? a.w.sn : a.K, BN / 2)) != cudaSuccess ||
      (e = tmap_view(&mo, a.out, a.M, a.N, a.out_sn ? a.out_sn : a.N, 32)) != cudaSuccess)
    return e;
  p.mtiles = (p.M + 255) / 256;
  p.ntiles = (p.N + BN - 1) / BN;
  const int64_t tiles = (int64_t)p.mtiles * p.ntiles;
  static std::atomic<uint64_t> smem_set{0};
  e = allow_smem((const void*)pair_kernel<BN, ACT>, PairCfg<BN>::kSmem, &smem_set);
  if (e != cudaSuccess) return e;
  // as many pairs as can be resident at once (a GPC with an odd number of SMs
  // leaves one out), each walking its share of the tiles
  static std::atomic<int> resident[64] = {};   // per device
  int dev = 0;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  int pairs = resident[dev & 63].load(std::memory_order_relaxed);
  if (pairs == 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(kPairThreads);
    cfg.dynamicSmemBytes = PairCfg<BN>::kSmem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(&pairs, pair_kernel<BN, ACT>, &cfg);
    if (e != cudaSuccess) return e;
    if (pairs < 1) return cudaErrorInvalidConfiguration;
    resident[dev & 63].store(pairs, std::memory_order_relaxed);
  }
  return launch(pair_kernel<BN, ACT>, 2 * (unsigned)(tiles < pairs ? tiles : pairs), kPairThreads,
                PairCfg<BN>::kSmem, s, 2, mx, mw, mo, p);
}

// CTAs that share a feature tile's K: as many as are resident at once, while
// each keeps four steps, and four at most (64×4096×4096: 14 µs with four, 17
// with eight, 16 with two, 24 unsplit).
int few_split(int64_t tiles, int kblocks, int64_t resident) {
  int split = 1;
  while (split < 4 && tiles * split * 2 <= resident && kblocks >= split * 8) split *= 2;
  return split;
}

template <int BT, int ACT>
cudaError_t launch_few(const LinearArgs& a, const LinParams& p, cudaStream_t s) {
  using C = FewCfg<BT>;
  CUtensorMap mx, mw;
  cudaError_t e;
  if ((e = tmap_view(&mx, a.x.data, a.M, a.K, a.x.sn ? a.x.sn : a.K, BT)) != cudaSuccess ||
      (e = tmap_view(&mw, a.w.data, a.N, a.K, a.w.sn ? a.w.sn : a.K, 128)) != cudaSuccess)
    return e;
  const int64_t ft = (a.N + 127) / 128, mt = (a.M + BT - 1) / BT;
  const int split = few_split(ft * mt, p.kblocks, C::kPerSm * (int64_t)a.num_sms);
  // A CTA alone on its SM has all stages; CTAs that share one have three each
  // (16×2048×8192: 8.4 µs, 9.2 with five; 16×4096×2048, alone: 7.9 with five or
  // eight, 9.0 with three).  No more stages than steps: a short K leaves room
  // for more CTAs per SM (777×128×4096: 6.6 µs against 11).
  const int steps = (p.kblocks + split - 1) / split;
  const int most = ft * mt * split <= a.num_sms ? C::kNum : C::kShared;
  const int stages = steps < most ? steps : most;
  if (ft * split * mt > INT32_MAX) return cudaErrorInvalidConfiguration;
  static std::atomic<uint64_t> smem_set{0};
  e = allow_smem((const void*)few_kernel<BT, ACT>, C::smem(C::kNum), &smem_set);
  if (e != cudaSuccess) return e;
  return launch(few_kernel<BT, ACT>, (unsigned)(ft * split * mt), kFewThreads,
                C::smem(stages), s, (unsigned)split, mx, mw, p, split, (int)ft, stages);
}

// Estimated time of few_kernel<BT>, in SM cycles: a CTA's launch, setup and
// drain, which grow with the tokens whose partial sums it writes and reads; the
// steps of K of the CTAs that an SM has, at 64 bytes a cycle into the SM; and
// the exchange between CTAs that split K.  In a CUDA graph, µs with BT = 32 / 64
// / 128: 200×64×2048 2.9 / 3.5 / 4.7; 1509×496×296 6.6 / 5.6 / 6.7; 250×1024×2048
// 8.1 / 6.8 / 8.6; 128×2048×8192 15.7 / 12.1 / 11.9.
template <int BT> double few_cycles(const LinearArgs& a, int kblocks) {
  const int64_t tiles = ((a.N + 127) / 128) * ((a.M + BT - 1) / BT);
  const int split = few_split(tiles, kblocks, FewCfg<BT>::kPerSm * (int64_t)a.num_sms);
  const double per_sm = (double)((tiles * split + a.num_sms - 1) / a.num_sms);
  const double fixed = 4300 + 36.5 * BT;
  return fixed * (0.6 + 0.4 * per_sm) + per_sm * kblocks / split * (FewCfg<BT>::kStage / 64.0) +
         (split > 1 ? 1000.0 * split : 0.0);
}

// The same for pair_kernel: the tiles that follow one another on a pair, by
// what a step of K measured where every SM has a tile.
template <int BN> double pair_cycles(const LinearArgs& a, int kblocks) {
  const int64_t tiles = ((a.M + 255) / 256) * ((a.N + BN - 1) / BN), pairs = a.num_sms / 2;
  return 11000 + (double)((tiles + pairs - 1) / pairs) * kblocks * (BN == 256 ? 540 : 460);
}

// The kernel for a product: few_kernel<16> to <128>, or pair_kernel<128> or <256>.
enum Choice { kFew16, kFew32, kFew64, kFew128, kPair128, kPair256 };

Choice choose(const LinearArgs& a) {
  const int kblocks = (int)((a.K + kBK - 1) / kBK);
  if (a.M <= 16) return kFew16;
  // tiles of at most twice the tokens there are
  const double none = 1e300;
  const double f32 = few_cycles<32>(a, kblocks);
  const double f64 = a.M > 32 ? few_cycles<64>(a, kblocks) : none;
  const double f128 = a.M > 64 ? few_cycles<128>(a, kblocks) : none;
  const double p128 = a.M > 128 ? pair_cycles<128>(a, kblocks) : none;
  const double p256 = a.M > 128 ? pair_cycles<256>(a, kblocks) : none;
  const double least = std::min({f32, f64, f128, p128, p256});
  if (f128 == least) return kFew128;
  if (f64 == least) return kFew64;
  if (f32 == least) return kFew32;
  return p256 == least ? kPair256 : kPair128;
}

template <int ACT>
cudaError_t by_shape(const LinearArgs& a, cudaStream_t s) {
  LinParams p{};
  p.bias = static_cast<const bf16*>(a.bias);
  p.residual = static_cast<const bf16*>(a.residual.data);
  p.res_sn = a.residual.sn;
  p.out = static_cast<bf16*>(a.out);
  p.out_sn = a.out_sn;
  p.M = (int)a.M;
  p.N = (int)a.N;
  p.kblocks = (int)((a.K + kBK - 1) / kBK);
  p.status = a.status;
  switch (choose(a)) {
    case kFew16: return launch_few<16, ACT>(a, p, s);
    case kFew32: return launch_few<32, ACT>(a, p, s);
    case kFew64: return launch_few<64, ACT>(a, p, s);
    case kFew128: return launch_few<128, ACT>(a, p, s);
    case kPair128: return launch_pair<128, ACT>(a, p, s);
    default: return launch_pair<256, ACT>(a, p, s);
  }
}

}  // namespace

const char* tc_linear_kernel(const LinearArgs& a) {
  static const char* const names[] = {"few16", "few32", "few64", "few128", "pair128", "pair256"};
  return names[choose(a)];
}

cudaError_t tc_linear(const LinearArgs& a, cudaStream_t s) {
  switch (a.act) {
    case LA_ACT_RELU: return by_shape<LA_ACT_RELU>(a, s);
    case LA_ACT_SILU: return by_shape<LA_ACT_SILU>(a, s);
    case LA_ACT_GELU: return by_shape<LA_ACT_GELU>(a, s);
    case LA_ACT_SOFTPLUS: return by_shape<LA_ACT_SOFTPLUS>(a, s);
    default: return by_shape<LA_ACT_NONE>(a, s);
  }
}

}  // namespace la
