// The gated delta rule in chunks of C = 64 tokens on the tcgen05 tensor cores.
//
// With b_i = Σ_{t≤i} log α_t within a chunk, S the state before it, and k, q of
// unit length (a factor r per row, so that the rows themselves stay bf16):
//   A_ij = β_i (k_i·k_j) e^{b_i − b_j} for j < i,   T = (1 + A)^{-1}
//   w    = T (β v − β e^b (k S))                      the chunk's corrected values
//   o_i  = scale·(e^{b_i} q_i S + Σ_{j≤i} (q_i·k_j) e^{b_i − b_j} w_j)
//   S'   = e^{b_C} S + Σ_j e^{b_C − b_j} k_jᵀ w_j
// Every row and column factor is folded into T, P, w or the output, so q, k and
// v go from TMA to the MMA as they are.
//
// One CTA per (sequence, value head, 128 columns of v) walks its chunks with S in
// fp32 registers.  All products on the way of S are transposed, with v's columns
// as the MMA's 128 rows and the chunk's tokens (or dk) as its columns: Sᵀ, (kS)ᵀ
// and wᵀ are then A operands in tensor memory, and their conversions never cross
// lanes.  A chunk is three dependent products: (kS)ᵀ = Sᵀkᵀ, wᵀ = vᵀT1ᵀ +
// (kS)ᵀT2ᵀ, and wᵀk for the new state; everything else (the gram matrix and the
// inverse of the chunk after next, the output) runs beside them.
//
// Rounding.  The state, sums, decays, A and T are fp32.  As MMA operands S, kS,
// T and w are split into two bf16 parts (2^-16 of a value is lost), so that the
// state stays within about 1e-5 of itself however long the sequence.  What only
// the output is made of (S in q·S, P, w in P·w) is rounded to bf16 once, as the
// output is.
//
// Roles: warps 0-7 S (two per quarter of the rows), 8-11 the chunk's T and P,
// 12-15 the output, 16 loads, 17 MMAs (18 and 19 complete a warpgroup).
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

constexpr int kC = 64;                        // tokens of a chunk
constexpr int kThreads = 20 * 32;
constexpr int kStateWarps = 8, kPrepWarp = 8, kOutWarp = 12, kLoadWarp = 16, kMmaWarp = 17;
constexpr int kKQ = 3, kVS = 2, kTok = 4;     // stages: k and q tiles, v tiles, token factors
constexpr int kSlab = kC * 128;               // 8 KB: 64 tokens × 64 features
constexpr int kAPitch = 68;                   // floats of a row of A

// Named barriers.
constexpr uint32_t kBarPrep = 1, kBarOut = 2;

struct TokenFactors {
  float4 pair[kC];      // b (two parts, log2), r_k; the factors of a column of A and P
  float left[kC];       // r_k e^{b_C − b}: a row of w for the state
  float out[kC];        // scale r_q e^b: a row of q·S
  float t1[kC], t2[kC]; // β and −β e^b r_k: a column of T
  float carry;          // e^{b_C}
};

struct Bars {
  uint64_t kq_full[kKQ], kq_empty[kKQ], v_full[kVS], v_empty[kVS];
  uint64_t kq_clean, v_clean;                 // the last chunk's rows past the length are zero
  uint64_t g_full, g_empty, t_ready, s_ready, ks_full, ks_ready, qs_full, qs_read, w_full, w_ready,
      upd_full, pv_full, done;
  uint32_t tmem;
  int abort;
  int kq_issued, v_issued;                    // loads
};

template <int DK> struct Cfg {
  static constexpr int kSlabs = DK / 64;
  static constexpr int kStage = 2 * kSlabs * kSlab;          // k and q: per 64 features, k's rows, then q's
  static constexpr int oV = kKQ * kStage;
  static constexpr int oT = oV + kVS * 2 * kSlab;            // T1 hi, lo, T2 hi, lo
  static constexpr int oP = oT + 4 * kSlab;                  // two
  static constexpr int oOut = oP + 2 * kSlab;
  static constexpr int oA = oOut + 2 * kSlab;
  static constexpr int oTok = oA + kC * kAPitch * 4;
  static constexpr int oBars = oTok + kTok * (int)sizeof(TokenFactors);
  static constexpr int kSmem = 1024 + oBars + (int)sizeof(Bars);
  static_assert(kSmem <= 227 * 1024, "shared memory of a CTA");
  // tensor memory columns
  static constexpr uint32_t SH = 0, SL = DK / 2, UPD = DK, KS = 2 * DK, W = KS + kC, PV = W + kC,
                            G = PV + kC;
  static_assert(G + kC <= 512, "tensor memory");
};

struct TcParams {
  Rows dt, beta;
  const float* a;
  const float* dt_bias;
  const float* state_in;
  float* state_out;
  const int32_t* lengths;
  bf16* out;
  int64_t out_sb, out_sn, out_sh;
  int n, Hk, Hv, dk, dv, tiles;
  int q_h, q_b, k_h, k_b, v_h, v_b, o_h, o_b;   // 0 for axes that are broadcast or single
  float scale;
  bool gates_f32, softplus, sigmoid, normalize;
  int* status;
};

// A pair of fp32 as two bf16 parts each: hi keeps the leading 8 bits, lo the next 8.
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  hi = pack_bf16x2(x, y);
  lo = pack_bf16x2(x - bf16lo_to_f32(hi), y - bf16hi_to_f32(hi));
}

// 32 lanes × 8 consecutive columns store (thread i writes lane lane_base + i).
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}

// The sum of two values that are kept in two parts each.
__device__ __forceinline__ float2 add_parts(float2 a, float2 b) {
  const float s = a.x + b.x, t = s - a.x;
  return make_float2(s, a.y + b.y + ((a.x - (s - t)) + (b.x - t)));
}

__device__ __forceinline__ float gate_value(const Rows& r, bool f32, int64_t at) {
  return f32 ? static_cast<const float*>(r.data)[at] : to_f32(static_cast<const bf16*>(r.data)[at]);
}

// Registers of a thread by role: at launch all have 96, and a warpgroup's share is
// moved where S is held: 2·120 + 104 + 64 + 72 = 5·96 (dk 128), 2·96 + 104 + 64 + 96.
template <int N> __device__ __forceinline__ void take_registers() {
  if constexpr (N > 96)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
  else
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

struct Ctx {
  uint8_t* sm;
  Bars* bars;
  TokenFactors* tok;
  uint32_t tmem;
  int b, h, tile, live, chunks;
  bool partial;           // rows of the last chunk lie past the length
};

// mbar_wait and mbar_wait_drain in line: the compiler refuses calls beside setmaxnreg.
__device__ __forceinline__ bool wait_in_line(uint64_t* bar, uint32_t parity, int* status,
                                             volatile int* abort) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  for (uint32_t it = 1; !mbar_try_wait(bar, parity); ++it) {
    if (it % 8) continue;
    if (*abort) return false;
    if (global_timer_ns() - t0 > 2000000000ull) {
      if (status) atomicCAS(status, 0, kStatusTimeout);
      *abort = 1;
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ bool warp_wait_in_line(uint64_t* bar, uint32_t parity, int* status,
                                                  volatile int* abort) {
  return __all_sync(0xffffffffu, wait_in_line(bar, parity, status, abort));
}

__device__ __forceinline__ void drain_in_line(uint64_t* bar, uint32_t parity) {
  const uint64_t t0 = global_timer_ns();
  for (uint32_t it = 1; !mbar_try_wait(bar, parity); ++it)
    if (it % 8 == 0 && global_timer_ns() - t0 > 500000000ull) return;
}

// A role that shares no barrier with other warps returns where a wait gives up;
// the others (LA_GO_ON) walk on through their remaining barriers, whose waits then
// end at once: what they write stays within their own buffers and the output.
#define LA_WAIT(bar, parity) \
  if (!warp_wait_in_line(&x.bars->bar, (parity) & 1, p.status, abort)) return
#define LA_GO_ON(bar, parity) warp_wait_in_line(&x.bars->bar, (parity) & 1, p.status, abort)

// ------------------------------------------------------------------ loads

// (whole warp)
template <int DK>
__device__ __forceinline__ void role_load(const Ctx& x, const TcParams& p, const CUtensorMap* mq,
                                          const CUtensorMap* mk, const CUtensorMap* mv, int lane) {
  using F = Cfg<DK>;
  volatile int* abort = &x.bars->abort;
  const int hk = x.h / (p.Hv / p.Hk);
  const int vslabs = p.dv - x.tile * 128 > 64 ? 2 : 1;
  for (int c = 0; c < x.chunks; ++c) {
    const int s = c % kKQ, vs = c % kVS, t = c * kC;
    if (c >= kKQ) LA_WAIT(kq_empty[s], c / kKQ - 1);
    if (lane == 0) {
      uint8_t* to = x.sm + s * F::kStage;
      mbar_arrive_expect_tx(&x.bars->kq_full[s], F::kStage);
#pragma unroll
      for (int i = 0; i < F::kSlabs; ++i) {
        tma_load_4d(to + i * 2 * kSlab, mk, &x.bars->kq_full[s], i * 64, hk * p.k_h, t, x.b * p.k_b);
        tma_load_4d(to + i * 2 * kSlab + kSlab, mq, &x.bars->kq_full[s], i * 64, hk * p.q_h, t, x.b * p.q_b);
      }
    }
    if (lane == 0) x.bars->kq_issued = c + 1;
    if (c >= kVS) LA_WAIT(v_empty[vs], c / kVS - 1);
    if (lane == 0) {
      uint8_t* to = x.sm + F::oV + vs * 2 * kSlab;
      mbar_arrive_expect_tx(&x.bars->v_full[vs], vslabs * kSlab);
      for (int i = 0; i < vslabs; ++i)
        tma_load_4d(to + i * kSlab, mv, &x.bars->v_full[vs], x.tile * 128 + i * 64, x.h * p.v_h, t, x.b * p.v_b);
    }
    if (lane == 0) x.bars->v_issued = c + 1;
  }
  // the rows past the length may hold anything: zeros, so that they add nothing
  if (!x.partial) return;
  const int c = x.chunks - 1, r0 = x.live - c * kC;
  auto clear = [&](uint8_t* slab) {
    for (int i = r0 * 8 + lane; i < kC * 8; i += 32)
      *reinterpret_cast<uint4*>(slab + i * 16) = make_uint4(0, 0, 0, 0);
  };
  LA_WAIT(kq_full[c % kKQ], c / kKQ);
  for (int i = 0; i < 2 * F::kSlabs; ++i) clear(x.sm + c % kKQ * F::kStage + i * kSlab);
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) mbar_arrive(&x.bars->kq_clean);
  LA_WAIT(v_full[c % kVS], c / kVS);
  for (int i = 0; i < vslabs; ++i) clear(x.sm + F::oV + (c % kVS * 2 + i) * kSlab);
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) mbar_arrive(&x.bars->v_clean);
}

// ------------------------------------------------------------------ products

// (one thread)
template <int DK>
__device__ __forceinline__ void role_mma(const Ctx& x, const TcParams& p) {
  using F = Cfg<DK>;
  Bars* bars = x.bars;
  volatile int* abort = &bars->abort;
  const uint32_t tmem = x.tmem, base = smem_u32(x.sm);
  constexpr uint32_t id_nn = idesc_bf16_f32(128, kC, false, false);   // K-major A and B, 64 columns
  constexpr uint32_t id_v = idesc_bf16_f32(128, kC, true, false);     // vᵀ from [token][column]
  constexpr uint32_t id_upd = idesc_bf16_f32(128, DK, false, true);   // k as [token][feature]
  constexpr int KD = DK / 16;
  const uint64_t dT = smem_desc(base + F::oT, 16, 1024, kSwizzle128B);
  // K-step k of a tile with 64 features per slab
  auto kstep = [](int k) { return (uint32_t)((k >> 2) * 2 * kSlab + (k & 3) * 32); };
  // K-step k of (kS)ᵀ or wᵀ: 32 tokens' hi parts, then their lo parts
  auto tokens = [](int k) { return (uint32_t)((k >> 1) * 32 + (k & 1) * 8); };
#define LA_MWAIT(bar, parity) \
  if (!wait_in_line(&bars->bar, (parity) & 1, p.status, abort)) return
  auto gram = [&](int c) -> bool {   // [k; q]·kᵀ
    if (!wait_in_line(&bars->kq_full[c % kKQ], (c / kKQ) & 1, p.status, abort)) return false;
    if (x.partial && c == x.chunks - 1 && !wait_in_line(&bars->kq_clean, 0, p.status, abort)) return false;
    if (c >= 1 && !wait_in_line(&bars->g_empty, (c - 1) & 1, p.status, abort)) return false;
    tc_fence_after();
    const uint64_t d = smem_desc(base + c % kKQ * F::kStage, 16, 1024, kSwizzle128B);
#pragma unroll
    for (int k = 0; k < KD; ++k)
      mma_ss(tmem + F::G, desc_at(d, kstep(k)), desc_at(d, kstep(k)), id_nn, k > 0);
    mma_commit(&bars->g_full);
    return true;
  };
  for (int c = 0; c < 2 && c < x.chunks; ++c)
    if (!gram(c)) return;
  for (int c = 0; c < x.chunks; ++c) {
    const uint32_t kq = base + c % kKQ * F::kStage;
    const uint64_t dK = smem_desc(kq, 16, 1024, kSwizzle128B);
    const uint64_t dQ = smem_desc(kq + kSlab, 16, 1024, kSwizzle128B);
    const uint64_t dKt = smem_desc(kq, 2 * kSlab, 1024, kSwizzle128B);
    const uint64_t dV = smem_desc(base + F::oV + c % kVS * 2 * kSlab, kSlab, 1024, kSwizzle128B);
    const uint64_t dP = smem_desc(base + F::oP + c % 2 * kSlab, 16, 1024, kSwizzle128B);
    // wᵀ = vᵀ T1ᵀ
    LA_MWAIT(t_ready, c);
    LA_MWAIT(v_full[c % kVS], c / kVS);
    if (x.partial && c == x.chunks - 1) LA_MWAIT(v_clean, 0);
    tc_fence_after();
#pragma unroll
    for (int part = 0; part < 2; ++part)
#pragma unroll
      for (int k = 0; k < kC / 16; ++k)
        mma_ss(tmem + F::W, desc_at(dV, k * 2048), desc_at(dT, part * kSlab + k * 32), id_v, part | k);
    mma_commit(&bars->v_empty[c % kVS]);
    // (kS)ᵀ = Sᵀ kᵀ, and (qS)ᵀ
    LA_MWAIT(s_ready, c);
    tc_fence_after();
#pragma unroll
    for (int part = 0; part < 2; ++part)
#pragma unroll
      for (int k = 0; k < KD; ++k)
        mma_ts(tmem + F::KS, tmem + (part ? F::SL : F::SH) + k * 8, desc_at(dK, kstep(k)), id_nn, part | k);
    mma_commit(&bars->ks_full);
#pragma unroll
    for (int k = 0; k < KD; ++k)
      mma_ts(tmem + F::UPD, tmem + F::SH + k * 8, desc_at(dQ, kstep(k)), id_nn, k > 0);
    mma_commit(&bars->qs_full);
    // wᵀ += (kS)ᵀ T2ᵀ
    LA_MWAIT(ks_ready, c);
    tc_fence_after();
#pragma unroll
    for (int part = 0; part < 3; ++part)   // hi·hi, hi·lo, lo·hi
#pragma unroll
      for (int k = 0; k < kC / 16; ++k)
        mma_ts(tmem + F::W, tmem + F::KS + tokens(k) + (part == 2 ? 16 : 0),
               desc_at(dT, (part == 1 ? 3 : 2) * kSlab + k * 32), id_nn, 1);
    mma_commit(&bars->w_full);
    if (c + 2 < x.chunks && !gram(c + 2)) return;
    // the state's wᵀk
    LA_MWAIT(w_ready, c);
    LA_MWAIT(qs_read, c);
    tc_fence_after();
#pragma unroll
    for (int part = 0; part < 2; ++part)
#pragma unroll
      for (int k = 0; k < kC / 16; ++k)
        mma_ts(tmem + F::UPD, tmem + F::KS + tokens(k) + part * 16, desc_at(dKt, k * 2048), id_upd, part | k);
    mma_commit(&bars->upd_full);
    mma_commit(&bars->kq_empty[c % kKQ]);
    // (P w)ᵀ on top of what the output's warps have put there
#pragma unroll
    for (int k = 0; k < kC / 16; ++k)
      mma_ts(tmem + F::PV, tmem + F::SL + k * 8, desc_at(dP, k * 32), id_nn, 1);
    mma_commit(&bars->pv_full);
  }
#undef LA_MWAIT
}

// ------------------------------------------------------------------ the state

// Warp w has rows 32(w % 4) … of Sᵀ (columns of v) and half of its columns.
template <int DK>
__device__ __forceinline__ void role_state(const Ctx& x, const TcParams& p, int warp, int lane) {
  using F = Cfg<DK>;
  constexpr int kCols = DK / 2;
  Bars* bars = x.bars;
  volatile int* abort = &bars->abort;
  const int half = warp / 4, k0 = half * kCols;
  const uint32_t at = tmem_addr(x.tmem, warp % 4 * 32, 0);
  const int col = x.tile * 128 + warp % 4 * 32 + lane;
  const int64_t head = (int64_t)x.b * p.Hv + x.h;
  float S[kCols];
#pragma unroll
  for (int i = 0; i < kCols; ++i)
    S[i] = p.state_in && col < p.dv && k0 + i < p.dk ? p.state_in[(head * p.dk + k0 + i) * p.dv + col] : 0.f;

  auto publish = [&] {   // S as the next products' operand
#pragma unroll
    for (int j = 0; j < kCols; j += 16) {
      uint32_t hi[8], lo[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) split2(S[j + 2 * i], S[j + 2 * i + 1], hi[i], lo[i]);
      tmem_st8(at + F::SH + (k0 + j) / 2, hi);
      tmem_st8(at + F::SL + (k0 + j) / 2, lo);
    }
    tmem_st_wait();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars->s_ready);
  };
  if (x.chunks) publish();
  for (int c = 0; c < x.chunks; ++c) {
    const TokenFactors& tok = x.tok[c % kTok];
    LA_WAIT(ks_full, c);
    tc_fence_after();
    {
      uint32_t r[32];
      tmem_ld32(at + F::KS + half * 32, r);
      tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < 16; j += 8) {
        uint32_t hi[8], lo[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          split2(__uint_as_float(r[2 * (j + i)]), __uint_as_float(r[2 * (j + i) + 1]), hi[i], lo[i]);
        tmem_st8(at + F::KS + half * 32 + j, hi);
        tmem_st8(at + F::KS + half * 32 + 16 + j, lo);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->ks_ready);
    }
    LA_WAIT(w_full, c);
    tc_fence_after();
    {
      uint32_t r[32];
      tmem_ld32(at + F::W + half * 32, r);
      tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < 16; j += 8) {
        uint32_t hi[8], lo[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          hi[i] = pack_bf16x2(__uint_as_float(r[2 * (j + i)]), __uint_as_float(r[2 * (j + i) + 1]));
        tmem_st8(at + F::SL + half * 16 + j, hi);   // for the output; (kS)ᵀ is done with S's lo parts
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          const uint32_t* v = r + 2 * (j + i);
          const float4 f = *reinterpret_cast<const float4*>(&tok.left[half * 32 + 2 * (j + i)]);
          split2(__uint_as_float(v[0]) * f.x, __uint_as_float(v[1]) * f.y, hi[i], lo[i]);
          split2(__uint_as_float(v[2]) * f.z, __uint_as_float(v[3]) * f.w, hi[i + 1], lo[i + 1]);
        }
        tmem_st8(at + F::KS + half * 32 + j, hi);
        tmem_st8(at + F::KS + half * 32 + 16 + j, lo);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->w_ready);
    }
    const float carry = tok.carry;
    LA_WAIT(upd_full, c);
    tc_fence_after();
#pragma unroll
    for (int j = 0; j < kCols; j += 32) {
      uint32_t r[32];
      tmem_ld32(at + F::UPD + k0 + j, r);
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 32; ++i) S[j + i] = fmaf(S[j + i], carry, __uint_as_float(r[i]));
    }
    LA_WAIT(pv_full, c);   // done with w where S's lo parts go
    if (c + 1 < x.chunks) publish();
  }
  if (p.state_out && col < p.dv) {
#pragma unroll
    for (int i = 0; i < kCols; ++i)
      if (k0 + i < p.dk) p.state_out[(head * p.dk + k0 + i) * p.dv + col] = S[i];
  }
}

// ------------------------------------------------------------------ the output

// Warp w has rows 32(w % 4) … of the transposed output (columns of v).
template <int DK>
__device__ __forceinline__ void role_out(const Ctx& x, const TcParams& p, const CUtensorMap* mo, int warp,
                                         int lane) {
  using F = Cfg<DK>;
  Bars* bars = x.bars;
  volatile int* abort = &bars->abort;
  const uint32_t at = tmem_addr(x.tmem, warp % 4 * 32, 0);
  const int d = warp % 4 * 32 + lane;
  const bool lead = warp == kOutWarp && lane == 0;
  uint8_t* stage = x.sm + F::oOut;
  const uint32_t mine = smem_u32(stage) + d / 64 * kSlab + d % 64 * 2;
  for (int c = 0; c < x.chunks; ++c) {
    const TokenFactors& tok = x.tok[c % kTok];
    // scale e^{b_i} q_i S is what P·w is added to
    LA_GO_ON(qs_full, c);
    tc_fence_after();
#pragma unroll
    for (int j = 0; j < kC; j += 32) {
      uint32_t r[32];
      tmem_ld32(at + F::UPD + j, r);
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 32; i += 4) {
        const float4 f = *reinterpret_cast<const float4*>(&tok.out[j + i]);
        r[i] = __float_as_uint(f.x * __uint_as_float(r[i]));
        r[i + 1] = __float_as_uint(f.y * __uint_as_float(r[i + 1]));
        r[i + 2] = __float_as_uint(f.z * __uint_as_float(r[i + 2]));
        r[i + 3] = __float_as_uint(f.w * __uint_as_float(r[i + 3]));
      }
      tmem_st32(at + F::PV + j, r);
    }
    tmem_st_wait();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars->qs_read);
    LA_GO_ON(pv_full, c);
    tc_fence_after();
    if (lead) tma_store_wait_read0();
    named_bar_sync(kBarOut, 128);
    const int rows = min(kC, x.live - c * kC);
#pragma unroll
    for (int j = 0; j < kC; j += 32) {
      uint32_t r[32];
      tmem_ld32(at + F::PV + j, r);
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const float o = j + i < rows ? __uint_as_float(r[i]) : 0.f;
        asm volatile("st.shared.b16 [%0], %1;" ::"r"(mine + (j + i) * 128),
                     "h"((uint16_t)(pack_bf16x2(o, 0.f) & 0xffffu))
                     : "memory");
      }
    }
    tc_fence_before();
    fence_proxy_async_smem();
    named_bar_sync(kBarOut, 128);
    if (lead) {
      for (int i = 0; i < 2; ++i) {
        const int col = x.tile * 128 + i * 64;
        if (col < p.dv && LA_DCHECK(p.status, c * kC < p.n, 61))
          tma_store_4d(mo, stage + i * kSlab, col, x.h * p.o_h, c * kC, x.b * p.o_b);
      }
      tma_store_commit();
    }
  }
  if (lead) tma_store_wait0();
  // chunks past the length
  const int cols = min(128, p.dv - x.tile * 128) / 8, lanes = (warp - kOutWarp) * 32 + lane;
  bf16* o = p.out + x.b * p.out_sb + x.h * p.out_sh + x.tile * 128;
  for (int64_t t = x.chunks * kC + lanes / 16; t < p.n; t += 8)
    if (lanes % 16 < cols) *reinterpret_cast<uint4*>(o + t * p.out_sn + lanes % 16 * 8) = make_uint4(0, 0, 0, 0);
}

// ------------------------------------------------------------------ T and P

// log2 α of a token, at least −2^20 (which any exponential takes to 0): sums of 64
// of them keep their differences.  A step of zero leaves the state alone.
__device__ __forceinline__ float log2_decay(const TcParams& p, float dt, float bias, float rate) {
  float d = dt + bias;
  if (p.softplus) d = softplus(d);
  const float g = d == 0.f ? 0.f : d * (rate * kLog2e);
  return g < -1048576.f ? -1048576.f : g;
}

// One column of the inverse of a unit lower triangular 16×16 block.
__device__ __forceinline__ void invert16(float* A, int lane) {
  float v[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float s = lane == i ? 1.f : 0.f;
#pragma unroll
    for (int j = 0; j < i; j += 4) {
      const float4 a = *reinterpret_cast<const float4*>(A + i * kAPitch + j);
      s = fmaf(-a.x, v[j], s);
      if (j + 1 < i) s = fmaf(-a.y, v[j + 1], s);
      if (j + 2 < i) s = fmaf(-a.z, v[j + 2], s);
      if (j + 3 < i) s = fmaf(-a.w, v[j + 3], s);
    }
    v[i] = s;
  }
  __syncwarp();
  if (lane < 16)
#pragma unroll
    for (int i = 0; i < 16; ++i) A[i * kAPitch + lane] = v[i];
}

// ROWS rows × 4 columns of X·Y over K of [K0, K1), all at the A's pitch.
template <int ROWS>
__device__ __forceinline__ void small_product(const float* X, const float* Y, int K0, int K1, float sign,
                                              float* Z) {
  float4 z[ROWS] = {};
#pragma unroll 2
  for (int k = K0; k < K1; k += 4) {
    float4 xs[ROWS], ys[4];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) xs[r] = *reinterpret_cast<const float4*>(X + r * kAPitch + k);
#pragma unroll
    for (int j = 0; j < 4; ++j) ys[j] = *reinterpret_cast<const float4*>(Y + (k + j) * kAPitch);
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const float xv[4] = {xs[r].x, xs[r].y, xs[r].z, xs[r].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        z[r].x = fmaf(xv[j], ys[j].x, z[r].x);
        z[r].y = fmaf(xv[j], ys[j].y, z[r].y);
        z[r].z = fmaf(xv[j], ys[j].z, z[r].z);
        z[r].w = fmaf(xv[j], ys[j].w, z[r].w);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < ROWS; ++r)
    *reinterpret_cast<float4*>(Z + r * kAPitch) =
        make_float4(sign * z[r].x, sign * z[r].y, sign * z[r].z, sign * z[r].w);
}

// Thread t < 64 has token t's row of k·kᵀ, thread 64 + t that of q·kᵀ.
template <int DK>
__device__ __forceinline__ void role_prep(const Ctx& x, const TcParams& p, int warp, int lane) {
  using F = Cfg<DK>;
  Bars* bars = x.bars;
  volatile int* abort = &bars->abort;
  const int t = (warp - kPrepWarp) * 32 + lane, row = t % kC;
  const bool keys = t < kC;
  const uint32_t at = tmem_addr(x.tmem, warp % 4 * 32, 0);
  float* A = reinterpret_cast<float*>(x.sm + F::oA);
  const float rate = p.a[x.h], bias = p.dt_bias ? p.dt_bias[x.h] : 0.f;
  // step and strength of tokens lane and lane + 32 of a chunk
  float dt[2], be[2];
  auto fetch = [&](int c) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t tt = (int64_t)c * kC + i * 32 + lane;
      const bool in = tt < x.live;
      dt[i] = in ? gate_value(p.dt, p.gates_f32, x.b * p.dt.sb + tt * p.dt.sn + x.h) : 0.f;
      be[i] = in ? gate_value(p.beta, p.gates_f32, x.b * p.beta.sb + tt * p.beta.sn + x.h) : 0.f;
    }
  };
  if (x.chunks) fetch(0);
  for (int c = 0; c < x.chunks; ++c) {
    TokenFactors& tok = x.tok[c % kTok];
    const bool live = c * kC + row < x.live;
    // b, inclusive, of both halves of the chunk
    float2 b[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      b[i] = make_float2(c * kC + i * 32 + lane < x.live ? log2_decay(p, dt[i], bias, rate) : 0.f, 0.f);
#pragma unroll
      for (int m = 1; m < 32; m *= 2) {
        const float2 o = make_float2(__shfl_up_sync(0xffffffffu, b[i].x, m), __shfl_up_sync(0xffffffffu, b[i].y, m));
        if (lane >= m) b[i] = add_parts(o, b[i]);
      }
    }
    b[1] = add_parts(b[1], make_float2(__shfl_sync(0xffffffffu, b[0].x, 31), __shfl_sync(0xffffffffu, b[0].y, 31)));
    const float2 last = make_float2(__shfl_sync(0xffffffffu, b[1].x, 31), __shfl_sync(0xffffffffu, b[1].y, 31));
    const float2 mine = row < 32 ? b[0] : b[1];
    float beta = row < 32 ? be[0] : be[1];
    if (p.sigmoid) beta = 1.f / (1.f + expf(-beta));
    if (!live) beta = 0.f;
    if (c + 1 < x.chunks) fetch(c + 1);
    // 1 / length of this thread's row of k or q
    LA_GO_ON(kq_full[c % kKQ], c / kKQ);
    float r = 1.f;
    if (p.normalize) {
      f32x2 s2 = 0;
#pragma unroll
      for (int i = 0; i < F::kSlabs; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          f32x2 v[4];
          unpack_pairs<bf16>(lds128(smem_u32(x.sm + c % kKQ * F::kStage + (2 * i + !keys) * kSlab) +
                                    sw_chunk(kC, row, 0, j)), v);
#pragma unroll
          for (int u = 0; u < 4; ++u) s2 = fma2(v[u], v[u], s2);
        }
      float lo, hi;
      unpack2(s2, lo, hi);
      r = rsqrtf(lo + hi + 1e-6f);
    }
    if (!live) r = 0.f;
    const float eb = ex2_f32(mine.x + mine.y);
    if (keys) {
      tok.pair[row] = make_float4(mine.x, mine.y, r, 0.f);
      tok.left[row] = r * ex2_f32((last.x - mine.x) + (last.y - mine.y));
      tok.t1[row] = beta;
      tok.t2[row] = -beta * eb * r;
      if (row == 0) tok.carry = ex2_f32(last.x + last.y);
    } else {
      tok.out[row] = p.scale * r * eb;
    }
    named_bar_sync(kBarPrep, 128);   // and the last chunk's T has been read from A
    // this row of A, or of P
    LA_GO_ON(g_full, c);
    tc_fence_after();
    uint32_t g[64];
    tmem_ld32(at + F::G, g);
    tmem_ld32(at + F::G + 32, g + 32);
    tmem_ld_wait();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars->g_empty);
    const float factor = keys ? beta * r : p.scale * r;
    const int upto = row - keys;      // A below the diagonal, P with it
    const int cols = row / 32 ? 64 : 32;
    uint32_t pk[32] = {};
#pragma unroll
    for (int j = 0; j < 64; j += 2) {
      if (j >= cols) break;           // (the same for the whole warp)
      float v[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float4 f = tok.pair[j + u];
        const float e = ex2_f32((mine.x - f.x) + (mine.y - f.y));
        v[u] = j + u <= upto ? factor * (__uint_as_float(g[j + u]) * f.z) * e : 0.f;
      }
      if (keys)
        *reinterpret_cast<float2*>(A + row * kAPitch + j) = make_float2(v[0], v[1]);
      else
        pk[j / 2] = pack_bf16x2(v[0], v[1]);
    }
    named_bar_sync(kBarPrep, 128);
    // T in A's place: blocks of 16, then 32, then 64; the upper blocks hold what is
    // between two products
    invert16(A + (t / 32) * 16 * (kAPitch + 1), lane);
    named_bar_sync(kBarPrep, 128);
    {
      const int o = t / 64 * 32, u = t % 64, r0 = u / 4, c0 = u % 4 * 4;
      float* B = A + o * (kAPitch + 1);
      small_product<1>(B + (16 + r0) * kAPitch, B + c0, 0, 16, 1.f, B + r0 * kAPitch + 16 + c0);
      named_bar_sync(kBarPrep, 128);
      small_product<1>(B + (16 + r0) * kAPitch + 16, B + 16 + c0, 0, 16, -1.f, B + (16 + r0) * kAPitch + c0);
    }
    named_bar_sync(kBarPrep, 128);
    {
      const int r0 = t / 8 * 2, c0 = t % 8 * 4;
      small_product<2>(A + (32 + r0) * kAPitch, A + c0, c0 < 16 ? 0 : 16, 32, 1.f, A + r0 * kAPitch + 32 + c0);
      named_bar_sync(kBarPrep, 128);
      small_product<2>(A + (32 + r0) * kAPitch + 32, A + 32 + c0, 0, r0 < 16 ? 16 : 32, -1.f,
                       A + (32 + r0) * kAPitch + c0);
    }
    named_bar_sync(kBarPrep, 128);
    // T1 and T2 where the last chunk's were, P where that of the one before was
    if (c >= 1) LA_GO_ON(w_full, c - 1);
    const uint32_t T = smem_u32(x.sm + F::oT);
    const int h0 = keys ? 0 : 32;     // half of the row's columns
#pragma unroll
    for (int j = 0; j < 32; j += 8) {
      uint4 o[4];
      uint32_t* w = reinterpret_cast<uint32_t*>(o);
#pragma unroll
      for (int i = 0; i < 8; i += 4) {
        const int k = h0 + j + i;
        const float4 a = *reinterpret_cast<const float4*>(A + row * kAPitch + k);
        const float4 f1 = *reinterpret_cast<const float4*>(&tok.t1[k]);
        const float4 f2 = *reinterpret_cast<const float4*>(&tok.t2[k]);
        const float v0 = k <= row ? a.x : 0.f, v1 = k + 1 <= row ? a.y : 0.f;
        const float v2 = k + 2 <= row ? a.z : 0.f, v3 = k + 3 <= row ? a.w : 0.f;
        split2(v0 * f1.x, v1 * f1.y, w[i / 2], w[4 + i / 2]);
        split2(v2 * f1.z, v3 * f1.w, w[i / 2 + 1], w[4 + i / 2 + 1]);
        split2(v0 * f2.x, v1 * f2.y, w[8 + i / 2], w[12 + i / 2]);
        split2(v2 * f2.z, v3 * f2.w, w[8 + i / 2 + 1], w[12 + i / 2 + 1]);
      }
#pragma unroll
      for (int m = 0; m < 4; ++m) sts128(T + m * kSlab + sw_chunk(kC, row, 0, (h0 + j) / 8), o[m]);
    }
    if (!keys) {
      const uint32_t P = smem_u32(x.sm + F::oP + c % 2 * kSlab);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        sts128(P + sw_chunk(kC, row, 0, j), make_uint4(pk[4 * j], pk[4 * j + 1], pk[4 * j + 2], pk[4 * j + 3]));
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars->t_ready);
  }
}

// ------------------------------------------------------------------ kernel

template <int DK>
__global__ void __launch_bounds__(kThreads, 1)
chunk_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
             const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mo, const TcParams p) {
  using F = Cfg<DK>;
  extern __shared__ uint8_t raw[];
  Ctx x;
  x.sm = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  x.tok = reinterpret_cast<TokenFactors*>(x.sm + F::oTok);
  x.bars = reinterpret_cast<Bars*>(x.sm + F::oBars);
  Bars* bars = x.bars;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kKQ; ++i) mbar_init(&bars->kq_full[i], 1), mbar_init(&bars->kq_empty[i], 1);
    for (int i = 0; i < kVS; ++i) mbar_init(&bars->v_full[i], 1), mbar_init(&bars->v_empty[i], 1);
    for (uint64_t* b : {&bars->kq_clean, &bars->v_clean, &bars->g_full, &bars->ks_full, &bars->qs_full,
                        &bars->w_full, &bars->upd_full, &bars->pv_full, &bars->done})
      mbar_init(b, 1);
    for (uint64_t* b : {&bars->g_empty, &bars->t_ready, &bars->qs_read}) mbar_init(b, 4);
    for (uint64_t* b : {&bars->s_ready, &bars->ks_ready, &bars->w_ready}) mbar_init(b, kStateWarps);
    bars->abort = bars->kq_issued = bars->v_issued = 0;
    fence_barrier_init();
    for (const CUtensorMap* m : {&mq, &mk, &mv, &mo}) tma_prefetch_desc(m);
  }
  // nothing reads v's second slab from global memory where the tile has one: zeros
  if (p.dv - (int)(blockIdx.x % p.tiles) * 128 <= 64)
    for (int i = threadIdx.x; i < kVS * kSlab / 16; i += kThreads)
      *reinterpret_cast<uint4*>(x.sm + F::oV + (2 * (i / (kSlab / 16)) + 1) * kSlab + i % (kSlab / 16) * 16) =
          make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  entry();
  if (warp == kMmaWarp) {
    tmem_alloc(&bars->tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  x.tmem = bars->tmem;
  x.tile = blockIdx.x % p.tiles;
  const int64_t bh = blockIdx.x / p.tiles;
  x.h = (int)(bh % p.Hv);
  x.b = (int)(bh / p.Hv);
  x.live = live_tokens(p.lengths, x.b, p.n);
  x.chunks = (x.live + kC - 1) / kC;
  x.partial = x.live % kC != 0 && x.live < p.n;

  if (warp < kStateWarps) {
    take_registers<DK == 128 ? 120 : 96>();
    role_state<DK>(x, p, warp, lane);
  } else if (warp < kOutWarp) {
    take_registers<104>();
    role_prep<DK>(x, p, warp, lane);
  } else if (warp < kLoadWarp) {
    take_registers<64>();
    role_out<DK>(x, p, &mo, warp, lane);
  } else {
    take_registers<DK == 128 ? 72 : 96>();
    if (warp == kLoadWarp)
      role_load<DK>(x, p, &mq, &mk, &mv, lane);
    else if (warp == kMmaWarp && lane == 0)
      role_mma<DK>(x, p);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (*(volatile int*)&bars->abort) {   // copies and products in flight end before the CTA does
    if (warp == kMmaWarp && lane == 0) {
      mma_commit(&bars->done);
      drain_in_line(&bars->done, 0);
    }
    if (warp == kLoadWarp && lane == 0) {
      const int kq_issued = bars->kq_issued, v_issued = bars->v_issued;
      for (int j = max(0, kq_issued - kKQ); j < kq_issued; ++j) drain_in_line(&bars->kq_full[j % kKQ], (j / kKQ) & 1);
      for (int j = max(0, v_issued - kVS); j < v_issued; ++j) drain_in_line(&bars->v_full[j % kVS], (j / kVS) & 1);
    }
    if (warp == kOutWarp && lane == 0) tma_store_wait0();
    __syncthreads();
  }
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(x.tmem, 512);
}

template <int DK>
cudaError_t launch_chunks(const DeltaArgs& a, const TcParams& p, cudaStream_t s) {
  CUtensorMap mq, mk, mv, mo;
  cudaError_t e;
  if ((e = tmap_heads(&mq, a.q, a.B, a.n, a.Hk, a.dk, kC, true)) != cudaSuccess ||
      (e = tmap_heads(&mk, a.k, a.B, a.n, a.Hk, a.dk, kC, true)) != cudaSuccess ||
      (e = tmap_heads(&mv, a.v, a.B, a.n, a.Hv, a.dv, kC, true)) != cudaSuccess ||
      (e = tmap_heads(&mo, a.out, a.B, a.n, a.Hv, a.dv, kC, false)) != cudaSuccess)
    return e;
  const int64_t ctas = a.B * a.Hv * p.tiles;
  if (ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
  static std::atomic<uint64_t> smem_set{0};
  if ((e = allow_smem((const void*)chunk_kernel<DK>, Cfg<DK>::kSmem, &smem_set)) != cudaSuccess) return e;
  return launch(chunk_kernel<DK>, (unsigned)ctas, kThreads, Cfg<DK>::kSmem, s, 1, mq, mk, mv, mo, p);
}

}  // namespace

bool tc_gated_delta_supported(const DeltaArgs& a) {
  // a tensor map has strides below 2^40 bytes; tokens that are all one row go by themselves
  for (const Heads* v : {&a.q, &a.k, &a.v, &a.out})
    if ((a.n > 1 && v->sn == 0) || v->sb >= ((int64_t)1 << 39) || v->sh >= ((int64_t)1 << 39)) return false;
  return a.bf16 && a.dk <= 128;
}

cudaError_t tc_gated_delta(const DeltaArgs& a, cudaStream_t s) {
  TcParams p{};
  p.dt = a.dt, p.beta = a.beta;
  p.a = a.a, p.dt_bias = a.dt_bias;
  p.state_in = a.state_in, p.state_out = a.state_out, p.lengths = a.lengths;
  p.out = static_cast<bf16*>(const_cast<void*>(a.out.data));
  p.out_sb = a.out.sb, p.out_sn = a.out.sn, p.out_sh = a.out.sh;
  p.n = (int)a.n, p.Hk = (int)a.Hk, p.Hv = (int)a.Hv, p.dk = a.dk, p.dv = a.dv;
  p.tiles = (a.dv + 127) / 128;
  p.q_h = a.q.sh != 0, p.q_b = a.q.sb != 0;
  p.k_h = a.k.sh != 0, p.k_b = a.k.sb != 0;
  p.v_h = a.v.sh != 0, p.v_b = a.v.sb != 0;
  p.o_h = a.out.sh != 0, p.o_b = a.out.sb != 0;
  p.scale = a.scale;
  p.gates_f32 = a.gates_f32, p.softplus = a.softplus, p.sigmoid = a.sigmoid, p.normalize = a.normalize;
  p.status = a.status;
  return a.dk <= 64 ? launch_chunks<64>(a, p, s) : launch_chunks<128>(a, p, s);
}

}  // namespace la
