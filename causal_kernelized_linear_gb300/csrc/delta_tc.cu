// The gated delta rule in chunks of C = 64 tokens on the tcgen05 tensor cores.
//
// With b_i = Σ_{t≤i} log α_t within a chunk, S the state before it, and k, q of
// unit length (a factor r per row, so that the rows themselves stay bf16):
//   A_ij = β_i (k_i·k_j) e^{b_i − b_j} for j < i,   T = (1 + A)^{-1}
//   w    = T β (v − e^b (k S))                        the chunk's corrected values
//   o_i  = scale·(e^{b_i} q_i S + Σ_{j≤i} (q_i·k_j) e^{b_i − b_j} w_j)
//   S'   = e^{b_C} S + Σ_j e^{b_C − b_j} k_jᵀ w_j
// Every row and column factor is folded into T, P, w or the output, so q, k and
// v go from TMA to the MMA as they are.
//
// One CTA per (sequence, value head, 128 columns of v) walks its chunks with S in
// fp32 registers.  All products on the way of S are transposed, with v's columns
// as the MMA's 128 rows and the chunk's tokens (or dk) as its columns: Sᵀ, (kS)ᵀ
// and wᵀ are then A operands in tensor memory, and their conversions never cross
// lanes.  A chunk is three dependent products: (kS)ᵀ = Sᵀkᵀ, wᵀ = (vᵀ −
// (kS)ᵀe^b)(Tβ)ᵀ, and wᵀk for the new state; everything else (the gram matrix and the
// inverse of the chunk after next, the output) runs beside them.
//
// Rounding.  The state, sums, decays, A and T are fp32.  As MMA operands S, kS, w and T
// are split into three bf16 parts, which keep 24 bits, and those of their products are
// taken that reach 2^-24.  What the output alone sees, which is bf16, goes by two parts
// (2^-16): S for q·S, w and P for P·w.  Whenever the tensor cores add to a sum they cut it
// towards zero, so small parts are added first: the state is then 1.5e-7 off after 4096 or
// 16384 tokens (fp32 products 1.7e-7), 1.0e-6 with the large parts first.  With two parts
// of S, kS and w and one of P it was 2.9e-6, the output off by 1.3 times its own
// rounding, and 4×4096 tokens of 32 heads took 283 µs, where three took 321.
//
// A NaN or infinity of a token would reach the earlier tokens of its chunk, as 0·NaN.  The
// warps of S look at w before anything goes by it, and walk a chunk in which it is not
// finite token by token instead (replay).  Columns of v that were spoilt before do not
// count, since they stay so: a sequence has few such chunks, 127 µs each.
//
// Roles: warps 0-7 S (two per quarter of the rows), 8-11 and 12-15 T and P of every
// other chunk, 16-19 the output, 20 loads, 21 MMAs, 22 and 23 decays and lengths.  Their loops
// are kept rolled where they can be: five roles at once run from one instruction
// cache, and unrolled throughout the kernel spent twice as long on fetching as on
// issuing (4×4096 tokens of 32 heads in 490 µs).
//
// What bounds it: the latency of a chunk's chain, since one CTA has an SM and a chunk waits
// for the state of the one before.  4×4096 tokens of 32 heads (64 chunks for each of 128
// CTAs) take 342 µs, 5.3 µs or some 10000 cycles a chunk, of which the tensor pipe is
// busy 4200, and the four conversions between products (S, k·S, w, and S
// again) with the signals around them take most of the rest; DRAM is at 13 %.
//
// The MMA warp issues what the chain waits for first, and the products beside it into
// its gaps: the small parts of v's share of w while k·S is converted, q·S and the next
// gram matrix while w is.
#include "block.cuh"
#include "internal.h"
#include "tc_pair.cuh"

#include <algorithm>
#include <atomic>
#include <type_traits>

namespace la {
namespace {

using namespace block;
using namespace tc;

using bf16 = __nv_bfloat16;

constexpr int kC = 64;                        // tokens of a chunk
constexpr int kThreads = 24 * 32;
constexpr int kStateWarps = 8, kPrepWarp = 8, kOutWarp = 16, kLoadWarp = 20, kMmaWarp = 21, kFactorWarp = 22;
constexpr int kKQ = 3, kVS = 1, kTok = 3, kPS = 2;   // stages: k and q tiles, v tiles, token factors, P
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kOutRows = 16;                  // tokens that are stored at once
constexpr int kSlab = kC * 128;               // 8 KB: 64 tokens × 64 features
constexpr int kAPitch = 68;                   // floats of a row of A

// Named barriers.
constexpr uint32_t kBarOut = 1, kBarPrep = 2 /* and 3 */, kBarState = 4;

struct alignas(16) TokenFactors {
  // Row i's b and column j's b − log2 r_k, each in two parts: e^{b_i − b_j} r_j is one
  // exponential of their difference.
  float bx[kC], by[kC], cx[kC], cy[kC];
  float far[kC];        // what rows from 32 on make of columns below: e^{b − b_31}, r_k e^{b_31 − b}
  float a[kC], q[kC];   // β r_k, scale r_q: a row of A, of P
  float beta[kC];       // a column of T
  float ks[kC];         // −e^b r_k: a row of k·S
  float left[kC];       // r_k e^{b_C − b}: a row of w for the state
  float out[kC];        // scale r_q e^b: a row of q·S
  Decay carry;          // e^{b_C}
};

struct Bars {
  uint64_t kq_full[kKQ], kq_empty[kKQ], v_full[kVS], v_empty[kVS], f_ready[kTok];
  // by the chunk's parity: each prep warpgroup sees every other one
  uint64_t g_full[2], w_full[2], p_empty[2];
  uint64_t kq_clean, v_clean;                 // the last chunk's rows past the length are zero
  uint64_t g_empty, t_ready, s_ready, ks_full, ks_ready, qs_full, qs_read, w_ready,
      upd_full, pv_full, pv_read, done;
  uint32_t tmem;
  int abort;
  int kq_issued, v_issued;                    // loads
  int replayed[2];                            // by parity: the last chunk that was walked token by token
};

// What the halves of a column of S exchange in replay: sums over their rows.
struct Sums {
  float4 part[32 * kStateWarps];              // k·S, q·S, k·k, q·q
  float qk[32 * kStateWarps];
};

template <int DK> struct Cfg {
  static constexpr int kSlabs = DK / 64;
  static constexpr int kStage = 2 * kSlabs * kSlab;          // k and q: per 64 features, k's rows, then q's
  static constexpr int oV = kKQ * kStage;
  static constexpr int oT = oV + kVS * 2 * kSlab;            // Tβ in three parts
  static constexpr int oP = oT + 3 * kSlab;                  // P in two parts
  static constexpr int oOut = oP + kPS * 2 * kSlab;          // kOutRows tokens, by 64 columns
  static constexpr int oA = oOut + 2 * kOutRows * 128;
  static constexpr int oTok = oA + 2 * kC * kAPitch * 4;     // of each prep warpgroup
  static constexpr int oSums = oTok + kTok * (int)sizeof(TokenFactors);
  static constexpr int oBars = oSums + (int)sizeof(Sums);
  static constexpr int kSmem = 1024 + oBars + (int)sizeof(Bars);
  static_assert(kSmem <= 227 * 1024, "shared memory of a CTA");
  // tensor memory columns
  static constexpr uint32_t SH = 0, SL = DK / 2, UPD = DK, KS = 2 * DK, W = KS + kC, PV = W + kC,
                            G = PV + kC;
  // third parts: of S and of k·S before the update takes their place, of w where S's
  // second part was (q·S has been taken)
  static constexpr uint32_t S3 = UPD, KS3 = UPD, W3 = SL;
  static_assert(G + kC <= 512, "tensor memory");
};

struct TcParams {
  Rows dt, beta;
  const float* a;
  const float* dt_bias;
  const float* state_in;
  float* state_out;
  const int32_t* lengths;
  // sequences in `segs` parts of seg_tokens each: what each but the last makes of a
  // zero state and of the identity, and the states that enter the others
  int segs, seg_tokens;
  float *added, *transition;
  const float* entering;
  const bf16* v;
  int64_t v_sb, v_sn, v_sh;
  bf16* out;
  int64_t out_sb, out_sn, out_sh;
  int n, Hk, Hv, dk, dv, tiles;
  int q_h, q_b, k_h, k_b, v_h, v_b, o_h, o_b;   // 0 for axes that are broadcast or single
  float scale;
  bool gates_f32, softplus, sigmoid, normalize;
  int* status;
};

// A pair of fp32 as two bf16 parts each: hi keeps the leading 8 bits, lo the next 8.
// Returns what hi leaves.
__device__ __forceinline__ f32x2 split1(f32x2 v, uint32_t& hi) {
  float x, y;
  unpack2(v, x, y);
  hi = pack_bf16x2(x, y);
  return fma2(pack2(bf16lo_to_f32(hi), bf16hi_to_f32(hi)), pack2(-1.f, -1.f), v);
}
__device__ __forceinline__ void split2(f32x2 v, uint32_t& hi, uint32_t& lo) {
  float x, y;
  unpack2(split1(v, hi), x, y);
  lo = pack_bf16x2(x, y);
}

// The same with a third part, which keeps the next 8.
__device__ __forceinline__ void split3(f32x2 v, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
  split2(split1(v, hi), mid, lo);
}

// 32 lanes × 8 consecutive columns store (thread i writes lane lane_base + i).
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
                 "=r"(r[7])
               : "r"(taddr));
}

// Two neighbours of what was loaded, as a pair of fp32.
__device__ __forceinline__ f32x2 pair_of(const uint32_t* r, int i) {
  return pack2(__uint_as_float(r[i]), __uint_as_float(r[i + 1]));
}

// The sum of two values that are kept in two parts each.
__device__ __forceinline__ float2 add_parts(float2 a, float2 b) {
  const float s = a.x + b.x, t = s - a.x;
  return make_float2(s, a.y + b.y + ((a.x - (s - t)) + (b.x - t)));
}

// A step size or strength as it is in memory, and its value: a load that is used a
// chunk later, and nothing before that would wait for it.
__device__ __forceinline__ uint32_t gate_bits(const Rows& r, bool f32, int64_t at) {
  return f32 ? static_cast<const uint32_t*>(r.data)[at] : static_cast<const uint16_t*>(r.data)[at];
}
__device__ __forceinline__ float gate_value(uint32_t bits, bool f32) {
  return __uint_as_float(f32 ? bits : bits << 16);
}

// Registers of a thread by role: at launch all have 80, and a warpgroup's share is
// moved where S is held: 2·120 + 2·64 + 56 + 56 = 6·80
// (dk 128), 2·112 + 2·72 + 48 + 64.
template <int N> __device__ __forceinline__ void take_registers() {
  if constexpr (N > 80)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
  else
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

struct Ctx {
  uint8_t* sm;
  Bars* bars;
  TokenFactors* tok;
  uint32_t tmem;
  // the CTA's part of a sequence: its first token, how many exist, how many count
  int b, h, tile, t0, end, live, chunks;
  bool partial;           // rows of the last chunk lie past the length
  bool identity;          // from the identity without v: the transition over the part
  const float* s_in;      // the state before and after, [dk, cols], or nullptr
  float* s_out;
  int cols;
};

// mbar_wait and mbar_wait_drain in line, since the compiler refuses calls beside
// setmaxnreg, and in few instructions.  The bound is a number of tests, of some 50
// cycles each; the kernel's end reports the timeout.
constexpr uint32_t kRounds = 20000;
__device__ __forceinline__ bool round_of_tests(uint64_t* bar, uint32_t parity) {   // 4096 at most
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .u32 n;\n\tmov.u32 n, 4096;\n"
      "W:\n\tmbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t@p bra D;\n\t"
      "sub.u32 n, n, 1;\n\tsetp.ne.u32 q, n, 0;\n\t@q bra W;\n"
      "D:\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool wait_in_line(uint64_t* bar, uint32_t parity, volatile int* abort) {
#pragma unroll 1
  for (uint32_t n = 0; !round_of_tests(bar, parity); ++n)
    if (*abort || n > kRounds) {
      *abort = 1;
      return false;
    }
  return true;
}
__device__ __forceinline__ bool warp_wait_in_line(uint64_t* bar, uint32_t parity, volatile int* abort) {
  return __all_sync(0xffffffffu, wait_in_line(bar, parity, abort));
}
__device__ __forceinline__ void drain_in_line(uint64_t* bar, uint32_t parity) {
#pragma unroll 1
  for (uint32_t n = 0; n < kRounds / 4 && !round_of_tests(bar, parity); ++n) {}
}

// A role that shares no barrier with other warps returns where a wait gives up;
// the others (LA_GO_ON) walk on through their remaining barriers, whose waits then
// end at once: what they write stays within their own buffers and the output.
#define LA_WAIT_AT(bar, parity) \
  if (!warp_wait_in_line(bar, (parity) & 1, abort)) return
#define LA_WAIT(bar, parity) LA_WAIT_AT(&x.bars->bar, parity)
#define LA_GO_ON(bar, parity) warp_wait_in_line(&x.bars->bar, (parity) & 1, abort)

// ------------------------------------------------------------------ loads

// (whole warp)
template <int DK, bool SUMMARY>
__device__ __forceinline__ void role_load(const Ctx& x, const TcParams& p, const CUtensorMap* mq,
                                          const CUtensorMap* mk, const CUtensorMap* mv, int lane) {
  using F = Cfg<DK>;
  volatile int* abort = &x.bars->abort;
  const int hk = x.h / (p.Hv / p.Hk);
  const int vslabs = p.dv - x.tile * 128 > 64 ? 2 : 1;
  // the rows past the length may hold anything: zeros, so that they add nothing
  const int last = x.live - (x.chunks - 1) * kC;
  auto clear = [&](uint8_t* slab) {
    for (int i = last * 8 + lane; i < kC * 8; i += 32)
      *reinterpret_cast<uint4*>(slab + i * 16) = make_uint4(0, 0, 0, 0);
  };
  // k and q a chunk ahead of v, whose one stage is given back in the middle of a chunk
#pragma unroll 1
  for (int g = 0; g <= x.chunks; ++g) {
    if (g < x.chunks) {
      const int s = g % kKQ, t = x.t0 + g * kC;
      if (g >= kKQ) LA_WAIT(kq_empty[s], g / kKQ - 1);
      if (lane == 0) {
        uint8_t* to = x.sm + s * F::kStage;
        const bool ok = LA_DCHECK(p.status, t >= x.t0 && t < x.t0 + x.live && hk < p.Hk, 62);
        mbar_arrive_expect_tx(&x.bars->kq_full[s], ok ? F::kStage : 0);
#pragma unroll
        for (int i = 0; ok && i < F::kSlabs; ++i) {
          tma_load_4d(to + i * 2 * kSlab, mk, &x.bars->kq_full[s], i * 64, hk * p.k_h, t, x.b * p.k_b);
          tma_load_4d(to + i * 2 * kSlab + kSlab, mq, &x.bars->kq_full[s], i * 64, hk * p.q_h, t, x.b * p.q_b);
        }
        x.bars->kq_issued = g + 1;
      }
      if (x.partial && g == x.chunks - 1) {   // (its gram matrix comes before its v)
        LA_WAIT(kq_full[s], g / kKQ);
        for (int i = 0; i < 2 * F::kSlabs; ++i) clear(x.sm + s * F::kStage + i * kSlab);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&x.bars->kq_clean);
      }
    }
    const int c = g - 1, vs = c % kVS, t = x.t0 + c * kC;
    if (c < 0 || (SUMMARY && x.identity)) continue;
    if (c >= kVS) LA_WAIT(v_empty[vs], c / kVS - 1);
    if (lane == 0) {
      uint8_t* to = x.sm + F::oV + vs * 2 * kSlab;
      const bool ok = LA_DCHECK(p.status, t >= x.t0 && t < x.t0 + x.live && x.tile * 128 + (vslabs - 1) * 64 < p.dv, 62);
      mbar_arrive_expect_tx(&x.bars->v_full[vs], ok ? vslabs * kSlab : 0);
      for (int i = 0; ok && i < vslabs; ++i)
        tma_load_4d(to + i * kSlab, mv, &x.bars->v_full[vs], x.tile * 128 + i * 64, x.h * p.v_h, t, x.b * p.v_b);
    }
    if (lane == 0) x.bars->v_issued = c + 1;
  }
  if (!x.partial || (SUMMARY && x.identity)) return;
  const int c = x.chunks - 1;
  LA_WAIT(v_full[c % kVS], c / kVS);
  for (int i = 0; i < vslabs; ++i) clear(x.sm + F::oV + (c % kVS * 2 + i) * kSlab);
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) mbar_arrive(&x.bars->v_clean);
}

// ------------------------------------------------------------------ products

// A shared-memory operand: of its descriptor (smem_desc) the low word, which holds the
// address, and the high one, which is the same for a layout.
struct Operand {
  uint32_t lo, hi;
  __device__ __forceinline__ Operand(uint32_t saddr, uint32_t lbo) {
    const uint64_t d = smem_desc(saddr, lbo, 1024, kSwizzle128B);
    lo = (uint32_t)d, hi = (uint32_t)(d >> 32);
  }
};

// D[tmem] (+)= A·B, B `at_b` bytes (and A `at_a`) into its operand.
template <bool ACC>
__device__ __forceinline__ void issue_ss(uint32_t d, const Operand& a, uint32_t at_a, const Operand& b, uint32_t at_b,
                                         uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tsetp.ne.b32 p, %6, 0;\n\tmov.b64 x, {%1, %2};\n\t"
      "mov.b64 y, {%3, %4};\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %5, p;\n\t}" ::"r"(d),
      "r"(a.lo + at_a / 16), "r"(a.hi), "r"(b.lo + at_b / 16), "r"(b.hi), "r"(idesc), "n"(ACC ? 1 : 0)
      : "memory");
}
template <bool ACC>
__device__ __forceinline__ void issue_ts(uint32_t d, uint32_t a, const Operand& b, uint32_t at_b, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b64 y, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b.lo + at_b / 16), "r"(b.hi), "r"(idesc), "n"(ACC ? 1 : 0)
      : "memory");
}
// (whole warp)  The loops over products are unrolled: an MMA of these takes 32 to 64
// cycles, and with its operands' addresses computed in a loop it is issued in 130.
template <int DK, bool SUMMARY>
__device__ __forceinline__ void role_mma(const Ctx& x, const TcParams& p) {
  using F = Cfg<DK>;
  Bars* bars = x.bars;
  volatile int* abort = &bars->abort;
  const uint32_t tmem = x.tmem, base = smem_u32(x.sm);
  constexpr uint32_t id_nn = idesc_bf16_f32(128, kC, false, false);   // K-major A and B, 64 columns
  constexpr uint32_t id_v = idesc_bf16_f32(128, kC, true, false);     // vᵀ from [token][column]
  constexpr uint32_t id_upd = idesc_bf16_f32(128, DK, false, true);   // k as [token][feature]
  constexpr int KD = DK / 16, KC = kC / 16;
  const uint32_t lead = elect_one();
  const Operand T(base + F::oT, 16);
  // K-step k of a tile with 64 features per slab
  auto kstep = [](int k) { return (uint32_t)((k >> 2) * 2 * kSlab + (k & 3) * 32); };
  // S's second and first parts with k (at 0) or q; the second on top of the third
  auto of_state = [&](auto acc, uint32_t to, const Operand& b, uint32_t at) {
    issue_ts<decltype(acc)::value>(to, tmem + F::SL, b, at, id_nn);
#pragma unroll
    for (int i = 1; i < KD; ++i) issue_ts<true>(to, tmem + F::SL + i * 8, b, at + kstep(i), id_nn);
#pragma unroll
    for (int i = 0; i < KD; ++i) issue_ts<true>(to, tmem + F::SH + i * 8, b, at + kstep(i), id_nn);
  };
  // S's third part is in two halves, each where its warps have read the update
  auto third = [](int k) { return (uint32_t)(k / (KD / 2) * (DK / 2) + k % (KD / 2) * 8); };
  // K-step k of (kS)ᵀ or wᵀ: 16 tokens' first parts, then their second parts
  auto tokens = [](int k) { return (uint32_t)(k * 16); };
#pragma unroll 1
  for (int c = -2; c < x.chunks; ++c) {
    if (c >= 0) {
      const uint32_t kq = base + c % kKQ * F::kStage;
      const Operand K(kq, 16);
      // (kS)ᵀ = Sᵀ kᵀ
      LA_WAIT(s_ready, c);
      tc_fence_after();
      if (lead) {
        issue_ts<false>(tmem + F::KS, tmem + F::S3, K, 0, id_nn);
#pragma unroll
        for (int i = 1; i < KD; ++i) issue_ts<true>(tmem + F::KS, tmem + F::S3 + third(i), K, kstep(i), id_nn);
        of_state(std::true_type(), tmem + F::KS, K, 0);
        mma_commit(&bars->ks_full);
      }
      __syncwarp();
      // the small parts of wᵀ = vᵀ (Tβ)ᵀ, whose columns (P w)ᵀ has read, while (kS)ᵀ is made an operand
      LA_WAIT(t_ready, c);
      if (!(SUMMARY && x.identity)) {
        LA_WAIT(v_full[c % kVS], c / kVS);
        if (x.partial && c == x.chunks - 1) LA_WAIT(v_clean, 0);
      }
      if (!SUMMARY && c >= 1) LA_WAIT(pv_full, c - 1);   // (else the state's warps have read them)
      tc_fence_after();
      if (lead) {
        const Operand V(base + F::oV + c % kVS * 2 * kSlab, kSlab);
        issue_ss<false>(tmem + F::W, V, 0, T, 2 * kSlab, id_v);
#pragma unroll
        for (int i = 1; i < 2 * KC; ++i)
          issue_ss<true>(tmem + F::W, V, i % KC * 2048, T, (2 - i / KC) * kSlab + i % KC * 32, id_v);
      }
      __syncwarp();
      // wᵀ −= (e^b kS)ᵀ (Tβ)ᵀ, of the parts whose products reach 2^-24, and v's large one
      LA_WAIT(ks_ready, c);
      tc_fence_after();
      if (lead) {
        const Operand V(base + F::oV + c % kVS * 2 * kSlab, kSlab);
#pragma unroll
        for (int sum = 2; sum >= 0; --sum)
#pragma unroll
          for (int a = sum; a >= 0; --a)
#pragma unroll
            for (int k = 0; k < KC; ++k)
              issue_ts<true>(tmem + F::W, tmem + (a < 2 ? F::KS + tokens(k) + a * 8 : F::KS3 + k * 8), T,
                             (sum - a) * kSlab + k * 32, id_nn);
#pragma unroll
        for (int k = 0; k < KC; ++k) issue_ss<true>(tmem + F::W, V, k * 2048, T, k * 32, id_v);
        mma_commit(&bars->v_empty[c % kVS]);
        mma_commit(&bars->w_full[c & 1]);
      }
      __syncwarp();
      // (qS)ᵀ
      if constexpr (!SUMMARY) {
        if (c >= 1) LA_WAIT(pv_read, c - 1);
        tc_fence_after();
        if (lead) {
          of_state(std::false_type(), tmem + F::PV, K, kSlab);
          mma_commit(&bars->qs_full);
        }
        __syncwarp();
      }
    }
    // while w is on its way: [k; q]·kᵀ of the chunk after next
    if (c + 2 < x.chunks) {
      const int g = c + 2;
      LA_WAIT(kq_full[g % kKQ], g / kKQ);
      if (x.partial && g == x.chunks - 1) LA_WAIT(kq_clean, 0);
      if (g >= 1) LA_WAIT(g_empty, g - 1);
      tc_fence_after();
      if (lead) {
        const Operand d(base + g % kKQ * F::kStage, 16);
        issue_ss<false>(tmem + F::G, d, 0, d, 0, id_nn);
#pragma unroll
        for (int k = 1; k < KD; ++k) issue_ss<true>(tmem + F::G, d, kstep(k), d, kstep(k), id_nn);
        mma_commit(&bars->g_full[g & 1]);
      }
      __syncwarp();
    }
    if (c >= 0) {
      // the state's wᵀk
      LA_WAIT(w_ready, c);
      tc_fence_after();
      if (lead) {
        const Operand Kt(base + c % kKQ * F::kStage, 2 * kSlab);
        issue_ts<false>(tmem + F::UPD, tmem + F::W3, Kt, 0, id_upd);
#pragma unroll
        for (int k = 1; k < KC; ++k) issue_ts<true>(tmem + F::UPD, tmem + F::W3 + k * 8, Kt, k * 2048, id_upd);
#pragma unroll
        for (int i = 0; i < 2 * KC; ++i)
          issue_ts<true>(tmem + F::UPD, tmem + F::KS + tokens(i % KC) + (1 - i / KC) * 8, Kt, i % KC * 2048, id_upd);
        mma_commit(&bars->upd_full);
        if (SUMMARY) mma_commit(&bars->kq_empty[c % kKQ]);
      }
      __syncwarp();
      // (P w)ᵀ on top of what the output's warps have put there
      if constexpr (!SUMMARY) {
        LA_WAIT(qs_read, c);
        tc_fence_after();
        if (lead) {
          // hi·lo, lo·hi, hi·hi
          const Operand P(base + F::oP + c % kPS * 2 * kSlab, 16);
#pragma unroll
          for (int i = 0; i < 3 * KC; ++i)
            issue_ts<true>(tmem + F::PV, tmem + F::W + tokens(i % KC) + (i / KC == 1 ? 8 : 0), P,
                           (i < KC ? kSlab : 0) + i % KC * 32, id_nn);
          mma_commit(&bars->pv_full);
          mma_commit(&bars->p_empty[c & 1]);
          mma_commit(&bars->kq_empty[c % kKQ]);   // and the chunk's factors
        }
        __syncwarp();
      }
    }
  }
}

// ------------------------------------------------------------------ the state

// Whether v holds for any thread of the state's warps.
__device__ __forceinline__ bool any_of_state(bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)v), "n"(kBarState), "n"(32 * kStateWarps)
      : "memory");
  return r != 0;
}

// (all the state's warps)  Chunk c token by token, outputs too, and what becomes of S: w_t =
// β_t(v_t − k_t(α_t S)), S = α_t S + k_tᵀ w_t, o_t = scale·q_t S.  A thread has a column of v
// (a row of Sᵀ) with half of dk, in tensor memory at `mine` so that all of this stays small
// beside the loop that it leaves, and exchanges its sums with the thread that has the other
// half.  k and q are still where the products read them.  Returns whether the column is spoilt.
template <int DK, bool SUMMARY>
__device__ __forceinline__ bool replay(const Ctx& x, const TcParams& p, int c, int row, int half, uint32_t mine) {
  using F = Cfg<DK>;
  constexpr int kCols = DK / 2;
  volatile int* abort = &x.bars->abort;
  Sums& sums = *reinterpret_cast<Sums*>(x.sm + F::oSums);
  // nothing of this is to be computed ahead, where it would take registers from the loop
  // (4×4096 tokens of 32 heads: 342 µs, 347 without this line)
  int h = x.h, b = x.b;
  asm volatile("" : "+r"(h), "+r"(b), "+r"(row), "+r"(half), "+r"(c), "+r"(mine));
  const int me = half * 128 + row, other = me ^ 128;
  const int col = x.tile * 128 + row, k0 = half * kCols;
  const bool valued = !(SUMMARY && x.identity) && col < p.dv;
  const float rate = p.a[h], bias = p.dt_bias ? p.dt_bias[h] : 0.f;
  const uint32_t stage = smem_u32(x.sm + c % kKQ * F::kStage) + k0 / 64 * 2 * kSlab;
  const int64_t t0 = (int64_t)x.t0 + c * kC;
  const bf16* v = p.v + b * p.v_sb + t0 * p.v_sn + h * p.v_sh + col;
  bf16* o = p.out + b * p.out_sb + t0 * p.out_sn + h * p.out_sh + col;
  const int rows = min(kC, x.end - c * kC), count = min(kC, x.live - c * kC);
  const f32x2 zero = pack2(0.f, 0.f);
  auto both = [](f32x2 v) {
    float lo, hi;
    unpack2(v, lo, hi);
    return lo + hi;
  };
  LA_GO_ON(kq_full[c % kKQ], c / kKQ);
#pragma unroll 1
  for (int t = 0; t < count; ++t) {
    float d = gate_value(gate_bits(p.dt, p.gates_f32, b * p.dt.sb + (t0 + t) * p.dt.sn + h), p.gates_f32) + bias;
    if (p.softplus) d = softplus(d);
    const Decay alpha = decay_of(d == 0.f ? 0.f : d * rate);
    float beta = gate_value(gate_bits(p.beta, p.gates_f32, b * p.beta.sb + (t0 + t) * p.beta.sn + h), p.gates_f32);
    if (p.sigmoid) beta = rcp_f32(1.f + ex2_f32(-kLog2e * beta));
    const float vt = valued ? __bfloat162float(v[t * p.v_sn]) : 0.f;
    f32x2 ks = 0, qs = 0, kk = 0, qq = 0, qk = 0;
#pragma unroll 1
    for (int i = 0; i < kCols; i += 8) {
      uint32_t r[8];
      tmem_ld8(mine + i, r);
      tmem_ld_wait();
      const uint32_t at = stage + sw_chunk(kC, t, 0, (k0 + i) / 8 % 8);
      const uint4 kv = lds128(at), qv = lds128(at + kSlab);
      const uint32_t kw[4] = {kv.x, kv.y, kv.z, kv.w}, qw[4] = {qv.x, qv.y, qv.z, qv.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const f32x2 k = pack2(bf16lo_to_f32(kw[j]), bf16hi_to_f32(kw[j]));
        const f32x2 q = pack2(bf16lo_to_f32(qw[j]), bf16hi_to_f32(qw[j]));
        ks = fma2(k, pair_of(r, 2 * j), ks), qs = fma2(q, pair_of(r, 2 * j), qs);
        kk = fma2(k, k, kk), qq = fma2(q, q, qq), qk = fma2(q, k, qk);
      }
    }
    float4 sum = make_float4(both(ks), both(qs), both(kk), both(qq));
    sums.part[me] = sum, sums.qk[me] = both(qk);
    named_bar_sync(kBarState, 32 * kStateWarps);
    const float4 more = sums.part[other];
    sum.x += more.x, sum.y += more.y, sum.z += more.z, sum.w += more.w;
    const float qks = both(qk) + sums.qk[other];
    named_bar_sync(kBarState, 32 * kStateWarps);   // before the next token's
    const float rk = p.normalize ? rsqrtf(sum.z + 1e-6f) : 1.f;
    const float rq = p.scale * (p.normalize ? rsqrtf(sum.w + 1e-6f) : 1.f);
    const float w = rk * (beta * (vt - decayed(alpha, rk * sum.x)));
    if (!SUMMARY && half == 0 && valued) o[t * p.out_sn] = __float2bfloat16_rn(rq * decayed(alpha, sum.y, qks * w));
    __syncwarp();
#pragma unroll 1
    for (int i = 0; i < kCols; i += 8) {
      uint32_t r[8];
      tmem_ld8(mine + i, r);
      tmem_ld_wait();
      const uint4 kv = lds128(stage + sw_chunk(kC, t, 0, (k0 + i) / 8 % 8));
      const uint32_t kw[4] = {kv.x, kv.y, kv.z, kv.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        r[2 * j] = __float_as_uint(decayed(alpha, __uint_as_float(r[2 * j]), bf16lo_to_f32(kw[j]) * w));
        r[2 * j + 1] = __float_as_uint(decayed(alpha, __uint_as_float(r[2 * j + 1]), bf16hi_to_f32(kw[j]) * w));
      }
      tmem_st8(mine + i, r);
    }
    tmem_st_wait();
  }
  if (!SUMMARY && half == 0 && valued)
    for (int t = count; t < rows; ++t) o[t * p.out_sn] = __float2bfloat16_rn(0.f);
  __syncwarp();
  f32x2 seen = 0;
#pragma unroll 1
  for (int i = 0; i < kCols; i += 8) {
    uint32_t r[8];
    tmem_ld8(mine + i, r);
    tmem_ld_wait();
#pragma unroll
    for (int j = 0; j < 4; ++j) seen = fma2(pair_of(r, 2 * j), zero, seen);
  }
  sums.qk[me] = both(seen);   // 0, or NaN
  named_bar_sync(kBarState, 32 * kStateWarps);
  const float found = both(seen) + sums.qk[other];
  named_bar_sync(kBarState, 32 * kStateWarps);
  return found != 0.f;
}

// Warp w has rows 32(w % 4) … of Sᵀ (columns of v) and half of its columns.
template <int DK, bool SUMMARY>
__device__ __forceinline__ void role_state(const Ctx& x, const TcParams& p, int warp, int lane) {
  using F = Cfg<DK>;
  constexpr int kCols = DK / 2;
  Bars* bars = x.bars;
  volatile int* abort = &bars->abort;
  const int half = warp / 4, k0 = half * kCols;
  const uint32_t at = tmem_addr(x.tmem, warp % 4 * 32, 0);
  const int col = (SUMMARY && x.identity ? 0 : x.tile * 128) + warp % 4 * 32 + lane;
  // between global memory and S by way of the columns of the update, so that these
  // loops stay small
  const uint32_t mine = at + F::UPD + k0;
  const int64_t first = (int64_t)k0 * x.cols + col;
  const int rows = min(kCols, p.dk - k0);   // multiples of 8
#pragma unroll 1
  for (int i = 0; i < kCols; i += 8) {
    uint32_t r[8] = {};
    if (SUMMARY && x.identity) {
#pragma unroll
      for (int j = 0; j < 8; ++j) r[j] = __float_as_uint(k0 + i + j == col ? 1.f : 0.f);
    } else if (x.s_in && col < x.cols && i < rows) {
#pragma unroll
      for (int j = 0; j < 8; ++j) r[j] = __float_as_uint(x.s_in[first + (int64_t)(i + j) * x.cols]);
    }
    __syncwarp();
    tmem_st8(mine + i, r);
  }
  tmem_st_wait();
  int c = 0;
  bool again = false;    // chunk c was walked token by token
  bool spoilt = false;   // this row of Sᵀ is known to hold a NaN or infinity
#pragma unroll 1
  while (true) {
    f32x2 S[kCols / 2];
#pragma unroll
    for (int j = 0; j < kCols; j += 32) {
      uint32_t r[32];
      tmem_ld32(mine + j, r);
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 16; ++i) S[j / 2 + i] = pair_of(r, 2 * i);
    }
    if (again) {   // its products go on, over what is not used
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->w_ready);
      LA_GO_ON(upd_full, c);
      tc_fence_after();
      again = false;
      ++c;
    }
#pragma unroll 1
    for (; c < x.chunks; ++c) {
      // S as the next products' operand
#pragma unroll
      for (int j = 0; j < kCols; j += 16) {
        uint32_t hi[8], mid[8], lo[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) split3(S[j / 2 + i], hi[i], mid[i], lo[i]);
        tmem_st8(at + F::SH + (k0 + j) / 2, hi);
        tmem_st8(at + F::SL + (k0 + j) / 2, mid);
        tmem_st8(at + F::S3 + k0 + j / 2, lo);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->s_ready);
      const TokenFactors& tok = x.tok[c % kTok];   // overwritten after the chunk's last product
      LA_GO_ON(f_ready[c % kTok], c / kTok);
      // (kS)ᵀ, then wᵀ, times a factor of each token as operands in three parts, 16 tokens at a time
      const f32x2 keep = pack2(tok.carry.keep, tok.carry.keep), more = pack2(tok.carry.more, tok.carry.more);
      f32x2 seen = 0;        // NaN once one of them is not finite
#pragma unroll 1
      for (int of_w = 0; of_w < 2; ++of_w) {
        warp_wait_in_line(of_w ? &bars->w_full[c & 1] : &bars->ks_full, (of_w ? c / 2 : c) & 1, abort);
        tc_fence_after();
        const float* factors = of_w ? tok.left : tok.ks;
#pragma unroll 1
        for (int t = half * 32; t < half * 32 + 32; t += 16) {
          uint32_t r[16], hi[8], mid[8], lo[8];
          tmem_ld16(at + (of_w ? F::W : F::KS) + t, r);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(factors + t + 2 * i);
            const f32x2 a = mul2(pair_of(r, 2 * i), f.x), b = mul2(pair_of(r, 2 * i + 2), f.y);
            split3(a, hi[i], mid[i], lo[i]);
            split3(b, hi[i + 1], mid[i + 1], lo[i + 1]);
            seen = fma2(a, pack2(0.f, 0.f), fma2(b, pack2(0.f, 0.f), seen));
          }
          tmem_st8(at + F::KS + t, hi);
          tmem_st8(at + F::KS + t + 8, mid);
          if (!SUMMARY && of_w) {   // for the output
#pragma unroll
            for (int i = 0; i < 8; ++i) split2(pair_of(r, 2 * i), hi[i], mid[i]);
            tmem_st8(at + F::W + t, hi);
            tmem_st8(at + F::W + t + 8, mid);
            LA_GO_ON(qs_full, c);   // (complete by now: q·S follows w on the tensor cores)
            tc_fence_after();
          }
          tmem_st8(at + (of_w ? F::W3 : F::KS3) + t / 2, lo);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (of_w) {
          float e, o;
          unpack2(seen, e, o);
          again = any_of_state(e + o != 0.f && !spoilt);
          if (again) break;
        }
        if (lane == 0) mbar_arrive(of_w ? &bars->w_ready : &bars->ks_ready);
      }
      if (again) break;
      LA_GO_ON(upd_full, c);
      tc_fence_after();
#pragma unroll
      for (int j = 0; j < kCols; j += 32) {
        uint32_t r[32];
        tmem_ld32(at + F::UPD + k0 + j, r);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; ++i)
          S[j / 2 + i] = fma2(S[j / 2 + i], keep, fma2(S[j / 2 + i], more, pair_of(r, 2 * i)));
      }
    }
#pragma unroll
    for (int j = 0; j < kCols; j += 8) {
      uint32_t r[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float lo, hi;
        unpack2(S[j / 2 + i], lo, hi);
        r[2 * i] = __float_as_uint(lo), r[2 * i + 1] = __float_as_uint(hi);
      }
      tmem_st8(mine + j, r);
    }
    tmem_st_wait();
    if (!again) break;
    if (threadIdx.x == 0) *(volatile int*)&bars->replayed[c & 1] = c;   // (its output is not to be stored)
    __syncwarp();
    spoilt = replay<DK, SUMMARY>(x, p, c, warp % 4 * 32 + lane, half, mine);
    __syncwarp();
  }
  if (!x.s_out) return;
#pragma unroll 1
  for (int i = 0; i < rows; i += 8) {
    uint32_t r[8];
    tmem_ld8(mine + i, r);
    tmem_ld_wait();
    if (col < x.cols)
#pragma unroll
      for (int j = 0; j < 8; ++j) x.s_out[first + (int64_t)(i + j) * x.cols] = __uint_as_float(r[j]);
    __syncwarp();
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
  const uint32_t mine = smem_u32(stage) + d / 64 * kOutRows * 128 + d % 64 * 2;
#pragma unroll 1
  for (int c = 0; c < x.chunks; ++c) {
    const TokenFactors& tok = x.tok[c % kTok];
    // scale e^{b_i} q_i S is what P·w is added to
    LA_GO_ON(f_ready[c % kTok], c / kTok);
    LA_GO_ON(qs_full, c);
    tc_fence_after();
#pragma unroll 1
    for (int j = 0; j < kC; j += 32) {
      uint32_t r[32];
      tmem_ld32(at + F::PV + j, r);
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
    const int rows = min(kC, x.live - c * kC);
    const bool stored = *(volatile int*)&bars->replayed[c & 1] == c;
#pragma unroll 1
    for (int j = 0; j < kC; j += kOutRows) {
      uint32_t v[kOutRows];
      tmem_ld16(at + F::PV + j, v);
      tmem_ld_wait();
      if (j + kOutRows == kC) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->pv_read);
      }
      if (lead) tma_store_wait_read0();
      named_bar_sync(kBarOut, 128);
#pragma unroll
      for (int i = 0; i < kOutRows; i += 2) {
        const uint32_t o = pack_bf16x2(__uint_as_float(v[i]), __uint_as_float(v[i + 1]));
        asm volatile("st.shared.b16 [%0], %1;" ::"r"(mine + i * 128), "h"((uint16_t)(o & 0xffffu)) : "memory");
        asm volatile("st.shared.b16 [%0], %1;" ::"r"(mine + i * 128 + 128), "h"((uint16_t)(o >> 16)) : "memory");
      }
      if (rows < kC)   // what q·S made of the rows past the length
#pragma unroll 1
        for (int i = max(0, rows - j); i < kOutRows; ++i)
          asm volatile("st.shared.b16 [%0], %1;" ::"r"(mine + i * 128), "h"((uint16_t)0) : "memory");
      fence_proxy_async_smem();
      named_bar_sync(kBarOut, 128);
      if (lead) {
        for (int i = 0; i < 2; ++i) {
          const int col = x.tile * 128 + i * 64;
          const int t = x.t0 + c * kC + j;
          if (!stored && col < p.dv && t < p.n && LA_DCHECK(p.status, t >= x.t0 && min(t + kOutRows, p.n) <= x.t0 + x.end, 61))
            tma_store_4d(mo, stage + i * kOutRows * 128, col, x.h * p.o_h, t, x.b * p.o_b);
        }
        tma_store_commit();
      }
    }
  }
  if (lead) tma_store_wait0();
  // chunks past the length
  const int cols = min(128, p.dv - x.tile * 128) / 8, lanes = (warp - kOutWarp) * 32 + lane;
  bf16* o = p.out + x.b * p.out_sb + x.t0 * p.out_sn + x.h * p.out_sh + x.tile * 128;
  for (int64_t t = x.chunks * kC + lanes / 16; t < x.end; t += 8)
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

// One column of the inverse of a unit lower triangular 16×16 block, whose diagonal
// holds zeros: v_i = [i is the column] − Σ_{j<i} A_ij v_j, two terms at a time.
__device__ __forceinline__ void invert16(float* A, int lane) {
  f32x2 v[8] = {};
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    f32x2 s = pack2(lane == i ? -1.f : 0.f, 0.f);
#pragma unroll
    for (int j = 0; j < i; j += 4) {
      const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(A + i * kAPitch + j);
      s = fma2(a.x, v[j / 2], s);
      if (j + 2 < i) s = fma2(a.y, v[j / 2 + 1], s);
    }
    float s0, s1, lo, hi;
    unpack2(s, s0, s1);
    unpack2(v[i / 2], lo, hi);
    v[i / 2] = i % 2 ? pack2(lo, -(s0 + s1)) : pack2(-(s0 + s1), 0.f);
  }
  __syncwarp();
  if (lane < 16)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float lo, hi;
      unpack2(v[i], lo, hi);
      A[2 * i * kAPitch + lane] = lo;
      A[(2 * i + 1) * kAPitch + lane] = hi;
    }
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

// Decays, strengths and lengths of each chunk's tokens, of k by warp 23 and of q by
// warp 22; lane i has tokens i and i + 32.
template <int DK>
__device__ __forceinline__ void role_factors(const Ctx& x, const TcParams& p, int warp, int lane) {
  using F = Cfg<DK>;
  volatile int* abort = &x.bars->abort;
  const bool keys = warp == kFactorWarp + 1;
  const float rate = p.a[x.h], bias = p.dt_bias ? p.dt_bias[x.h] : 0.f;
  uint32_t dt[2], be[2];
  auto fetch = [&](int c) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const bool in = c * kC + i * 32 + lane < x.live;
      const int64_t t = (int64_t)x.t0 + c * kC + i * 32 + lane;
      dt[i] = in ? gate_bits(p.dt, p.gates_f32, x.b * p.dt.sb + t * p.dt.sn + x.h) : 0u;
      be[i] = in ? gate_bits(p.beta, p.gates_f32, x.b * p.beta.sb + t * p.beta.sn + x.h) : 0u;
    }
  };
  if (x.chunks) fetch(0);
#pragma unroll 1
  for (int c = 0; c < x.chunks; ++c) {
    TokenFactors& tok = x.tok[c % kTok];
    const int count = x.live - c * kC;
    float2 b[2];                        // inclusive sums
    float beta[2], r[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const bool live = i * 32 + lane < count;
      b[i] = make_float2(live ? log2_decay(p, gate_value(dt[i], p.gates_f32), bias, rate) : 0.f, 0.f);
      const float strength = gate_value(be[i], p.gates_f32);
      beta[i] = !live ? 0.f : p.sigmoid ? rcp_f32(1.f + ex2_f32(-kLog2e * strength)) : strength;
    }
    if (c + 1 < x.chunks) fetch(c + 1);
#pragma unroll 1
    for (int m = 1; m < 32; m *= 2)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float2 o = make_float2(__shfl_up_sync(0xffffffffu, b[i].x, m), __shfl_up_sync(0xffffffffu, b[i].y, m));
        if (lane >= m) b[i] = add_parts(o, b[i]);
      }
    const float2 mid = make_float2(__shfl_sync(0xffffffffu, b[0].x, 31), __shfl_sync(0xffffffffu, b[0].y, 31));
    b[1] = add_parts(b[1], mid);
    const float2 last = make_float2(__shfl_sync(0xffffffffu, b[1].x, 31), __shfl_sync(0xffffffffu, b[1].y, 31));
    LA_WAIT(kq_full[c % kKQ], c / kKQ);
    r[0] = r[1] = 1.f;
    if (p.normalize) {
      const uint32_t slab = smem_u32(x.sm + c % kKQ * F::kStage + !keys * kSlab);
      f32x2 sum[2][2] = {};
#pragma unroll 2
      for (int j = 0; j < 8 * F::kSlabs; ++j) {
        const uint32_t at = slab + (j / 8) * 2 * kSlab + sw_chunk(kC, lane, 0, j % 8);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint4 v = lds128(at + i * 32 * 128);
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const f32x2 f = pack2(bf16lo_to_f32(w[e]), bf16hi_to_f32(w[e]));
            sum[i][e & 1] = fma2(f, f, sum[i][e & 1]);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float lo, hi;
        unpack2(add2(sum[i][0], sum[i][1]), lo, hi);
        r[i] = rsqrtf(lo + hi + 1e-6f);
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int t = i * 32 + lane;
      if (t >= count) r[i] = 0.f;
      const float eb = ex2_f32(b[i].x + b[i].y);
      if (keys) {
        const float off = (mid.x - b[i].x) + (mid.y - b[i].y);
        tok.bx[t] = tok.cx[t] = b[i].x;
        tok.by[t] = b[i].y;
        tok.cy[t] = b[i].y - lg2_f32(r[i]);
        tok.far[t] = i ? ex2_f32(-off) : r[i] * ex2_f32(off);
        tok.a[t] = beta[i] * r[i];
        tok.beta[t] = beta[i];
        tok.ks[t] = -eb * r[i];
        tok.left[t] = r[i] * ex2_f32((last.x - b[i].x) + (last.y - b[i].y));
      } else {
        tok.out[t] = p.scale * r[i] * eb;
        tok.q[t] = p.scale * r[i];
      }
    }
    if (keys && lane == 0) tok.carry = decay_of(kLn2 * (last.x + last.y));
    __syncwarp();
    if (lane == 0) mbar_arrive(&x.bars->f_ready[c % kTok]);
  }
}

// Thread t < 64 has token t's row of k·kᵀ, thread 64 + t that of q·kᵀ.
template <int DK, bool SUMMARY>
__device__ __forceinline__ void role_prep(const Ctx& x, const TcParams& p, int warp, int lane) {
  using F = Cfg<DK>;
  Bars* bars = x.bars;
  volatile int* abort = &bars->abort;
  const int group = (warp - kPrepWarp) / 4, t = warp % 4 * 32 + lane, row = t % kC;
  const uint32_t bar = kBarPrep + group;
  const bool keys = t < kC;
  const uint32_t at = tmem_addr(x.tmem, warp % 4 * 32, 0);
  float* A = reinterpret_cast<float*>(x.sm + F::oA) + group * kC * kAPitch;
#pragma unroll 1
  for (int c = group; c < x.chunks; c += 2) {
    const TokenFactors& tok = x.tok[c % kTok];
    LA_GO_ON(f_ready[c % kTok], c / kTok);
    const float bx = tok.bx[row], by = tok.by[row];
    const float factor = keys ? tok.a[row] : tok.q[row];
    const int upto = row - keys;      // A below the diagonal, P with it
    const uint32_t P = smem_u32(x.sm + F::oP + c % kPS * 2 * kSlab);
    named_bar_sync(bar, 128);    // the last chunk's T has been read from A
    // this row of A, or of P, 16 columns at a time
    LA_GO_ON(g_full[c & 1], c / 2);
    if (!SUMMARY && !keys && c >= kPS) LA_GO_ON(p_empty[c & 1], c / kPS - 1);
    tc_fence_after();
    const float far = factor * tok.far[row];
    const f32x2 f2 = pack2(factor, factor), bx2 = pack2(bx, bx), by2 = pack2(by, by), minus = pack2(-1.f, -1.f);
#pragma unroll 1
    for (int j0 = 0; j0 < kC; j0 += 16) {
      float v[16] = {};
      if (j0 <= (row | 31)) {         // (the same for the whole warp)
        uint32_t g[16];
        tmem_ld16(at + F::G + j0, g);
        tmem_ld_wait();
        if (row >= 32 && j0 < 32) {
          const f32x2 far2 = pack2(far, far);
#pragma unroll
          for (int j = 0; j < 16; j += 4) {
            const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(&tok.far[j0 + j]);
            unpack2(mul2(far2, mul2(pair_of(g, j), f.x)), v[j], v[j + 1]);
            unpack2(mul2(far2, mul2(pair_of(g, j + 2), f.y)), v[j + 2], v[j + 3]);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 16; j += 4) {
            const ulonglong2 cx = *reinterpret_cast<const ulonglong2*>(&tok.cx[j0 + j]);
            const ulonglong2 cy = *reinterpret_cast<const ulonglong2*>(&tok.cy[j0 + j]);
            const f32x2 d0 = add2(fma2(cx.x, minus, bx2), fma2(cy.x, minus, by2));
            const f32x2 d1 = add2(fma2(cx.y, minus, bx2), fma2(cy.y, minus, by2));
            float e[4];
            unpack2(d0, e[0], e[1]);
            unpack2(d1, e[2], e[3]);
            unpack2(mul2(mul2(pair_of(g, j), f2), pack2(ex2_f32(e[0]), ex2_f32(e[1]))), v[j], v[j + 1]);
            unpack2(mul2(mul2(pair_of(g, j + 2), f2), pack2(ex2_f32(e[2]), ex2_f32(e[3]))), v[j + 2], v[j + 3]);
          }
#pragma unroll
          for (int j = 0; j < 16; ++j) v[j] = j0 + j <= upto ? v[j] : 0.f;
        }
      }
      if (keys) {
        float4* to = reinterpret_cast<float4*>(A + row * kAPitch + j0);
#pragma unroll
        for (int j = 0; j < 4; ++j) to[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
      } else if (!SUMMARY) {
#pragma unroll
        for (int j = 0; j < 16; j += 8) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) split2(pack2(v[j + 2 * i], v[j + 2 * i + 1]), hi[i], lo[i]);
          const uint32_t to = P + sw_chunk(kC, row, 0, (j0 + j) / 8);
          sts128(to, make_uint4(hi[0], hi[1], hi[2], hi[3]));
          sts128(to + kSlab, make_uint4(lo[0], lo[1], lo[2], lo[3]));
        }
      }
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars->g_empty);
    named_bar_sync(bar, 128);
    // T in A's place: blocks of 16, then 32, then 64; the upper blocks hold what is
    // between two products
    invert16(A + (t / 32) * 16 * (kAPitch + 1), lane);
    named_bar_sync(bar, 128);
    {
      const int o = t / 64 * 32, u = t % 64, r0 = u / 4, c0 = u % 4 * 4;
      float* B = A + o * (kAPitch + 1);
      small_product<1>(B + (16 + r0) * kAPitch, B + c0, 0, 16, 1.f, B + r0 * kAPitch + 16 + c0);
      named_bar_sync(bar, 128);
      small_product<1>(B + (16 + r0) * kAPitch + 16, B + 16 + c0, 0, 16, -1.f, B + (16 + r0) * kAPitch + c0);
    }
    named_bar_sync(bar, 128);
    {
      const int r0 = t / 8 * 2, c0 = t % 8 * 4;
      small_product<2>(A + (32 + r0) * kAPitch, A + c0, c0 < 16 ? 0 : 16, 32, 1.f, A + r0 * kAPitch + 32 + c0);
      named_bar_sync(bar, 128);
      small_product<2>(A + (32 + r0) * kAPitch + 32, A + 32 + c0, 0, r0 < 16 ? 16 : 32, -1.f,
                       A + (32 + r0) * kAPitch + c0);
    }
    named_bar_sync(bar, 128);
    // Tβ where the last chunk's was; its w is complete
    if (c >= 1) LA_GO_ON(w_full[(c - 1) & 1], (c - 1) / 2);
    const uint32_t T = smem_u32(x.sm + F::oT);
    const int h0 = keys ? 0 : 32;     // half of the row's columns
#pragma unroll 1
    for (int j = h0; j < h0 + 32; j += 8) {
      uint4 o[3] = {};
      if (j / 16 <= row / 16) {       // (above, blocks hold what was between two products)
        uint32_t* u = reinterpret_cast<uint32_t*>(o);
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
          const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(A + row * kAPitch + j + i);
          const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(&tok.beta[j + i]);
          split3(mul2(a.x, f.x), u[i / 2], u[4 + i / 2], u[8 + i / 2]);
          split3(mul2(a.y, f.y), u[i / 2 + 1], u[4 + i / 2 + 1], u[8 + i / 2 + 1]);
        }
      }
#pragma unroll
      for (int m = 0; m < 3; ++m) sts128(T + m * kSlab + sw_chunk(kC, row, 0, j / 8), o[m]);
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars->t_ready);
  }
}

// ------------------------------------------------------------------ kernel

// SUMMARY: no output, and one more CTA for each part, which starts from the identity.
template <int DK, bool SUMMARY>
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
    for (uint64_t* b : {&bars->kq_clean, &bars->v_clean, &bars->g_full[0], &bars->g_full[1], &bars->p_empty[0],
                        &bars->p_empty[1], &bars->ks_full, &bars->qs_full, &bars->w_full[0], &bars->w_full[1], &bars->upd_full, &bars->pv_full, &bars->done})
      mbar_init(b, 1);
    for (int i = 0; i < kTok; ++i) mbar_init(&bars->f_ready[i], 2);
    for (uint64_t* b : {&bars->g_empty, &bars->t_ready, &bars->qs_read, &bars->pv_read}) mbar_init(b, 4);
    for (uint64_t* b : {&bars->s_ready, &bars->ks_ready, &bars->w_ready}) mbar_init(b, kStateWarps);
    bars->abort = bars->kq_issued = bars->v_issued = 0;
    bars->replayed[0] = bars->replayed[1] = -1;
    fence_barrier_init();
    for (const CUtensorMap* m : {&mq, &mk, &mv, &mo}) tma_prefetch_desc(m);
  }
  const int tiles = p.tiles + SUMMARY, parts = p.segs - SUMMARY;
  x.tile = blockIdx.x % tiles;
  x.identity = SUMMARY && x.tile == p.tiles;
  const int part = blockIdx.x / tiles % parts;
  const int64_t bh = blockIdx.x / tiles / parts;
  // what is not loaded of the v tiles: zeros
  const int rest = x.identity ? 0 : p.dv - x.tile * 128 <= 64 ? 1 : 2;
  for (int i = threadIdx.x; i < kVS * 2 * kSlab / 16; i += kThreads)
    if (i / (kSlab / 16) % 2 >= rest) *reinterpret_cast<uint4*>(x.sm + F::oV + i * 16) = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  entry();
  if (warp == kMmaWarp) {
    tmem_alloc(&bars->tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  x.tmem = __shfl_sync(0xffffffffu, bars->tmem, 0);   // (known to be the same for the warp)
  x.h = (int)(bh % p.Hv);
  x.b = (int)(bh / p.Hv);
  x.t0 = part * p.seg_tokens;
  x.end = min(p.n - x.t0, p.seg_tokens);
  x.live = max(0, min(live_tokens(p.lengths, x.b, p.n) - x.t0, x.end));
  x.chunks = (x.live + kC - 1) / kC;
  x.partial = x.live % kC != 0 && x.t0 + x.live < p.n;
  const int64_t state = (int64_t)p.dk * p.dv;
  x.cols = x.identity ? p.dk : p.dv;
  if (SUMMARY) {
    x.s_in = nullptr;
    x.s_out = x.identity ? p.transition + (bh * parts + part) * p.dk * p.dk : p.added + (bh * parts + part) * state;
  } else {
    x.s_in = part ? p.entering + (bh * (parts - 1) + part - 1) * state
                  : p.state_in ? p.state_in + bh * state : nullptr;
    x.s_out = part == parts - 1 && p.state_out ? p.state_out + bh * state : nullptr;
  }

  if (warp < kStateWarps) {
    take_registers<DK == 128 ? 120 : 112>();
    role_state<DK, SUMMARY>(x, p, warp, lane);
  } else if (warp < kOutWarp) {
    take_registers<DK == 128 ? 64 : 72>();
    role_prep<DK, SUMMARY>(x, p, warp, lane);
  } else if (warp < kLoadWarp) {
    take_registers<DK == 128 ? 56 : 48>();
    if (!SUMMARY) role_out<DK>(x, p, &mo, warp, lane);
  } else {
    take_registers<DK == 128 ? 56 : 64>();
    if (warp == kLoadWarp)
      role_load<DK, SUMMARY>(x, p, &mq, &mk, &mv, lane);
    else if (warp == kMmaWarp)
      role_mma<DK, SUMMARY>(x, p);
    else
      role_factors<DK>(x, p, warp, lane);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (*(volatile int*)&bars->abort) {   // a wait gave up: copies and products in flight end before the CTA does
    if (warp == kMmaWarp && lane == 0) {
      mma_commit(&bars->done);
      drain_in_line(&bars->done, 0);
    }
    if (warp == kLoadWarp && lane == 0) {
      const int kq_issued = bars->kq_issued, v_issued = bars->v_issued;
      for (int j = max(0, kq_issued - kKQ); j < kq_issued; ++j) drain_in_line(&bars->kq_full[j % kKQ], (j / kKQ) & 1);
      for (int j = max(0, v_issued - kVS); j < v_issued; ++j) drain_in_line(&bars->v_full[j % kVS], (j / kVS) & 1);
    }
    if (warp == kOutWarp && lane == 0) {
      tma_store_wait0();
      atomicCAS(p.status, 0, kStatusTimeout);
    }
    __syncthreads();
  }
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(x.tmem, 512);
}

// The states that enter the parts of a sequence, S ← M·S + N over them: a CTA has
// kJoinCols columns of a head's state, and the next part's M under way while it
// multiplies with this one's.
constexpr int kJoinCols = 16, kJoinThreads = 256, kMPitch = 132;
constexpr int kJoinSmem = (2 * 128 * kMPitch + 2 * 128 * kJoinCols) * 4;

__global__ void __launch_bounds__(kJoinThreads) join_kernel(const float* state_in, const float* added,
                                                            const float* transition, float* entering, int dk, int dv,
                                                            int parts) {
  extern __shared__ float sm[];
  float* S = sm + 2 * 128 * kMPitch;        // [2][128][kJoinCols]
  entry();
  const int blocks = (dv + kJoinCols - 1) / kJoinCols;
  const int64_t bh = blockIdx.x / blocks;
  const int c0 = blockIdx.x % blocks * kJoinCols;
  const int k = threadIdx.x / 2, c = threadIdx.x % 2 * 8;   // this thread's row and columns
  const bool in = k < dk && c0 + c < dv;                    // dv is a multiple of 8
  auto fetch = [&](int g) {
    const float* M = transition + (bh * parts + g) * dk * dk;
    for (int i = threadIdx.x; i < dk * dk / 4; i += kJoinThreads)
      cp_async16(smem_u32(sm + (g & 1) * 128 * kMPitch + i / (dk / 4) * kMPitch + i % (dk / 4) * 4), M + i * 4);
    cp_commit();
  };
  auto load8 = [&](const float* p, float (&v)[8]) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  };
  auto store8 = [&](float* p, const float (&v)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  };
  const int64_t at = (int64_t)k * dv + c0 + c, state = (int64_t)dk * dv;
  float v[8] = {};
  if (state_in && in) load8(state_in + bh * state + at, v);
  store8(S + k * kJoinCols + c, v);
  fetch(0);
  for (int g = 0; g < parts; ++g) {
    if (g + 1 < parts) fetch(g + 1);
    if (in) load8(added + (bh * parts + g) * state + at, v);
    if (g + 1 < parts) cp_wait<1>(); else cp_wait<0>();
    __syncthreads();
    const float* M = sm + (g & 1) * 128 * kMPitch + k * kMPitch;
    const float* from = S + (g & 1) * 128 * kJoinCols + c;
    if (in) {
      for (int j = 0; j < dk; j += 4) {
        const float4 m = *reinterpret_cast<const float4*>(M + j);
        const float mv[4] = {m.x, m.y, m.z, m.w};
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          float w[8];
          load8(from + (j + u) * kJoinCols, w);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = fmaf(mv[u], w[i], v[i]);
        }
      }
      store8(entering + (bh * parts + g) * state + at, v);
    }
    store8(S + ((g + 1) & 1) * 128 * kJoinCols + k * kJoinCols + c, v);
    __syncthreads();   // before this part's M is overwritten
  }
}

// Parts of a sequence: with few heads most SMs would have none, so each sequence is
// walked twice, first for what every part makes of a state (one CTA more for each
// part, and no output), then with the states that enter them.  By the µs of a chunk
// (5.1, and 4.3 without the output), of joining two parts (4.8) and of two launches more:
// 8 heads of 4096 tokens take 123 µs in 8 parts, 180 in 4 and 329 undivided, of 1024
// tokens 67, 69 and 89.
int parts_of(const DeltaArgs& a, int tiles) {
  const int64_t heads = a.B * a.Hv, chunks = (a.n + kC - 1) / kC;
  auto rounds = [&](int64_t ctas) { return (double)((ctas + a.num_sms - 1) / a.num_sms); };
  int best = 1;
  double least = rounds(heads * tiles) * chunks * 5.1;
  for (int g = 2; g <= 64 && g * 4 <= chunks; ++g) {
    const int64_t part = (chunks + g - 1) / g;
    if ((chunks + part - 1) / part != g) continue;
    const double t = rounds(heads * (g - 1) * (tiles + 1)) * part * 4.3 + rounds(heads * g * tiles) * part * 5.1 +
                     15.0 + rounds(heads * ((a.dv + kJoinCols - 1) / kJoinCols)) * (g - 1) * 4.8;
    if (t < least) least = t, best = g;
  }
  return best;
}

template <int DK>
cudaError_t launch_chunks(const DeltaArgs& a, TcParams p, cudaStream_t s) {
  CUtensorMap mq, mk, mv, mo;
  cudaError_t e;
  if ((e = tmap_heads(&mq, a.q, a.B, a.n, a.Hk, a.dk, kC, true)) != cudaSuccess ||
      (e = tmap_heads(&mk, a.k, a.B, a.n, a.Hk, a.dk, kC, true)) != cudaSuccess ||
      (e = tmap_heads(&mv, a.v, a.B, a.n, a.Hv, a.dv, kC, true)) != cudaSuccess ||
      (e = tmap_heads(&mo, a.out, a.B, a.n, a.Hv, a.dv, kOutRows, false)) != cudaSuccess)
    return e;
  const int64_t heads = a.B * a.Hv;
  p.segs = parts_of(a, p.tiles);
  p.seg_tokens = (int)(((a.n + kC - 1) / kC + p.segs - 1) / p.segs) * kC;
  const int64_t ctas = heads * p.segs * p.tiles, first = heads * (p.segs - 1) * (p.tiles + 1);
  if (ctas > INT32_MAX || first > INT32_MAX) return cudaErrorInvalidConfiguration;
  static std::atomic<uint64_t> smem_set[2];
  constexpr int kSmem = Cfg<DK>::kSmem;
  if ((e = allow_smem((const void*)chunk_kernel<DK, false>, kSmem, smem_set)) != cudaSuccess) return e;
  DeltaParts w{};
  if (p.segs > 1) {
    if ((e = allow_smem((const void*)chunk_kernel<DK, true>, kSmem, smem_set + 1)) != cudaSuccess ||
        (e = delta_parts(a, p.segs, &w, s)) != cudaSuccess)
      return e;
    p.added = w.added, p.transition = w.transition, p.entering = w.entering;
    e = launch(chunk_kernel<DK, true>, (unsigned)first, kThreads, kSmem, s, 1, mq, mk, mv, mo, p);
    if (e == cudaSuccess) e = delta_join(a, p.segs, w, s);
  }
  if (e == cudaSuccess)
    e = launch(chunk_kernel<DK, false>, (unsigned)ctas, kThreads, kSmem, s, 1, mq, mk, mv, mo, p);
  if (w.added) {
    const cudaError_t f = cudaFreeAsync(w.added, s);
    if (e == cudaSuccess) e = f;
  }
  return e;
}

}  // namespace

cudaError_t delta_parts(const DeltaArgs& a, int parts, DeltaParts* w, cudaStream_t s) {
  const int64_t each = a.B * a.Hv * (parts - 1), state = (int64_t)a.dk * a.dv;
  const cudaError_t e = ws_alloc((void**)&w->added, each * (2 * state + (int64_t)a.dk * a.dk) * sizeof(float), s);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return e;
  }
  w->entering = w->added + each * state;
  w->transition = w->entering + each * state;
  return e;
}

cudaError_t delta_join(const DeltaArgs& a, int parts, const DeltaParts& w, cudaStream_t s) {
  static std::atomic<uint64_t> smem_set{0};
  const cudaError_t e = allow_smem((const void*)join_kernel, kJoinSmem, &smem_set);
  if (e != cudaSuccess) return e;
  const int64_t ctas = a.B * a.Hv * ((a.dv + kJoinCols - 1) / kJoinCols);
  if (ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
  return launch(join_kernel, (unsigned)ctas, kJoinThreads, kJoinSmem, s, 1, a.state_in, w.added, w.transition,
                w.entering, a.dk, a.dv, parts - 1);
}

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
  p.v = static_cast<const bf16*>(a.v.data);
  p.v_sb = a.v.sb, p.v_sn = a.v.sn, p.v_sh = a.v.sh;
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
