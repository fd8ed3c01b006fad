// The selective state-space recurrence over a prompt and for one token:
//   Δ = softplus(dt + dt_bias);  h_s ← exp(Δ·a_s)·h_s + Δ·x·B_s;
//   y = (Σ_s C_s·h_s + skip·x)·silu(gate),
// for every channel (a row of a) with S states.
//
// Per (token, channel, state): one 2^x (4 cycles a warp) and four fp32
// multiply-adds (4 cycles as two packed pairs), against half a byte moved: bound
// by the latency of a few warps' dependent instructions and by the shared-memory
// reads of B and C, with HBM at a fifth.  So a state element is computed once where possible, and every other
// cost is kept off its path.  A group of G = S/K lanes owns two neighbouring
// channels, K states of each per lane, in registers over the whole prompt,
// packed in pairs (one instruction for two multiply-adds).  Tokens go in
// batches of G: each lane of a group prepares one token's Δ and Δ·x, the group
// shares them through shared memory, and the G partial readouts are summed so
// that lane i ends with token i, gates it and writes it.  A stage of tokens is
// prepared while the one before it is scanned (215 µs against 260).
//
// A warp is a CTA and waits for nobody: it keeps two stages of its inputs in
// flight with cp.async in a ring of its own.  Where channels alone give too few
// warps, the sequence is cut into chunks: a first launch reaches each chunk's
// end state from zero (no readout), and the second starts every chunk from the
// states before it, combined as h ← exp(a·ΣΔ)·h + end.  That costs 0.6 of the
// work again.
//
// Measured, bf16 with gate, 16 states: 4×2048×4096 (1024 warps, uncut) in
// 213 µs = 2.5 T state elements/s (issue 52 %, shared-memory pipe 50 %, ex2
// pipe 32 %; 1.7 warps per scheduler); 1×65536×2048 (cut) in 1.05 ms.
#include "block.cuh"
#include "internal.h"

#include <atomic>
#include <type_traits>

namespace la {
namespace {

using namespace block;

constexpr float kLargest = 3.0e38f;

// a·log2 e, the decay's exponent per Δ.  Kept finite below: a step of zero, a
// masked token's among them, leaves the state alone, and 0·(−inf) is not 0.
__device__ __forceinline__ float rate(float a) {
  const float r = a * kLog2e;
  return r < -kLargest ? -kLargest : r;   // keeps NaN
}

// Added to every decay's exponent.  The hardware's 2^x is low by 2e-8 on average
// for x in [−0.1, −0.003], a third of an ulp, which a state with a memory of
// hundreds of tokens adds up (2e-6 after 130 tokens).  With this its mean error
// is within 1.2e-8 of zero for x in [−0.3, 0], and 2^0 is still 1.
constexpr float kCentre = 2.0e-8f;

// 2^e·h over a whole chunk of growth (a > 0 or negative steps), where 2^e can be
// past fp32's range although the states are not: h is tiny, or 0 until later tokens.
__device__ __forceinline__ float grown(float e, float h) {
  const float half = tc::ex2_f32(0.5f * e);
  return h == 0.f ? h : half * (half * h);
}

constexpr int kTok = 16;      // tokens per stage of the ring
constexpr int kRing = 3;      // stages: one in use, two in flight

template <typename T, int S> struct Cfg {
  // States per lane and channel.  Fewer give more warps and cost more per element
  // (sharing and summing over G lanes).  2×2048×4096: 32 states in 193 µs with
  // four, 255 with eight; 4×2048×4096: 8 states in 178 µs with two, 240 with
  // four, 16 states in 238 µs with two, 213 with four.  With 64, four would leave
  // a warp less than 16 bytes of a row.
  static constexpr int K = S == 8 ? 2 : (S <= 32 ? 4 : 8);
  static constexpr int G = S / K;                  // lanes per channel pair, tokens per batch
  static constexpr int kPairs = 32 / G;            // channel pairs per warp
  static constexpr int kCh = 2 * kPairs;           // channels per warp
  static constexpr int kRowB = kCh * (int)sizeof(T);      // bytes of a token's x, dt or gate
  static constexpr int kStB = S * (int)sizeof(T);         // bytes of a token's B or C
  static constexpr int kStage = kTok * (3 * kRowB + 2 * kStB);
  static constexpr int kDu = kTok * kPairs * 16;          // Δ and Δ·x of a stage
  static constexpr int kPrep = kDu + 2 * kTok * S * 4;    // and B, C as fp32
  static constexpr int kSmem = kRing * kStage + 2 * kPrep;
  static_assert(kRowB % 16 == 0 && kStB % 16 == 0 && kTok % G == 0, "scan layout");
  static_assert(32 % (kRowB / 16) == 0 && 32 % (kStB / 16) == 0, "pieces per row");
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

// Two neighbouring values in shared memory.
template <typename T>
__device__ __forceinline__ float2 load2s(const T* p) {
  if constexpr (sizeof(T) == 2) {
    const uint32_t r = *reinterpret_cast<const uint32_t*>(p);
    return make_float2(tc::bf16lo_to_f32(r), tc::bf16hi_to_f32(r));
  } else {
    return *reinterpret_cast<const float2*>(p);
  }
}

// K fp32 values (2 or a multiple of 4) as pairs, from shared or global memory.
template <int K>
__device__ __forceinline__ void load_pairs(const void* at, f32x2 (&p)[K / 2]) {
  if constexpr (K == 2) {
    p[0] = *reinterpret_cast<const f32x2*>(at);
  } else {
#pragma unroll
    for (int q = 0; q < K / 4; ++q) {
      const ulonglong2 v = reinterpret_cast<const ulonglong2*>(at)[q];
      p[2 * q] = v.x;
      p[2 * q + 1] = v.y;
    }
  }
}

template <int K>
__device__ __forceinline__ void store_pairs(void* at, const f32x2 (&p)[K / 2]) {
  if constexpr (K == 2) {
    *reinterpret_cast<f32x2*>(at) = p[0];
  } else {
#pragma unroll
    for (int q = 0; q < K / 4; ++q)
      reinterpret_cast<ulonglong2*>(at)[q] = make_ulonglong2(p[2 * q], p[2 * q + 1]);
  }
}

struct Chunks {
  int count;           // chunks per sequence
  int len;             // tokens per chunk, a multiple of kTok
  float* end;          // [B][count][D][S]: state reached from zero
  float* step;         // [B][count][D]: ΣΔ
};

// ENDS: the first launch of a cut sequence (end states and ΣΔ of the chunks,
// the last one excepted); otherwise the outputs.
template <typename T, int S, bool ENDS>
__global__ void __launch_bounds__(32) scan_kernel(const ScanArgs a, const int cblocks,
                                                  const Chunks ch) {
  using C = Cfg<T, S>;
  constexpr int K = C::K, G = C::G;
  extern __shared__ __align__(16) uint8_t smem[];
  const uint32_t ring = tc::smem_u32(smem);
  const int cb = blockIdx.x % cblocks;
  const int k = (blockIdx.x / cblocks) % (ENDS ? ch.count - 1 : ch.count);
  const int64_t b = blockIdx.x / cblocks / (ENDS ? ch.count - 1 : ch.count);
  const int lane = threadIdx.x, lg = lane / C::kPairs, pair = lane % C::kPairs;
  // No early trigger for the next kernel: its CTAs would take their places on the
  // SMs that have room first.
  tc::grid_dependency_wait();
  const int D = (int)a.D, n = (int)a.n;
  const int c0 = cb * C::kCh, cw = c0 + 2 * pair;
  const bool on = cw < D;         // D is even: both channels or none
  const int c = on ? cw : 0;
  const int len = live_tokens(a.lengths, b, n);
  const int t_lo = k * ch.len;                              // this chunk: [t_lo, t_hi)
  const int t_hi = ch.count - 1 - k > 0 ? t_lo + ch.len : n;
  const int live = min(t_hi, len);                          // the tokens of it that count

  f32x2 A[2][K / 2], h[2][K / 2];
  const f32x2 centre = pack2(kCentre, kCentre);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    load_pairs<K>(a.a + (int64_t)(c + j) * S + lg * K, A[j]);
#pragma unroll
    for (int q = 0; q < K / 2; ++q) {
      float a0, a1;
      unpack2(A[j][q], a0, a1);
      A[j][q] = pack2(rate(a0), rate(a1));
      h[j][q] = 0ull;
    }
    if ((!ENDS || k == 0) && a.state_in)
      load_pairs<K>(a.state_in + (b * D + c + j) * S + lg * K, h[j]);
  }
  float bias[2] = {0.f, 0.f}, skip[2] = {0.f, 0.f};
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    if (a.dt_bias) bias[j] = a.dt_bias[c + j];
    if (a.skip) skip[j] = a.skip[c + j];
  }
  const char* src[5] = {
      reinterpret_cast<const char*>(static_cast<const T*>(a.x.data) + b * a.x.sb + c0),
      reinterpret_cast<const char*>(static_cast<const T*>(a.dt.data) + b * a.dt.sb + c0),
      reinterpret_cast<const char*>(static_cast<const T*>(a.b.data) + b * a.b.sb),
      reinterpret_cast<const char*>(static_cast<const T*>(a.c.data) + b * a.c.sb),
      reinterpret_cast<const char*>(static_cast<const T*>(a.gate.data) + b * a.gate.sb + c0)};
  const bool gated = a.gate.data != nullptr;
  const int row_ok = min(C::kRowB, (D - c0) * (int)sizeof(T));   // bytes of a row inside D

  // A stage's 16-byte pieces of each tensor are dealt to the lanes; absent
  // ones are written as zeros.  Every lane keeps the address of its first
  // piece of the next stage.
  const char* next_piece[5];
  const int64_t sn[5] = {a.x.sn * (int64_t)sizeof(T), a.dt.sn * (int64_t)sizeof(T),
                         a.b.sn * (int64_t)sizeof(T), a.c.sn * (int64_t)sizeof(T),
                         a.gate.sn * (int64_t)sizeof(T)};
#pragma unroll
  for (int i = 0; i < 5; ++i) {
    const int per = (i == 2 || i == 3 ? C::kStB : C::kRowB) / 16;
    next_piece[i] = src[i] + (t_lo + lane / per) * sn[i] + (lane % per) * 16;
  }
  auto fetch = [&](auto rb, auto which, uint32_t dst, int ok, int t0, bool whole) {
    constexpr int RB = decltype(rb)::value, PER = RB / 16, I = decltype(which)::value;
#pragma unroll
    for (int e0 = 0; e0 < kTok * PER; e0 += 32) {
      const int e = e0 + lane;
      const char* from = next_piece[I] + (e0 / PER) * sn[I];
      if (kTok * PER % 32 == 0 || e < kTok * PER) {
        if (whole) {
          cp_async16(dst + e * 16, from);
        } else {
          const bool take = t0 + e / PER < live && (e % PER) * 16 < ok;
          cp_async16(dst + e * 16, take ? from : src[I], take ? 16 : 0);
        }
      }
    }
    next_piece[I] += kTok * sn[I];
  };
  auto fetch_stage = [&](int slot, int t0) {
    if (t0 < live) {
      const uint32_t st = ring + slot * C::kStage;
      const bool whole = t0 + kTok <= live && row_ok == C::kRowB;
      std::integral_constant<int, C::kRowB> rb;
      std::integral_constant<int, C::kStB> sb;
      fetch(rb, std::integral_constant<int, 0>(), st, row_ok, t0, whole);
      fetch(rb, std::integral_constant<int, 1>(), st + kTok * C::kRowB, row_ok, t0, whole);
      fetch(sb, std::integral_constant<int, 2>(), st + 3 * kTok * C::kRowB, C::kStB, t0, whole);
      if (!ENDS) {
        if (gated)
          fetch(rb, std::integral_constant<int, 4>(), st + 2 * kTok * C::kRowB, row_ok, t0, whole);
        fetch(sb, std::integral_constant<int, 3>(), st + 3 * kTok * C::kRowB + kTok * C::kStB,
              C::kStB, t0, whole);
      }
    }
    cp_commit();
  };
#pragma unroll
  for (int i = 0; i < kRing - 1; ++i) fetch_stage(i, t_lo + i * kTok);

  if (!ENDS && k > 0) {
    // the state entering this chunk; a chunk past the length has ΣΔ = 0 and a
    // zero end state, and leaves it alone
    auto enter = [&](auto growing) {
#pragma unroll 4
      for (int p = 0; p < k; ++p) {
        const int64_t at = (b * ch.count + p) * D + c;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float sd = p > 0 ? ch.step[at + j] : 0.f;
          const f32x2 s2 = pack2(sd, sd);
#pragma unroll
          for (int q = 0; q < K / 2; ++q) {
            const float2 e = *reinterpret_cast<const float2*>(ch.end + (at + j) * S + lg * K + 2 * q);
            float e0, e1;
            unpack2(mul2(s2, A[j][q]), e0, e1);
            // the first chunk's end state was reached from state_in
            if (p == 0) {
              h[j][q] = pack2(e.x, e.y);
            } else if constexpr (decltype(growing)::value) {
              float h0, h1;
              unpack2(h[j][q], h0, h1);
              h[j][q] = add2(pack2(grown(e0, h0), grown(e1, h1)), pack2(e.x, e.y));
            } else {
              h[j][q] = fma2(pack2(tc::ex2_f32(e0), tc::ex2_f32(e1)), h[j][q], pack2(e.x, e.y));
            }
          }
        }
      }
    };
    enter(std::false_type());
    // a factor past fp32's range leaves no finite state behind
    bool lost = false;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int q = 0; q < K / 2; ++q) {
        float h0, h1;
        unpack2(h[j][q], h0, h1);
        lost |= !(fabsf(h0) <= kLargest) || !(fabsf(h1) <= kLargest);
      }
    if (lost) enter(std::true_type());
  }

  float sum[2] = {0.f, 0.f};   // ΣΔ of this lane's tokens (ENDS)
  T* op = ENDS ? nullptr : static_cast<T*>(a.out) + b * a.out_sb + c;

  // A stage is prepared while the one before it is scanned, so that the two
  // chains of dependent instructions fill each other's gaps.  prep: [token]
  // [pair] Δ and Δ·x, then B and C as fp32; two of them, used in turn.
  uint8_t* const prep0 = smem + kRing * C::kStage;
  auto widen = [&](const uint8_t* st, uint8_t* prep) {
    constexpr int V = kVec<T>, PER = S / V;
#pragma unroll
    for (int e = lane; e < kTok * PER; e += 32)
#pragma unroll
      for (int w = 0; w < (ENDS ? 1 : 2); ++w) {
        float f[V];
        unpack<T>(*reinterpret_cast<const uint4*>(st + 3 * kTok * C::kRowB + w * kTok * C::kStB + e * 16), f);
        float4* to = reinterpret_cast<float4*>(prep + C::kDu + w * kTok * S * 4 + e * V * 4);
#pragma unroll
        for (int i = 0; i < V; i += 4) to[i / 4] = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
      }
  };
  // token bi·G + lg of the stage that starts at t0: Δ and Δ·x for the group;
  // the skip term and the gate stay with the lane
  float xs[2][kTok / G][2], zs[2][kTok / G][2];
  auto prepare = [&](const uint8_t* st, uint8_t* prep, int t0, int bi, float (&x1)[2], float (&z1)[2]) {
    const int ti = bi * G + lg;
    const T* at = reinterpret_cast<const T*>(st + ti * C::kRowB) + 2 * pair;
    const float2 x = load2s(at);
    float2 dt = load2s(at + kTok * C::kCh);
    dt.x += bias[0];
    dt.y += bias[1];
    if (a.softplus) dt = softplus2(dt);
    if (t0 + ti >= live) dt = make_float2(0.f, 0.f);   // a step of zero changes nothing
    if constexpr (ENDS) {
      sum[0] += dt.x;
      sum[1] += dt.y;
    } else {
      x1[0] = skip[0] * x.x;
      x1[1] = skip[1] * x.y;
      z1[0] = z1[1] = 1.f;
      if (gated) {
        const float2 z = load2s(at + 2 * kTok * C::kCh);
        z1[0] = silu(z.x);
        z1[1] = silu(z.y);
      }
    }
    return make_float4(dt.x, dt.y, dt.x * x.x, dt.y * x.y);
  };
  auto put = [&](uint8_t* prep, int bi, const float4& v) {
    *reinterpret_cast<float4*>(prep + ((bi * G + lg) * C::kPairs + pair) * 16) = v;
  };
  // scans the stage prepared in `prep` and prepares the next one from `st`
  auto stage = [&](int t0, const uint8_t* prep, uint8_t* next, const uint8_t* st,
                   const float (&x0)[kTok / G][2], const float (&z0)[kTok / G][2],
                   float (&x1)[kTok / G][2], float (&z1)[kTok / G][2]) {
    const uint8_t *bt = prep + C::kDu, *ct = bt + kTok * S * 4;
#pragma unroll
    for (int bi = 0; bi < kTok / G; ++bi) {
      float4 du[G];
      f32x2 B2[G][K / 2], C2[G][K / 2];
#pragma unroll
      for (int i = 0; i < G; ++i) {
        const int ti = bi * G + i;
        du[i] = *reinterpret_cast<const float4*>(prep + (ti * C::kPairs + pair) * 16);
        load_pairs<K>(bt + (ti * S + lg * K) * 4, B2[i]);
        if (!ENDS) load_pairs<K>(ct + (ti * S + lg * K) * 4, C2[i]);
      }
      const float4 nx = prepare(st, next, t0 + kTok, bi, x1[bi], z1[bi]);
      float y[2][G];
#pragma unroll
      for (int i = 0; i < G; ++i) {
        const f32x2 d2[2] = {pack2(du[i].x, du[i].x), pack2(du[i].y, du[i].y)};
        const f32x2 u2[2] = {pack2(du[i].z, du[i].z), pack2(du[i].w, du[i].w)};
        f32x2 acc[2] = {0ull, 0ull};
#pragma unroll
        for (int q = 0; q < K / 2; ++q)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float e0, e1;
            unpack2(fma2(d2[j], A[j][q], centre), e0, e1);
            const f32x2 dec = pack2(tc::ex2_f32(e0), tc::ex2_f32(e1));
            h[j][q] = fma2(dec, h[j][q], mul2(u2[j], B2[i][q]));
            if (!ENDS) acc[j] = q == 0 ? mul2(C2[i][q], h[j][q]) : fma2(C2[i][q], h[j][q], acc[j]);
          }
        if constexpr (!ENDS) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float lo, hi;
            unpack2(acc[j], lo, hi);
            y[j][i] = lo + hi;
          }
        }
      }
      if constexpr (!ENDS) {
        // lane i of the group keeps token i: halve the tokens per exchange
#pragma unroll
        for (int m = G / 2; m >= 1; m /= 2) {
          const bool up = (lg & m) != 0;
#pragma unroll
          for (int i = 0; i < m; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const float give = up ? y[j][i] : y[j][i + m];
              const float keep = up ? y[j][i + m] : y[j][i];
              y[j][i] = keep + __shfl_xor_sync(0xffffffffu, give, m * C::kPairs);
            }
        }
        const int t = t0 + bi * G + lg;
        if (on && t < live)
          store2(op + t * a.out_sn, (y[0][0] + x0[bi][0]) * z0[bi][0],
                 (y[1][0] + x0[bi][1]) * z0[bi][1]);
      }
      put(next, bi, nx);
    }
    widen(st, next);
    __syncwarp();
  };
  if (t_lo < live) {
    cp_wait<kRing - 2>();
    __syncwarp();
    widen(smem, prep0);
#pragma unroll
    for (int bi = 0; bi < kTok / G; ++bi)
      put(prep0, bi, prepare(smem, prep0, t_lo, bi, xs[0][bi], zs[0][bi]));
    __syncwarp();
  }
  int slot = 0;   // ring slot of the stage that is scanned
  auto advance = [&](int t0) {
    // the prepared stage's slot is free; the next one has to be there
    fetch_stage((slot + kRing - 1) % kRing, t0 + (kRing - 1) * kTok);
    cp_wait<kRing - 2>();
    __syncwarp();
    slot = (slot + 1) % kRing;
  };
  for (int t0 = t_lo; t0 < live; t0 += 2 * kTok) {
    advance(t0);
    stage(t0, prep0, prep0 + C::kPrep, smem + slot * C::kStage, xs[0], zs[0], xs[1], zs[1]);
    if (t0 + kTok >= live) break;
    advance(t0 + kTok);
    stage(t0 + kTok, prep0 + C::kPrep, prep0, smem + slot * C::kStage, xs[1], zs[1], xs[0], zs[0]);
  }
  cp_wait<0>();
  float* to = ENDS ? ch.end + ((b * ch.count + k) * D + c) * S
                   : (a.state_out && k == ch.count - 1 ? a.state_out + (b * D + c) * S : nullptr);
  if (on && to) {
#pragma unroll
    for (int j = 0; j < 2; ++j) store_pairs<K>(to + j * S + lg * K, h[j]);
  }
  if constexpr (ENDS) {
#pragma unroll
    for (int m = G / 2; m >= 1; m /= 2) {
      sum[0] += __shfl_xor_sync(0xffffffffu, sum[0], m * C::kPairs);
      sum[1] += __shfl_xor_sync(0xffffffffu, sum[1], m * C::kPairs);
    }
    if (on && lg == 0) {
      ch.step[(b * ch.count + k) * D + c] = sum[0];
      ch.step[(b * ch.count + k) * D + c + 1] = sum[1];
    }
  } else if (on) {
    // tokens past the length
    for (int t = max(t_lo, live) + lg; t < t_hi; t += G) store2(op + t * a.out_sn, 0.f, 0.f);
  }
}

// One token: a lane owns four states of a channel (G = S/4 lanes a channel) in
// R batch entries, so that it reads a once for all of them and has R loads of
// the state in flight.  The state's read and write are nearly all of the
// traffic (8 bytes per state element); a warp touches 512 contiguous bytes.
// The lanes of a channel share the work per entry: each prepares the entries
// R/G apart (or one), and passes Δ and Δ·x on by shuffles (32 µs without).
// Measured: 256×4096×16 bf16 in 22.4 µs = 6.4 TB/s, 0.95 of the copy bandwidth.
constexpr int kStepThreads = 256;

template <typename T, int S, int R>
__global__ void __launch_bounds__(kStepThreads) step_kernel(const ScanArgs a, uint32_t cblocks) {
  constexpr int G = S / 4;
  constexpr int P = G < R ? R / G : 1;              // entries a lane prepares
  const int e = (int)(blockIdx.x % cblocks) * kStepThreads + (int)threadIdx.x;
  const int64_t b0 = (int64_t)(blockIdx.x / cblocks) * R;
  const bool on = e < (int)a.D * G;
  const int q = e % G, c = on ? e / G : 0;
  const int rows = (int)min((int64_t)R, a.B - b0);
  entry();
  float* const hp = a.state_out + (b0 * a.D + c) * S + 4 * q;
  const int64_t hs = a.D * S;
  float4 h[R];
#pragma unroll
  for (int r = 0; r < R; ++r)
    h[r] = __ldcs(reinterpret_cast<const float4*>(hp + (r < rows ? r : 0) * hs));
  float x[P], dt[P], z[P], u[P];
  int row[P];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    row[p] = G < R ? p * G + q : q % R;
    const int64_t b = b0 + (row[p] < rows ? row[p] : 0);
    x[p] = to_f32(static_cast<const T*>(a.x.data)[b * a.x.sb + c]);
    dt[p] = to_f32(static_cast<const T*>(a.dt.data)[b * a.dt.sb + c]);
    z[p] = a.gate.data ? to_f32(static_cast<const T*>(a.gate.data)[b * a.gate.sb + c]) : 0.f;
  }
  float2 Bv[R][2], Cv[R][2];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int64_t b = b0 + (r < rows ? r : 0);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      Bv[r][i] = load2(static_cast<const T*>(a.b.data) + b * a.b.sb + 4 * q + 2 * i);
      Cv[r][i] = load2(static_cast<const T*>(a.c.data) + b * a.c.sb + 4 * q + 2 * i);
    }
  }
  float4 A = *reinterpret_cast<const float4*>(a.a + (int64_t)c * S + 4 * q);
  A.x = rate(A.x), A.y = rate(A.y), A.z = rate(A.z), A.w = rate(A.w);
  const float bias = a.dt_bias ? a.dt_bias[c] : 0.f, skip = a.skip ? a.skip[c] : 0.f;
#pragma unroll
  for (int p = 0; p < P; ++p) {
    dt[p] += bias;
    if (a.softplus) dt[p] = softplus(dt[p]);
    u[p] = dt[p] * x[p];
  }
  float own[P];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int from = G < R ? r % G : r, slot = G < R ? r / G : 0;
    const float d = __shfl_sync(0xffffffffu, dt[slot], from, G);
    const float v = __shfl_sync(0xffffffffu, u[slot], from, G);
    float4 n;
    n.x = fmaf(tc::ex2_f32(fmaf(d, A.x, kCentre)), h[r].x, v * Bv[r][0].x);
    n.y = fmaf(tc::ex2_f32(fmaf(d, A.y, kCentre)), h[r].y, v * Bv[r][0].y);
    n.z = fmaf(tc::ex2_f32(fmaf(d, A.z, kCentre)), h[r].z, v * Bv[r][1].x);
    n.w = fmaf(tc::ex2_f32(fmaf(d, A.w, kCentre)), h[r].w, v * Bv[r][1].y);
    if (on && r < rows) __stcs(reinterpret_cast<float4*>(hp + r * hs), n);
    float y = fmaf(n.x, Cv[r][0].x, fmaf(n.y, Cv[r][0].y, fmaf(n.z, Cv[r][1].x, n.w * Cv[r][1].y)));
#pragma unroll
    for (int m = G / 2; m >= 1; m /= 2) y += __shfl_xor_sync(0xffffffffu, y, m);
    if (r == row[slot]) own[slot] = y;
  }
#pragma unroll
  for (int p = 0; p < P; ++p) {
    if (!on || q >= R || row[p] >= rows) continue;
    float y = fmaf(skip, x[p], own[p]);
    if (a.gate.data) y *= silu(z[p]);
    static_cast<T*>(a.out)[(b0 + row[p]) * a.out_sb + c] = from_f32<T>(y);
  }
}

// Sequences are cut where they give fewer than kWarpsWanted warps per SM
// (2×2048×4096, 3.4 per SM: 147 µs cut, 158 whole; 4×2048×4096, 6.7 per SM:
// 265 µs cut, 213 whole), into chunks that give kWarpsCut of them (1×65536×2048:
// 1114 µs at 16, 1059 at 24, 1076 at 32) and have at least kChunkMin tokens
// (1×300×2048: 17 µs at 64, 20 at 96; 4×500×1024: 26 at 64, 32 at 32).  Short
// ones are not worth a second launch: with less than two warps per SM
// 1×130×2048 takes 16 µs cut, 14 whole, and 1×200×2048 16 and 19; with more,
// 7×333×520 (fp32, 32 states) takes 32 cut and 26 whole, and 2×2048×4096 gains;
// the border between was not measured closer.
constexpr int kCutMin = 160, kCutMinFull = 1024;   // tokens: below and from two warps per SM
constexpr int kWarpsWanted = 4;
constexpr int kWarpsCut = 24;
constexpr int kChunkMin = 64;

template <typename T, int S>
cudaError_t launch_scan(const ScanArgs& a, cudaStream_t s) {
  using C = Cfg<T, S>;
  const int64_t cblocks = (a.D + C::kCh - 1) / C::kCh;
  const int64_t warps = cblocks * a.B;
  if (warps > INT32_MAX) return cudaErrorInvalidConfiguration;
  Chunks ch{1, (int)a.n, nullptr, nullptr};
  const int64_t wanted = (int64_t)kWarpsWanted * a.num_sms;
  if (warps < wanted && a.n >= (warps < 2 * a.num_sms ? kCutMin : kCutMinFull)) {
    int64_t count = (kWarpsCut * (int64_t)a.num_sms + warps - 1) / warps;
    count = count < a.n / kChunkMin ? count : a.n / kChunkMin;
    int64_t len = (a.n + count - 1) / count;
    len = (len + kTok - 1) / kTok * kTok;
    ch.len = (int)len;
    ch.count = (int)((a.n + len - 1) / len);
  }
  static std::atomic<uint64_t> set_all{0}, set_ends{0};
  cudaError_t e = allow_smem((const void*)scan_kernel<T, S, false>, kSmemMax, &set_all);
  if (e != cudaSuccess) return e;
  float* ws = nullptr;
  if (ch.count > 1) {
    e = allow_smem((const void*)scan_kernel<T, S, true>, kSmemMax, &set_ends);
    if (e != cudaSuccess) return e;
    const size_t rows = (size_t)a.B * ch.count * a.D;
    e = ws_alloc(reinterpret_cast<void**>(&ws), rows * (S + 1) * sizeof(float), s);
    if (e != cudaSuccess) {
      cudaGetLastError();
      return e;
    }
    ch.end = ws;
    ch.step = ws + rows * S;
    const int64_t ctas = warps * (ch.count - 1);
    e = launch(scan_kernel<T, S, true>, (unsigned)ctas, 32, even_smem(C::kSmem, ctas, a.num_sms), s, 1,
               a, (int)cblocks, ch);
  }
  // An even share of the CTAs per SM, wherever the predecessor's tail leaves room:
  // after a convolution or a product 4×2048×4096 takes 210 µs, without 352;
  // 4×500×2048 41 and 90.
  const int64_t ctas = warps * ch.count;
  if (e == cudaSuccess)
    e = launch(scan_kernel<T, S, false>, (unsigned)ctas, 32, even_smem(C::kSmem, ctas, a.num_sms), s, 1,
               a, (int)cblocks, ch);
  if (ws) {
    const cudaError_t f = cudaFreeAsync(ws, s);
    if (e == cudaSuccess) e = f;
  }
  return e;
}

// Batch entries per lane of the step: four where that leaves a thousand threads per
// SM (256×4096×16: 32 µs against 39 for one entry, before the lanes shared work);
// one otherwise, where latency counts.
int step_rows(const ScanArgs& a) {
  return a.B >= 4 && a.B / 4 * a.D * (a.S / 4) >= (int64_t)1024 * a.num_sms ? 4 : 1;
}

template <typename T, int S, int R>
cudaError_t launch_step_rows(const ScanArgs& a, cudaStream_t s) {
  const int64_t cblocks = (a.D * (S / 4) + kStepThreads - 1) / kStepThreads;
  const int64_t blocks = (a.B + R - 1) / R * cblocks;
  if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
  return launch(step_kernel<T, S, R>, (unsigned)blocks, kStepThreads, 0, s, 1, a,
                (uint32_t)cblocks);
}

template <typename T, int S>
cudaError_t launch_step(const ScanArgs& a, cudaStream_t s) {
  return step_rows(a) == 4 ? launch_step_rows<T, S, 4>(a, s) : launch_step_rows<T, S, 1>(a, s);
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

const char* selective_step_kernel(const ScanArgs& a) { return step_rows(a) == 4 ? "step4" : "step1"; }

cudaError_t selective_step(const ScanArgs& a, cudaStream_t s) {
  return a.bf16 ? by_states<__nv_bfloat16>(a, true, s) : by_states<float>(a, true, s);
}

}  // namespace la
