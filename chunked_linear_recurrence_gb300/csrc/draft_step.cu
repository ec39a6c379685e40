// draft_step.cu -- several tokens of every sequence on the paged pool of FP32 states [V,K]
// (include/sf_decode.h): accepted tokens advance the state, drafted ones read it.
//
// Chunk form over m tokens from the state S0, with lam_i = e^{gate_i} (e^{decay_h}),
// c_i = lam_1 .. lam_i and R_ij = lam_{j+1} .. lam_i:
//     u_i   = beta_i (v_i - c_i S0 k_i - sum_{j<i} R_ij (k_i . k_j) u_j)      (u_i = v_i without delta)
//     out_i = scale (c_i S0 q_i + sum_{j<=i} R_ij (q_i . k_j) u_j)
//     S_m   = c_m S0 + sum_j R_mj u_j k_j^T
// The R_ij are products, not exponentials of differences of sums, so that a gate of -inf gives 0
// and not NaN.  The state is touched twice a token by the drafts, and twice and once more by the
// accepted ones, against four times each by the rule itself.
//
// Tokens go in groups of up to 8, the state advanced between them; a group of accepted BF16 tokens and
// one of drafts take one pass over the state before both (both()).  A warp holds 16 rows of a state
// in registers and needs no other warp: with g = lane / 4, t = lane % 4 a lane holds of rows g and
// g + 8 the columns 32 j + 8 t .. + 7.  That is at once
//  * an accumulator of 16x8 products and the left operand of 16x8x16 products, if column pair e of
//    every lane is taken as one tile of 8 columns (the sum's order is free);
//  * for a token g in BF16, the right operand of those (S k, S q of 8 tokens), both operands of the
//    tokens' own products, and through movmatrix the right operand of the update W K.
// So nothing passes through shared memory but the tokens' 8x8 products and 16x8 results, for the
// solve, one row to a lane, and what is copied ahead: the tokens, and the next strip's state.
//
// Precision: FP32.  The state that k and q read and the rows' weights W are split into three BF16
// summands (24 bits), and the update's sum is formed apart and added to the state by one FP32
// multiply-add with rounding to nearest, so that the state has no bias of the tensor core's sums.
// (Drafts that read two summands, 16 bits, lose what cancels: where a token takes the place of one 2^13
// times larger, outputs were off by 2.0e-2 for 1.1e-3.  128 sequences, 5 + 5 tokens 93.4 -> 94.3 us, 64 with
// 16 + 16 79 -> 86.)  FP32 tokens are split into three summands themselves, and the six products
// down to 2^-24 are formed everywhere.
//
// A warp takes four strips of a head in a row, with their tokens and what those are to each other in
// shared memory, then four strips of the head that comes next in the whole grid's order: the grid moves
// through the pool as one window.
//
// Bound by memory, 4 V K bytes read and as many written (if a token was accepted), and by the chain
// of a strip's steps (1270 instructions with both kinds of tokens, two warps to a scheduler).  Measured,
// K = 128: 128 sequences of 32 heads, 5 + 5 tokens 94.3 us (537 MB, 5.8 TB/s, 85 % of the copy rate),
// 256 of 16 heads, 8 + 8 tokens by linear attention 96.5 us, a commit of 8 tokens 92 us, 5 tokens with
// nothing pending 56 us and by linear attention 52 (of 40 for the states' bytes); one sequence
// of 16 heads 4.5 us.  The same movement without any tokens' work takes 88 us.  What it came
// from: FP32 pipes with shared-memory tokens 156, 148, 120 us; states loaded where they are used
// 164, 149, 113; copied ahead 158, 146, 121; factors and tokens of a run of strips kept 100, 114,
// 102; whole rows to a copy and whole lines to a store, eight warps an SM and a window 96-98, 98, 92;
// one pass for both kinds of tokens 93.5, 96; the state read in three summands 94.3, 96.5.  With two:
// twelve warps an SM (168 registers, some spilled) 98, 109, 95; runs of one strip 115, 102, 88; summands by
// truncation and byte permutes instead of conversions: the same.  FP32 tokens, 64 sequences of 32 heads: 5 + 5 tokens 88 us, a commit of 8 51 us (on the FP32 pipes 85, 68; floor 41).
#include <cuda_bf16.h>

#include "common.cuh"
#include "decode.cuh"
#include "f32x2.cuh"

namespace sfg {
namespace {

constexpr int GROUP = 8;      // tokens
constexpr int STRIP = 16;     // rows of a state to a warp
template <typename T>
constexpr int PLANES = sizeof(T) == 2 ? 1 : 3;     // BF16 summands of a token
// CTAs of one warp each on an SM; G groups of tokens in their shared memory.
template <int D, typename T, int G>
constexpr int CTAS = sizeof(T) == 2 ? (D == 128 ? 8 : G == 1 ? 14 : 13)
                                    : (D == 128 ? (G == 1 ? 7 : 4) : G == 1 ? 12 : 7);
// Whether pending and fresh tokens take one pass over the state (both()): at the most 8 of each, BF16.
// (FP32 tokens, whose pass would keep more than fits in registers and shared memory: 91 -> 128 us.)
template <typename T, int G>
constexpr bool ONE_PASS = sizeof(T) == 2 && G == 1;
constexpr int RUN = 4;        // strips of a head that a warp takes in a row
constexpr int LD = 12;        // floats between rows of 8 in shared memory: 8 lanes' 16 bytes in distinct banks

// A group's tokens in shared memory.  q and k as a lane reads them (token g, columns 32 j + 8 t .. + 7).
template <int D, typename T>
struct Tokens {
  uint4 k[PLANES<T>][D / 32][32];
  float gate[GROUP], beta[GROUP];
};
// What a group's tokens are to each other.
struct Factors {
  float A[GROUP * GROUP];                     // R_ij (k_i . k_j), column j together
  float c[GROUP], rest[GROUP];                // c_i, R_mi
};
template <int D, typename T, int G>
struct Scratch {                              // of a warp
  float4 state[STRIP][D / 4];                 // the next strip's; in odd rows 16-byte units 2 i, 2 i + 1 swapped
  Tokens<D, T> pend[G], fresh[G];
  uint4 q[G][PLANES<T>][D / 32][32];
  Factors fp[G], ff[G];
  T v[2][2][G][GROUP][STRIP];                 // values of this strip and the next, pending and fresh
  float B[G][GROUP * GROUP];                  // R_ij (q_i . k_j) of fresh tokens
  float X[ONE_PASS<T, G> ? 2 : 1][ONE_PASS<T, G> ? GROUP * GROUP : 4];     // k_i . k_j, q_i . k_j of fresh i and pending j (both())
  float dk[STRIP * LD], dq[STRIP * LD];       // S k, then the rows' weights; S q
  float df[ONE_PASS<T, G> ? STRIP * LD : 4];          // S k of fresh tokens where dk is of pending ones
};

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The same for FP32 results, added outside: the tensor core cuts its sums instead of rounding them,
// and a row of them would add up to ten FP32 roundings.
__device__ __forceinline__ void add_mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  float x[4] = {};
  mma_bf16(x, a, b0, b1);
#pragma unroll
  for (int i = 0; i < 4; ++i) d[i] += x[i];
}
// (from zero)
__device__ __forceinline__ void mma_bf16_k8(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t b0) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5}, {%6}, {%7,%7,%7,%7};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(b0), "f"(0.f));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
template <int BYTES>
__device__ __forceinline__ void copy(void* to, const void* from) {
  const uint32_t s = (uint32_t)__cvta_generic_to_shared(to);
  if (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(s), "l"(from) : "memory");
  else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(s), "l"(from), "n"(BYTES) : "memory");
}
// The same, or zeros in its place (`from` is not read then).
template <int BYTES>
__device__ __forceinline__ void copy_or_zero(void* to, const void* from, bool on) {
  const uint32_t s = (uint32_t)__cvta_generic_to_shared(to), n = on ? BYTES : 0;
  if (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(s), "l"(from), "r"(n) : "memory");
  else asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;" ::"r"(s), "l"(from), "r"(n), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits for all but the LEFT last groups of copies.
template <int LEFT>
__device__ __forceinline__ void wait() { asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory"); }

// 32 bytes of a lane: four lanes write a whole line.
__device__ __forceinline__ void store32(float* to, float2 a, float2 b, float2 c, float2 d) {
  asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(to), "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y),
               "f"(c.x), "f"(c.y), "f"(d.x), "f"(d.y) : "memory");
}

// A strip: its number, its sequence's slot and accepted and drafted tokens (both 0: nothing to do).
struct Strip {
  unsigned at;
  int slot, a, m;
};
struct Place {
  int n, h, row0;
};
template <int D>
__device__ __forceinline__ Place place_of(const DraftParams& p, unsigned at) {
  const int nh = (int)(at / (D / STRIP)), n = p.by_head(nh);
  return {n, nh - n * p.H, (int)(at % (D / STRIP)) * STRIP};
}
template <int D>
__device__ __forceinline__ Strip strip_at(const DraftParams& p, unsigned at, unsigned strips) {
  Strip s{at, 0, 0, 0};
  if (at >= strips) return s;
  const int n = p.by_head((int)(s.at / (D / STRIP)));
  s.slot = p.idx ? p.idx[n] : n;
  if (p.idx ? s.slot > 0 && s.slot < p.num_slots : s.slot < p.num_slots) {
    s.a = p.pend.num ? min(max(p.pend.num[n], 0), p.pend.rows) : p.pend.rows;
    s.m = p.fresh.num ? min(max(p.fresh.num[n], 0), p.fresh.rows) : p.fresh.rows;
  }
  return s;
}
template <int D>
__device__ __forceinline__ float* state_of(const DraftParams& p, const Strip& s) {
  const Place at = place_of<D>(p, s.at);
  return p.pool + (((int64_t)s.slot * p.H + at.h) * D + at.row0) * D;
}
// (Whole rows to a copy.)
template <int D, typename W>
__device__ __forceinline__ void fetch_state(const DraftParams& p, const Strip& s, W& w) {
  if (s.a | s.m) {
    constexpr int U = D / 4, R = 32 / U > 0 ? 32 / U : 1;    // units of a row, rows of a copy
    const int lane = threadIdx.x & 31, r = lane / U, c = lane % U;
    const float* S = state_of<D>(p, s) + lane * 4;
#pragma unroll
    for (int i = 0; i < STRIP / R; ++i) copy<16>(&w.state[i * R + r][c ^ ((i * R + r) & 1)], S + i * R * D);
  }
}
// Eight FP32 values of a lane as three BF16 summands each (zeros if not `on`).
template <int J>
__device__ __forceinline__ void split_to(uint4 (*to)[J][32], int j, const float* from, bool on) {
  const float4 a = on ? *reinterpret_cast<const float4*>(from) : make_float4(0.f, 0.f, 0.f, 0.f);
  const float4 b = on ? *reinterpret_cast<const float4*>(from + 4) : make_float4(0.f, 0.f, 0.f, 0.f);
  float2 x[4] = {make_float2(a.x, a.y), make_float2(a.z, a.w), make_float2(b.x, b.y), make_float2(b.z, b.w)};
#pragma unroll
  for (int l = 0; l < 3; ++l) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      u[i] = pack2(x[i]);
      x[i] = sub2(x[i], unpack2(u[i]));
    }
    to[l][j][threadIdx.x & 31] = make_uint4(u[0], u[1], u[2], u[3]);
  }
}
// The queries, keys and gates of the group from token `first` of `count` on; what lies behind its last
// token is zero.
template <int D, bool kDelta, bool kFresh, typename T>
__device__ __forceinline__ void fetch_tokens(const DraftParams& p, const DraftTokens& tok, Tokens<D, T>& to,
                                             uint4 (*q)[D / 32][32], unsigned strip, int first, int count) {
  const int m = min(count - first, GROUP);
  if (m > 0) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const Place at = place_of<D>(p, strip);
    const int64_t token0 = (int64_t)at.n * tok.rows + first;
    // (a token behind the last one of the sequence is not read: any address of the tensor does)
    const int64_t mine = ((token0 + (g < m ? g : 0)) * p.HK + p.by_group(at.h)) * D + 8 * t;
    const T* k = reinterpret_cast<const T*>(tok.k) + mine;
    const T* x = kFresh ? reinterpret_cast<const T*>(tok.q) + mine : nullptr;
#pragma unroll
    for (int j = 0; j < D / 32; ++j) {
      if constexpr (PLANES<T> == 1) {
        copy_or_zero<16>(&to.k[0][j][lane], k + j * 32, g < m);
        if (kFresh) copy_or_zero<16>(&q[0][j][lane], x + j * 32, g < m);
      } else {
        split_to(to.k, j, k + j * 32, g < m);
        if (kFresh) split_to(q, j, x + j * 32, g < m);
      }
    }
    const int i = lane & 7;
    if (kDelta && lane < 2 * GROUP && i < m)
      copy<4>(lane < GROUP ? &to.gate[i] : &to.beta[i],
              (lane < GROUP ? tok.gate : tok.beta) + (token0 + i) * p.H + at.h);
  }
}
// The values of a group of the strip's rows.
template <int D, typename T>
__device__ __forceinline__ void fetch_values(const DraftParams& p, const DraftTokens& tok, T (*v)[STRIP],
                                             unsigned strip, int first, int count) {
  const int m = min(count - first, GROUP);
  if (m > 0) {
    constexpr int E = 16 / sizeof(T), UNITS = STRIP / E;      // units of a token's values
    const int lane = threadIdx.x & 31, i = lane / UNITS, part = lane % UNITS * E;
    const Place at = place_of<D>(p, strip);
    const int64_t token = (int64_t)at.n * tok.rows + first + (i < m ? i : 0);
    if (lane < GROUP * UNITS)
      copy_or_zero<16>(&v[i][part],
                       reinterpret_cast<const T*>(tok.v) + (token * p.H + at.h) * D + at.row0 + part, i < m);
  }
}
// All the groups that the buffers hold, if they are to be loaded.
template <int D, bool kDelta, bool kFresh, typename W>
__device__ __forceinline__ void fetch_groups(const DraftParams& p, W& w, unsigned strip, int count, bool on) {
  constexpr int G = sizeof(w.fp) / sizeof(Factors);
  if (on) {
#pragma unroll
    for (int i = 0; i < G; ++i) {
      if (kFresh) fetch_tokens<D, kDelta, true>(p, p.fresh, w.fresh[i], w.q[i], strip, i * GROUP, count);
      else fetch_tokens<D, kDelta, false>(p, p.pend, w.pend[i], w.q[0], strip, i * GROUP, count);
    }
  }
  commit();
}
// A strip's state and values.
template <int D, typename W>
__device__ __forceinline__ void fetch_strip(const DraftParams& p, const Strip& s, W& w, int side) {
  constexpr int G = sizeof(w.fp) / sizeof(Factors);
  fetch_state<D>(p, s, w);
#pragma unroll
  for (int i = 0; i < G; ++i) {
    fetch_values<D>(p, p.pend, w.v[side][0][i], s.at, i * GROUP, s.a);
    fetch_values<D>(p, p.fresh, w.v[side][1][i], s.at, i * GROUP, s.m);
  }
  commit();
}

// k_i . x_j (rows g) and q_i . x_j (rows g + 8) for j = 2 t, 2 t + 1.
template <int D, bool kQueries, typename T>
__device__ __forceinline__ void token_products(float (&c)[4], const uint4 (*ks)[D / 32][32], const uint4 (*qs)[D / 32][32],
                                               const uint4 (*xs)[D / 32][32]) {
  const int lane = threadIdx.x & 31;
  float small[4] = {};
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = 0.f;
#pragma unroll
  for (int l = 0; l < PLANES<T>; ++l)
#pragma unroll
    for (int o = 0; o + l < PLANES<T>; ++o)
#pragma unroll
      for (int j = 0; j < D / 32; ++j) {
        const uint4 k = ks[l][j][lane], q = kQueries ? qs[l][j][lane] : make_uint4(0, 0, 0, 0), z = xs[o][j][lane];
        const uint32_t x[4] = {k.x, q.x, k.y, q.y}, y[4] = {k.z, q.z, k.w, q.w};
        if (PLANES<T> == 1) {
          mma_bf16(c, x, z.x, z.y);
          mma_bf16(c, y, z.z, z.w);
        } else if (l + o == 0) {
          add_mma(c, x, z.x, z.y);
          add_mma(c, y, z.z, z.w);
        } else {
          mma_bf16(small, x, z.x, z.y);
          mma_bf16(small, y, z.z, z.w);
        }
      }
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] += small[i];
}
// The products of fresh tokens with pending keys.
template <int D, typename T, typename W>
__device__ __forceinline__ void cross_products(W& w) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  float c[4];
  token_products<D, true, T>(c, w.fresh[0].k, w.q[0], w.pend[0].k);
  w.X[0][2 * t * GROUP + g] = c[0];
  w.X[0][(2 * t + 1) * GROUP + g] = c[1];
  w.X[1][2 * t * GROUP + g] = c[2];
  w.X[1][(2 * t + 1) * GROUP + g] = c[3];
  __syncwarp();
}

// The factors of a group of m tokens.
template <int D, bool kDelta, bool kFresh, typename T>
__device__ __forceinline__ void factors(const DraftParams& p, const Tokens<D, T>& tok, const uint4 (*qs)[D / 32][32],
                                        Factors& f, float* B, unsigned strip, int m) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  // the decay of token lane % 8
  float lam = 1.f;
  if ((lane & 7) < m) lam = expf(kDelta ? tok.gate[lane & 7] : p.decay[place_of<D>(p, strip).h]);
  if (kDelta || kFresh) {
    float c[4];
    token_products<D, kFresh, T>(c, tok.k, qs, tok.k);
    float R0 = 1.f, R1 = 1.f;
#pragma unroll
    for (int l = 1; l < GROUP; ++l) {
      const float x = __shfl_sync(0xffffffffu, lam, l);
      if (l <= g && l > 2 * t) R0 *= x;
      if (l <= g && l > 2 * t + 1) R1 *= x;
    }
    if (kDelta) {
      f.A[2 * t * GROUP + g] = R0 * c[0];
      f.A[(2 * t + 1) * GROUP + g] = R1 * c[1];
    }
    if (kFresh) {
      B[2 * t * GROUP + g] = R0 * c[2];
      B[(2 * t + 1) * GROUP + g] = R1 * c[3];
    }
  }
  // products of the decays up to a token and from behind it to the last one
  float c = lam, rest = __shfl_down_sync(0xffffffffu, lam, 1, 8);
  if ((lane & 7) == 7) rest = 1.f;
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) {
    const float x = __shfl_up_sync(0xffffffffu, c, o, 8), y = __shfl_down_sync(0xffffffffu, rest, o, 8);
    if ((lane & 7) >= o) c *= x;
    if ((lane & 7) + o < 8) rest *= y;
  }
  if (lane < GROUP) {
    f.c[lane] = c;
    f.rest[lane] = rest;
  }
  __syncwarp();
}

// s[j][e][i]: row g + 8 i, columns 32 j + 8 t + 2 e, + 1 of a strip's state.
template <int D>
using State = float2[D / 32][4][2];

// S k of up to 8 pending tokens (to dk) and S k, S q of up to 8 fresh ones (to df and dq).
template <int D, bool kDelta, bool kPend, bool kFresh, typename T>
__device__ __forceinline__ void read_state(const State<D>& s, const uint4 (*pk)[D / 32][32], const uint4 (*fk)[D / 32][32],
                                           const uint4 (*fq)[D / 32][32], float* dk, float* df, float* dq) {
  constexpr int NP = PLANES<T>;
  constexpr bool kP = kPend && kDelta, kF = kFresh && kDelta;
  constexpr int SUMMANDS = 3;     // of the state
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  float cp[2][4] = {}, cf[2][4] = {}, cq[2][4] = {};
  const uint4 none = make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int j = 0; j < D / 32; ++j) {
    uint4 k[NP], f[NP], q[NP];
#pragma unroll
    for (int o = 0; o < NP; ++o) {
      k[o] = kP ? pk[o][j][lane] : none;
      f[o] = kF ? fk[o][j][lane] : none;
      q[o] = kFresh ? fq[o][j][lane] : none;
    }
#pragma unroll
    for (int e = 0; e < 4; e += 2) {
      float2 x[4] = {s[j][e][0], s[j][e][1], s[j][e + 1][0], s[j][e + 1][1]};
#pragma unroll
      for (int l = 0; l < SUMMANDS; ++l) {
        uint32_t a[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          a[i] = pack2(x[i]);
          if (l + 1 < SUMMANDS) x[i] = sub2(x[i], unpack2(a[i]));
        }
        // (products of summands l and o below 2^-24 of the whole are left out)
#pragma unroll
        for (int o = 0; o < NP && o + l < 3; ++o) {
          auto add = [&](float (&c)[2][4], const uint4& y) {
            const uint32_t b0 = e ? y.z : y.x, b1 = e ? y.w : y.y;
            if (NP > 1 && l + o == 0) add_mma(c[0], a, b0, b1);
            else mma_bf16(c[NP > 1 ? 1 : l & 1], a, b0, b1);       // (FP32: the small products together)
          };
          if (kP) add(cp, k[o]);
          if (kF) add(cf, f[o]);
          if (kFresh) add(cq, q[o]);
        }
      }
    }
  }
  auto store = [&](float* to, const float (&c)[2][4]) {
    *reinterpret_cast<float2*>(&to[g * LD + 2 * t]) = make_float2(c[0][0] + c[1][0], c[0][1] + c[1][1]);
    *reinterpret_cast<float2*>(&to[(g + 8) * LD + 2 * t]) = make_float2(c[0][2] + c[1][2], c[0][3] + c[1][3]);
  };
  if (kP) store(dk, cp);
  if (kF) store(df, cf);
  if (kFresh) store(dq, cq);
  __syncwarp();
}

__device__ __forceinline__ void load8(float (&x)[GROUP], const float* from) {
  *reinterpret_cast<float4*>(x) = *reinterpret_cast<const float4*>(from);
  *reinterpret_cast<float4*>(x + 4) = *reinterpret_cast<const float4*>(from + 4);
}

// u of row lane % 16 from S k (both halves of the warp the same); with queries the outputs, from S q to
// `out` (a token every `step`), column by column of A and B.
template <bool kDelta, bool kFresh, typename T>
__device__ __forceinline__ void solve(float (&u)[GROUP], float (&o)[GROUP], const float (&c)[GROUP], const T (*v)[STRIP],
                                      const float* beta, const float* A, const float* B, int m, T* out, int step,
                                      float scale) {
  const int lane = threadIdx.x & 31, r = lane & 15;
#pragma unroll
  for (int i = 0; i < GROUP; ++i) {
    const float x = to_f(v[i][r]);
    u[i] = kDelta ? fmaf(-c[i], u[i], x) : x;
    if (kFresh) o[i] *= c[i];
  }
#pragma unroll
  for (int j = 0; j < GROUP; ++j) {
    if (j >= m) break;
    float x[GROUP];
    if (kDelta) {
      u[j] *= beta[j];
      load8(x, &A[j * GROUP]);
#pragma unroll
      for (int i = j + 1; i < GROUP; ++i) u[i] = fmaf(-x[i], u[j], u[i]);
    }
    if (kFresh) {
      load8(x, &B[j * GROUP]);
#pragma unroll
      for (int i = j; i < GROUP; ++i) o[i] = fmaf(x[i], u[j], o[i]);
      if (lane >> 4 == (j & 1)) *out = from_f<T>(scale * o[j]);
      out += step;
    }
  }
}

// u becomes the rows' weights R_mj u_j, a copy of them in shared memory.
__device__ __forceinline__ void weights(float (&u)[GROUP], const float* rest, int m, float* to) {
  const int lane = threadIdx.x & 31;
  float x[GROUP];
  load8(x, rest);
#pragma unroll
  for (int i = 0; i < GROUP; ++i) u[i] = i < m ? u[i] * x[i] : 0.f;
  __syncwarp();
  if (lane < STRIP) {
    *reinterpret_cast<float4*>(&to[lane * LD]) = make_float4(u[0], u[1], u[2], u[3]);
    *reinterpret_cast<float4*>(&to[lane * LD + 4]) = make_float4(u[4], u[5], u[6], u[7]);
  }
  __syncwarp();
}

// S = c S + W K.
template <int D, typename T>
__device__ __forceinline__ void update(State<D>& s, float c, const float* W, const uint4 (*ks)[D / 32][32]) {
  constexpr int NP = PLANES<T>;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  uint32_t a[4], last[2];     // rows g, g + 8: the first two summands as 16 columns, and the third
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float2 x = *reinterpret_cast<const float2*>(&W[(g + 8 * i) * LD + 2 * t]);
    a[i] = pack2(x);
    x = sub2(x, unpack2(a[i]));
    a[i + 2] = pack2(x);
    last[i] = pack2(sub2(x, unpack2(a[i + 2])));
  }
  const float2 c2 = make_float2(c, c);
  const uint32_t ends[4] = {last[0], last[1], a[0], a[1]};     // the third summand, and the first once more
#pragma unroll
  for (int j = 0; j < D / 32; ++j) {
    uint32_t pairs[NP][4];
#pragma unroll
    for (int o = 0; o < NP; ++o) {
      const uint4 k = ks[o][j][lane];
      pairs[o][0] = k.x; pairs[o][1] = k.y; pairs[o][2] = k.z; pairs[o][3] = k.w;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float d[4];
      const uint32_t x = transpose8(pairs[0][e]);
      if constexpr (NP == 1) {
        mma_bf16_k8(d, last[0], last[1], x);
      } else {
        const uint32_t y = transpose8(pairs[1][e]), z = transpose8(pairs[2][e]);
        d[0] = d[1] = d[2] = d[3] = 0.f;
        mma_bf16(d, ends, x, z);
        mma_bf16(d, a, y, y);
      }
      mma_bf16(d, a, x, x);
      s[j][e][0] = fma2(c2, s[j][e][0], make_float2(d[0], d[1]));
      s[j][e][1] = fma2(c2, s[j][e][1], make_float2(d[2], d[3]));
    }
  }
  __syncwarp();
}

// A strip's rows of the outputs from token `first` on, its lane's row.
template <int D, typename T>
__device__ __forceinline__ T* out_of(const DraftParams& p, unsigned strip, int first) {
  const Place at = place_of<D>(p, strip);
  return reinterpret_cast<T*>(p.out) +
         (((int64_t)at.n * p.fresh.rows + first) * p.H + at.h) * D + at.row0 + (threadIdx.x & 15);
}
template <int D>
__device__ __forceinline__ void store_state(const DraftParams& p, const Strip& at, const State<D>& s) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  float* S = state_of<D>(p, at) + g * D + 8 * t;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < D / 32; ++j) store32(S + i * 8 * D + j * 32, s[j][0][i], s[j][1][i], s[j][2][i], s[j][3][i]);
}

// Group b of up to 8 pending tokens, m of them: the state is advanced.
template <int D, bool kDelta, typename T, typename W>
__device__ __forceinline__ void pending(State<D>& s, W& w, int side, int b, int m) {
  const int r = threadIdx.x & 15;
  if (kDelta)
    read_state<D, true, true, false, T>(s, w.pend[b].k, nullptr, nullptr, w.dk, nullptr, nullptr);
  float u[GROUP], c[GROUP];
  if (kDelta) load8(u, &w.dk[r * LD]);
  load8(c, w.fp[b].c);
  solve<kDelta, false, T>(u, u, c, w.v[side][0][b], w.pend[b].beta, w.fp[b].A, nullptr, m, nullptr, 0, 0.f);
  weights(u, w.fp[b].rest, m, w.dk);
  update<D, T>(s, c[GROUP - 1], w.dk, w.pend[b].k);
}

// The same for fresh ones: their outputs, and the state for the group behind them if there is one.
template <int D, bool kDelta, typename T, typename W>
__device__ __forceinline__ void fresh(const DraftParams& p, State<D>& s, W& w, unsigned strip, int side, int b, int first,
                                      int m, bool more) {
  const int r = threadIdx.x & 15;
  read_state<D, kDelta, false, true, T>(s, nullptr, w.fresh[b].k, w.q[b], nullptr, w.dk, w.dq);
  float u[GROUP], o[GROUP], c[GROUP];
  if (kDelta) load8(u, &w.dk[r * LD]);
  load8(o, &w.dq[r * LD]);
  load8(c, w.ff[b].c);
  solve<kDelta, true, T>(u, o, c, w.v[side][1][b], w.fresh[b].beta, w.ff[b].A, w.B[b], m, out_of<D, T>(p, strip, first),
                         p.H * D, p.scale);
  if (more) {
    weights(u, w.ff[b].rest, m, w.dk);
    update<D, T>(s, c[GROUP - 1], w.dk, w.fresh[b].k);
  }
  __syncwarp();
}

// A group of a pending tokens and one of m fresh ones in one pass over the state before both: with W the
// pending rows' weights, S' x = c S x + W (K x) for the fresh k and q.
template <int D, bool kDelta, typename T, typename W>
__device__ __forceinline__ void both(const DraftParams& p, State<D>& s, W& w, const Strip& at, int side) {
  const int r = threadIdx.x & 15;
  read_state<D, kDelta, true, true, T>(s, w.pend[0].k, w.fresh[0].k, w.q[0], w.dk, w.df, w.dq);
  float u[GROUP], c[GROUP];
  if (kDelta) load8(u, &w.dk[r * LD]);
  load8(c, w.fp[0].c);
  solve<kDelta, false, T>(u, u, c, w.v[side][0][0], w.pend[0].beta, w.fp[0].A, nullptr, at.a, nullptr, 0, 0.f);
  weights(u, w.fp[0].rest, at.a, w.dk);
  const float ce = c[GROUP - 1];
  update<D, T>(s, ce, w.dk, w.pend[0].k);
  store_state<D>(p, at, s);

  float f[GROUP], o[GROUP];
  if (kDelta) load8(f, &w.df[r * LD]);
  load8(o, &w.dq[r * LD]);
#pragma unroll
  for (int i = 0; i < GROUP; ++i) {
    if (kDelta) f[i] *= ce;
    o[i] *= ce;
  }
#pragma unroll
  for (int j = 0; j < GROUP; ++j) {
    if (j >= at.a) break;
    float x[GROUP];
    if (kDelta) {
      load8(x, &w.X[0][j * GROUP]);
#pragma unroll
      for (int i = 0; i < GROUP; ++i) f[i] = fmaf(x[i], u[j], f[i]);
    }
    load8(x, &w.X[1][j * GROUP]);
#pragma unroll
    for (int i = 0; i < GROUP; ++i) o[i] = fmaf(x[i], u[j], o[i]);
  }
  load8(c, w.ff[0].c);
  solve<kDelta, true, T>(f, o, c, w.v[side][1][0], w.fresh[0].beta, w.ff[0].A, w.B[0], at.m, out_of<D, T>(p, at.at, 0),
                         p.H * D, p.scale);
  __syncwarp();
}

template <int D, bool kDelta, typename T, int G>
__global__ void __launch_bounds__(32, CTAS<D, T, G>) draft_kernel(const DraftParams p) {
  constexpr int J = D / 32;
  extern __shared__ __align__(16) char smem[];
  const int lane = threadIdx.x, g = lane >> 2, t = lane & 3;
  Scratch<D, T, G>& w = *reinterpret_cast<Scratch<D, T, G>*>(smem);
  // A warp takes `run` strips of a head in a row, then the run as many warps on: the tokens and their
  // factors stay for a run.
  const unsigned run = p.run;     // a power of two
  const unsigned strips = (unsigned)p.N * p.H * (D / STRIP), ahead = gridDim.x * run;
  unsigned where = blockIdx.x * run;
  auto next_at = [&](unsigned x) { return (x + 1) & (run - 1) ? x + 1 : x + 1 - run + ahead; };
  Strip at = strip_at<D>(p, where, strips), next = strip_at<D>(p, next_at(where), strips);
  // Copies are committed in the order of a strip's state and values, its pending tokens, its fresh
  // tokens (the last two with the first strip of a run alone): each where the buffer is free, a phase or
  // two ahead of its use.
  int side = 0;
  fetch_strip<D>(p, at, w, side);
  fetch_groups<D, kDelta, false>(p, w, at.at, at.a, true);
  fetch_groups<D, kDelta, true>(p, w, at.at, at.m, true);
  bool new_pend = true, new_fresh = true;   // the buffers hold tokens whose factors are not formed yet
#pragma unroll 1
  for (; where < strips; where = next_at(where)) {
    Strip after = next;
    after.at = next_at(next.at);
    if ((after.at & (run - 1)) == 0) after = strip_at<D>(p, after.at, strips);
    if (at.m < p.fresh.rows) {
      T* out = out_of<D, T>(p, where, at.m + (lane >> 4));
      for (int i = at.m + (lane >> 4); i < p.fresh.rows; i += 2, out += 2 * p.H * D) *out = from_f<T>(0.f);
    }
    const bool last = ((where + 1) & (run - 1)) == 0, one_pass = ONE_PASS<T, G> && at.a > 0 && at.m > 0;
    State<D> s;
    if (one_pass) wait<0>();
    else wait<1>();
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
          const float4 x = w.state[g + 8 * i][(8 * j + 2 * t + e / 2) ^ (g & 1)];
          s[j][e][i] = make_float2(x.x, x.y);
          s[j][e + 1][i] = make_float2(x.z, x.w);
        }
    __syncwarp();
    fetch_strip<D>(p, next, w, side ^ 1);
    if (one_pass) {
      if constexpr (ONE_PASS<T, G>) {
        if (new_pend) {      // (both kinds are new at once)
          factors<D, kDelta, false>(p, w.pend[0], w.q[0], w.fp[0], w.B[0], at.at, at.a);
          factors<D, kDelta, true>(p, w.fresh[0], w.q[0], w.ff[0], w.B[0], at.at, at.m);
          cross_products<D, T>(w);
        }
        both<D, kDelta, T>(p, s, w, at, side);
        new_pend = new_fresh = last;
        fetch_groups<D, kDelta, false>(p, w, next.at, next.a, last);
        fetch_groups<D, kDelta, true>(p, w, next.at, next.m, last);
      }
    } else {
#pragma unroll 1
      for (int first = 0; first < at.a; first += GROUP) {
        const int i = first / GROUP % G, m = min(at.a - first, GROUP);
        const bool late = first >= G * GROUP;        // a group that the buffers do not hold yet
        if (late) {
          fetch_tokens<D, kDelta, false>(p, p.pend, w.pend[i], w.q[0], at.at, first, at.a);
          fetch_values<D>(p, p.pend, w.v[side][0][i], at.at, first, at.a);
          commit();
          wait<0>();
          __syncwarp();
        }
        if (late || new_pend) factors<D, kDelta, false>(p, w.pend[i], w.q[0], w.fp[i], w.B[0], at.at, m);
        pending<D, kDelta, T>(s, w, side, i, m);
      }
      new_pend = last || at.a > G * GROUP;
      fetch_groups<D, kDelta, false>(p, w, next.at, next.a, new_pend);
      if (at.a > 0) store_state<D>(p, at, s);
      wait<2>();
      __syncwarp();
#pragma unroll 1
      for (int first = 0; first < at.m; first += GROUP) {
        const int i = first / GROUP % G, m = min(at.m - first, GROUP);
        const bool late = first >= G * GROUP;
        if (late) {
          fetch_tokens<D, kDelta, true>(p, p.fresh, w.fresh[i], w.q[i], at.at, first, at.m);
          fetch_values<D>(p, p.fresh, w.v[side][1][i], at.at, first, at.m);
          commit();
          wait<0>();
          __syncwarp();
        }
        if (late || new_fresh) factors<D, kDelta, true>(p, w.fresh[i], w.q[i], w.ff[i], w.B[i], at.at, m);
        fresh<D, kDelta, T>(p, s, w, at.at, side, i, first, m, first + GROUP < at.m);
      }
      new_fresh = last || at.m > G * GROUP;
      fetch_groups<D, kDelta, true>(p, w, next.at, next.m, new_fresh);
    }
    at = next;
    next = after;
    side ^= 1;
  }
}

template <int D, bool kDelta, typename T, int G>
cudaError_t go(DraftParams p, cudaStream_t st) {
  const int strips = p.N * p.H * (D / STRIP);
  // Strips in a row save work, but the CTAs take whole runs in turns.  The costs of a strip in runs of one
  // and two, to those in runs of four, are those of 5 + 5 BF16 tokens, K = 128 (1.17, 1.02 by other sizes; 115
  // us, 102, 96 as first measured).  Others differ, measured with 64 or 96 sequences of 32 heads: 16 + 16 tokens
  // 1.15, 1.07; linear attention 1.09, 0.98; drafts alone 1.10, 0.99; commits 0.97, 0.96; K = 64 1.16, 1.01; FP32
  // 1.43, 1.17, and 1.65, 1.29 with two groups.
  constexpr int kSlots = 152 * CTAS<D, T, G>;
  double best = 0;
  for (int run = 1; run <= RUN; run *= 2) {
    const int turns = (strips / run + kSlots - 1) / kSlots;
    const double time = turns * run * (run == 1 ? 1.18 : run == 2 ? 1.06 : 1.0);
    if (run == 1 || time < best) {
      best = time;
      p.run = run;
    }
  }
  const int want = strips / p.run, grid = want < kSlots ? want : kSlots;
  constexpr int bytes = (int)sizeof(Scratch<D, T, G>);
  static_assert(CTAS<D, T, G> * (bytes + 1024) <= 228 * 1024, "shared memory of an SM");
  auto kernel = draft_kernel<D, kDelta, T, G>;
  if (bytes > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
  }
  kernel<<<grid, 32, bytes, st>>>(p);
  return cudaGetLastError();
}

template <int D, typename T, int G>
cudaError_t rule(const DraftParams& p, cudaStream_t st) {
  return p.decay ? go<D, false, T, G>(p, st) : go<D, true, T, G>(p, st);
}
// Two groups in shared memory where a sequence may have them: otherwise each strip would load its
// tokens again (64 sequences of 32 heads, 16 + 16 tokens, delta rule and linear attention, BF16 93 and
// 75 us against 86 and 66, FP32 268 and 164 against 222 and 136).
template <int D, typename T>
cudaError_t groups(const DraftParams& p, cudaStream_t st) {
  return p.pend.rows > GROUP || p.fresh.rows > GROUP ? rule<D, T, 2>(p, st) : rule<D, T, 1>(p, st);
}

}  // namespace

cudaError_t launch_draft_step(const DraftParams& p, bool bf16, int D, cudaStream_t st) {
  if (p.N < 1 || p.pend.rows + p.fresh.rows == 0) return cudaSuccess;
  if (bf16) return D == 128 ? groups<128, __nv_bfloat16>(p, st) : groups<64, __nv_bfloat16>(p, st);
  return D == 128 ? groups<128, float>(p, st) : groups<64, float>(p, st);
}

}  // namespace sfg
