// draft_step.cu -- several FP32 tokens of every sequence on the paged pool of FP32 states [V,K]
// (include/sf_decode.h): accepted tokens advance the state, drafted ones read it.
//
// Chunk form over m tokens from the state S0, with lam_i = e^{gate_i} (e^{decay_h}),
// c_i = lam_1 .. lam_i and R_ij = lam_{j+1} .. lam_i:
//     u_i   = beta_i (v_i - c_i S0 k_i - sum_{j<i} R_ij (k_i . k_j) u_j)      (u_i = v_i without delta)
//     out_i = scale (c_i S0 q_i + sum_{j<=i} R_ij (q_i . k_j) u_j)
//     S_m   = c_m S0 + sum_j R_mj u_j k_j^T
// The R_ij are products, not exponentials of differences of sums, so that a gate of -inf gives 0
// and not NaN.  The state is touched 2 m times for the drafts and 2 m + 1 for the accepted ones,
// against 4 m for each by the rule itself.
#include "common.cuh"
#include "decode.cuh"

namespace sfg {
namespace {

constexpr int ROWS = 64;      // rows of a state that a CTA holds
constexpr int THREADS = 128;  // 4 warps of 16 rows; 8 lanes share a row
constexpr int RL = 4;         // rows of a lane

__device__ __forceinline__ float4 ld4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float dot4(float4 a, float4 b, float c) {
  return fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, c))));
}

// Sums 4 values over 8 lanes; a lane ends with value (lane / 2) % 4.
__device__ __forceinline__ float sum_rows(float (&x)[RL], int lane) {
  const bool b4 = lane & 4, b2 = lane & 2;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float send = b4 ? x[i] : x[i + 2], keep = b4 ? x[i + 2] : x[i];
    x[i] = keep + __shfl_xor_sync(0xffffffffu, send, 4);
  }
  const float send = b2 ? x[0] : x[1], keep = b2 ? x[1] : x[0];
  const float y = keep + __shfl_xor_sync(0xffffffffu, send, 2);
  return y + __shfl_xor_sync(0xffffffffu, y, 1);
}

// A CTA's tokens in shared memory, FP32.
struct Tok {
  float *k, *q, *v;          // [rows][D], [rows][D], [rows][ROWS]
  float *A, *B;              // [rows][rows]: R_ij (k_i . k_j), R_ij (q_i . k_j)
  float *lam, *beta, *c;     // [rows]
  float *dk, *dq;            // [rows][ROWS]: S0 k_i (then u_i), S0 q_i
};
constexpr size_t tok_floats(int rows, int D, bool reads, bool delta) {
  const size_t n = (size_t)rows * (D + ROWS + 3 + ROWS) + (delta ? (size_t)rows * rows : 0) +
                   (reads ? (size_t)rows * (D + ROWS + rows) : 0);
  return (n + 3) / 4 * 4;
}
__device__ __forceinline__ float* carve(float* s, Tok& t, int rows, int D, bool reads, bool delta) {
  t.k = s; s += rows * D;
  t.v = s; s += rows * ROWS;
  t.dk = s; s += rows * ROWS;
  t.q = t.dq = t.A = t.B = nullptr;
  if (reads) {
    t.q = s; s += rows * D;
    t.dq = s; s += rows * ROWS;
    t.B = s; s += rows * rows;
  }
  if (delta) { t.A = s; s += rows * rows; }
  t.lam = s; s += rows;
  t.beta = s; s += rows;
  t.c = s; s += rows;
  return s;
}

template <int D, bool kDelta>
__device__ __forceinline__ void load_tokens(const DraftTokens& g, const Tok& t, int m, int n, int h, int hk,
                                            int row0, const DraftParams& p) {
  constexpr int LK = D / 4;
  for (int i = threadIdx.x; i < m * LK; i += THREADS) {
    const int r = i / LK, c = (i % LK) * 4;
    const size_t at = (((size_t)n * g.rows + r) * p.HK + hk) * D + c;
    *reinterpret_cast<float4*>(t.k + r * D + c) = ld4(static_cast<const float*>(g.k) + at);
    if (t.q) *reinterpret_cast<float4*>(t.q + r * D + c) = ld4(static_cast<const float*>(g.q) + at);
  }
  for (int i = threadIdx.x; i < m * (ROWS / 4); i += THREADS) {
    const int r = i / (ROWS / 4), c = (i % (ROWS / 4)) * 4;
    const size_t at = (((size_t)n * g.rows + r) * p.H + h) * D + row0 + c;
    *reinterpret_cast<float4*>(t.v + r * ROWS + c) = ld4(static_cast<const float*>(g.v) + at);
  }
  for (int r = threadIdx.x; r < m; r += THREADS) {
    const size_t at = ((size_t)n * g.rows + r) * p.H + h;
    t.lam[r] = expf(kDelta ? g.gate[at] : p.decay[h]);
    t.beta[r] = kDelta ? g.beta[at] : 1.f;
  }
}

// A, B and c.
template <int D, bool kDelta>
__device__ __forceinline__ void products(const Tok& t, int m, int rows) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int e = warp; e < m * m; e += THREADS / 32) {
    const int i = e / m, j = e % m;
    if (j > i || (!t.B && (j == i || !kDelta))) continue;
    float kk = 0.f, qk = 0.f;
#pragma unroll
    for (int c = lane; c < D; c += 32) {
      const float b = t.k[j * D + c];
      if (kDelta) kk = fmaf(t.k[i * D + c], b, kk);
      if (t.B) qk = fmaf(t.q[i * D + c], b, qk);
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
      kk += __shfl_xor_sync(0xffffffffu, kk, o);
      qk += __shfl_xor_sync(0xffffffffu, qk, o);
    }
    float R = 1.f;
    for (int l = j + 1; l <= i; ++l) R *= t.lam[l];
    if (lane == 0) {
      if (kDelta) t.A[i * rows + j] = R * kk;
      if (t.B) t.B[i * rows + j] = R * qk;
    }
  }
  for (int i = threadIdx.x; i < m; i += THREADS) {
    float c = 1.f;
    for (int l = 0; l <= i; ++l) c *= t.lam[l];
    t.c[i] = c;
  }
}

// dk, dq: the dot products of the CTA's rows of S with the tokens.
template <int D, bool kDelta>
__device__ __forceinline__ void read_state(const float4 (&s)[RL][D / 32], const Tok& t, int m) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = (lane & 7) * 4, row = warp * 16 + (lane >> 3) * RL + ((lane >> 1) & 3);
  for (int i = 0; i < m; ++i) {
#pragma unroll
    for (int what = 0; what < 2; ++what) {
      const float* x = what ? t.q : t.k;
      if (what ? !t.q : !kDelta) continue;
      float a[RL] = {};
#pragma unroll
      for (int b = 0; b < D / 32; ++b) {
        const float4 y = ld4(x + i * D + b * 32 + c);
#pragma unroll
        for (int r = 0; r < RL; ++r) a[r] = dot4(s[r][b], y, a[r]);
      }
      const float y = sum_rows(a, lane);
      if (!(lane & 1)) (what ? t.dq : t.dk)[i * ROWS + row] = y;
    }
  }
}

// dk becomes u.
template <bool kDelta>
__device__ __forceinline__ void solve(const Tok& t, int m, int rows) {
  const int r = threadIdx.x;
  if (r >= ROWS) return;
  for (int i = 0; i < m; ++i) {
    float u = t.v[i * ROWS + r];
    if (kDelta) {
      u = fmaf(-t.c[i], t.dk[i * ROWS + r], u);
      for (int j = 0; j < i; ++j) u = fmaf(-t.A[i * rows + j], t.dk[j * ROWS + r], u);
      u *= t.beta[i];
    }
    t.dk[i * ROWS + r] = u;
  }
}

template <int D, bool kDelta>
__global__ void __launch_bounds__(THREADS) draft_step_kernel(const DraftParams p) {
  extern __shared__ __align__(16) float smem[];
  constexpr int CPS = D / ROWS;       // CTAs of a state
  constexpr int CV = D / 32;
  const int part = blockIdx.x % CPS;
  const int nh = blockIdx.x / CPS, n = nh / p.H, h = nh % p.H, hk = h / (p.H / p.HK);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, row0 = part * ROWS;
  const int P = p.pend.rows, M = p.fresh.rows;
  float* out = static_cast<float*>(p.out);
  const int slot = p.idx ? p.idx[n] : n;
  const bool live = p.idx ? slot > 0 && slot < p.num_slots : slot < p.num_slots;
  int a = !live ? 0 : p.pend.num ? min(max(p.pend.num[n], 0), P) : P;
  int m = !live ? 0 : p.fresh.num ? min(max(p.fresh.num[n], 0), M) : M;
  for (int i = m * ROWS + threadIdx.x; i < M * ROWS; i += THREADS)
    out[(((size_t)n * M + i / ROWS) * p.H + h) * D + row0 + i % ROWS] = 0.f;
  if (a == 0 && m == 0) return;

  const int r0 = warp * 16 + (lane >> 3) * RL, c = (lane & 7) * 4;
  float* S = p.pool + (((size_t)slot * p.H + h) * D + row0 + r0) * D + c;
  float4 s[RL][CV];
#pragma unroll
  for (int r = 0; r < RL; ++r)
#pragma unroll
    for (int b = 0; b < CV; ++b) s[r][b] = ld4(S + (size_t)r * D + b * 32);

  Tok tp, tm;
  float* next = carve(smem, tp, P, D, false, kDelta);
  next += -(next - smem) & 3;
  carve(next, tm, M, D, true, kDelta);
  load_tokens<D, kDelta>(p.pend, tp, a, n, h, hk, row0, p);
  load_tokens<D, kDelta>(p.fresh, tm, m, n, h, hk, row0, p);
  __syncthreads();
  products<D, kDelta>(tp, a, P);
  products<D, kDelta>(tm, m, M);
  if (a > 0) {
    read_state<D, kDelta>(s, tp, a);
    __syncthreads();
    solve<kDelta>(tp, a, P);
    __syncthreads();
    const float ce = tp.c[a - 1];
#pragma unroll
    for (int r = 0; r < RL; ++r)
#pragma unroll
      for (int b = 0; b < CV; ++b) { s[r][b].x *= ce; s[r][b].y *= ce; s[r][b].z *= ce; s[r][b].w *= ce; }
    float R = 1.f;
    for (int i = a - 1; i >= 0; --i) {
      float w[RL];
#pragma unroll
      for (int r = 0; r < RL; ++r) w[r] = R * tp.dk[i * ROWS + r0 + r];
#pragma unroll
      for (int b = 0; b < CV; ++b) {
        const float4 y = ld4(tp.k + i * D + b * 32 + c);
#pragma unroll
        for (int r = 0; r < RL; ++r) {
          s[r][b].x = fmaf(w[r], y.x, s[r][b].x);
          s[r][b].y = fmaf(w[r], y.y, s[r][b].y);
          s[r][b].z = fmaf(w[r], y.z, s[r][b].z);
          s[r][b].w = fmaf(w[r], y.w, s[r][b].w);
        }
      }
      R *= tp.lam[i];
    }
#pragma unroll
    for (int r = 0; r < RL; ++r)
#pragma unroll
      for (int b = 0; b < CV; ++b) *reinterpret_cast<float4*>(S + (size_t)r * D + b * 32) = s[r][b];
  }
  if (m == 0) return;
  read_state<D, kDelta>(s, tm, m);
  __syncthreads();
  solve<kDelta>(tm, m, M);
  __syncthreads();
  for (int e = threadIdx.x; e < m * ROWS; e += THREADS) {
    const int i = e / ROWS, r = e % ROWS;
    float o = tm.c[i] * tm.dq[i * ROWS + r];
    for (int j = 0; j <= i; ++j) o = fmaf(tm.B[i * M + j], tm.dk[j * ROWS + r], o);
    out[(((size_t)n * M + i) * p.H + h) * D + row0 + r] = p.scale * o;
  }
}

template <int D, bool kDelta>
cudaError_t go(const DraftParams& p, cudaStream_t st) {
  const int grid = p.N * p.H * (D / ROWS);
  const size_t bytes = 4 * (tok_floats(p.pend.rows, D, false, kDelta) + tok_floats(p.fresh.rows, D, true, kDelta));
  auto kernel = draft_step_kernel<D, kDelta>;
  if (bytes > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != cudaSuccess) return e;
  }
  kernel<<<grid, THREADS, bytes, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_draft_step(const DraftParams& p, bool bf16, int D, cudaStream_t st) {
  if (p.N < 1 || p.pend.rows + p.fresh.rows == 0) return cudaSuccess;
  if (bf16) return launch_draft_mma(p, D, st);
  if (D == 128) return p.decay ? go<128, false>(p, st) : go<128, true>(p, st);
  return p.decay ? go<64, false>(p, st) : go<64, true>(p, st);
}

}  // namespace sfg
