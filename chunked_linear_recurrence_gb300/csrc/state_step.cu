// state_step.cu -- one token of every sequence on the paged pool of FP32 states [V,K]
// (include/sf_linattn.h): linear attention with a decay, and the gated delta rule.
//
//     linear attention   S' = lam S + v k^T                    out = scale S' q
//     delta rule         S' = e^g S + r k^T, r = beta (v - e^g S k)
// The read of the updated state needs no second pass: S' q = lam (S q) + r (k . q), so each
// row takes its one or two dot products with the old state while it is in registers.
//
// Bound by memory: 8 V K bytes of state per (sequence, head) against ~5 V K operations.  A
// warp holds 8 row-loads in flight (one float4 per lane each; two rows a load at K = 64), and
// the rows of a state are independent, so a CTA takes 64 of them: even one sequence of 16
// heads gives 32 CTAs at K = 128.  Sums over a row's lanes are
// butterflies that halve the number of values with every exchange (9 shuffles for 8 rows
// instead of 40).  Outputs are rounded once, to the token type; the state stays FP32.
// Measured, BF16, K = 128: 256 sequences of 16 heads 82 us, 6.5 TB/s (537 MB; 96 % of the copy
// rate), the delta rule on 128 of 32 heads the same; one sequence of 16 heads 2.8 us, the
// latency of a launch.
#include <cuda_bf16.h>

#include "common.cuh"
#include "linattn.cuh"

namespace sfg {
namespace {

constexpr int NL = 8;     // row loads of a warp
constexpr int ROWS = 64;  // rows of a CTA

__device__ __forceinline__ float4 ldv(const float* p, int c) { return *reinterpret_cast<const float4*>(p + c); }
__device__ __forceinline__ float4 ldv(const __nv_bfloat16* p, int c) {
  const uint2 u = *reinterpret_cast<const uint2*>(p + c);
  const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.x));
  const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.y));
  return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ float dot4(float4 a, float4 b) {
  return fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, a.w * b.w)));
}

// Sums the NL values of every lane over the LPR lanes of a row.  The lane ends with the sum
// of one of them: value `slot`, the same for LPR / NL lanes.
template <int LPR>
__device__ __forceinline__ float reduce_rows(float (&x)[NL], int lane, int& slot) {
  slot = 0;
#pragma unroll
  for (int m = LPR / 2, cnt = NL / 2; m >= 1; m >>= 1, cnt >>= 1) {
    if (cnt >= 1) {
      const bool up = lane & m;
#pragma unroll
      for (int i = 0; i < NL / 2; ++i)
        if (i < cnt) {
          const float send = up ? x[i] : x[i + cnt];
          const float keep = up ? x[i + cnt] : x[i];
          x[i] = keep + __shfl_xor_sync(0xffffffffu, send, m);
        }
      if (up) slot += cnt;
    } else {
      x[0] += __shfl_xor_sync(0xffffffffu, x[0], m);
    }
  }
  return x[0];
}
// The lane (of the LPR of a row) that ends with value i.
template <int LPR>
__device__ __forceinline__ int lane_of(int i) {
  int l = 0;
#pragma unroll
  for (int m = LPR / 2, cnt = NL / 2; cnt >= 1; m >>= 1, cnt >>= 1)
    if (i & cnt) l |= m;
  return l;
}

// Threads of a CTA: 8 warps at K = 128, 4 at K = 64.
template <int D>
constexpr int kThreads = ROWS / (NL * (128 / D)) * 32;

template <typename T, int D, bool kDelta>
__global__ void __launch_bounds__(kThreads<D>) state_step_kernel(const StepParams p) {
  constexpr int LPR = D / 4;          // lanes of a row
  constexpr int R = 32 / LPR;         // rows of a load
  constexpr int CPS = D / ROWS;       // CTAs of a state
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int part = blockIdx.x % CPS;
  const int nh = blockIdx.x / CPS, n = nh / p.H, h = nh % p.H;
  const int hk = h / (p.H / p.HK);
  const int row0 = part * ROWS + warp * NL * R + lane / LPR;   // row of load i: row0 + i R
  const int c = (lane % LPR) * 4;
  T* out = reinterpret_cast<T*>(p.out) + (size_t)nh * D;
  const int slot = p.idx ? p.idx[n] : n;
  if (p.idx ? slot <= 0 || slot >= p.num_slots : slot >= p.num_slots) {   // padding
    if (threadIdx.x < ROWS) out[part * ROWS + threadIdx.x] = from_f<T>(0.f);
    return;
  }
  float* S = p.pool + ((size_t)slot * p.H + h) * D * D + c;
  float4 s[NL];
#pragma unroll
  for (int i = 0; i < NL; ++i) s[i] = *reinterpret_cast<const float4*>(S + (size_t)(row0 + i * R) * D);
  const size_t qk = ((size_t)n * p.HK + hk) * D;
  const float4 q = ldv(reinterpret_cast<const T*>(p.q) + qk, c);
  const float4 k = ldv(reinterpret_cast<const T*>(p.k) + qk, c);
  const float lam = expf(kDelta ? p.gate[nh] : p.decay[h]);
  const float beta = kDelta ? p.beta[nh] : 1.f;
  float kq = dot4(k, q);
#pragma unroll
  for (int m = LPR / 2; m >= 1; m >>= 1) kq += __shfl_xor_sync(0xffffffffu, kq, m);
#pragma unroll
  for (int i = 0; i < NL; ++i) { s[i].x *= lam; s[i].y *= lam; s[i].z *= lam; s[i].w *= lam; }
  float dq[NL];
#pragma unroll
  for (int i = 0; i < NL; ++i) dq[i] = dot4(s[i], q);
  int mine;
  const float sq = reduce_rows<LPR>(dq, lane % LPR, mine);
  const int row = row0 + mine * R;    // the row whose sums this lane holds
  float r = to_f(reinterpret_cast<const T*>(p.v)[(size_t)nh * D + row]);
  if (kDelta) {
    float dk[NL];
#pragma unroll
    for (int i = 0; i < NL; ++i) dk[i] = dot4(s[i], k);
    int same;
    r = beta * (r - reduce_rows<LPR>(dk, lane % LPR, same));
  }
  if (lane % (LPR / NL) == 0) out[row] = from_f<T>(p.scale * fmaf(r, kq, sq));
#pragma unroll
  for (int i = 0; i < NL; ++i) {
    const float ri = __shfl_sync(0xffffffffu, r, (lane / LPR) * LPR + lane_of<LPR>(i));
    s[i].x = fmaf(ri, k.x, s[i].x);
    s[i].y = fmaf(ri, k.y, s[i].y);
    s[i].z = fmaf(ri, k.z, s[i].z);
    s[i].w = fmaf(ri, k.w, s[i].w);
    *reinterpret_cast<float4*>(S + (size_t)(row0 + i * R) * D) = s[i];
  }
}

template <typename T, int D>
cudaError_t go(const StepParams& p, cudaStream_t st) {
  const int64_t grid = (int64_t)p.N * p.H * (D / ROWS);
  if (grid <= 0) return cudaSuccess;
  if (grid > 0x7fffffff) return cudaErrorInvalidValue;
  if (p.decay) state_step_kernel<T, D, false><<<(unsigned)grid, kThreads<D>, 0, st>>>(p);
  else state_step_kernel<T, D, true><<<(unsigned)grid, kThreads<D>, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_state_step(const StepParams& p, bool bf16, int D, cudaStream_t st) {
  if (bf16) return D == 128 ? go<__nv_bfloat16, 128>(p, st) : go<__nv_bfloat16, 64>(p, st);
  return D == 128 ? go<float, 128>(p, st) : go<float, 64>(p, st);
}

}  // namespace sfg
