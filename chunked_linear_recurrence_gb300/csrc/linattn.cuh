// linattn.cuh -- parameters and launchers of the decayed linear attention, the single-token
// steps and the norm-and-rotate pass (include/sf_linattn.h).
//
// One product serves the forward and all three gradients of the linear attention.  For rows
// r, s of a sequence and lam = exp(decay),
//     out_r = a sum_s lam^|r-s| (x_r . y_s) z_s  +  b lam^e(r) S x_r
//     S'    = lam^L S + c sum_s lam^f(s) z_s y_s^T
// chunk by chunk (L rows, local r, s = 0 .. L-1), S [z][y] the FP32 state that enters the chunk:
//     forward walk   s <= r   e(r) = r + 1      f(s) = L - 1 - s
//     reverse walk   s >= r   e(r) = L - 1 - r  f(s) = s + 1     (chunks from the last row)
//     out:  x, y, z = q, k, v       forward   a = b = scale, c = 1   S = state
//     dq:   do, v, k                forward   a = b = scale, c = 1   S = state^T
//     dv:   k, q, do                reverse   a = c = scale, b = 1   S = cotangent
//     dk:   v, do, q                reverse   a = c = scale, b = 1   S = cotangent^T
//
// A long walk is cut into segments of `seg` rows (in walk order) that run side by side: a
// first launch computes what each segment adds to the state, a second carries the entry
// states over the segments, a third runs the segments from them.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/sf_linattn.h"

namespace sfg {

struct LaPass {
  const void* x;
  const void* y;
  const void* z;
  void* out;            // [rows, H, D]: the token type, or FP32 (out_f32)
  const float* s_in;    // [N,H,D,D] or NULL (zeros)
  float* s_out;         // [N,H,D,D] or NULL
  float* seg_state;     // [units,H,D,D] (z rows): segment sums, then segment entry states
  int hx, hy, hz;       // heads of x, y, z (each divides H)
  int s_t;              // the state is stored as [y][z] (s_in, s_out)
  int out_f32;
  int reverse;
  float a, b, c;
};

struct LaParams {
  LaPass pass[3];
  int npass;
  const float* decay;   // [H]
  const int32_t* cu;    // [N+1] or NULL
  float* pool;          // paged states (pass 0), or NULL
  const int32_t* state_idx;
  const uint8_t* has_init;
  int num_slots;
  int B, T, H, N;
  int seg;              // rows of a segment, a multiple of 64
  int units;            // launched (sequence, segment) units; packed: an upper bound
  int* status;
};

constexpr int LA_CHUNK = 64;

// (sequence, segment) units of a launch whose segments have `seg` rows.
inline int64_t la_units(int B, int T, int N, bool packed, int seg) {
  const int64_t per = T > 0 ? (T + (int64_t)seg - 1) / seg : 1;
  return packed ? (int64_t)T / seg + N : (int64_t)N * (per > 0 ? per : 1);
}

#ifdef __CUDACC__
// Unit u -> sequence n and its segment w in walk order; a warp calls it together.  False
// when the unit holds nothing.  bos, eos: the sequence's rows, clamped into [0, B T].
__device__ __forceinline__ bool la_locate(int u, const LaParams& p, int& n, int& w, int64_t& bos,
                                          int64_t& eos) {
  const int64_t total = (int64_t)p.B * p.T;
  if (!p.cu) {
    const int per = p.T > 0 ? (p.T + p.seg - 1) / p.seg : 1;
    n = u / per;
    w = u % per;
    if (n >= p.N) return false;
    bos = (int64_t)n * p.T;
    eos = bos + p.T;
    return true;
  }
  const int lane = threadIdx.x & 31;
  int base = 0;
  for (int m0 = 0; m0 < p.N; m0 += 32) {
    const int m = m0 + lane;
    int64_t b = 0, e = 0;
    int cnt = 0;
    if (m < p.N) {
      b = p.cu[m];
      e = p.cu[m + 1];
      b = b < 0 ? 0 : (b > total ? total : b);
      e = e < b ? b : (e > total ? total : e);
      cnt = e > b ? (int)((e - b + p.seg - 1) / p.seg) : 1;
    }
    int incl = cnt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += t;
    }
    const bool mine = m < p.N && u >= base + incl - cnt && u < base + incl;
    const unsigned hit = __ballot_sync(0xffffffffu, mine);
    if (hit) {
      const int src = __ffs(hit) - 1;
      n = m0 + src;
      w = u - __shfl_sync(0xffffffffu, base + incl - cnt, src);
      bos = __shfl_sync(0xffffffffu, b, src);
      eos = __shfl_sync(0xffffffffu, e, src);
      return true;
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
  }
  return false;
}

// lam^n for a natural-log decay d (n = 0: 1 even for d = -inf).
__device__ __forceinline__ double la_pow(float d, int64_t n) {
  return n == 0 ? 1.0 : exp((double)d * (double)n);
}

// The entry state's slot of sequence n, head h: NULL for zeros; `skip` marks padding.
__device__ __forceinline__ const float* la_entry(const LaParams& p, const LaPass& q, int n, int h,
                                                 int D, bool& skip) {
  skip = false;
  const size_t sz = (size_t)D * D;
  if (p.pool) {
    const int idx = p.state_idx[n];
    skip = idx <= 0 || idx >= p.num_slots;
    if (skip || (p.has_init && !p.has_init[n])) return nullptr;
    return p.pool + ((size_t)idx * p.H + h) * sz;
  }
  return q.s_in ? q.s_in + ((size_t)n * p.H + h) * sz : nullptr;
}
__device__ __forceinline__ float* la_exit(const LaParams& p, const LaPass& q, int n, int h, int D) {
  const size_t sz = (size_t)D * D;
  if (p.pool) return p.pool + ((size_t)p.state_idx[n] * p.H + h) * sz;
  return q.s_out ? q.s_out + ((size_t)n * p.H + h) * sz : nullptr;
}
#endif

// The CUDA-core kernel (FP32 or BF16 tokens, D 64 or 128): state_only computes the segments'
// sums into seg_state, otherwise the outputs.
cudaError_t launch_la_simt(const LaParams& p, bool bf16, int D, bool state_only, cudaStream_t st);
// The tcgen05 kernel (BF16 tokens, D = 128; needs tc_fwd_available()).
cudaError_t launch_la_tc(const LaParams& p, bool state_only, cudaStream_t st);
// seg_state: segment sums -> entry states of every segment but the walk's first.
cudaError_t launch_la_carry(const LaParams& p, int D, cudaStream_t st);

struct StepParams {
  const void* q;
  const void* k;
  const void* v;
  const float* decay;   // [H] (linear attention), or NULL
  const float* gate;    // [N,H] (delta rule)
  const float* beta;    // [N,H]
  float* pool;
  const int32_t* idx;   // [N] or NULL
  void* out;
  int N, H, HK, num_slots;
  float scale;
};
cudaError_t launch_state_step(const StepParams& p, bool bf16, int D, cudaStream_t st);

struct QkParams {
  const void* q;
  const void* k;
  const float* qw;
  const float* kw;
  const float* cs;
  const int32_t* pos;
  void* q_out;
  void* k_out;
  const void* dqo;      // backward: cotangents of q_out, k_out
  const void* dko;
  float* part;          // backward: per-CTA sums of the weights' gradients [blocks][D]
  int64_t rows, sq, sk; // tokens; element strides between tokens of q and k
  int H, HK, half, inter, table_rows, axes, l2;
  int q_blocks;         // CTAs that take queries; the rest take keys
  int bound[4];         // pairs below bound[a] belong to axes 0 .. a
  float eps;
};
// Most CTAs of the backward: parts of the weights' gradients, [QK_PARTS][D].
constexpr int QK_PARTS = 152 * 4;
cudaError_t launch_qk_norm_rope(const QkParams& p, bool bf16, int D, cudaStream_t st);
cudaError_t launch_qk_norm_rope_bwd(const QkParams& p, bool bf16, int D, float* dqw, float* dkw,
                                    cudaStream_t st);

}  // namespace sfg
