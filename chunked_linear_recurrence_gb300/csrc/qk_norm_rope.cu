// qk_norm_rope.cu -- norm of each query and key head with the position rotation in the same
// pass, and its backward (include/sf_linattn.h).
//
//     y = x r w;  (out_a, out_b) = (y_a c - y_b s, y_b c + y_a s) for each rotary pair
//     backward: dy = the rotation by the opposite angle of d_out;  g = dy w;
//               dx = r (g - x t <g, x>),  t = r^2 / D (RMS), r^2 (L2 above eps), 0 (L2 below)
//               dw = sum over tokens and heads of dy x r
//
// Bound by memory: every element is read and written once (the backward reads two).  A row of
// D elements belongs to D / 8 lanes, each with both members of its four pairs (two groups of
// four consecutive elements; eight consecutive ones where the pairs are neighbours), so norm
// and rotation stay in registers.  A group of lanes takes UNROLL heads of one token at a
// time: its loads are in flight together, and the token's cosines and sines are read once
// for all of them.  The weights' gradients are summed per lane over everything a CTA takes,
// then over its lanes, then (a second kernel) over the CTAs, each in a fixed order.
#include <cuda_bf16.h>

#include "common.cuh"
#include "linattn.cuh"

namespace sfg {
namespace {

constexpr int NT = 256;
constexpr int UNROLL = 4;

__device__ __forceinline__ void ld4(const float* p, float* x) {
  const float4 v = *reinterpret_cast<const float4*>(p);
  x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
}
__device__ __forceinline__ void ld4(const __nv_bfloat16* p, float* x) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.x));
  const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.y));
  x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
}
__device__ __forceinline__ void st4(float* p, const float* x) {
  *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
}
__device__ __forceinline__ void st4(__nv_bfloat16* p, const float* x) {
  __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
  uint2 u;
  u.x = *reinterpret_cast<uint32_t*>(&a);
  u.y = *reinterpret_cast<uint32_t*>(&b);
  *reinterpret_cast<uint2*>(p) = u;
}

// What a lane holds of a row: elements [a, a+4) and [b, b+4), and its first pair (or no pair).
struct Lane {
  int a, b, pair;
  bool turns;
};
__device__ __forceinline__ Lane lane_of(int l, const QkParams& p) {
  Lane t;
  const int lanes = p.half / 4;             // lanes that hold pairs
  t.turns = l < lanes;
  t.pair = 4 * l;
  if (t.turns && !p.inter) {
    t.a = 4 * l;
    t.b = p.half + 4 * l;
  } else {
    t.a = 8 * l;
    t.b = 8 * l + 4;
  }
  return t;
}

// Cosines and sines of the lane's four pairs at a token.
__device__ __forceinline__ void load_turn(const QkParams& p, const Lane& t, int64_t row, float* c,
                                          float* s) {
  if (!t.turns) return;
  int axis = 0;
  while (axis + 1 < p.axes && t.pair >= p.bound[axis]) ++axis;
  auto at = [&](int ax) {
    int pos = p.pos[(size_t)ax * p.rows + row];
    pos = pos < 0 ? 0 : (pos >= p.table_rows ? p.table_rows - 1 : pos);
    return p.cs + ((size_t)pos * p.half + t.pair) * 2;
  };
  const float* cs = at(axis);
  if (t.pair + 4 <= p.bound[axis]) {        // one axis for all four
    const float4 u = *reinterpret_cast<const float4*>(cs), v = *reinterpret_cast<const float4*>(cs + 4);
    c[0] = u.x; s[0] = u.y; c[1] = u.z; s[1] = u.w;
    c[2] = v.x; s[2] = v.y; c[3] = v.z; s[3] = v.w;
    return;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    while (axis + 1 < p.axes && t.pair + e >= p.bound[axis]) cs = at(++axis);
    const float2 u = *reinterpret_cast<const float2*>(cs + 2 * e);
    c[e] = u.x;
    s[e] = u.y;
  }
}

// Rotates the lane's eight elements by its four angles (sign -1: the opposite ones).
__device__ __forceinline__ void turn(float* x, const Lane& t, bool inter, const float* c,
                                     const float* s, float sign) {
  if (!t.turns) return;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float sn = sign * s[e];
    if (inter) {
      const float a = x[2 * e], b = x[2 * e + 1];
      x[2 * e] = a * c[e] - b * sn;
      x[2 * e + 1] = b * c[e] + a * sn;
    } else {
      const float a = x[e], b = x[e + 4];
      x[e] = a * c[e] - b * sn;
      x[e + 4] = b * c[e] + a * sn;
    }
  }
}

template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int m = LPR / 2; m >= 1; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
  return x;
}

__device__ __forceinline__ void load_weight(const float* w, const Lane& t, float* x) {
  if (w) {
    ld4(w + t.a, x);
    ld4(w + t.b, x + 4);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = 1.f;
  }
}

// Item -> token and its UNROLL heads [h0, h0 + cnt) of q, or of k.
struct Item {
  int64_t row;
  int h0, cnt;
  bool is_q;
};
__device__ __forceinline__ Item item_of(int64_t id, const QkParams& p, int per, int nq) {
  Item it;
  it.row = id / per;
  const int g = (int)(id % per);
  it.is_q = g < nq;
  it.h0 = (it.is_q ? g : g - nq) * UNROLL;
  const int left = (it.is_q ? p.H : p.HK) - it.h0;
  it.cnt = left < UNROLL ? left : UNROLL;
  return it;
}

template <typename T, int D>
__global__ void __launch_bounds__(NT) qk_fwd_kernel(const QkParams p) {
  constexpr int LPR = D / 8, GROUPS = NT / LPR;
  const int l = threadIdx.x % LPR, grp = threadIdx.x / LPR;
  const Lane t = lane_of(l, p);
  const int nq = (p.H + UNROLL - 1) / UNROLL, per = nq + (p.HK + UNROLL - 1) / UNROLL;
  const int64_t items = p.rows * per, rounds = (items + (int64_t)gridDim.x * GROUPS - 1) / ((int64_t)gridDim.x * GROUPS);
  float wq[8], wk[8];
  load_weight(p.qw, t, wq);
  load_weight(p.kw, t, wk);
  for (int64_t rd = 0; rd < rounds; ++rd) {
    const int64_t id = (rd * gridDim.x + blockIdx.x) * GROUPS + grp;
    const bool live = id < items;            // whole warps stay for the shuffles
    const Item it = item_of(live ? id : 0, p, per, nq);
    const int heads = it.is_q ? p.H : p.HK;
    const T* src = reinterpret_cast<const T*>(it.is_q ? p.q : p.k) +
                   (size_t)it.row * (it.is_q ? p.sq : p.sk) + (size_t)it.h0 * D;
    T* dst = reinterpret_cast<T*>(it.is_q ? p.q_out : p.k_out) + ((size_t)it.row * heads + it.h0) * D;
    float x[UNROLL][8], c[4], s[4];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u)
      if (live && u < it.cnt) {
        ld4(src + u * D + t.a, x[u]);
        ld4(src + u * D + t.b, x[u] + 4);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[u][e] = 0.f;
      }
    load_turn(p, t, it.row, c, s);
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(x[u][e], x[u][e], ss);
      ss = row_sum<LPR>(ss);
      const float r = p.l2 ? 1.f / fmaxf(sqrtf(ss), p.eps) : rsqrtf(ss * (1.f / D) + p.eps);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[u][e] *= r * (it.is_q ? wq[e] : wk[e]);
      turn(x[u], t, p.inter, c, s, 1.f);
      if (live && u < it.cnt) {
        st4(dst + u * D + t.a, x[u]);
        st4(dst + u * D + t.b, x[u] + 4);
      }
    }
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(NT) qk_bwd_kernel(const QkParams p) {
  constexpr int LPR = D / 8, GROUPS = NT / LPR;
  __shared__ float red[GROUPS][D];
  const int l = threadIdx.x % LPR, grp = threadIdx.x / LPR;
  const Lane t = lane_of(l, p);
  const int nq = (p.H + UNROLL - 1) / UNROLL, per = nq + (p.HK + UNROLL - 1) / UNROLL;
  const int64_t items = p.rows * per, rounds = (items + (int64_t)gridDim.x * GROUPS - 1) / ((int64_t)gridDim.x * GROUPS);
  float wq[8], wk[8], gq[8], gk[8];
  load_weight(p.qw, t, wq);
  load_weight(p.kw, t, wk);
#pragma unroll
  for (int e = 0; e < 8; ++e) gq[e] = gk[e] = 0.f;
  for (int64_t rd = 0; rd < rounds; ++rd) {
    const int64_t id = (rd * gridDim.x + blockIdx.x) * GROUPS + grp;
    const bool live = id < items;
    const Item it = item_of(live ? id : 0, p, per, nq);
    const int heads = it.is_q ? p.H : p.HK;
    const T* src = reinterpret_cast<const T*>(it.is_q ? p.q : p.k) +
                   (size_t)it.row * (it.is_q ? p.sq : p.sk) + (size_t)it.h0 * D;
    const size_t at = ((size_t)it.row * heads + it.h0) * D;
    const T* dsrc = reinterpret_cast<const T*>(it.is_q ? p.dqo : p.dko) + at;
    T* dst = reinterpret_cast<T*>(it.is_q ? p.q_out : p.k_out) + at;
    float x[UNROLL][8], d[UNROLL][8], c[4], s[4];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u)
      if (live && u < it.cnt) {
        ld4(src + u * D + t.a, x[u]);
        ld4(src + u * D + t.b, x[u] + 4);
        ld4(dsrc + u * D + t.a, d[u]);
        ld4(dsrc + u * D + t.b, d[u] + 4);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[u][e] = d[u][e] = 0.f;
      }
    load_turn(p, t, it.row, c, s);
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      turn(d[u], t, p.inter, c, s, -1.f);
      float ss = 0.f, gx = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        ss = fmaf(x[u][e], x[u][e], ss);
        gx = fmaf(d[u][e] * (it.is_q ? wq[e] : wk[e]), x[u][e], gx);
      }
      ss = row_sum<LPR>(ss);
      gx = row_sum<LPR>(gx);
      float r, f;
      if (p.l2) {
        const float nrm = sqrtf(ss);
        r = 1.f / fmaxf(nrm, p.eps);
        f = nrm > p.eps ? r * r * gx : 0.f;
      } else {
        r = rsqrtf(ss * (1.f / D) + p.eps);
        f = r * r * (1.f / D) * gx;
      }
      const bool on = live && u < it.cnt;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float dw = on ? d[u][e] * (x[u][e] * r) : 0.f;
        if (it.is_q) gq[e] += dw;
        else gk[e] += dw;
        d[u][e] = r * (d[u][e] * (it.is_q ? wq[e] : wk[e]) - x[u][e] * f);
      }
      if (on) {
        st4(dst + u * D + t.a, d[u]);
        st4(dst + u * D + t.b, d[u] + 4);
      }
    }
  }
  if (!p.part) return;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 8; ++e) red[grp][(e < 4 ? t.a : t.b) + (e & 3)] = which ? gk[e] : gq[e];
    __syncthreads();
    if (threadIdx.x < D) {
      float sum = 0.f;
#pragma unroll
      for (int g = 0; g < GROUPS; ++g) sum += red[g][threadIdx.x];
      p.part[((size_t)blockIdx.x * 2 + which) * D + threadIdx.x] = sum;
    }
  }
}

// dw[c] = sum over the parts of part[.][which][c]: 32 columns a CTA, 32 threads a column.
__global__ void __launch_bounds__(1024) qk_weight_kernel(const float* part, int parts, int D,
                                                         float* dqw, float* dkw) {
  __shared__ float red[32][33];
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + x;       // of 2 D
  float s = 0.f;
  for (int i = y; i < parts; i += 32) s += part[(size_t)i * 2 * D + col];
  red[y][x] = s;
  __syncthreads();
  s = red[x][y];
#pragma unroll
  for (int m = 16; m; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
  const int c = blockIdx.x * 32 + y;
  float* dst = c < D ? dqw : dkw;
  if (x == 0 && dst) dst[c % D] = s;
}

// CTAs for the tokens' items, at most `cap`.
unsigned qk_grid(const QkParams& p, int D, int64_t cap) {
  const int per = (p.H + UNROLL - 1) / UNROLL + (p.HK + UNROLL - 1) / UNROLL;
  const int64_t want = (p.rows * per + NT / (D / 8) - 1) / (NT / (D / 8));
  return (unsigned)(want < cap ? want : cap);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const QkParams& p, bool bf16, int D, cudaStream_t st) {
  if (p.rows <= 0) return cudaSuccess;
  const unsigned g = qk_grid(p, D, 152 * 8);
  if (bf16) {
    if (D == 128) qk_fwd_kernel<__nv_bfloat16, 128><<<g, NT, 0, st>>>(p);
    else qk_fwd_kernel<__nv_bfloat16, 64><<<g, NT, 0, st>>>(p);
  } else {
    if (D == 128) qk_fwd_kernel<float, 128><<<g, NT, 0, st>>>(p);
    else qk_fwd_kernel<float, 64><<<g, NT, 0, st>>>(p);
  }
  return cudaGetLastError();
}

cudaError_t launch_qk_norm_rope_bwd(const QkParams& p, bool bf16, int D, float* dqw, float* dkw,
                                    cudaStream_t st) {
  const unsigned g = p.rows > 0 ? qk_grid(p, D, QK_PARTS) : 0;
  if (g > 0) {
    if (bf16) {
      if (D == 128) qk_bwd_kernel<__nv_bfloat16, 128><<<g, NT, 0, st>>>(p);
      else qk_bwd_kernel<__nv_bfloat16, 64><<<g, NT, 0, st>>>(p);
    } else {
      if (D == 128) qk_bwd_kernel<float, 128><<<g, NT, 0, st>>>(p);
      else qk_bwd_kernel<float, 64><<<g, NT, 0, st>>>(p);
    }
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (dqw || dkw) qk_weight_kernel<<<2 * D / 32, 1024, 0, st>>>(p.part, (int)g, D, dqw, dkw);
  return cudaGetLastError();
}

}  // namespace sfg
