// qk_norm_rope.cu -- norm of each query and key head with the position rotation in the same
// pass, and its backward (include/sf_linattn.h).
//
//     y = x r w;  (out_a, out_b) = (y_a c - y_b s, y_b c + y_a s) for each rotary pair
//     backward: dy = the rotation by the opposite angle of d_out;  g = dy w;
//               dx = r (g - x t <g, x>),  t = r^2 / D (RMS), r^2 (L2 above eps), 0 (L2 below)
//               dw = sum over tokens and heads of dy x r
//
// Bound by memory: every element is read and written once (the backward reads two).  A row of
// D elements belongs to D / (2 VEC) lanes, each with both members of its VEC pairs: two groups of
// VEC consecutive elements (2 VEC consecutive ones where the pairs are neighbours), so norm and
// rotation stay in registers.  VEC is 8 (16-byte accesses of BF16) unless the rotated part ends
// inside such a group.  A group of lanes takes U heads of one token at a time: its loads are in
// flight together and the token's cosines and sines serve all of them.  A CTA takes queries or
// keys, not both (the grid is shared in proportion), so it keeps one weight and one gradient of
// it.  Arithmetic goes two elements an instruction.  The weights' gradients are summed per lane
// over everything a CTA takes, then over its lanes, then (a second kernel) over the CTAs, each
// in a fixed order.  Everything is FP32 until the results are rounded to the tokens' type.
// Measured, BF16, D = 128: forward of 32769 tokens of 16 + 16 heads with three axes 88.7 us (92 %
// of the copy rate; one head at a time 109 us, eight 112-117), backward of 16384 tokens of 16 + 16
// heads 70.0 us (87 %), 74.3 with the weights, whose launch waits for the first one's end (77.5 when
// it started after it; one head at a time 96 us, three 101-106).  Two
// CTAs of 256 threads an SM instead of four of 128 are level in the forward (88.8 us).
#include <cuda_bf16.h>

#include "common.cuh"
#include "f32x2.cuh"
#include "linattn.cuh"

namespace sfg {
namespace {

constexpr int NT = 128;   // four CTAs an SM: persistent, 512 threads with 64 KB on the way

// VEC consecutive elements as they come from memory, and as VEC / 2 pairs of floats.
template <typename T, int VEC>
struct Raw {
  static constexpr int W = VEC * sizeof(T) / 8;   // 8-byte words
  uint2 u[W];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (W % 2 == 0) {
#pragma unroll
      for (int i = 0; i < W; i += 2) {
        const uint4 v = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint2*>(p) + i);
        u[i] = make_uint2(v.x, v.y);
        u[i + 1] = make_uint2(v.z, v.w);
      }
    } else {
      u[0] = *reinterpret_cast<const uint2*>(p);
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < W; ++i) u[i] = make_uint2(0, 0);
  }
  __device__ __forceinline__ void get(float2* x) const {
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int i = 0; i < W; ++i) {
        x[2 * i] = unpack2(u[i].x);
        x[2 * i + 1] = unpack2(u[i].y);
      }
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i) x[i] = make_float2(__uint_as_float(u[i].x), __uint_as_float(u[i].y));
    }
  }
  __device__ __forceinline__ void put(const float2* x) {
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int i = 0; i < W; ++i) u[i] = make_uint2(pack2(x[2 * i]), pack2(x[2 * i + 1]));
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i) u[i] = make_uint2(__float_as_uint(x[i].x), __float_as_uint(x[i].y));
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (W % 2 == 0) {
#pragma unroll
      for (int i = 0; i < W; i += 2)
        *reinterpret_cast<uint4*>(reinterpret_cast<uint2*>(p) + i) =
            make_uint4(u[i].x, u[i].y, u[i + 1].x, u[i + 1].y);
    } else {
      *reinterpret_cast<uint2*>(p) = u[0];
    }
  }
};

// What a lane holds of a row: elements [a, a + VEC) and [b, b + VEC), and its first pair.
struct Lane {
  int a, b, pair;
  bool turns;
};
template <int VEC>
__device__ __forceinline__ Lane lane_of(int l, const QkParams& p) {
  Lane t;
  t.turns = l * VEC < p.half;
  t.pair = VEC * l;
  const bool halves = t.turns && !p.inter;
  t.a = halves ? VEC * l : 2 * VEC * l;
  t.b = halves ? p.half + VEC * l : 2 * VEC * l + VEC;
  return t;
}

// Cosines and sines of the lane's VEC pairs at a token, two pairs to a float2.
template <int VEC>
__device__ __forceinline__ void load_turn(const QkParams& p, const Lane& t, int64_t row, float2* c,
                                          float2* s) {
  if (!t.turns) return;
  int axis = 0;
  while (axis + 1 < p.axes && t.pair >= p.bound[axis]) ++axis;
  auto at = [&](int ax) {
    int pos = p.pos[(size_t)ax * p.rows + row];
    pos = pos < 0 ? 0 : (pos >= p.table_rows ? p.table_rows - 1 : pos);
    return p.cs + ((size_t)pos * p.half + t.pair) * 2;
  };
  const float* cs = at(axis);
  if (t.pair + VEC <= p.bound[axis]) {        // one axis for all of them
#pragma unroll
    for (int e = 0; e < VEC / 2; ++e) {
      const float4 v = *reinterpret_cast<const float4*>(cs + 4 * e);
      c[e] = make_float2(v.x, v.z);
      s[e] = make_float2(v.y, v.w);
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    while (axis + 1 < p.axes && t.pair + e >= p.bound[axis]) cs = at(++axis);
    const float2 v = *reinterpret_cast<const float2*>(cs + 2 * e);
    if (e & 1) c[e / 2].y = v.x, s[e / 2].y = v.y;
    else c[e / 2].x = v.x, s[e / 2].x = v.y;
  }
}

// Rotates the lane's elements by its angles (kBack: the opposite ones); xa, xb its two groups.
template <int VEC, bool kBack>
__device__ __forceinline__ void turn(float2* xa, float2* xb, const Lane& t, bool inter, const float2* c,
                                     const float2* s) {
  if (!t.turns) return;
  if (!inter) {
#pragma unroll
    for (int e = 0; e < VEC / 2; ++e) {
      const float2 a = xa[e], b = xb[e], n = make_float2(-s[e].x, -s[e].y);
      xa[e] = fma2(a, c[e], mul2(b, kBack ? s[e] : n));
      xb[e] = fma2(b, c[e], mul2(a, kBack ? n : s[e]));
    }
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {            // pair e is one float2
      float2& v = e < VEC / 2 ? xa[e] : xb[e - VEC / 2];
      const float ce = e & 1 ? c[e / 2].y : c[e / 2].x;
      float se = e & 1 ? s[e / 2].y : s[e / 2].x;
      if (kBack) se = -se;
      v = make_float2(v.x * ce - v.y * se, v.y * ce + v.x * se);
    }
  }
}

template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int m = LPR / 2; m >= 1; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
  return x;
}

// max(x, least), NaN where x is NaN (fmaxf would give `least`, and a head that holds a NaN finite
// results).
__device__ __forceinline__ float at_least(float x, float least) { return x < least ? least : x; }

template <int VEC>
__device__ __forceinline__ void load_weight(const float* w, const Lane& t, float2* x) {
#pragma unroll
  for (int e = 0; e < VEC / 2; ++e) {
    x[e] = w ? *reinterpret_cast<const float2*>(w + t.a + 2 * e) : make_float2(1.f, 1.f);
    x[VEC / 2 + e] = w ? *reinterpret_cast<const float2*>(w + t.b + 2 * e) : make_float2(1.f, 1.f);
  }
}

// The part of the grid that takes the queries, and the walk of one group of lanes over its
// (token, U heads) items.
struct Share {
  bool is_q;
  int block, blocks, heads, per;
  int64_t items;
};
template <int U>
__device__ __forceinline__ Share share_of(const QkParams& p) {
  Share w;
  w.is_q = (int)blockIdx.x < p.q_blocks;
  w.block = w.is_q ? blockIdx.x : blockIdx.x - p.q_blocks;
  w.blocks = w.is_q ? p.q_blocks : gridDim.x - p.q_blocks;
  w.heads = w.is_q ? p.H : p.HK;
  w.per = (w.heads + U - 1) / U;
  w.items = p.rows * w.per;
  return w;
}

template <typename T, int D, int VEC, int U>
__global__ void __launch_bounds__(NT) qk_fwd_kernel(const QkParams p) {
  constexpr int LPR = D / (2 * VEC), GROUPS = NT / LPR, NP = VEC / 2;
  const int l = threadIdx.x % LPR, grp = threadIdx.x / LPR;
  const Lane t = lane_of<VEC>(l, p);
  const Share w = share_of<U>(p);
  const T* const base = reinterpret_cast<const T*>(w.is_q ? p.q : p.k);
  T* const obase = reinterpret_cast<T*>(w.is_q ? p.q_out : p.k_out);
  const int64_t stride = w.is_q ? p.sq : p.sk;
  float2 wt[VEC];
  load_weight<VEC>(w.is_q ? p.qw : p.kw, t, wt);
  for (int64_t first = (int64_t)w.block * GROUPS; first < w.items; first += (int64_t)w.blocks * GROUPS) {
    const bool live = first + grp < w.items;       // whole warps stay for the shuffles
    const int64_t id = live ? first + grp : w.items - 1;
    const int64_t row = (id >> 31) ? id / w.per : (int64_t)((uint32_t)id / (uint32_t)w.per);
    const int h0 = (int)(id - row * w.per) * U, cnt = live ? w.heads - h0 : 0;
    const T* src = base + (size_t)row * stride + (size_t)h0 * D;
    T* dst = obase + ((size_t)row * w.heads + h0) * D;
    Raw<T, VEC> ra[U], rb[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (u < cnt) {
        ra[u].load(src + u * D + t.a);
        rb[u].load(src + u * D + t.b);
      } else {
        ra[u].zero();
        rb[u].zero();
      }
    float2 c[NP], s[NP];
    load_turn<VEC>(p, t, row, c, s);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float2 x[VEC];
      ra[u].get(x);
      rb[u].get(x + NP);
      float2 q = mul2(x[0], x[0]);
#pragma unroll
      for (int e = 1; e < VEC; ++e) q = fma2(x[e], x[e], q);
      const float ss = row_sum<LPR>(q.x + q.y);
      const float r = p.l2 ? 1.f / at_least(sqrtf(ss), p.eps) : rsqrtf(ss * (1.f / D) + p.eps);
#pragma unroll
      for (int e = 0; e < VEC; ++e) x[e] = mul2(x[e], mul2(wt[e], make_float2(r, r)));
      turn<VEC, false>(x, x + NP, t, p.inter, c, s);
      if (u < cnt) {
        ra[u].put(x);
        rb[u].put(x + NP);
        ra[u].store(dst + u * D + t.a);
        rb[u].store(dst + u * D + t.b);
      }
    }
  }
}

template <typename T, int D, int VEC, int U>
__global__ void __launch_bounds__(NT) qk_bwd_kernel(const QkParams p) {
  launch_next();
  constexpr int LPR = D / (2 * VEC), GROUPS = NT / LPR, NP = VEC / 2;
  __shared__ float red[GROUPS][D];
  const int l = threadIdx.x % LPR, grp = threadIdx.x / LPR;
  const Lane t = lane_of<VEC>(l, p);
  const Share w = share_of<U>(p);
  const T* const base = reinterpret_cast<const T*>(w.is_q ? p.q : p.k);
  const T* const dbase = reinterpret_cast<const T*>(w.is_q ? p.dqo : p.dko);
  T* const obase = reinterpret_cast<T*>(w.is_q ? p.q_out : p.k_out);
  const int64_t stride = w.is_q ? p.sq : p.sk;
  float2 wt[VEC], dw[VEC];
  load_weight<VEC>(w.is_q ? p.qw : p.kw, t, wt);
#pragma unroll
  for (int e = 0; e < VEC; ++e) dw[e] = make_float2(0.f, 0.f);
  for (int64_t first = (int64_t)w.block * GROUPS; first < w.items; first += (int64_t)w.blocks * GROUPS) {
    const bool live = first + grp < w.items;
    const int64_t id = live ? first + grp : w.items - 1;
    const int64_t row = (id >> 31) ? id / w.per : (int64_t)((uint32_t)id / (uint32_t)w.per);
    const int h0 = (int)(id - row * w.per) * U, cnt = live ? w.heads - h0 : 0;
    const T* src = base + (size_t)row * stride + (size_t)h0 * D;
    const size_t at = ((size_t)row * w.heads + h0) * D;
    Raw<T, VEC> ra[U], rb[U], da[U], db[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (u < cnt) {
        ra[u].load(src + u * D + t.a);
        rb[u].load(src + u * D + t.b);
        da[u].load(dbase + at + u * D + t.a);
        db[u].load(dbase + at + u * D + t.b);
      } else {                                     // adds nothing to the weight's gradient
        ra[u].zero();
        rb[u].zero();
        da[u].zero();
        db[u].zero();
      }
    float2 c[NP], s[NP];
    load_turn<VEC>(p, t, row, c, s);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float2 x[VEC], d[VEC];
      ra[u].get(x);
      rb[u].get(x + NP);
      da[u].get(d);
      db[u].get(d + NP);
      turn<VEC, true>(d, d + NP, t, p.inter, c, s);
      float2 q = mul2(x[0], x[0]), g = mul2(mul2(d[0], wt[0]), x[0]);
#pragma unroll
      for (int e = 1; e < VEC; ++e) {
        q = fma2(x[e], x[e], q);
        g = fma2(mul2(d[e], wt[e]), x[e], g);
      }
      const float ss = row_sum<LPR>(q.x + q.y), gx = row_sum<LPR>(g.x + g.y);
      float r, f;
      if (p.l2) {
        const float nrm = sqrtf(ss);
        r = 1.f / at_least(nrm, p.eps);
        f = nrm <= p.eps ? 0.f : r * r * gx;
      } else {
        r = rsqrtf(ss * (1.f / D) + p.eps);
        f = r * r * (1.f / D) * gx;
      }
      if (u >= cnt) continue;
      const float2 r2 = make_float2(r, r), nrf = make_float2(-r * f, -r * f);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float2 dr = mul2(d[e], r2);
        dw[e] = fma2(dr, x[e], dw[e]);
        d[e] = fma2(dr, wt[e], mul2(x[e], nrf));   // r (g - x f)
      }
      ra[u].put(d);
      rb[u].put(d + NP);
      ra[u].store(obase + at + u * D + t.a);
      rb[u].store(obase + at + u * D + t.b);
    }
  }
  if (!p.part) return;
#pragma unroll
  for (int e = 0; e < NP; ++e) {
    *reinterpret_cast<float2*>(&red[grp][t.a + 2 * e]) = dw[e];
    *reinterpret_cast<float2*>(&red[grp][t.b + 2 * e]) = dw[NP + e];
  }
  __syncthreads();
  if (threadIdx.x < D) {
    float sum = 0.f;
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) sum += red[g][threadIdx.x];
    p.part[(size_t)blockIdx.x * D + threadIdx.x] = sum;
  }
}

// dw[c] = sum of part[.][c] over the query blocks (dqw) and over the key blocks (dkw): 32 columns
// a CTA, 32 threads a column.  (304 rows of 512 bytes in L2: latency, ~3 us, of which its early
// start hides half.)
__global__ void __launch_bounds__(1024) qk_weight_kernel(const float* part, int q_blocks, int blocks,
                                                         int D, float* dqw, float* dkw) {
  __shared__ float red[32][33];
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  const bool is_q = (int)blockIdx.x < D / 32;
  const int col = (blockIdx.x % (D / 32)) * 32;
  const int lo = is_q ? 0 : q_blocks, hi = is_q ? q_blocks : blocks;
  float* dst = is_q ? dqw : dkw;
  launch_wait();                                  // the partial sums
  if (!dst) return;
  float s = 0.f;
#pragma unroll 4
  for (int i = lo + y; i < hi; i += 32) s += part[(size_t)i * D + col + x];
  red[y][x] = s;
  __syncthreads();
  s = red[x][y];
#pragma unroll
  for (int m = 16; m; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
  if (x == 0) dst[col + y] = s;
}

// Blocks for the queries' and the keys' items, at most `cap` together.
template <int U>
void share(QkParams& p, int groups, int64_t cap, unsigned& blocks) {
  const int64_t qi = (p.rows * ((p.H + U - 1) / U) + groups - 1) / groups;
  const int64_t ki = (p.rows * ((p.HK + U - 1) / U) + groups - 1) / groups;
  int64_t qb = qi, kb = ki;
  if (qi + ki > cap) {
    qb = cap * qi / (qi + ki);
    qb = qb < 1 ? 1 : qb > cap - 1 ? cap - 1 : qb;
    kb = cap - qb;
  }
  p.q_blocks = (int)qb;
  blocks = (unsigned)(qb + kb);
}

constexpr int FWD_U = 4, BWD_U = 2;

template <typename T, int D, int VEC>
cudaError_t fwd(QkParams p, cudaStream_t st) {
  unsigned blocks;
  share<FWD_U>(p, NT / (D / (2 * VEC)), 152 * 4, blocks);
  qk_fwd_kernel<T, D, VEC, FWD_U><<<blocks, NT, 0, st>>>(p);
  return cudaGetLastError();
}
template <typename T, int D, int VEC>
cudaError_t bwd(QkParams p, float* dqw, float* dkw, cudaStream_t st) {
  unsigned blocks = 0;
  cudaError_t e = cudaSuccess;
  if (p.rows > 0) {
    share<BWD_U>(p, NT / (D / (2 * VEC)), QK_PARTS, blocks);
    qk_bwd_kernel<T, D, VEC, BWD_U><<<blocks, NT, 0, st>>>(p);
    e = cudaGetLastError();
  }
  if (e == cudaSuccess && (dqw || dkw))
    e = launch_after(p.rows > 0, qk_weight_kernel, 2 * D / 32, 1024, 0, st, (const float*)p.part, p.q_blocks,
                     (int)blocks, D, dqw, dkw);
  return e;
}

}  // namespace

// Groups of 8 elements need a rotated part of a multiple of 16 elements.
cudaError_t launch_qk_norm_rope(const QkParams& p, bool bf16, int D, cudaStream_t st) {
  if (p.rows <= 0) return cudaSuccess;
  const bool wide = p.half % 8 == 0;
  if (bf16) {
    if (D == 128) return wide ? fwd<__nv_bfloat16, 128, 8>(p, st) : fwd<__nv_bfloat16, 128, 4>(p, st);
    return wide ? fwd<__nv_bfloat16, 64, 8>(p, st) : fwd<__nv_bfloat16, 64, 4>(p, st);
  }
  return D == 128 ? fwd<float, 128, 4>(p, st) : fwd<float, 64, 4>(p, st);
}

cudaError_t launch_qk_norm_rope_bwd(const QkParams& p, bool bf16, int D, float* dqw, float* dkw,
                                    cudaStream_t st) {
  const bool wide = p.half % 8 == 0;
  if (bf16) {
    if (D == 128)
      return wide ? bwd<__nv_bfloat16, 128, 8>(p, dqw, dkw, st) : bwd<__nv_bfloat16, 128, 4>(p, dqw, dkw, st);
    return wide ? bwd<__nv_bfloat16, 64, 8>(p, dqw, dkw, st) : bwd<__nv_bfloat16, 64, 4>(p, dqw, dkw, st);
  }
  return D == 128 ? bwd<float, 128, 4>(p, dqw, dkw, st) : bwd<float, 64, 4>(p, dqw, dkw, st);
}

}  // namespace sfg
