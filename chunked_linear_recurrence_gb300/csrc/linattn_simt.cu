// linattn_simt.cu -- the decayed linear attention's product (linattn.cuh) on the CUDA cores, for
// FP32 tokens: FP32 multiply-adds throughout.
//
// One CTA of 256 threads walks one (segment, head, 64-column slice of z).  Per 64-row chunk
//     P  = a (X Y^T) o lam^|r-s|       64 x 64, each thread 4 x 4
//     O  = b lam^e diag (X S^T) + P Z  64 x 64, each thread 4 x 4
//     S' = lam^L S + c (lam^f Y)^T Z   D x 64, each thread D/16 x 4, kept in registers
// Every product reads one operand as rows that sixteen threads share (a broadcast) and the
// other as consecutive float4 of the row that the sixteen divide among them.  P is computed
// and used up to the diagonal's 16 x 16 blocks alone.  The state is copied to shared memory
// once a chunk for the second product.  lam^64 is formed in FP64 and carried as a sum of two
// floats, so that a state kept over thousands of chunks does not drift by the rounding of one
// factor.
// Bound by multiply-adds and the shared-memory loads that feed them (8 warps an SM, half of the
// FP32 rate): about 1.9 C D + 2 D^2 multiply-adds a row at C = 64, D = 128, against 2 KB of
// tokens.  Measured, one CTA on every SM, a chunk: D = 128 12.4 us and 4.0 us (states alone), D =
// 64 8.1 us and 2.7 us.  2 x 2048 tokens of 16 heads: 35 + 199 us (86 us at the full FP32 rate) and
// 23 + 60 us; 200 tokens of 2 heads, where every chunk is a segment: 32 us and 24 us a call.
#include "common.cuh"
#include "f32x2.cuh"
#include "linattn.cuh"

namespace sfg {
namespace {

constexpr int ZT = 64;   // columns of z per CTA
constexpr int C = LA_CHUNK;

__device__ __forceinline__ float4 ld4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ void st4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
// Chunks in flight: at D = 128 one CTA fills an SM, so the next chunk's rows travel under the
// present one's products; at D = 64 two CTAs share an SM and cover for one another.
template <int D>
constexpr int kStages = D == 128 ? 2 : 1;

template <int D>
struct Smem {
  float X[kStages<D>][C][D + 4], Y[kStages<D>][C][D + 4], Z[kStages<D>][C][ZT + 4];
  float P[C][ZT + 4], S[D][ZT + 4], tab[C + 4], wr[2][C], carry[4];
};

// Copies rows [r0, r0 + L) of one head's columns [c0, c0 + W) to dst (leading dimension ld); the
// other rows of the 64 become zero.  Asynchronous: part of the thread's next commit.
template <int W>
__device__ __forceinline__ void copy_rows(float* dst, int ld, const float* src, int64_t r0, int L,
                                          int heads, int head, int D, int c0, int tid) {
  for (int idx = tid; idx < C * (W / 4); idx += 256) {
    const int r = idx / (W / 4), c = (idx % (W / 4)) * 4;
    const float* from = src + ((size_t)(r0 + (r < L ? r : 0)) * heads + head) * D + c0 + c;
    const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(dst + r * ld + c));
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(r < L ? 16 : 0)
                 : "memory");
  }
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int D, bool kState>
__global__ void __launch_bounds__(256, D == 128 ? 1 : 2) la_simt_kernel(const LaParams p) {
  extern __shared__ __align__(16) uint8_t raw[];
  Smem<D>& sm = *reinterpret_cast<Smem<D>*>(raw);
  constexpr int NZ = D / ZT, YR = D / 16;
  launch_next();
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int zt = blockIdx.x % NZ;
  int pi, h, u;
  la_place(blockIdx.x / NZ, p, pi, h, u);
  const LaPass& q = p.pass[pi];
  LaUnit t;
  if (!la_locate<kState>(u, p, t)) return;
  const int n = t.n;
  const bool split = p.seg < p.T && !(t.last && t.off == 0);
  const int64_t rows = t.rows;
  const int64_t sb = q.reverse ? t.eos - t.off - rows : t.bos + t.off, se = sb + rows;
  bool skip;
  const float* s_in = la_entry(p, q, n, h, D, skip);
  const int zc = zt * ZT;
  if (skip) {                                     // padding of the paged pool
    if (kState) return;
    float* o = static_cast<float*>(q.out);
    for (int64_t idx = tid; idx < rows * (ZT / 4); idx += 256)
      st4(o + ((size_t)(sb + idx / (ZT / 4)) * p.H + h) * D + zc + (int)(idx % (ZT / 4)) * 4,
          make_float4(0.f, 0.f, 0.f, 0.f));
    return;
  }
  const float d = p.decay[h];
  const int nc = (int)((rows + C - 1) / C);
  const int tail = (int)(rows - (int64_t)(nc - 1) * C);
  const int hx = la_head(h, q.hx, p), hy = la_head(h, q.hy, p), hz = la_head(h, q.hz, p);
  constexpr int NB = kStages<D>;
  auto fetch = [&](int ci) {
    const int64_t done = (int64_t)ci * C;
    const int L = (int)(rows - done < C ? rows - done : C);
    const int64_t r0 = q.reverse ? se - done - L : sb + done;
    const int b = ci % NB;
    if (!kState)
      copy_rows<D>(&sm.X[b][0][0], D + 4, static_cast<const float*>(q.x), r0, L, q.hx, hx, D, 0, tid);
    copy_rows<D>(&sm.Y[b][0][0], D + 4, static_cast<const float*>(q.y), r0, L, q.hy, hy, D, 0, tid);
    copy_rows<ZT>(&sm.Z[b][0][0], ZT + 4, static_cast<const float*>(q.z), r0, L, q.hz, hz, D, zc, tid);
    copies_commit();
  };
  if (nc > 0) fetch(0);
  auto pw = [&](int e) { return e <= 0 ? 1.f : expf(d * (float)e); };
  if (tid <= C) sm.tab[tid] = pw(tid);
  if (tid >= 128) {                               // weights of a full chunk's rows, and of the last's
    const int r = tid & 63, at = (tid - 128) >> 6, n = at ? tail : C;
    sm.wr[at][r] = r < n ? q.c * pw(q.reverse ? r + 1 : n - 1 - r) : 0.f;
  }
  if (tid == 96 || tid == 97) {                  // lam^64 and lam^tail as sums of two floats
    const double f = la_pow(d, tid == 96 ? C : tail);
    sm.carry[2 * (tid - 96)] = (float)f;
    sm.carry[2 * (tid - 96) + 1] = (float)(f - (double)(float)f);
  }

  // S[y = ty YR + e][z = zc + 4 tx ..]: zeros, the caller's state, or the segment's entry
  float4 s[YR];
  const size_t uoff = ((size_t)t.at * p.H + h) * D * D;
  const float* src = kState ? nullptr : split ? q.entry + uoff : s_in;
  if (!src) {
#pragma unroll
    for (int e = 0; e < YR; ++e) s[e] = make_float4(0.f, 0.f, 0.f, 0.f);
  } else if (q.s_t && !split) {
#pragma unroll
    for (int e = 0; e < YR; ++e) s[e] = ld4(src + (size_t)(ty * YR + e) * D + zc + 4 * tx);
  } else {                                        // four y of one z at a time
    const int zs = split ? 4 : D, ys = split ? D : 1;
#pragma unroll
    for (int e = 0; e < YR; e += 4) {
      const float* v = src + (ty * YR + e) * ys + (zc + 4 * tx) * zs;
      const float4 c0 = ld4(v), c1 = ld4(v + zs), c2 = ld4(v + 2 * zs), c3 = ld4(v + 3 * zs);
      s[e] = make_float4(c0.x, c1.x, c2.x, c3.x);
      s[e + 1] = make_float4(c0.y, c1.y, c2.y, c3.y);
      s[e + 2] = make_float4(c0.z, c1.z, c2.z, c3.z);
      s[e + 3] = make_float4(c0.w, c1.w, c2.w, c3.w);
    }
  }
  // A thread's four rows (and columns) of P and O lie in the chunk's four 16-row blocks, taken
  // in walk order: row block i meets column blocks 0 .. i alone.
  const int turn = q.reverse ? -16 : 16, first = q.reverse ? 48 : 0;
  const int row0 = ty + first, col0 = tx + first;
  for (int ci = 0; ci < nc; ++ci) {
    const int64_t done = (int64_t)ci * C;
    const bool end = ci + 1 == nc;
    const int L = end ? tail : C;
    const int64_t r0 = q.reverse ? se - done - L : sb + done;
    __syncthreads();                              // the last chunk's readers; the tables
    if (NB == 1 ? ci > 0 : !end) fetch(NB == 1 ? ci : ci + 1);
    if (!kState) {
#pragma unroll
      for (int e = 0; e < YR; ++e) st4(&sm.S[ty * YR + e][4 * tx], s[e]);
    }
    if (NB > 1 && !end) copies_wait<1>();
    else copies_wait<0>();
    __syncthreads();
    const auto& X = sm.X[ci % NB];
    const auto& Y = sm.Y[ci % NB];
    const auto& Z = sm.Z[ci % NB];
    if (!kState) {
      // P rows row0 + turn i, columns col0 + turn j
      float2 acc[4][4] = {};                      // sums over even and odd c
#pragma unroll 8
      for (int c = 0; c < D; c += 4) {
        float4 xv[4], yv[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) xv[i] = ld4(&X[row0 + turn * i][c]);
#pragma unroll
        for (int j = 0; j < 4; ++j) yv[j] = ld4(&Y[col0 + turn * j][c]);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j <= i; ++j)
            acc[i][j] = fma2(make_float2(xv[i].x, xv[i].y), make_float2(yv[j].x, yv[j].y),
                             fma2(make_float2(xv[i].z, xv[i].w), make_float2(yv[j].z, yv[j].w), acc[i][j]));
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j <= i; ++j) {
          const int r = row0 + turn * i, c = col0 + turn * j, gap = q.reverse ? c - r : r - c;
          sm.P[r][c] = gap >= 0 ? (acc[i][j].x + acc[i][j].y) * (q.a * sm.tab[gap]) : 0.f;
        }
      __syncthreads();
      // O rows row0 + turn i, columns 4 tx ..
      float2 o[4][2] = {};
      auto add = [](float2 (&o)[2], float x, float4 v) {   // o += x v
        o[0] = fma2(make_float2(x, x), make_float2(v.x, v.y), o[0]);
        o[1] = fma2(make_float2(x, x), make_float2(v.z, v.w), o[1]);
      };
#pragma unroll 4
      for (int c = 0; c < D; c += 4) {
        float4 sv[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) sv[e] = ld4(&sm.S[c + e][4 * tx]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 xv = ld4(&X[row0 + turn * i][c]);
          add(o[i], xv.x, sv[0]);
          add(o[i], xv.y, sv[1]);
          add(o[i], xv.z, sv[2]);
          add(o[i], xv.w, sv[3]);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = row0 + turn * i;
        const float f = r < L ? q.b * sm.tab[q.reverse ? L - 1 - r : r + 1] : 0.f;
        o[i][0] = mul2(o[i][0], make_float2(f, f));
        o[i][1] = mul2(o[i][1], make_float2(f, f));
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll 4
      for (int c4 = 0; c4 < 16; c4 += 4) {
        const int c = col0 - tx + turn * j + c4;
        float4 zv[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) zv[e] = ld4(&Z[c + e][4 * tx]);
#pragma unroll
        for (int i = j; i < 4; ++i) {
          const float4 pv = ld4(&sm.P[row0 + turn * i][c]);
          add(o[i], pv.x, zv[0]);
          add(o[i], pv.y, zv[1]);
          add(o[i], pv.z, zv[2]);
          add(o[i], pv.w, zv[3]);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = row0 + turn * i;
        if (r >= L) continue;
        const size_t at = ((size_t)(r0 + r) * p.H + h) * D + zc + 4 * tx;
        st4(static_cast<float*>(q.out) + at, make_float4(o[i][0].x, o[i][0].y, o[i][1].x, o[i][1].y));
      }
    }
    // S = lam^L S + c sum_r lam^f(r) y_r z_r
    const float hi = sm.carry[end ? 2 : 0], lo = sm.carry[end ? 3 : 1];
    const float* wr = sm.wr[end];
    float2 acc[YR / 2][4] = {};                   // rows 2 e, 2 e + 1 of the state, columns 4 tx + j
#pragma unroll 8
    for (int r = 0; r < C; ++r) {                 // (rows past L are zero)
      const float wgt = wr[r];
      const float4 z4 = ld4(&Z[r][4 * tx]);
      const float zv[4] = {z4.x * wgt, z4.y * wgt, z4.z * wgt, z4.w * wgt};
      float2 yv[YR / 2];
#pragma unroll
      for (int e = 0; e < YR / 2; e += 2) *reinterpret_cast<float4*>(&yv[e]) = ld4(&Y[r][ty * YR + 2 * e]);
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < YR / 2; ++e) acc[e][j] = fma2(yv[e], make_float2(zv[j], zv[j]), acc[e][j]);
    }
#pragma unroll
    for (int e = 0; e < YR; ++e) {
      s[e].x = fmaf(hi, s[e].x, fmaf(lo, s[e].x, e & 1 ? acc[e / 2][0].y : acc[e / 2][0].x));
      s[e].y = fmaf(hi, s[e].y, fmaf(lo, s[e].y, e & 1 ? acc[e / 2][1].y : acc[e / 2][1].x));
      s[e].z = fmaf(hi, s[e].z, fmaf(lo, s[e].z, e & 1 ? acc[e / 2][2].y : acc[e / 2][2].x));
      s[e].w = fmaf(hi, s[e].w, fmaf(lo, s[e].w, e & 1 ? acc[e / 2][3].y : acc[e / 2][3].x));
    }
  }
  float* dst = kState ? q.sums + uoff : t.last ? la_exit(p, q, n, h, D) : nullptr;
  if (!dst) return;
  if (q.s_t && !kState) {
#pragma unroll
    for (int e = 0; e < YR; ++e) st4(dst + (size_t)(ty * YR + e) * D + zc + 4 * tx, s[e]);
    return;
  }
  const int zs = kState ? 4 : D, ys = kState ? D : 1;
#pragma unroll
  for (int e = 0; e < YR; e += 4) {
    float* v = dst + (ty * YR + e) * ys + (zc + 4 * tx) * zs;
    st4(v, make_float4(s[e].x, s[e + 1].x, s[e + 2].x, s[e + 3].x));
    st4(v + zs, make_float4(s[e].y, s[e + 1].y, s[e + 2].y, s[e + 3].y));
    st4(v + 2 * zs, make_float4(s[e].z, s[e + 1].z, s[e + 2].z, s[e + 3].z));
    st4(v + 3 * zs, make_float4(s[e].w, s[e + 1].w, s[e + 2].w, s[e + 3].w));
  }
}

// Entry states of the segments of one (sequence, head, pass): e = the caller's state, then
// e = lam^pre e + sum over the pieces, kept at every segment's start.  Each thread carries one
// float4 of the state, and sixteen CTAs share a state at D = 128.  Bound by the latency of L2, which
// the early copies of the launch behind it stretch to microseconds: AHEAD pieces' sums are in
// flight together, 32 where the walks leave each CTA an SM, else 8, whose registers leave room for
// more CTAs.  Measured, all three launches (8, 32 ahead): 4 walks of 35 pieces 156.6, 146.4 us, 6 of
// 24 68.6, 62.5 us; 16 walks 82.9, 85.0 us, 64 walks of 2 pieces 76.8, 91.2 us.  (Loading a piece as
// another is used: 37.8 -> 58.4 us for one walk of 127.)  Both kernels' walks use it.
template <int D, int AHEAD>
__global__ void __launch_bounds__(256) la_carry_kernel(const LaParams p) {
  launch_next();
  const int tid = threadIdx.x;
  constexpr int PARTS = D * D / 1024;
  const int part = blockIdx.x % PARTS;
  int pi, h, n;                                        // packed: the n-th walk that is cut
  la_place(blockIdx.x / PARTS, p, pi, h, n);
  const LaPass& q = p.pass[pi];
  const int k = p.per_seg;
  int64_t len = p.T;
  int u0, s0;
  if (!p.cu) {
    const int S = p.cuts;
    u0 = n * S;
    s0 = n * (S - 1) * k;
  } else {
    const int lane = tid & 31;
    const int nth = n;
    int found = -1, sum = 0;                           // its sequence; segments of the ones before it
    for (int m0 = 0; m0 < p.N && found < 0; m0 += 32) {
      const int m = m0 + lane;
      int64_t b = 0, e = 0;
      if (m < p.N) seq_span(m, p.B, p.T, p.cu, b, e);
      unsigned hit = __ballot_sync(0xffffffffu, e - b > p.seg);
      int upto = 32;
      if (n < __popc(hit)) {
        for (; n > 0; --n) hit &= hit - 1;
        upto = __ffs(hit) - 1;
        found = m0 + upto;
        len = __shfl_sync(0xffffffffu, e - b, upto);
      } else {
        n -= __popc(hit);
      }
      if (lane < upto && e - b > p.seg) sum += la_segments(e - b, p);
    }
    if (found < 0) {                                   // fewer walks are cut
      launch_wait();                                   // (the launch before may still read the offsets)
      return;
    }
    n = found;
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    u0 = sum;
    s0 = (sum - nth) * k;
  }
  const int S = la_segments(len, p), pieces = (S - 1) * k;
  bool skip;
  const float* s_in = la_entry(p, q, n, h, D, skip);
  // padding; malformed offsets
  if (skip || u0 + S > p.entries || s0 + pieces > p.pre_units) {
    launch_wait();
    return;
  }
  const int at = (part * 256 + tid) * 4, z = at / 4 % D, y = at / (4 * D) * 4;
  float4 e = make_float4(0.f, 0.f, 0.f, 0.f);
  if (s_in) {
    if (q.s_t) e = make_float4(s_in[(size_t)y * D + z], s_in[(size_t)(y + 1) * D + z],
                               s_in[(size_t)(y + 2) * D + z], s_in[(size_t)(y + 3) * D + z]);
    else e = ld4(s_in + (size_t)z * D + y);
  }
  __shared__ float pow_s[2];
  if (tid == 0) {
    const double full = la_pow(p.decay[h], p.pre);
    pow_s[0] = (float)full;
    pow_s[1] = (float)(full - (double)pow_s[0]);
  }
  const size_t step = (size_t)p.H * D * D;
  float* out = q.entry + ((size_t)u0 * p.H + h) * D * D + at;
  const float* in = q.sums + ((size_t)s0 * p.H + h) * D * D + at;
  launch_wait();                                       // the sums
  st4(out, e);
  __syncthreads();
  const float hi = pow_s[0], lo = pow_s[1];
  int until = k;                                       // pieces to the next segment's start
  for (int i = 0; i < pieces; i += AHEAD) {
    float4 x[AHEAD];
#pragma unroll
    for (int j = 0; j < AHEAD; ++j)
      if (i + j < pieces) x[j] = ld4(in + (size_t)(i + j) * step);
#pragma unroll
    for (int j = 0; j < AHEAD; ++j)
      if (i + j < pieces) {
        e.x = fmaf(hi, e.x, fmaf(lo, e.x, x[j].x));
        e.y = fmaf(hi, e.y, fmaf(lo, e.y, x[j].y));
        e.z = fmaf(hi, e.z, fmaf(lo, e.z, x[j].z));
        e.w = fmaf(hi, e.w, fmaf(lo, e.w, x[j].w));
        if (--until == 0) {
          out += step;
          st4(out, e);
          until = k;
        }
      }
  }
}

template <int D, bool kState>
cudaError_t go(const LaParams& p, cudaStream_t st) {
  const int64_t grid = (int64_t)(kState ? p.pre_units : p.units) * p.H * p.npass * (D / ZT);
  if (grid <= 0) return cudaSuccess;
  if (grid > 0x7fffffff) return cudaErrorInvalidValue;
  auto kern = la_simt_kernel<D, kState>;
  const cudaError_t e = allow_smem(kern, sizeof(Smem<D>));
  if (e != cudaSuccess) return e;
  // (not early: CTAs placed beside the last ones of the launch before would share their SMs)
  return launch_after(false, kern, (unsigned)grid, 256, sizeof(Smem<D>), st, p);
}

}  // namespace

cudaError_t launch_la_simt(const LaParams& p, int D, bool state_only, cudaStream_t st) {
  if (D == 64) return state_only ? go<64, true>(p, st) : go<64, false>(p, st);
  return state_only ? go<128, true>(p, st) : go<128, false>(p, st);
}

cudaError_t launch_la_carry(const LaParams& p, int D, cudaStream_t st) {
  // (a walk that is cut has more than `seg` rows: of packed ones there are T / seg at most)
  const int walks = p.cu && p.T / p.seg < p.N ? p.T / p.seg : p.N;
  const int64_t grid = (int64_t)walks * p.H * p.npass * (D * D / 1024);
  if (grid <= 0) return cudaSuccess;
  if (grid > 0x7fffffff) return cudaErrorInvalidValue;
  // pieces of a walk (of packed ones that are cut: of an average one)
  const int pieces = p.cu ? p.pre_units / walks : (p.cuts - 1) * p.per_seg;
  const bool deep = pieces > 8 && grid <= 152;
  auto kern = D == 64 ? (deep ? la_carry_kernel<64, 32> : la_carry_kernel<64, 8>)
                      : (deep ? la_carry_kernel<128, 32> : la_carry_kernel<128, 8>);
  return launch_after(true, kern, (unsigned)grid, 256, 0, st, p);
}

}  // namespace sfg
