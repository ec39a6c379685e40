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
// A long walk is cut into segments of `seg` rows (in walk order) that run side by side: a first
// launch computes what each piece of `pre` rows (seg / pre to a segment) adds to the state, a
// second carries the entry states over the pieces, a third runs the segments from them.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/sf_linattn.h"

namespace sfg {

// Division of 0 <= n < 2^31 by a constant of the launch, d >= 1 (Granlund and Montgomery 1994): with
// 2^(sh-1) < d <= 2^sh and mul = floor(2^32 (2^sh - d) / d) + 1, n / d = (n mul / 2^32 + n) / 2^sh.
// A unit's place takes six divisions in a row before its first copy can start, and one by a
// variable costs ~150 cycles.
struct FastDiv {
  uint32_t mul, sh;
  static FastDiv of(uint32_t d) {
    uint32_t sh = 0;
    while ((1ull << sh) < d) ++sh;
    return {(uint32_t)((((1ull << sh) - d) << 32) / d + 1), sh};
  }
#ifdef __CUDACC__
  __device__ __forceinline__ int operator()(int n) const {
    return (int)((__umulhi((uint32_t)n, mul) + (uint32_t)n) >> sh);
  }
#endif
};

struct LaPass {
  const void* x;
  const void* y;
  const void* z;
  void* out;            // [rows, H, D]: the token type, or FP32 (out_f32)
  const float* s_in;    // [N,H,D,D] or NULL (zeros)
  float* s_out;         // [N,H,D,D] or NULL
  float* entry;         // [entries,H,D/4,D,4] (y / 4, z, y % 4): entry states of cut walks' segments
  float* sums;          // [pre_units,H,D/4,D,4]: what each piece adds to the state
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
  int seg, pre;         // rows of a segment and of a piece, multiples of 64; pre divides seg
  int per_seg, cuts;    // pieces of a segment; segments of a walk (not packed)
  FastDiv by_pass, by_head, by_group, by_n, by_seg, by_pieces;   // npass, H, H / HK, N, seg, pieces of a walk
  int units, pre_units; // launched (sequence, segment) and (sequence, piece) units; packed: bounds
  int entries;          // segments of walks that are cut; packed: a bound
  int* status;
  int tries;            // of a wait in a launch that a test makes give up (linattn_tc.cu), else 0
};

constexpr int LA_CHUNK = 64;

// (sequence, segment) units of a launch whose segments have `seg` rows, and (sequence, piece)
// units of all segments but each walk's last.
inline int64_t la_units(int64_t T, int64_t N, bool packed, int64_t seg) {
  const int64_t per = T > seg ? (T + seg - 1) / seg : 1;
  return packed ? T / seg + N : N * per;
}
inline int64_t la_pre_units(int64_t T, int64_t N, bool packed, int64_t seg, int64_t pre) {
  const int64_t cuts = packed ? T / seg : N * ((T > seg ? (T + seg - 1) / seg : 1) - 1);
  return cuts * (seg / pre);
}
// Segments of the walks that are cut (the others take their states from the caller).  Packed: such
// a walk's S segments but the last are whole, T / seg of them in all, and S <= 2 (S - 1).
inline int64_t la_entries(int64_t T, int64_t N, bool packed, int64_t seg) {
  if (T <= seg) return 0;
  const int64_t whole = T / seg;
  return packed ? whole + (whole < N ? whole : N) : N * ((T + seg - 1) / seg);
}

#ifdef __CUDACC__
struct LaUnit {
  int n;                // sequence
  int64_t bos, eos;     // its rows, clamped into [0, B T]
  int64_t off, rows;    // the unit's rows in walk order
  int at;               // its place in `entry` (segments of a cut walk) or `sums` (pieces)
  bool last;            // the walk ends with it
};

__device__ __forceinline__ int la_segments(int64_t len, const LaParams& p) {
  return len > p.seg ? p.by_seg((int)len + p.seg - 1) : 1;   // (fewer than 2^26 rows)
}
// Entry states of a walk of S segments.
__device__ __forceinline__ int la_kept(int S) { return S > 1 ? S : 0; }
// A CTA's pass, head and unit.
__device__ __forceinline__ void la_place(int id, const LaParams& p, int& pass, int& h, int& u) {
  const int a = p.by_pass(id), b = p.by_head(a);
  pass = id - a * p.npass;
  h = a - b * p.H;
  u = b;
}
// The head that value head h reads of a tensor with `heads` of them (H or HK).
__device__ __forceinline__ int la_head(int h, int heads, const LaParams& p) {
  return heads == p.H ? h : p.by_group(h);
}

// Unit u of a launch; a warp calls it together.  False when the unit holds nothing.  Whole
// segments come first, then the walks' remainders -- the longest first, for up to 64 packed
// sequences -- so that the launch ends evenly.
template <bool kPieces>
__device__ __forceinline__ bool la_locate(int u, const LaParams& p, LaUnit& t) {
  const int64_t total = (int64_t)p.B * p.T;
  const int k = p.per_seg;
  if (!p.cu) {
    const int S = p.cuts;
    int w;
    if (kPieces) {
      t.n = p.by_pieces(u);
      w = u - t.n * (S - 1) * k;
      t.at = u;
    } else {
      w = p.by_n(u);
      t.n = u - w * p.N;
      t.at = t.n * S + w;
      if (w >= S) return false;
    }
    if (t.n >= p.N) return false;
    t.bos = (int64_t)t.n * p.T;
    t.eos = t.bos + p.T;
    t.off = (int64_t)w * (kPieces ? p.pre : p.seg);
    t.last = !kPieces && w + 1 == S;
    t.rows = t.last ? p.T - t.off : (kPieces ? p.pre : p.seg);
    return true;
  }
  const int lane = threadIdx.x & 31;
  auto span = [&](int m, int64_t& b, int64_t& e) {
    b = p.cu[m];
    e = p.cu[m + 1];
    b = b < 0 ? 0 : (b > total ? total : b);
    e = e < b ? b : (e > total ? total : e);
  };
  // the place of u among the whole segments (pieces), or past them among the remainders
  int base = 0, at = 0, found = -1, w = 0;
#pragma unroll 1
  for (int m0 = 0; m0 < p.N; m0 += 32) {
    const int m = m0 + lane;
    int64_t b = 0, e = 0;
    int S = 0;
    if (m < p.N) {
      span(m, b, e);
      S = la_segments(e - b, p);
    }
    const int cnt = S > 0 ? (kPieces ? (S - 1) * k : S - 1) : 0;
    int incl = cnt, slots = kPieces ? cnt : la_kept(S);   // before the walk's last segment; stored
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, incl, o), y = __shfl_up_sync(0xffffffffu, slots, o);
      if (lane >= o) incl += x, slots += y;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, u >= base + incl - cnt && u < base + incl);
    if (hit) {
      const int src = __ffs(hit) - 1;
      found = m0 + src;
      w = u - __shfl_sync(0xffffffffu, base + incl - cnt, src);
      at += __shfl_sync(0xffffffffu, slots - (kPieces ? cnt : la_kept(S)), src) + w;
      break;
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
    at += __shfl_sync(0xffffffffu, slots, 31);
  }
  if (kPieces) {
    if (found < 0) return false;
    t.n = found;
    span(found, t.bos, t.eos);
    t.off = (int64_t)w * p.pre;
    t.rows = p.pre;
    t.at = at;
    t.last = false;
    return true;
  }
  t.last = found < 0;
  if (found < 0) {
    const int r = u - base;                            // the r-th remainder
    if (r >= p.N) return false;
    found = r;
    if (p.N <= 64) {
      auto rem = [&](int m) {
        int64_t b, e;
        span(m, b, e);
        return e - b - (int64_t)(la_segments(e - b, p) - 1) * p.seg;
      };
#pragma unroll 1
      for (int m0 = 0; m0 < p.N; m0 += 32) {
        const int m = m0 + lane;
        int rank = -1;
        if (m < p.N) {
          const int64_t mine = rem(m);
          rank = 0;
#pragma unroll 1
          for (int o = 0; o < p.N; ++o) {
            const int64_t other = rem(o);
            rank += other > mine || (other == mine && o < m);
          }
        }
        const unsigned hit = __ballot_sync(0xffffffffu, rank == r);
        if (hit) found = m0 + __ffs(hit) - 1;
      }
    }
    span(found, t.bos, t.eos);
    const int S = la_segments(t.eos - t.bos, p);
    w = S - 1;
    at = 0;                                            // entry states of the sequences before it
#pragma unroll 1
    for (int m = lane; m < found; m += 32) {
      int64_t b, e;
      span(m, b, e);
      at += la_kept(la_segments(e - b, p));
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) at += __shfl_xor_sync(0xffffffffu, at, o);
    at += w;
  }
  t.n = found;
  span(found, t.bos, t.eos);
  t.off = (int64_t)w * p.seg;
  t.rows = t.last ? t.eos - t.bos - t.off : p.seg;
  t.at = at;
  return (t.last && w == 0) || at < p.entries;         // (malformed offsets could ask for more)
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

// The CUDA-core kernel (FP32 tokens, D 64 or 128): state_only computes the pieces' sums,
// otherwise the outputs.
cudaError_t launch_la_simt(const LaParams& p, int D, bool state_only, cudaStream_t st);
// The tcgen05 kernel (BF16 tokens, D 64 or 128; needs tc_fwd_available()).
cudaError_t launch_la_tc(const LaParams& p, int D, bool state_only, cudaStream_t st);
// sums -> entry: the entry state of every segment.
cudaError_t launch_la_carry(const LaParams& p, int D, cudaStream_t st);

// Lets `kern` take `bytes` of dynamic shared memory: once for each device and kernel (the call
// costs a microsecond; a small problem's whole launch takes a few).
template <typename K>
inline cudaError_t allow_smem(K kern, size_t bytes) {
  constexpr int DEVICES = 64;
  static std::atomic<const void*> done[DEVICES][8];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const void* id = reinterpret_cast<const void*>(kern);
  if (dev < DEVICES)
    for (auto& d : done[dev])
      if (d.load(std::memory_order_relaxed) == id) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e != cudaSuccess || dev >= DEVICES) return e;
  for (auto& d : done[dev]) {
    const void* none = nullptr;
    if (d.compare_exchange_strong(none, id, std::memory_order_relaxed)) break;
  }
  return cudaSuccess;
}

// The launches of one call follow one another closely: each may start while the one before it
// ends (its start needs none of that one's results), and waits for them (launch_wait) where it
// does.  Only launches after a call's first do so: `early`.
template <typename... P, typename... A>
inline cudaError_t launch_after(bool early, void (*kern)(P...), dim3 grid, unsigned threads,
                                size_t smem, cudaStream_t st, const A&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = early ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}
#ifdef __CUDACC__
__device__ __forceinline__ void launch_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void launch_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
#endif

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
