// draft_verify.cu -- drafted tokens against the target's probabilities (include/sf_decode.h).
//
// A cluster of CTAs takes a sequence: every CTA finds the first rejected draft a (a gather of two
// values a draft), then sums its slice of the weights w = max(p_a - q_a, 0); the slices' sums meet
// in shared memory, and the warp whose slice crosses u * total reads it again (from L2) to find
// the token.  Bound by memory: one row of p and one of q.
//
// The comparison and the search have to give what exact arithmetic gives, however the sums are
// split: the test is one product in FP64 (exact for FP32 factors); a thread sums in two floats
// (the rounding error of every difference and sum is kept: FP64 at a fraction of its cost on this
// machine), and the threads' sums are joined in FP64 in a fixed order.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include "common.cuh"
#include "decode.cuh"

namespace sfg {
namespace {

namespace cg = cooperative_groups;
constexpr int THREADS = 256;
constexpr int WARPS = THREADS / 32;
constexpr int MAX_CLUSTER = 8;

enum Weight { kTarget, kLess, kOthers };   // p, max(p - q, 0), p but for the drafted token

// w as two floats (the second one the rounding error of the difference); not positive: zero.
template <typename T>
__device__ __forceinline__ float2 weight(const T* p, const T* q, int y, int skip, Weight how) {
  const float a = to_f(p[y]);
  if (how == kLess) {
    const float b = to_f(q[y]);
    const float d = __fsub_rn(a, b), t = __fsub_rn(d, a);
    const float e = __fsub_rn(__fsub_rn(a, __fsub_rn(d, t)), __fadd_rn(b, t));
    return d > 0.f ? make_float2(d, e) : make_float2(0.f, 0.f);
  }
  return make_float2(a > 0.f && !(how == kOthers && y == skip) ? a : 0.f, 0.f);
}

__device__ __forceinline__ void add(float2& s, float2 w) {
  const float n = __fadd_rn(s.x, w.x), t = __fsub_rn(n, s.x);
  s.y += __fadd_rn(__fsub_rn(s.x, __fsub_rn(n, t)), __fsub_rn(w.x, t)) + w.y;
  s.x = n;
}

__device__ __forceinline__ double warp_sum(double x) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

template <typename T>
__global__ void __launch_bounds__(THREADS) draft_verify_kernel(const VerifyParams p) {
  __shared__ double sums[2][MAX_CLUSTER * WARPS];    // of every warp of the cluster, in order
  __shared__ int accepted;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
  const int n = blockIdx.x / ranks;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const T* target = reinterpret_cast<const T*>(p.target) + n * p.target_seq;
  const T* draft = reinterpret_cast<const T*>(p.draft) + (p.draft ? n * p.draft_seq : 0);
  int32_t* tokens = p.tokens + (size_t)n * (p.T + 1);
  const float* u = p.u + (size_t)n * (p.T + 1);
  const int32_t* x = p.x + (size_t)n * p.T;
  const int nd = p.num ? min(p.num[n], p.T) : p.T;
  if (nd < 0) {       // padding: the whole cluster leaves
    if (rank == 0) {
      for (int i = threadIdx.x; i <= p.T; i += THREADS) tokens[i] = -1;
      if (threadIdx.x == 0) p.count[n] = 0;
    }
    return;
  }
  cluster.barrier_arrive();   // waited for before the first store into another CTA
  if (warp == 0) {
    int a = 0;
    while (a < nd) {
      const int i = a + lane;
      bool ok = false;
      if (i < nd) {
        const int y = x[i];
        if (y >= 0 && y < p.V) {
          const double q = p.draft ? (double)to_f(draft[i * p.draft_row + y]) : 1.0;
          ok = (double)u[i] * q < (double)to_f(target[i * p.target_row + y]);
        }
      }
      const unsigned no = ~__ballot_sync(0xffffffffu, ok);
      if (no) { a += __ffs(no) - 1; break; }
      a += 32;
    }
    if (lane == 0) accepted = min(a, nd);
  }
  __syncthreads();
  const int a = accepted;
  if (rank == 0) {
    for (int i = threadIdx.x; i <= p.T; i += THREADS)
      if (i != a) tokens[i] = i < a ? x[i] : -1;
    if (threadIdx.x == 0) p.count[n] = a + 1;
  }
  const T* pr = target + a * p.target_row;
  const T* qr = a < nd && p.draft ? draft + a * p.draft_row : nullptr;
  const int skip = a < nd ? x[a] : -1;
  Weight how = a == nd ? kTarget : qr ? kLess : kOthers;

  const int64_t workers = (int64_t)ranks * WARPS, me = (int64_t)rank * WARPS + warp;
  const int lo = (int)(p.V * me / workers), hi = (int)(p.V * (me + 1) / workers);
  for (int pass = 0;; ++pass) {
    float2 s = make_float2(0.f, 0.f);
#pragma unroll 8
    for (int y = lo + lane; y < hi; y += 32) add(s, weight(pr, qr, y, skip, how));
    const double mine = warp_sum((double)s.x + (double)s.y);
    if (pass == 0) cluster.barrier_wait();
    if (lane < ranks) cluster.map_shared_rank(&sums[pass][0], lane)[me] = mine;
    cluster.sync();
    double total = 0.0, before = 0.0;
    for (int w = 0; w < workers; ++w) {
      const double v = sums[pass][w];
      if (w == me) before = total;
      total += v;
    }
    if (!(total > 0.0) && how != kTarget && total == 0.0) {   // nothing is left: draw from p
      how = kTarget;
      continue;
    }
    if (!(total > 0.0) || isinf(total)) {
      if (rank == 0 && threadIdx.x == 0) tokens[a] = -1;
      return;
    }
    const double aim = (double)u[p.T] * total;
    // the first warp whose slice passes the aim; the last one with any weight if rounding or a u
    // outside [0,1) leaves none
    int pick = -1, any = -1;
    double run = 0.0;
    for (int w = 0; w < workers; ++w) {
      const double v = sums[pass][w];
      run += v;
      if (v > 0.0) any = w;
      if (v > 0.0 && run > aim) { pick = w; break; }
    }
    if (pick < 0) pick = any;
    if (pick != me) return;
    // this warp's slice once more, a run of neighbours to a lane
    const int len = hi - lo, per = (len + 31) / 32;
    const int b = min(lo + lane * per, hi), e = min(b + per, hi);
    double sum = 0.0;
    for (int y = b; y < e; ++y) {
      const float2 w = weight(pr, qr, y, skip, how);
      sum += (double)w.x + (double)w.y;
    }
    double incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double t = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += t;
    }
    const unsigned over = __ballot_sync(0xffffffffu, sum > 0.0 && before + incl > aim);
    const unsigned some = __ballot_sync(0xffffffffu, sum > 0.0);
    const int who = over ? __ffs(over) - 1 : 31 - __clz(some);
    if (lane != who) return;
    double at = before + (incl - sum);
    int y = -1;
    for (int i = b; i < e; ++i) {
      const float2 w = weight(pr, qr, i, skip, how);
      const double v = (double)w.x + (double)w.y;
      if (!(v > 0.0)) continue;
      at += v;
      y = i;
      if (at > aim) break;
    }
    tokens[a] = y;
    return;
  }
}

template <typename T>
cudaError_t go(const VerifyParams& p, cudaStream_t st) {
  int ranks = MAX_CLUSTER;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.N * ranks));
  cfg.blockDim = dim3(THREADS);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = ranks;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, draft_verify_kernel<T>, p);
}

}  // namespace

cudaError_t launch_draft_verify(const VerifyParams& p, bool bf16, cudaStream_t st) {
  if (p.N < 1) return cudaSuccess;
  return bf16 ? go<__nv_bfloat16>(p, st) : go<float>(p, st);
}

}  // namespace sfg
