// draft_verify.cu -- drafted tokens against the target's probabilities (include/sf_decode.h).
//
// A cluster of CTAs takes a sequence: every CTA finds the first rejected draft a (a gather of two
// values a draft), then each warp sums its slice of the weights w = max(p_a - q_a, 0); the slices'
// sums meet in the shared memory of all CTAs, and the CTA of the slice that crosses u * total reads
// it again (from L2) to find the token.  Bound by memory: one row of p and one of q.
//
// The comparison and the search have to give what exact arithmetic gives, however the sums are
// split: the test is one product in FP64 (exact for FP32 factors), and sums are two floats, a sum
// and the rounding errors of its additions and differences (48 bits, kept over long rows by Sum; FP64 would be exact
// enough, but this machine does two FP64 operations a clock and SM, and a warp's scan in it takes
// 1.5 us).
//
// Measured, 128 sequences, 7 drafts, 100003 tokens, FP32: 26.8 us (floor 13.0: one row of p, most of q)
// of which, by the clock of its CTAs (two of 16 warps a sequence), the test 1.5, the stream 13 for the
// median CTA and 18 for the last one, the sums' way and the pick among the warps 2, the search 3.5.
// Rows of BF16 23 us, of looked-up drafts 22 and (BF16) 20.  Of many rows
// instructions take more: 600 sequences with 2 drafts 76 us (floor 46), 45 M instructions, 59 % of the issue slots;
// in BF16 59 us (floor 23), 42 M, 72 %.
// With 8 warps: copies of 16 bytes to shared memory against 4-byte loads to registers (rows start at any
// multiple of an element) stream 22 -> 13-19; sums sent with st.async to a barrier against a cluster barrier
// with release and acquire 28.3 -> 26.9 us; five CTAs an SM 26.9, 3, 4, 6: 32.0, 27.5, 31-35 (six leave
// clusters for a second wave).
#include <cuda_bf16.h>

#include "common.cuh"
#include "decode.cuh"
#include "tc_ptx.cuh"

namespace sfg {
namespace {

constexpr int MAX_CLUSTER = 8;
// CTAs of WARPS warps on an SM.  Long rows take 16 warps: fewer rows are under way at a time, and each
// is read faster (600 sequences of 100003 tokens 117 us with 8 warps, 73 with 16; of 65536 72, 53; 128
// sequences the same either way).  Short ones end sooner with 8 (32000 tokens, 600 sequences 32, 36; 2000 82,
// 104).  Of 50000 tokens 600 sequences take 51, 44, 2000 128, 118: many rows could change over from there on.
template <int WARPS>
constexpr int CTAS = WARPS == 8 ? 5 : 2;
constexpr int LONG_ROW = 65536;
constexpr int DEEP_ROW = 1 << 20;  // longer ones than that sum in three levels
constexpr int STAGES = 2;         // chunks of a warp's slice in flight
constexpr int CHUNK_BYTES = 1024; // of a row
constexpr int STAGE = STAGES * 2 * (CHUNK_BYTES + 16);
constexpr int kSlice = 1024;      // elements that are worth a CTA

constexpr int kNone = -1, kAgain = -2, kLate = -3;     // in place of the picked warp

enum Weight { kTarget, kLess, kOthers };   // p, max(p - q, 0), p but for the drafted token

// w as two floats (the second one the rounding error of the difference, exact where the first is
// positive and the draft's value is not negative); not positive: zero.
template <Weight how>
__device__ __forceinline__ float2 weight(float a, float b, bool skip) {
  if (how == kLess) {
    const float d = __fsub_rn(a, b);
    return d > 0.f ? make_float2(d, __fsub_rn(__fsub_rn(a, d), b)) : make_float2(0.f, 0.f);
  }
  return make_float2(a > 0.f && !(how == kOthers && skip) ? a : 0.f, 0.f);
}

__device__ __forceinline__ void add(float2& s, float2 w) {
  const float n = __fadd_rn(s.x, w.x), t = __fsub_rn(n, s.x);
  s.y = __fadd_rn(s.y, __fadd_rn(__fadd_rn(__fsub_rn(s.x, __fsub_rn(n, t)), __fsub_rn(w.x, t)), w.y));
  s.x = n;
}
__device__ __forceinline__ float2 sum(float2 a, float2 b) {
  add(a, b);
  return a;
}
// The sum of a long run of non-negative weights.  add() rounds what the low parts gather to 24 bits, and
// they grow with the number of additions (0.7 262144 times: off by 2^-18).  So up to 17 weights are added from
// zero (m of them: off by m^2 2^-48 at the worst), such sums in runs of 64, the runs' sums in runs of 64, and
// those, each with its low part brought below half a step of the high one: 64 x 2^-47 a level, 2^-38
// in all.  (Against additions in one run 26.5 -> 26.7 us in the batch below.)
template <bool kDeep>      // (up to 2^20 tokens one level does: 256 chunks a lane)
struct Sum {
  static constexpr int LEVELS = kDeep ? 3 : 1;
  float2 s[LEVELS] = {};
  int n = 0;
  static __device__ __forceinline__ void fold(float2& s, float2 w) {
    add(s, w);
    const float h = __fadd_rn(s.x, s.y);
    s.y = __fsub_rn(s.y, __fsub_rn(h, s.x));
    s.x = h;
  }
  __device__ __forceinline__ void operator+=(float2 w) {
    fold(s[0], w);
    if (kDeep && (++n & 63) == 0) {
      fold(s[1 % LEVELS], s[0]);
      s[0] = make_float2(0.f, 0.f);
      if ((n & 4095) == 0) {
        fold(s[LEVELS - 1], s[1 % LEVELS]);
        s[1 % LEVELS] = make_float2(0.f, 0.f);
      }
    }
  }
  __device__ __forceinline__ float2 total() const {
    float2 t = s[0];
    if (kDeep && n >= 64) {
      fold(t, s[1 % LEVELS]);
      fold(t, s[LEVELS - 1]);
    }
    return t;
  }
};
// a > b, of sums of non-negative weights; false with a NaN.
__device__ __forceinline__ bool more(float2 a, float2 b) {
  const float ah = __fadd_rn(a.x, a.y), al = __fadd_rn(__fsub_rn(a.x, ah), a.y);
  const float bh = __fadd_rn(b.x, b.y), bl = __fadd_rn(__fsub_rn(b.x, bh), b.y);
  return ah > bh || (ah == bh && al > bl);
}
__device__ __forceinline__ float2 shfl(float2 s, int lane) {
  return make_float2(__shfl_sync(0xffffffffu, s.x, lane), __shfl_sync(0xffffffffu, s.y, lane));
}
// (Behind the stream, once: kept out of the stream's registers.)
__device__ __noinline__ float2 warp_sum(float2 s) {
#pragma unroll 1
  for (int o = 16; o >= 1; o >>= 1)
    add(s, make_float2(__shfl_xor_sync(0xffffffffu, s.x, o), __shfl_xor_sync(0xffffffffu, s.y, o)));
  return shfl(s, 0);     // (the lanes' low parts may differ)
}

__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}

// A warp's sum of the weights [lo, hi).  Rows start anywhere: whole chunks are copied in
// 16-byte units from the unit that holds their first element to the one behind their last, which lie
// within the slice because 16 bytes at least of it are left at either end; those ends are loaded.
template <typename T, Weight how, bool kDeep>
__device__ __forceinline__ float2 sum_slice(const T* p, const T* q, int lo, int hi, int skip, char* buf) {
  constexpr int E = 16 / sizeof(T), C = CHUNK_BYTES / sizeof(T);
  constexpr int ROW = CHUNK_BYTES + 16, UNITS = ROW / 16;
  const int lane = threadIdx.x & 31;
  const int chunks = hi - lo >= C + 2 * E ? (hi - lo - 2 * E) / C : 0;
  const char* pa = reinterpret_cast<const char*>(p + lo + E);
  const char* qa = reinterpret_cast<const char*>(q + lo + E);
  const int ps = (int)(reinterpret_cast<uintptr_t>(pa) & 15), qs = (int)(reinterpret_cast<uintptr_t>(qa) & 15);
  const uint32_t to = (uint32_t)__cvta_generic_to_shared(buf);
  auto fetch = [&](int c) {
    if (c < chunks) {
      const uint32_t s = to + (c % STAGES) * 2 * ROW;
#pragma unroll
      for (int i = 0; i < (UNITS + 31) / 32; ++i) {
        const int j = lane + i * 32;
        if (j < UNITS) {
          copy16(s + j * 16, pa - ps + (size_t)c * CHUNK_BYTES + j * 16);
          if (how == kLess) copy16(s + ROW + j * 16, qa - qs + (size_t)c * CHUNK_BYTES + j * 16);
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int c = 0; c < STAGES; ++c) fetch(c);
  Sum<kDeep> all;
  float2 s = make_float2(0.f, 0.f);
  const int ends = hi - lo - chunks * C;       // (at most C + 2 E)
#pragma unroll 4
  for (int t = lane; t < ends; t += 32) {
    const int y = lo + t + (t >= E ? chunks * C : 0);
    add(s, weight<how>(to_f(p[y]), how == kLess ? to_f(q[y]) : 0.f, y == skip));
  }
  all += s;
  for (int c = 0; c < chunks; ++c) {
    asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 1) : "memory");
    __syncwarp();
    const char* at = buf + (c % STAGES) * 2 * ROW;
    const T* a = reinterpret_cast<const T*>(at + ps) + lane;
    const T* b = reinterpret_cast<const T*>(at + ROW + qs) + lane;
    const int y = lo + E + c * C + lane;
    s = weight<how>(to_f(a[0]), how == kLess ? to_f(b[0]) : 0.f, y == skip);
#pragma unroll
    for (int i = 1; i < C / 32; ++i)
      add(s, weight<how>(to_f(a[i * 32]), how == kLess ? to_f(b[i * 32]) : 0.f, y + i * 32 == skip));
    all += s;
    __syncwarp();
    fetch(c + STAGES);
  }
  return all.total();
}

// The CTAs of a cluster.  Arrivals order nothing by themselves: a release would wait for every store
// in flight (1.3 to 6 thousand cycles here).
__device__ __forceinline__ int cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return (int)r;
}
__device__ __forceinline__ int cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return (int)r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }
// Eight bytes to the same place of another CTA of the cluster, counted by its barrier.
__device__ __forceinline__ void send(float2* to, uint64_t* bar, int rank, float2 v) {
  asm volatile(
      "{\n .reg .b32 a, b;\n mapa.shared::cluster.u32 a, %0, %2;\n mapa.shared::cluster.u32 b, %1, %2;\n"
      " st.async.shared::cluster.mbarrier::complete_tx::bytes.b64 [a], %3, [b];\n}"
      ::"r"(tc::smem_u32(to)), "r"(tc::smem_u32(bar)), "r"(rank), "l"(*reinterpret_cast<uint64_t*>(&v)) : "memory");
}

// One weight, in a search.
template <typename T>
__device__ __forceinline__ float2 one(const T* p, const T* q, int y, int skip, Weight how) {
  const float a = to_f(p[y]), b = how == kLess ? to_f(q[y]) : 0.f;
  return how == kLess ? weight<kLess>(a, b, false) : weight<kOthers>(a, b, how == kOthers && y == skip);
}

// The first lane whose sum (in the lanes' order, behind `before`) passes the aim, and what lies
// before it; the last lane with any weight where rounding, or a u outside [0,1), leaves none (lane 0
// if there is none).
struct Pick {
  float2 before;
  int who;
};
__device__ __noinline__ Pick pick_lane(float2 mine, float2 before, float2 aim) {
  const int lane = threadIdx.x & 31;
  float2 incl = mine;
#pragma unroll 1
  for (int o = 1; o < 32; o <<= 1) {
    const float2 t = make_float2(__shfl_up_sync(0xffffffffu, incl.x, o), __shfl_up_sync(0xffffffffu, incl.y, o));
    if (lane >= o) incl = sum(t, incl);
  }
  float2 excl = make_float2(__shfl_up_sync(0xffffffffu, incl.x, 1), __shfl_up_sync(0xffffffffu, incl.y, 1));
  if (lane == 0) excl = make_float2(0.f, 0.f);
  const unsigned over = __ballot_sync(0xffffffffu, mine.x > 0.f && more(sum(before, incl), aim));
  const unsigned some = __ballot_sync(0xffffffffu, mine.x > 0.f);
  const int who = over ? __ffs(over) - 1 : max(31 - __clz(some), 0);
  return {sum(before, shfl(excl, who)), who};
}

template <typename T, int WARPS, bool kDeep>
__global__ void __launch_bounds__(32 * WARPS, CTAS<WARPS>) draft_verify_kernel(const VerifyParams p) {
  constexpr int THREADS = 32 * WARPS;
  constexpr int EACH = MAX_CLUSTER * WARPS / 32;     // warps of a cluster to a lane
  extern __shared__ __align__(16) char stages[];     // STAGE bytes a warp
  __shared__ float2 sums[2][MAX_CLUSTER * WARPS];    // of every warp of the cluster, in order
  __shared__ float2 runs[WARPS];                     // of the picked slice
  __shared__ float2 found[2];                        // what lies before the picked warp, and the aim
  __shared__ int accepted, rejected, picked, range[2];
  __shared__ uint64_t arrived[2];                    // the sums of a pass
  const int rank = cluster_rank(), ranks = cluster_size();
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
  const int64_t workers = (int64_t)ranks * WARPS, me = (int64_t)rank * WARPS + warp;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) tc::mbar_init(&arrived[i], 1);
    tc::fence_mbar_init();
    for (int i = 0; i < 2; ++i) tc::mbar_arrive_expect_tx(&arrived[i], (uint32_t)(workers * sizeof(float2)));
  }
  __syncwarp();
  cluster_arrive();   // the barriers are there; waited for before the first sum is sent
  float final_u = 0.f;
  if (warp == 0) {
    final_u = u[p.T];
    int a = 0;
    while (a < nd) {
      // (loaded for all T drafts: nothing waits for num)
      const int i = a + lane;
      int y = -1;
      bool ok = false;
      if (i < p.T) {
        y = x[i];
        if (y >= 0 && y < p.V) {
          const double q = p.draft ? (double)to_f(draft[i * p.draft_row + y]) : 1.0;
          ok = i < nd && (double)u[i] * q < (double)to_f(target[i * p.target_row + y]);
        }
      }
      const unsigned no = ~__ballot_sync(0xffffffffu, ok);
      if (no) {
        const int f = __ffs(no) - 1;
        if (lane == f) rejected = y;
        a += f;
        break;
      }
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
  const int skip = a < nd ? rejected : -1;
  Weight how = a == nd ? kTarget : qr ? kLess : kOthers;

  const int lo = (int)(p.V * me / workers), hi = (int)(p.V * (me + 1) / workers);
  for (int pass = 0;; ++pass) {
    float2 s = how == kLess     ? sum_slice<T, kLess, kDeep>(pr, qr, lo, hi, skip, stages + warp * STAGE)
               : how == kOthers ? sum_slice<T, kOthers, kDeep>(pr, pr, lo, hi, skip, stages + warp * STAGE)
                                : sum_slice<T, kTarget, kDeep>(pr, pr, lo, hi, skip, stages + warp * STAGE);
    s = warp_sum(s);
    __syncwarp();
    if (pass == 0) cluster_wait();
    if (lane < ranks) send(&sums[pass][me], &arrived[pass], lane, s);
    if (warp == 0) {
      const bool late = (p.give_up && rank == 0) || !tc::mbar_wait(&arrived[pass], 0);
      __syncwarp();
      float2 v[EACH], all = make_float2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < EACH; ++i) {
        const int w = lane * EACH + i;
        v[i] = w < workers ? sums[pass][w] : make_float2(0.f, 0.f);
        add(all, v[i]);
      }
      const float2 total = warp_sum(all);
      int pick = kNone;
      if (__any_sync(0xffffffffu, late)) pick = kLate;
      else if (total.x == 0.f && how != kTarget) pick = kAgain;
      else if (total.x > 0.f && isfinite(total.x) && isfinite(total.y)) {
        const float ut = final_u < -1.f ? -1.f : final_u;     // (-1 draws as any below 0, but its aim is finite)
        const float hi_u = __fmul_rn(ut, total.x);
        const float2 aim = make_float2(hi_u, __fmaf_rn(ut, total.y, __fmaf_rn(ut, total.x, -hi_u)));
        const Pick lanes = pick_lane(all, make_float2(0.f, 0.f), aim);
        // the same rule over the lane's own
        int at = -1;
        float2 before = lanes.before, lower = before;
#pragma unroll
        for (int i = 0; i < EACH; ++i)
          if (v[i].x > 0.f && (at < 0 || !more(before, aim))) {
            at = lane * EACH + i;
            lower = before;
            add(before, v[i]);
          }
        pick = __shfl_sync(0xffffffffu, at, lanes.who);
        lower = shfl(lower, lanes.who);
        if (lane == 0) {
          found[0] = lower;
          found[1] = aim;
        }
      }
      if (lane == 0) picked = pick;
    }
    __syncthreads();
    if (picked == kAgain) {     // nothing is left: draw from p
      how = kTarget;
      continue;
    }
    if (picked == kNone) {
      if (rank == 0 && threadIdx.x == 0) tokens[a] = -1;
      return;
    }
    if (picked == kLate) {
      // A CTA that is behind still sends its sums here: this one outlives all that have not left (their
      // waits are bounded too, and those that have left are not waited for), and what they sent last.
      // Only then does it say so: the first CTA may not have written its number before.
      cluster_arrive();
      cluster_wait();
      for (int b = 0; b < 2; ++b)
        for (int i = 0; i < 1000 && !tc::mbar_try_wait(&arrived[b], 0); ++i) {}
      if (threadIdx.x == 0) p.count[n] = -1;
      return;
    }
    if (picked / WARPS != rank) return;
    // that slice once more, by the whole CTA: a run of neighbours to a thread, until the run with
    // the token has a lane for each
    float2 before = found[0];
    const float2 aim = found[1];
    int from = (int)(p.V * (int64_t)picked / workers), to = (int)(p.V * (int64_t)(picked + 1) / workers);
    for (;;) {
      const int per = (to - from + THREADS - 1) / THREADS;
      const int b = min(from + (int)threadIdx.x * per, to), e = min(b + per, to);
      Sum<kDeep> run;
      for (int y = b; y < e; y += 8) {
        float2 s = one(pr, qr, y, skip, how);
#pragma unroll
        for (int i = 1; i < 8; ++i)
          if (y + i < e) add(s, one(pr, qr, y + i, skip, how));
        run += s;
      }
      float2 mine = run.total();
      const float2 r = warp_sum(mine);
      if (lane == 0) runs[warp] = r;
      __syncthreads();
      const Pick warps = pick_lane(lane < WARPS ? runs[lane] : make_float2(0.f, 0.f), before, aim);
      if (warp == warps.who) {
        const Pick lanes = pick_lane(mine, warps.before, aim);
        from = __shfl_sync(0xffffffffu, b, lanes.who);
        to = __shfl_sync(0xffffffffu, e, lanes.who);
        if (per <= 32) {
          mine = from + lane < to ? one(pr, qr, from + lane, skip, how) : make_float2(0.f, 0.f);
          const Pick last = pick_lane(mine, lanes.before, aim);
          if (lane == last.who) tokens[a] = from + lane;
        } else if (lane == 0) {
          range[0] = from;
          range[1] = to;
          found[0] = lanes.before;
        }
      }
      if (per <= 32) return;
      __syncthreads();
      from = range[0];
      to = range[1];
      before = found[0];
    }
  }
}

template <typename T, int WARPS, bool kDeep>
cudaError_t go(const VerifyParams& p, cudaStream_t st) {
  // as many CTAs to a sequence as one wave holds, each with a slice worth its start
  int ranks = MAX_CLUSTER;
  const int wave = 152 * CTAS<WARPS>;
  if (ranks > wave / p.N) ranks = wave / p.N;
  if (ranks > (p.V + kSlice - 1) / kSlice) ranks = (p.V + kSlice - 1) / kSlice;
  if (ranks < 1) ranks = 1;
  auto kernel = draft_verify_kernel<T, WARPS, kDeep>;
  constexpr int bytes = WARPS * STAGE;
  if (bytes > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.N * ranks));
  cfg.blockDim = dim3(32 * WARPS);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = ranks;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}
template <typename T>
cudaError_t sized(const VerifyParams& p, cudaStream_t st) {
  return p.V > DEEP_ROW ? go<T, 16, true>(p, st) : p.V >= LONG_ROW ? go<T, 16, false>(p, st) : go<T, 8, false>(p, st);
}

}  // namespace

cudaError_t launch_draft_verify(const VerifyParams& p, bool bf16, cudaStream_t st) {
  if (p.N < 1) return cudaSuccess;
  return bf16 ? sized<__nv_bfloat16>(p, st) : sized<float>(p, st);
}

}  // namespace sfg
