// state_pool.cu -- copies, forks and compaction of the slots of a pool of states
// (include/sf_decode.h).
//
// A plan turns indices into pairs (source, destination) and the rows' new slots; the copy moves the
// slots of every cache.  The plan works on bitmaps of the slots in shared memory with a running
// count a word, so that "the r-th free slot" is a search and not a scan; its results depend on the
// order of rows and slots alone.  In small pools every CTA of the copy makes the plan for itself, in one
// launch and without a workspace's traffic; where that takes longer, where it would hold too much shared
// memory, or where the new indices go where the old ones are read, one CTA makes it in a launch before.
//
// The copies are bound by memory.  Measured: 59 slots in 8 caches of 1 MB (990 MB) 148 us, 99 % of
// the copy rate; a compaction's 48 (805 MB) 129 us, 92 %; one slot copied three times 4.7 us.  Pieces of
// 16 KB, 16 CTAs of 128 threads an SM; 8 KB 153, 133; 32 KB, 8 CTAs of 256 threads 150, 130; the last
// turn's pieces cut for the CTAs that have none 150, 130.  One launch and two, forks of slots of 64 KB: 9
// slots and 4 rows 3.8 and 6.0 us; 160 and 96 4.4, 6.3; 4096 and 64 4.8, 6.4; 300 and 150 5.9, 6.4; 4096 and 256 8.0,
// 7.9; 400 and 300 8.6, 7.5; 1000 and 400 17.0, 8.4; 4096 and 1024 32.7, 12.0 (128 threads plan for longer,
// and with 25 KB eight CTAs fit an SM, so that a second wave plans again); of 1 MB: 96 slots, 48 rows 9.4, 9.4;
// 300 and 150 29.3, 29.7; 600 and 300 55.7, 53.4; 1000 and 400 75.8, 69.2.
#include "common.cuh"
#include "decode.cuh"
#include "linattn.cuh"

namespace sfg {
namespace {

constexpr int PLAN = 1024;            // threads of the plan
constexpr int COPY = 128;
constexpr int PIECE = 1024;           // 16-byte units of a piece: 16 KB
constexpr int CACHES = 64;            // caches of a copy launch
constexpr int CTAS = 152 * 16;
constexpr int FUSED_SLOTS = 4096, FUSED_ROWS = 1024;   // of a plan in every CTA, at the most: 25 KB ...
constexpr int FAST_ROWS = 256;                         // ... and where it is faster than a launch of its own

// Exclusive prefix sums over a CTA's TH threads, and their total.
template <int TH>
__device__ __forceinline__ int block_scan(int x, int* warp_sums, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int s = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += t;
  }
  if (lane == 31) warp_sums[warp] = s;
  __syncthreads();
  if (warp == 0) {
    int w = lane < TH / 32 ? warp_sums[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += t;
    }
    if (lane < TH / 32) warp_sums[lane] = w;
  }
  __syncthreads();
  total = warp_sums[TH / 32 - 1];
  const int r = s - x + (warp ? warp_sums[warp - 1] : 0);
  __syncthreads();
  return r;
}

// before[w]: bits set in words 0 .. w - 1; returns the number of all.
template <int TH>
__device__ __forceinline__ int count_words(const uint32_t* bits, int* before, int words, int* warp_sums) {
  int base = 0;
  for (int w0 = 0; w0 < words; w0 += TH) {
    const int w = w0 + threadIdx.x;
    int total;
    const int r = block_scan<TH>(w < words ? __popc(bits[w]) : 0, warp_sums, total);
    if (w < words) before[w] = base + r;
    base += total;
  }
  __syncthreads();
  return base;
}
// The place of the r-th set bit of a word (r below their number), by halves.
__device__ __forceinline__ int nth_bit(uint32_t x, int r) {
  int at = 0;
#pragma unroll
  for (int half = 16; half >= 1; half >>= 1) {
    const int n = __popc(x & ((1u << half) - 1u));
    if (r >= n) {
      r -= n;
      x >>= half;
      at += half;
    }
  }
  return at;
}
// The slot of the r-th set bit (r below their number).
__device__ __forceinline__ int select_bit(const uint32_t* bits, const int* before, int words, int r) {
  int lo = 0, hi = words - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (before[mid] <= r) lo = mid;
    else hi = mid - 1;
  }
  return lo * 32 + nth_bit(bits[lo], r - before[lo]);
}
__device__ __forceinline__ int rank_bit(const uint32_t* bits, const int* before, int s) {
  return before[s >> 5] + __popc(bits[s >> 5] & ((1u << (s & 31)) - 1u));
}
__device__ __forceinline__ bool bit(const uint32_t* bits, int s) { return bits[s >> 5] >> (s & 31) & 1u; }
__device__ __forceinline__ void set_bit(uint32_t* bits, int s) { atomicOr(&bits[s >> 5], 1u << (s & 31)); }

// Slots that may be given out: not slot 0, not reserved.
template <int TH>
__device__ __forceinline__ void usable_bits(uint32_t* bits, const PoolPlan& p, int words) {
  for (int w = threadIdx.x >> 5; w < words; w += TH / 32) {
    const int s = w * 32 + (threadIdx.x & 31);
    const bool ok = s > 0 && s < p.num_slots && !(p.reserved && p.reserved[s]);
    const uint32_t b = __ballot_sync(0xffffffffu, ok);
    if (!(threadIdx.x & 31)) bits[w] = b;
  }
}

// The pairs to copy (p.src, p.dst) and, if `write`, the rows' new slots; returns the number of pairs.
// smem: 2 words for 32 slots (a fork), 4 (a compaction).
template <int TH>
__device__ __forceinline__ int fork_plan(const PoolPlan& p, uint32_t* smem, int* warp_sums, bool write) {
  const int words = (p.num_slots + 31) / 32;
  uint32_t* open = smem;                                    // slots to give out
  int* before = reinterpret_cast<int*>(open + words);
  for (int s = threadIdx.x; s < p.num_slots; s += TH) p.first[s] = 0x7fffffff;
  usable_bits<TH>(open, p, words);
  __syncthreads();
  // the row's present slot, kept in dst until its place is known (out may be an input)
  for (int i = threadIdx.x; i < p.M; i += TH) {
    const int a = p.parents[i];
    int s = a >= 0 && a < p.N ? p.idx[a] : -1;
    if (s <= 0 || s >= p.num_slots) s = -1;
    p.dst[i] = s;
    if (s > 0) atomicMin(&p.first[s], i);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < p.M; i += TH) {
    const int s = p.dst[i];
    if (s > 0 && p.first[s] == i && !(p.reserved && p.reserved[s])) atomicAnd(&open[s >> 5], ~(1u << (s & 31)));
  }
  __syncthreads();
  const int room = count_words<TH>(open, before, words, warp_sums);
  int base = 0;
  for (int i0 = 0; i0 < p.M; i0 += TH) {
    const int i = i0 + threadIdx.x;
    int s = -1;
    bool need = false;
    if (i < p.M) {
      s = p.dst[i];
      need = s > 0 && (p.first[s] != i || (p.reserved && p.reserved[s]));
    }
    int total;
    const int r = base + block_scan<TH>(need, warp_sums, total);    // (its barriers part reads of dst from writes)
    base += total;
    if (i < p.M) {
      int to = s;
      if (need) {
        to = r < room ? select_bit(open, before, words, r) : -1;
        if (to > 0) { p.src[r] = s; p.dst[r] = to; }
      }
      if (write) p.out[i] = to;
    }
  }
  __syncthreads();
  return min(base, room);
}

template <int TH>
__device__ __forceinline__ int compact_plan(const PoolPlan& p, uint32_t* smem, int* warp_sums, bool write) {
  const int words = (p.num_slots + 31) / 32;
  uint32_t* ok = smem;                                      // usable, then: to leave
  uint32_t* live = ok + words;                              // then: to fill
  int* before = reinterpret_cast<int*>(live + words);
  int* gaps = before + words;
  usable_bits<TH>(ok, p, words);
  for (int w = threadIdx.x; w < words; w += TH) live[w] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < p.N; i += TH) {
    const int s = p.idx[i];
    if (s > 0 && s < p.num_slots && bit(ok, s)) set_bit(live, s);
  }
  __syncthreads();
  const int L = count_words<TH>(live, gaps, words, warp_sums);
  count_words<TH>(ok, before, words, warp_sums);
  // the low slots are the first L usable ones
  for (int w = threadIdx.x; w < words; w += TH) {
    uint32_t low = ok[w];
    const int keep = min(max(L - before[w], 0), 32);
    if (keep < __popc(low)) low = keep == 0 ? 0u : low & (0xffffffffu >> (31 - nth_bit(low, keep - 1)));
    const uint32_t v = live[w];
    ok[w] = v & ~low;
    live[w] = low & ~v;
  }
  __syncthreads();
  const int moves = count_words<TH>(ok, before, words, warp_sums);
  count_words<TH>(live, gaps, words, warp_sums);
  for (int r = threadIdx.x; r < moves; r += TH) {
    p.src[r] = select_bit(ok, before, words, r);
    p.dst[r] = select_bit(live, gaps, words, r);
  }
  for (int i = threadIdx.x; i < p.N; i += TH) {
    const int s = p.idx[i];
    int to = s;
    if (s > 0 && s < p.num_slots && bit(ok, s)) to = select_bit(live, gaps, words, rank_bit(ok, before, s));
    if (write) p.out[i] = to;
  }
  __syncthreads();
  return moves;
}

__global__ void __launch_bounds__(PLAN) plan_kernel(const PoolPlan p) {
  extern __shared__ __align__(16) uint32_t smem[];
  __shared__ int warp_sums[32];
  const int n = p.parents ? fork_plan<PLAN>(p, smem, warp_sums, true) : compact_plan<PLAN>(p, smem, warp_sums, true);
  if (threadIdx.x == 0) *p.count = n;
}

struct CopyParams {
  const int32_t* src;
  const int32_t* dst;
  const int32_t* count;
  int rows, num_slots, caches;
  int pieces[CACHES + 1];             // of a slot, before cache c
  uint4* base[CACHES];
  int64_t units[CACHES];              // 16-byte units of a slot
};

// Copies of p.src[i] to p.dst[i], i < rows.
__device__ __forceinline__ void copy_rows(const CopyParams& p, const int32_t* src, const int32_t* dst, int rows) {
  const int per = p.pieces[p.caches];
  const int64_t work = (int64_t)rows * per;
  for (int64_t at = blockIdx.x; at < work; at += gridDim.x) {
    const int row = (int)(at / per), piece = (int)(at % per);
    const int s = src[row], d = dst[row];
    if (s <= 0 || d <= 0 || s >= p.num_slots || d >= p.num_slots || s == d) continue;
    int c = 0;
    while (piece >= p.pieces[c + 1]) ++c;
    const int64_t from = (int64_t)(piece - p.pieces[c]) * PIECE;
    const int64_t left = p.units[c] - from;
    const int len = left < PIECE ? (int)left : PIECE;
    const uint4* a = p.base[c] + s * p.units[c] + from;
    uint4* b = p.base[c] + d * p.units[c] + from;
    uint4 x[PIECE / COPY];
#pragma unroll
    for (int i = 0; i < PIECE / COPY; ++i) {
      const int j = threadIdx.x + i * COPY;
      if (j < len) x[i] = a[j];
    }
#pragma unroll
    for (int i = 0; i < PIECE / COPY; ++i) {
      const int j = threadIdx.x + i * COPY;
      if (j < len) b[j] = x[i];
    }
  }
}

__global__ void __launch_bounds__(COPY) copy_kernel(const __grid_constant__ CopyParams p) {
  copy_rows(p, p.src, p.dst, p.count ? min(*p.count, p.rows) : p.rows);
}

__global__ void __launch_bounds__(COPY) plan_copy_kernel(PoolPlan plan, const __grid_constant__ CopyParams p) {
  extern __shared__ __align__(16) uint32_t smem[];
  __shared__ int warp_sums[32];
  const int words = (plan.num_slots + 31) / 32;
  uint32_t* at = smem + words * (plan.parents ? 2 : 4);
  plan.src = reinterpret_cast<int32_t*>(at);
  plan.dst = plan.src + p.rows;
  plan.first = plan.dst + p.rows;
  const bool write = blockIdx.x == 0;
  const int n = plan.parents ? fork_plan<COPY>(plan, smem, warp_sums, write)
                             : compact_plan<COPY>(plan, smem, warp_sums, write);
  copy_rows(p, plan.src, plan.dst, n);
}

CopyParams copy_params(int num_slots, int num_caches, void* const* caches, const size_t* slot_bytes, int rows) {
  CopyParams p;
  p.src = p.dst = p.count = nullptr;
  p.rows = rows;
  p.num_slots = num_slots;
  p.caches = num_caches < CACHES ? num_caches : CACHES;
  p.pieces[0] = 0;
  for (int c = 0; c < p.caches; ++c) {
    p.base[c] = reinterpret_cast<uint4*>(caches[c]);
    p.units[c] = (int64_t)(slot_bytes[c] / 16);
    p.pieces[c + 1] = p.pieces[c] + (int)((p.units[c] + PIECE - 1) / PIECE);
  }
  return p;
}
int copy_grid(const CopyParams& p) {
  const int64_t work = (int64_t)p.rows * p.pieces[p.caches];
  return (int)(work < CTAS ? work : CTAS);
}
}  // namespace

cudaError_t launch_pool_copy(int num_slots, int num_caches, void* const* caches,
                             const size_t* slot_bytes, const int32_t* src, const int32_t* dst,
                             const int32_t* count, int rows, cudaStream_t st) {
  if (rows < 1) return cudaSuccess;
  for (int c = 0; c < num_caches; c += CACHES) {
    CopyParams p = copy_params(num_slots, num_caches - c, caches + c, slot_bytes + c, rows);
    p.src = src;
    p.dst = dst;
    p.count = count;
    if (p.pieces[p.caches] == 0) continue;
    copy_kernel<<<copy_grid(p), COPY, 0, st>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

bool pool_move_needs_workspace(const PoolPlan& plan, int num_caches) {
  const int rows = plan.parents ? plan.M : plan.N;
  const size_t out = (size_t)rows * 4;
  return num_caches > CACHES || plan.num_slots > FUSED_SLOTS || rows > FUSED_ROWS ||
         overlap(plan.out, out, plan.idx, (size_t)plan.N * 4) ||
         overlap(plan.out, out, plan.parents, (size_t)plan.M * 4) ||
         overlap(plan.out, out, plan.reserved, (size_t)plan.num_slots);
}

bool pool_move_likes_workspace(const PoolPlan& plan) {
  return (plan.parents ? plan.M : plan.N) > FAST_ROWS;
}

cudaError_t launch_pool_move(const PoolPlan& plan, int num_caches, void* const* caches,
                             const size_t* slot_bytes, cudaStream_t st) {
  const int words = (plan.num_slots + 31) / 32, rows = plan.parents ? plan.M : plan.N;
  const size_t bits = (size_t)words * 4 * (plan.parents ? 2 : 4), out = (size_t)rows * 4;
  if (!plan.count) {
    const CopyParams p = copy_params(plan.num_slots, num_caches, caches, slot_bytes, rows);
    const int grid = copy_grid(p);
    const size_t bytes = bits + 2 * out + (plan.parents ? (size_t)plan.num_slots * 4 : 0);
    plan_copy_kernel<<<grid > 0 ? grid : 1, COPY, bytes, st>>>(plan, p);
    return cudaGetLastError();
  }
  if (bits > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bits);
    if (e != cudaSuccess) return e;
  }
  plan_kernel<<<1, PLAN, bits, st>>>(plan);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_pool_copy(plan.num_slots, num_caches, caches, slot_bytes, plan.src, plan.dst, plan.count, rows, st);
}

}  // namespace sfg
