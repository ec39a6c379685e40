// state_pool.cu -- copies, forks and compaction of the slots of a pool of states
// (include/sf_decode.h).
//
// A plan (one CTA) turns indices into pairs (source, destination) and the rows' new slots; a copy
// kernel moves the slots of every cache.  The plan works on bitmaps of the slots in shared memory
// with a running count a word, so that "the r-th free slot" is a search and not a scan; its results
// depend on the order of rows and slots alone.  The copies are bound by memory.
#include "common.cuh"
#include "decode.cuh"
#include "linattn.cuh"

namespace sfg {
namespace {

constexpr int PLAN = 1024;            // threads of the plan
constexpr int COPY = 256;
constexpr int PIECE = 2048;           // 16-byte units of a piece: 32 KB
constexpr int CACHES = 64;            // caches of a copy launch

// Exclusive prefix sums over a CTA's threads, and their total.
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
    int w = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += t;
    }
    warp_sums[lane] = w;
  }
  __syncthreads();
  total = warp_sums[31];
  const int r = s - x + (warp ? warp_sums[warp - 1] : 0);
  __syncthreads();
  return r;
}

// before[w]: bits set in words 0 .. w - 1; returns the number of all.
__device__ int count_words(const uint32_t* bits, int* before, int words, int* warp_sums) {
  int base = 0;
  for (int w0 = 0; w0 < words; w0 += PLAN) {
    const int w = w0 + threadIdx.x;
    int total;
    const int r = block_scan(w < words ? __popc(bits[w]) : 0, warp_sums, total);
    if (w < words) before[w] = base + r;
    base += total;
  }
  __syncthreads();
  return base;
}
// The slot of the r-th set bit (r below their number).
__device__ __forceinline__ int select_bit(const uint32_t* bits, const int* before, int words, int r) {
  int lo = 0, hi = words - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (before[mid] <= r) lo = mid;
    else hi = mid - 1;
  }
  return lo * 32 + (int)__fns(bits[lo], 0, r - before[lo] + 1);
}
__device__ __forceinline__ int rank_bit(const uint32_t* bits, const int* before, int s) {
  return before[s >> 5] + __popc(bits[s >> 5] & ((1u << (s & 31)) - 1u));
}
__device__ __forceinline__ bool bit(const uint32_t* bits, int s) { return bits[s >> 5] >> (s & 31) & 1u; }
__device__ __forceinline__ void set_bit(uint32_t* bits, int s) { atomicOr(&bits[s >> 5], 1u << (s & 31)); }

// Slots that may be given out: not slot 0, not reserved.
__device__ __forceinline__ void usable_bits(uint32_t* bits, const PoolPlan& p, int words) {
  for (int w = threadIdx.x >> 5; w < words; w += PLAN / 32) {
    const int s = w * 32 + (threadIdx.x & 31);
    const bool ok = s > 0 && s < p.num_slots && !(p.reserved && p.reserved[s]);
    const uint32_t b = __ballot_sync(0xffffffffu, ok);
    if (!(threadIdx.x & 31)) bits[w] = b;
  }
}

__global__ void __launch_bounds__(PLAN) fork_plan_kernel(const PoolPlan p) {
  extern __shared__ __align__(16) uint32_t smem[];
  __shared__ int warp_sums[32];
  const int words = (p.num_slots + 31) / 32;
  uint32_t* open = smem;                                    // slots to give out
  int* before = reinterpret_cast<int*>(open + words);
  for (int s = threadIdx.x; s < p.num_slots; s += PLAN) p.first[s] = 0x7fffffff;
  usable_bits(open, p, words);
  __syncthreads();
  // the row's present slot, kept in dst until its place is known (out may be an input)
  for (int i = threadIdx.x; i < p.M; i += PLAN) {
    const int a = p.parents[i];
    int s = a >= 0 && a < p.N ? p.idx[a] : -1;
    if (s <= 0 || s >= p.num_slots) s = -1;
    p.dst[i] = s;
    if (s > 0) atomicMin(&p.first[s], i);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < p.M; i += PLAN) {
    const int s = p.dst[i];
    if (s > 0 && p.first[s] == i && !(p.reserved && p.reserved[s])) atomicAnd(&open[s >> 5], ~(1u << (s & 31)));
  }
  __syncthreads();
  const int room = count_words(open, before, words, warp_sums);
  int base = 0;
  for (int i0 = 0; i0 < p.M; i0 += PLAN) {
    const int i = i0 + threadIdx.x;
    int s = -1;
    bool need = false;
    if (i < p.M) {
      s = p.dst[i];
      need = s > 0 && (p.first[s] != i || (p.reserved && p.reserved[s]));
    }
    int total;
    const int r = base + block_scan(need, warp_sums, total);    // (its barriers part reads of dst from writes)
    base += total;
    if (i < p.M) {
      int to = s;
      if (need) {
        to = r < room ? select_bit(open, before, words, r) : -1;
        if (to > 0) { p.src[r] = s; p.dst[r] = to; }
      }
      p.out[i] = to;
    }
  }
  if (threadIdx.x == 0) *p.count = min(base, room);
}

__global__ void __launch_bounds__(PLAN) compact_plan_kernel(const PoolPlan p) {
  extern __shared__ __align__(16) uint32_t smem[];
  __shared__ int warp_sums[32];
  const int words = (p.num_slots + 31) / 32;
  uint32_t* ok = smem;                                      // usable, then: to leave
  uint32_t* live = ok + words;                              // then: to fill
  int* before = reinterpret_cast<int*>(live + words);
  int* gaps = before + words;
  usable_bits(ok, p, words);
  for (int w = threadIdx.x; w < words; w += PLAN) live[w] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < p.N; i += PLAN) {
    const int s = p.idx[i];
    if (s > 0 && s < p.num_slots && bit(ok, s)) set_bit(live, s);
  }
  __syncthreads();
  const int L = count_words(live, gaps, words, warp_sums);
  count_words(ok, before, words, warp_sums);
  // the low slots are the first L usable ones
  for (int w = threadIdx.x; w < words; w += PLAN) {
    uint32_t low = ok[w];
    const int keep = min(max(L - before[w], 0), 32);
    if (keep < __popc(low)) low = keep == 0 ? 0u : low & (0xffffffffu >> (31 - __fns(low, 0, keep)));
    const uint32_t v = live[w];
    ok[w] = v & ~low;
    live[w] = low & ~v;
  }
  __syncthreads();
  const int moves = count_words(ok, before, words, warp_sums);
  count_words(live, gaps, words, warp_sums);
  for (int r = threadIdx.x; r < moves; r += PLAN) {
    p.src[r] = select_bit(ok, before, words, r);
    p.dst[r] = select_bit(live, gaps, words, r);
  }
  for (int i = threadIdx.x; i < p.N; i += PLAN) {
    const int s = p.idx[i];
    int to = s;
    if (s > 0 && s < p.num_slots && bit(ok, s)) to = select_bit(live, gaps, words, rank_bit(ok, before, s));
    p.out[i] = to;
  }
  if (threadIdx.x == 0) *p.count = moves;
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

__global__ void __launch_bounds__(COPY) pool_copy_kernel(const __grid_constant__ CopyParams p) {
  const int rows = p.count ? min(*p.count, p.rows) : p.rows;
  const int per = p.pieces[p.caches];
  const int64_t work = (int64_t)rows * per;
  for (int64_t at = blockIdx.x; at < work; at += gridDim.x) {
    const int row = (int)(at / per), piece = (int)(at % per);
    const int s = p.src[row], d = p.dst[row];
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

}  // namespace

cudaError_t launch_pool_plan(const PoolPlan& p, cudaStream_t st) {
  const int words = (p.num_slots + 31) / 32;
  const size_t bytes = (size_t)words * 4 * (p.parents ? 2 : 4);
  auto kernel = p.parents ? fork_plan_kernel : compact_plan_kernel;
  if (bytes > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != cudaSuccess) return e;
  }
  kernel<<<1, PLAN, bytes, st>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_pool_copy(int num_slots, int num_caches, void* const* caches,
                             const size_t* slot_bytes, const int32_t* src, const int32_t* dst,
                             const int32_t* count, int rows, cudaStream_t st) {
  if (rows < 1) return cudaSuccess;
  for (int c0 = 0; c0 < num_caches; c0 += CACHES) {
    CopyParams p{};
    p.src = src;
    p.dst = dst;
    p.count = count;
    p.rows = rows;
    p.num_slots = num_slots;
    p.caches = num_caches - c0 < CACHES ? num_caches - c0 : CACHES;
    for (int c = 0; c < p.caches; ++c) {
      p.base[c] = reinterpret_cast<uint4*>(caches[c0 + c]);
      p.units[c] = (int64_t)(slot_bytes[c0 + c] / 16);
      p.pieces[c + 1] = p.pieces[c] + (int)((p.units[c] + PIECE - 1) / PIECE);
    }
    if (p.pieces[p.caches] == 0) continue;
    const int64_t work = (int64_t)rows * p.pieces[p.caches];
    const int grid = (int)(work < 152 * 8 ? work : 152 * 8);
    pool_copy_kernel<<<grid, COPY, 0, st>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace sfg
