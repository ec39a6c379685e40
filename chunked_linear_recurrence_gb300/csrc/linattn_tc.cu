// linattn_tc.cu -- the decayed linear attention's product (linattn.cuh) on tcgen05: BF16 tokens,
// head sizes D = 128 and 64.
//
// One CTA walks one (segment, head) in 64-row chunks.  Rows r, s of a chunk, the state S [z][y]:
//     QK  = [Y; X] Y^T           M = 128, N = 64, K = D     (rows 64-127: X Y^T)
//     P   = a QK o lam^|r-s|     BF16, by two warps, to shared memory
//     E   = (lam^f c Z)^T Y      M = 128, N = D,  K = 64    three times (below)
//     O1^T = S X^T               M = 128, N = 64, K = D     (S as BF16 in TMEM)
//     O2^T = Z^T P^T             M = 128, N = 64, K = 64
//     out = b lam^e O1 + O2,     S <- lam^L S + E           (FP32)
// Everything is laid out as the TMA brings it: [rows][D] BF16 tiles of swizzled 64-column panels,
// read K-major or MN-major as each product needs.  (At D = 64 the products' M = 128 is half
// empty; the warps of the empty lanes have no work.)
//
// The state stays in the registers of eight warps (D / 2 floats a thread), not in TMEM: every
// chunk's E is a product of its own, so E of the next chunks never waits for S, no FP32 state
// is read and written back around the products, and the sum over the chunks is rounded in
// FP32 to nearest.  E's left operand is exact enough to keep FP32 accuracy of the state: the
// weighted rows are split into three BF16 summands (8 bits each, 24 together) in TMEM, each
// multiplied with the exact Y.  A launch that returns no state takes two of them (16 bits): its
// state only ever reaches BF16 results.  (The parts as an MN-major operand in shared memory
// needed 48 KB of stores and loads a chunk more: slower.)
//
// Roundings to BF16: S before O1 and P before O2, where the results are BF16 themselves.  Their
// error against FP64 is 2.35e-3 (2-norm) with them, 1.66e-3, the result's own rounding, without;
// both in two parts, 16 bits, took 223 us for 167 (backward of 2 x 8192 tokens of 16 heads) and 500
// for 378 (65536 packed tokens of 32 heads), measured with the work alone.  P keeps 16 bits in walks
// of one chunk, whose results may come from one or two elements.
//
// Twenty warps: 0 loads (four stages) and issues E, in two halves of 32 rows so that the split
// refills one under the other; 1 issues QK, O1 and O2; 2-3 form P; 4-11 hold the state (two
// warpgroups: columns y of either half); 12-15 split the weighted rows; 16-19 write the
// results, turned in shared memory into 16-byte stores.  A batch of products costs ~170 cycles
// beyond its products' own time, so O1 and O2 go together, and the next chunk's QK goes while the
// last results are read.  A launch that computes pieces' states alone has E only: warp 1 loads,
// two buffers of E and of the parts, and warps 16-19 split every other chunk.
// Products are issued behind elect.sync in warp-uniform code (a lane test costs 62 cycles a
// product instead of 32-64), and the loops are kept from unrolling: the roles run at the speed
// of instruction fetch.  Register shares of the five warpgroups: 56, 128, 128, 72, 96.
//
// Warps meet through mbarriers alone; every wait is bounded, and a thread that gives up writes
// SF_ERR_TIMEOUT to the status word and raises the CTA's abort flag; copies and products in
// flight land before the CTA leaves.
//
// Bound by the chain of roles that a chunk passes through, not by one unit: at D = 128 the tensor
// pipe is active 54 % of a CTA's time (1410 of ~2500 cycles a chunk; QK 8 products, E 12, O1 8, O2
// 4, four batches' starts between them), and the same backward takes 190-194 us for 167 with
// the products of O1 and O2, those of QK or P's work done twice, 218 with the state's copy (where
// it spills).  At D = 64 the pipe is active 39 %.  With a CTA on every SM and no state to wait for
// memory is near: 131072 tokens of 4 heads read and write 5.9 TB/s in the walks, 5.5 in the pieces'
// states.  Measured, D = 128: 96 walks of 128 chunks 167 us (3.6 TB/s on 96 SMs), 256 walks of 32
// chunks 110 us (5.2 TB/s), 4 x 4096 tokens of 16 heads 19 us of pieces' states and 50 us, one
// prompt of 130 tokens 9 us; a chunk takes 1.2 us (0.58 us of a piece's states) with few CTAs, 1.5
// (0.88) with one on every SM.  D = 64: 96 walks of 128 chunks 131 us.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <type_traits>

#include "common.cuh"
#include "f32x2.cuh"
#include "linattn.cuh"
#include "tc_ptx.cuh"
#include "tmap.cuh"

namespace sfg {
namespace {

using namespace tc;

constexpr int C = LA_CHUNK, NT = 640, NS = 4;
constexpr uint32_t PANEL = 8192;                 // 64 rows x 128 bytes
constexpr int PQ_LD = 136;
// Shared memory for head size D (one or two panels a tile).
template <int D>
struct Mem {
  static constexpr uint32_t NP = D / 64;
  static constexpr uint32_t Y = 0, X = PANEL;      // panel 0 of Y and X; panel 1 two panels on
  static constexpr uint32_t Z = 2 * NP * PANEL, STAGE = 3 * NP * PANEL;
  static constexpr uint32_t P = NS * STAGE;        // P [64][64], two buffers
  static constexpr uint32_t OUT = P + 2 * PANEL;   // results, [32 rows][32 columns] of each of four warps
  // b lam^e and c lam^f of a full chunk and of the walk's last one [64] each, carry [6] (padded to 16), the
  // weights of P by 64 + s - r in four copies, each a word further on, 8 banks apart
  static constexpr uint32_t TAB = OUT + 8192;
  static constexpr uint32_t BAR = TAB + 3328;
  static constexpr uint32_t SIZE = BAR + 320 + 1024;
};
static_assert(Mem<128>::SIZE <= 232448, "shared memory");
static_assert(256 * 4 + 64 + 4 * PQ_LD * 4 <= 3328 && Mem<128>::BAR % 256 == 0 && Mem<64>::BAR % 256 == 0,
              "tables");

// TMEM columns: E, the state's BF16 copy, QK, O1, O2, the weighted rows' parts (32 columns
// each); a launch that computes states alone has two buffers of E and of the parts.
constexpr uint32_t TM_E = 0, TM_SB = 128, TM_P = 192, TM_O1 = 256, TM_O2 = 320;
template <bool kState>
__device__ __forceinline__ uint32_t tm_w(int buf) { return kState ? 256 + 96 * buf : 384; }

constexpr uint32_t ID_QK = idesc_bf16(128, 64, false, false);
constexpr uint32_t ID_O1 = idesc_bf16(128, 64, false, false);   // A in TMEM
constexpr uint32_t ID_O2 = idesc_bf16(128, 64, true, false);

enum { FULL = 0, LANDED = FULL + NS, FREE = LANDED + 1, QKDONE = FREE + NS, PREADY,
       PFREE = PREADY + 2, SPLIT, EHALF = SPLIT + 4, EDONE = EHALF + 2, EFREE = EDONE + 2,
       O1DONE = EFREE + 2, ODONE, OFREE, GO, TBL, DRAIN, NBAR = DRAIN + 2 };
static_assert(8 * NBAR + 40 <= 320 && NBAR <= 32, "barriers");

// Tries of a wait before it gives up: each may suspend the thread for up to 20 us (at the least
// it takes the ~50 ns of the instruction), so between 50 ms and 20 s, where a wait that ends takes
// microseconds.  (A count and not a clock: the waits are inlined into every role's loop, and
// the loops run at the speed of instruction fetch.  It lies in shared memory, TRIES words behind
// the abort flag, so that a test can shorten it.)
constexpr int WAIT_TRIES = 1000000, TRIES = 8;

struct Maps {
  CUtensorMap m[3][3];   // x, y, z of each pass
};

// False when the wait gave up, or another thread of the CTA did (`abort`: where, once).
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile uint32_t* abort) {
  if (mbar_try_wait(bar, parity)) return true;
  int i = 0;
#pragma unroll 1
  do {
    if (mbar_try_wait_sleep(bar, parity, 20000u)) return true;
    if (*abort) return false;
  } while (++i < (int)abort[TRIES]);
  *abort = 0x40000000u | ((threadIdx.x >> 5) << 6) | ((smem_u32(bar) & 255u) >> 3);
  return false;
}
// The lanes of a warp wait together and agree on the outcome.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile uint32_t* cx) {
  return __all_sync(0xffffffffu, wait_bar(bar, parity, cx));
}
__device__ __forceinline__ void warp_arrive(uint64_t* bar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

__device__ __forceinline__ uint64_t kstep_k(int kk) {   // panels 16 KB apart
  return (uint64_t)(((uint32_t)(kk >> 2) * 2 * PANEL + (uint32_t)(kk & 3) * 32u) >> 4);
}
__device__ __forceinline__ uint64_t kstep_mn(int kk) { return (uint64_t)(kk * 2048 >> 4); }

template <int D, bool kState, int NSP>
__global__ void __launch_bounds__(NT, 1) la_tc_kernel(const __grid_constant__ Maps maps,
                                                      const LaParams p) {
  using M = Mem<D>;
  constexpr int NP = D / 64, KD = D / 16, WL = D / 32;   // panels, K steps over D, warps of D lanes
  constexpr uint32_t ID_E = idesc_bf16(128, D, false, true);   // A in TMEM
  extern __shared__ __align__(1024) uint8_t raw[];
  uint8_t* sm = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  const uint32_t sb = smem_u32(sm);
  float* rd = reinterpret_cast<float*>(sm + M::TAB);   // [2][64]
  float* wr = rd + 128;                               // [2][64]
  float* carry = rd + 256;
  float* pq = rd + 272;                               // [4][PQ_LD]
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + M::BAR);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(sm + M::BAR + 8 * NBAR);
  volatile uint32_t* cx = reinterpret_cast<uint32_t*>(sm + M::BAR + 8 * NBAR + 4);
  launch_next();
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;

  int pi, h, u;
  la_place(blockIdx.x, p, pi, h, u);
  const LaPass& q = p.pass[pi];
  const bool rev = q.reverse != 0;
  constexpr int NE = kState ? 2 : 1;              // buffers of E and of the weighted rows
  // The unit, found by one warp: whether there is one (2: padding of the paged pool), its rows
  // [s0, s1), its sequence, its place, whether the walk ends with it, whether it is cut.
  int* unit = reinterpret_cast<int*>(sm + M::BAR + 8 * NBAR + 8);
  if (warp == 0) {
    LaUnit t;
    int code = la_locate<kState>(u, p, t);
    if (code) {
      bool skip;
      la_entry(p, q, t.n, h, D, skip);
      if (skip) code = 2;
      const int first = (int)(rev ? t.eos - t.off - t.rows : t.bos + t.off);
      if (lane == 0) {
        unit[1] = first;
        unit[2] = first + (int)t.rows;
        unit[3] = t.n;
        unit[4] = t.at;
        unit[5] = t.last;
        unit[6] = p.seg < p.T && !(t.last && t.off == 0);
      }
    }
    if (lane == 0) unit[0] = code, *cx = 0, cx[TRIES] = p.tries > 0 ? p.tries : WAIT_TRIES;
    if (lane < NBAR) {
      const int i = lane;
      mbar_init(&bars[i], i >= PREADY && i <= PFREE ? 2 : (i >= SPLIT && i < SPLIT + 4) || i == OFREE ? WL
                          : i == GO || i == EFREE || i == EFREE + 1 ? 2 * WL : i >= FREE && i < FREE + NS && !kState ? 2 : 1);
    }
    fence_mbar_init();
    fence_proxy_async_smem();
    __syncwarp();
  }
  auto pw = [&](int e) { return e <= 0 ? 1.f : expf(p.decay[h] * (float)e); };
  if (warp != 0) {                                // what does not depend on the unit
    if (warp == 1) tmem_alloc(tslot, 512);
    if (tid >= 128 && tid < 256) {
      const int j = tid - 128;
      if (j < C) {
        rd[j] = q.b * pw(rev ? C - 1 - j : j + 1);
        wr[j] = q.c * pw(rev ? j + 1 : C - 1 - j);
      }
      const int gap = rev ? j - 64 : 64 - j;          // |r - s| where s may contribute to r
      const float f = gap >= 0 ? q.a * pw(gap) : 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) pq[k * PQ_LD + j + k] = f;
    }
    if (!kState && tid >= 256)   // P on the far side of the diagonal stays zero
#pragma unroll 1
      for (int i = tid - 256; i < 2 * (int)PANEL / 16; i += NT - 256)
        *reinterpret_cast<uint4*>(sm + M::P + 16 * i) = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();                              // warp 0: once the first chunk is on its way
  }
  // (the shuffles tell the compiler that these are the same in every lane: they stay out of the
  // roles' registers)
  const int s0 = __shfl_sync(0xffffffffu, unit[1], 0), s1 = __shfl_sync(0xffffffffu, unit[2], 0);
  const int nc = (s1 - s0 + C - 1) / C;
  const int tail = s1 - s0 - (nc - 1) * C;        // rows of the walk's last chunk
  const int hx = la_head(h, q.hx, p), hy = la_head(h, q.hy, p), hz = la_head(h, q.hz, p);
  int issued = 0;
  auto load = [&](int c) {
    const int b = c % NS, L = c + 1 == nc ? tail : C;
    const int r0 = rev ? s1 - c * C - L : s0 + c * C;
    uint8_t* st = sm + b * M::STAGE;
    uint64_t* bar = L < C ? &bars[LANDED] : &bars[FULL + b];   // (the last chunk only)
    if (elect_one()) {
      mbar_arrive_expect_tx(bar, (kState ? 2 : 3) * NP * PANEL);
#pragma unroll
      for (int pp = 0; pp < NP; ++pp) {
        tma_load_3d(st + M::Y + 2 * pp * PANEL, &maps.m[pi][1], bar, 64 * pp, hy, r0);
        tma_load_3d(st + M::Z + pp * PANEL, &maps.m[pi][2], bar, 64 * pp, hz, r0);
        if (!kState) tma_load_3d(st + M::X + 2 * pp * PANEL, &maps.m[pi][0], bar, 64 * pp, hx, r0);
      }
    }
    __syncwarp();
    issued = c + 1;
  };
  auto land = [&]() {   // the copies in flight, when a wait has failed
#pragma unroll 1
    for (int c = issued > NS ? issued - NS : 0; c < issued; ++c) {
      if (c + 1 == nc && tail < C) mbar_wait(&bars[LANDED], 0, 100000000ull);
      else mbar_wait(&bars[FULL + c % NS], (c / NS) & 1, 100000000ull);
    }
  };
  if (warp == 0) {
    if (unit[0] == 1 && nc > 0) load(0);
    __syncthreads();
  }
  tc_fence_after();
  const uint32_t tm = *tslot;
  if (unit[0] != 1) {
    if (warp == 1) {
      tmem_relinquish();
      tmem_dealloc(tm, 512);
    }
    if (!kState && p.seg < p.T) launch_wait();
    if (kState || unit[0] == 0) return;
    uint4* o = reinterpret_cast<uint4*>(q.out);   // padding: zero rows
#pragma unroll 1
    for (int i = tid; i < (s1 - s0) * (D / 8); i += NT)
      o[((size_t)(s0 + i / (D / 8)) * p.H + h) * (D / 8) + i % (D / 8)] = make_uint4(0, 0, 0, 0);
    return;
  }
  if (tid >= 512 && tid < 576) {                  // the last chunk's weights
    const int i = tid - 512;
    rd[64 + i] = i < tail ? q.b * pw(rev ? tail - 1 - i : i + 1) : 0.f;
    wr[64 + i] = i < tail ? q.c * pw(rev ? i + 1 : tail - 1 - i) : 0.f;
  }
  __syncthreads();

  // ------------------------------------------------------------------ weighted rows in BF16 parts
  // (four warps; chunks first, first + step, ..)
  auto split_rows = [&](int first, int step) {
    // Each warp weights and splits the 32 columns z of its TMEM lanes: 16 at a time, transposed
    // on the way from shared memory (8 x 8 tiles), the rows j along the TMEM columns.
    const uint32_t tl = tm + ((uint32_t)((warp & 3) * 32) << 16);
    const int m = lane >> 3, i = lane & 7;
    // lane's source row of K step 0: j = 8 (m / 2) + i, columns z0 + 8 (m % 2) ..; z0 of either
    // half differs in bit 1 of the 16-byte chunk
    const uint32_t ch = (uint32_t)(4 * (warp & 1) + (m & 1));
    const uint32_t src = sb + M::Z + (uint32_t)((warp & 3) >> 1) * PANEL + (uint32_t)(8 * (m >> 1) + i) * 128u;
    const uint32_t c0 = (ch ^ (uint32_t)i) << 4, c1 = ((ch + 2) ^ (uint32_t)i) << 4;
#pragma unroll 1
    for (int c = first; c < nc; c += step) {
      const int b = c % NS, eb = c % NE;
      if (!warp_wait(&bars[FULL + b], (c / NS) & 1, cx)) break;
      const float2* wt = reinterpret_cast<const float2*>(wr + (c + 1 == nc ? 64 : 0)) + (lane & 3);
      uint32_t from = src + b * M::STAGE, to = tl + tm_w<kState>(eb);
      bool ok = true;
#pragma unroll 1
      for (int hf = 0; hf < 2; ++hf) {
        // the products of the chunk that had this half of the buffer are done
        if (c >= NE && !(ok = warp_wait(&bars[(hf ? EDONE : EHALF) + eb], ((c / NE) & 1) ^ 1, cx))) break;
        tc_fence_after();
#pragma unroll 1
        for (int kk = 0; kk < 2; ++kk) {
          // 16 rows: 2 (lane % 4), + 1 and 8 more
          const float2 wv[2] = {wt[0], wt[4]};
#pragma unroll
          for (int hz = 0; hz < 2; ++hz) {
            uint32_t v[4], o[NSP][4];
            ldmatrix_x4_trans(from + (hz ? c1 : c0), v);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float2 x = mul2(unpack2(v[e]), wv[e >> 1]);
#pragma unroll
              for (int sp = 0; sp < NSP; ++sp) {
                o[sp][e] = pack2(x);
                if (sp + 1 < NSP) x = sub2(x, unpack2(o[sp][e]));
              }
            }
#pragma unroll
            for (int sp = 0; sp < NSP; ++sp)
              tmem_st_16x8(to + ((uint32_t)(16 * hz) << 16) + 32 * sp, o[sp][0], o[sp][1], o[sp][2],
                           o[sp][3]);
          }
          wt += 8;
          from += 2048;
          to += 8;
        }
        tmem_st_wait();
        tc_fence_before();
        warp_arrive(&bars[SPLIT + 2 * eb + hf], lane);
      }
      if (!ok) break;
    }
  };

  if (warp < 4) {
    reg_dealloc<56>();
    if (warp == 0) {
      // -------------------------------------------------------------- loader, issuer of E
      // A short last chunk: rows past the end (other tokens, or NaN padding) must not reach the
      // products.
      auto trim = [&]() {
        const int b = (nc - 1) % NS;
        if (!warp_wait(&bars[LANDED], 0, cx)) return false;
        uint8_t* st = sm + b * M::STAGE;
#pragma unroll 1
        for (int at = tail * 128 + lane * 16; at < (int)PANEL; at += 512)
#pragma unroll
          for (int pp = 0; pp < NP; ++pp) {
            *reinterpret_cast<uint4*>(st + M::Y + 2 * pp * PANEL + at) = make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4*>(st + M::Z + pp * PANEL + at) = make_uint4(0, 0, 0, 0);
          }
        fence_proxy_async_smem();
        warp_arrive(&bars[FULL + b], lane);
        return true;
      };
#pragma unroll 1
      for (int c = 1; !kState && c < NS && c < nc; ++c) load(c);
      bool ok = kState || nc != 1 || tail == C || trim();
#pragma unroll 1
      for (int c = 0; c < nc && ok; ++c) {
        const int b = c % NS;
        const int eb = c % NE, ph = (c / NE) & 1;
        const uint64_t dy = sdesc_sw128(sb + b * M::STAGE + M::Y, 2 * PANEL, 1024);
        if (c >= NE && !(ok = warp_wait(&bars[EFREE + eb], ph ^ 1, cx))) break;
        // E in two halves of 32 rows: the split warps refill the first under the second.  (They
        // have waited for the rows themselves.)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          if (!(ok = warp_wait(&bars[SPLIT + 2 * eb + hf], ph, cx))) break;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int sp = 0; sp < NSP; ++sp)
#pragma unroll
              for (int kk = 2 * hf; kk < 2 * hf + 2; ++kk)
                mma_bf16_ta(tm + TM_E + 128 * eb, tm + tm_w<kState>(eb) + 32 * sp + 8 * kk,
                            dy + kstep_mn(kk), ID_E, kk + sp > 0);
            mma_commit(&bars[(hf ? EDONE : EHALF) + eb]);
            if (hf) mma_commit(&bars[FREE + b]);
          }
          __syncwarp();
        }
        if (!ok) break;
        if (!kState && c + 2 == nc && tail < C && !(ok = trim())) break;
        if (!kState && c > 0 && c + NS - 1 < nc) {
          if (!(ok = warp_wait(&bars[FREE + (c - 1) % NS], ((c - 1) / NS) & 1, cx))) break;
          load(c + NS - 1);
        }
      }
      if (!kState && !ok) land();
      if (elect_one()) mma_commit(&bars[DRAIN]);
      mbar_wait(&bars[DRAIN], 0, 100000000ull);
      __syncwarp();
    } else if (warp == 1) {
      // -------------------------------------------------------------- issuer of QK, O1, O2
      // (the whole warp waits; one elected lane issues).  A batch of products costs ~170 cycles
      // beyond its products' own time, so O1 and O2 go together.  The next chunk's QK goes
      // first, while the results of the last chunk are being read, if its rows are there (P takes
      // as long as the rest of a step), else in its own turn.
      int qn = 0;                                      // chunks whose QK is issued
      auto put_qk = [&]() {                            // by the elected lane
        const uint64_t dy = sdesc_sw128(sb + (qn % NS) * M::STAGE + M::Y, 0, 1024);
#pragma unroll
        for (int kk = 0; kk < KD; ++kk)
          mma_bf16(tm + TM_P, dy + kstep_k(kk), dy + kstep_k(kk), ID_QK, kk > 0);
        mma_commit(&bars[QKDONE]);
      };
      bool ok = true;
      if (kState) {                                    // the loader, where E is the only product
        issued = 1;                                    // (by warp 0)
#pragma unroll 1
        for (int c = 1; c < nc; ++c) {
          if (c >= NS && !(ok = warp_wait(&bars[FREE + c % NS], ((c - NS) / NS) & 1, cx))) break;
          load(c);
        }
        land();                                        // also where other warps give up on them
      }
#pragma unroll 1
      for (int c = 0; !kState && c < nc && ok; ++c) {
        const int b = c % NS;
        const uint32_t st = sb + b * M::STAGE;
        if (qn == c) {                                 // its own turn
          if (!(ok = warp_wait(&bars[FULL + b], (c / NS) & 1, cx))) break;
          tc_fence_after();
          if (elect_one()) put_qk();
          __syncwarp();
          ++qn;
        }
        if (qn < nc) {
          if (!(ok = warp_wait(&bars[PFREE], c & 1, cx))) break;   // P of this chunk has been read
          if (__all_sync(0xffffffffu, mbar_test(&bars[FULL + qn % NS], (qn / NS) & 1))) {
            tc_fence_after();
            if (elect_one()) put_qk();
            __syncwarp();
            ++qn;
          }
        }
        if (!(ok = warp_wait(&bars[GO], c & 1, cx))) break;
        if (!(ok = warp_wait(&bars[PREADY + (c & 1)], (c >> 1) & 1, cx))) break;
        if (c > 0 && !(ok = warp_wait(&bars[OFREE], (c - 1) & 1, cx))) break;   // the last to come
        tc_fence_after();
        const uint64_t dx = sdesc_sw128(st + M::X, 0, 1024);
        const uint64_t dz = sdesc_sw128(st + M::Z, PANEL, 1024);
        const uint64_t dp = sdesc_sw128(sb + M::P + (c & 1) * PANEL, 0, 1024);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < KD; ++kk)
            mma_bf16_ta(tm + TM_O1, tm + TM_SB + kk * 8, dx + kstep_k(kk), ID_O1, kk > 0);
          mma_commit(&bars[O1DONE]);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_bf16(tm + TM_O2, dz + kstep_mn(kk), dp + (uint64_t)(kk * 2), ID_O2, kk > 0);
          if (__builtin_expect(nc == 1, 0))
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_bf16(tm + TM_O2, dz + kstep_mn(kk), dp + (uint64_t)((PANEL >> 4) + kk * 2), ID_O2, true);
          mma_commit(&bars[ODONE]);
          mma_commit(&bars[FREE + b]);
        }
        __syncwarp();
      }
      if (elect_one()) mma_commit(&bars[DRAIN + 1]);
      mbar_wait(&bars[DRAIN + 1], 0, 100000000ull);
      __syncwarp();
    } else {
      // -------------------------------------------------------------- P
      if (!kState) {
        // row r of P.  A walk of one chunk has its rounding's rest in the second buffer: there a
        // result may come from one or two elements, whose rounding to BF16 would show as much as
        // the result's own.  The half on the far side of the diagonal (32 columns of one warp) is
        // never touched: it stays zero.
        const int r = (warp - 2) * 32 + lane;          // TMEM lane 64 + r
        // a lam^|r-s|, or 0, at f[s] (the copy in which that is 16-byte aligned)
        const float* f = pq + (r & 3) * (PQ_LD + 1) + 64 - r;
        const uint32_t tl = tm + TM_P + ((uint32_t)(warp * 32) << 16);
        const int s0 = rev && warp == 3 ? 32 : 0, s1 = !rev && warp == 2 ? 32 : 64;
        auto weigh = [&](int s, uint8_t* row, bool last, auto rest) {   // 16 columns
          float x[16];
          tmem_ld16(tl + s, x);
          float4 g[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) g[e] = *reinterpret_cast<const float4*>(f + s + 4 * e);
          tmem_ld_wait();
          if (last) {
            tc_fence_before();
            warp_arrive(&bars[PFREE], lane);
          }
#pragma unroll
          for (int ch = 0; ch < 2; ++ch) {
            uint32_t v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float4 w = g[2 * ch + (e >> 1)];
              const float2 t = mul2(make_float2(x[8 * ch + 2 * e], x[8 * ch + 2 * e + 1]),
                                    e & 1 ? make_float2(w.z, w.w) : make_float2(w.x, w.y));
              v[e] = pack2(t);
              if (rest.value) v[e] = pack2(sub2(t, unpack2(v[e])));
            }
            *reinterpret_cast<uint4*>(row + ((((s >> 3) + ch) ^ (r & 7)) << 4)) =
                make_uint4(v[0], v[1], v[2], v[3]);
          }
        };
#pragma unroll 1
        for (int c = 0; c < nc; ++c) {
          if (!warp_wait(&bars[QKDONE], c & 1, cx)) break;
          tc_fence_after();
          uint8_t* row = sm + M::P + (c & 1) * PANEL + r * 128;
#pragma unroll 1
          for (int s = s0; s < s1; s += 16) weigh(s, row, s + 16 >= s1, std::false_type());
          if (__builtin_expect(nc == 1, 0))
#pragma unroll 1
            for (int s = s0; s < s1; s += 16) weigh(s, row + PANEL, false, std::true_type());
          fence_proxy_async_smem();
          warp_arrive(&bars[PREADY + (c & 1)], lane);
        }
      }
    }
  } else if (warp < 12) {
    reg_alloc<128>();
    if ((warp & 3) < WL) {                              // (the others have no lanes)
    // ---------------------------------------------------------------- state
    const int wg = (warp - 4) >> 2;
    const int z = ((warp & 3) << 5) + lane;
    const uint32_t tl = tm + ((uint32_t)((warp & 3) * 32) << 16);
    if (!kState && unit[6]) launch_wait();              // the entry states
    float2 s[D / 4];                                    // columns D / 2 wg + 2 e, + 1 of row z
    {
      bool skip;
      const bool split = unit[6];
      const float* src = kState ? nullptr : split ? q.entry + ((size_t)unit[4] * p.H + h) * D * D
                                         : la_entry(p, q, unit[3], h, D, skip);
      if (!src) {
#pragma unroll
        for (int e = 0; e < D / 4; ++e) s[e] = make_float2(0.f, 0.f);
      } else if (split) {
        const float4* v = reinterpret_cast<const float4*>(src) + D / 8 * wg * D + z;
#pragma unroll
        for (int e = 0; e < D / 8; ++e) {
          const float4 f = v[e * D];
          s[2 * e] = make_float2(f.x, f.y);
          s[2 * e + 1] = make_float2(f.z, f.w);
        }
      } else if (q.s_t) {                             // stored [y][z]
#pragma unroll
        for (int e = 0; e < D / 4; ++e)
          s[e] = make_float2(src[(size_t)(D / 2 * wg + 2 * e) * D + z], src[(size_t)(D / 2 * wg + 2 * e + 1) * D + z]);
      } else {
        const float4* v = reinterpret_cast<const float4*>(src + (size_t)z * D + D / 2 * wg);
#pragma unroll
        for (int e = 0; e < D / 8; ++e) {
          const float4 f = v[e];
          s[2 * e] = make_float2(f.x, f.y);
          s[2 * e + 1] = make_float2(f.z, f.w);
        }
      }
    }
    auto put_state = [&]() {                          // BF16 copy, the A operand of S X^T
#pragma unroll
      for (int k = 0; k < NP; ++k) {
        uint32_t v[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = pack_bf16x2(s[16 * k + e].x, s[16 * k + e].y);
        tmem_st16(tl + TM_SB + D / 4 * wg + 16 * k, v);
      }
    };
    if (!kState && nc > 0) {
      put_state();
      tmem_st_wait();
      tc_fence_before();
      warp_arrive(&bars[GO], lane);
    }
    bool ok = nc == 0 || warp_wait(&bars[TBL], 0, cx);
    // lam^64 lies between two floats.  Each chunk takes the one of them that keeps the product of
    // the factors nearest to the power (error diffusion): rows of any age are off by an ulp of the
    // factor at most and by nothing on average, at no cost to the elements.  The last chunk makes
    // good what is left.  (One float alone, with its lack given back every 16 chunks, left younger
    // rows up to 1e-6 off.)
    float lack = 0.f;                                   // of the factors so far, relative
#pragma unroll 1
    for (int c = 0; c < nc && ok; ++c) {
      const bool end = c + 1 == nc;
      if (!(ok = warp_wait(&bars[EDONE + c % NE], (c / NE) & 1, cx))) break;
      tc_fence_after();
      const bool other = fabsf(lack + carry[5]) < fabsf(lack + carry[1]);
      const int at = end ? 2 : other ? 4 : 0;
      lack += carry[at + 1];
      const float f = carry[at];
      const float2 fh = make_float2(f, f), fl = make_float2(f * lack, f * lack);
#pragma unroll
      for (int k = 0; k < NP; ++k) {
        float x[32];
        tmem_ld32(tl + TM_E + 128 * (c % NE) + D / 2 * wg + 32 * k, x);
        tmem_ld_wait();
        if (k == NP - 1) {
          tc_fence_before();
          warp_arrive(&bars[EFREE + c % NE], lane);
        }
        if (end) {
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 t = fma2(fl, s[16 * k + e], make_float2(x[2 * e], x[2 * e + 1]));
            x[2 * e] = t.x;
            x[2 * e + 1] = t.y;
          }
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          float2& v = s[16 * k + e];
          v = fma2(fh, v, make_float2(x[2 * e], x[2 * e + 1]));
        }
      }
      if (kState || end) continue;
      // S X^T of this chunk has read the old copy
      if (!(ok = warp_wait(&bars[O1DONE], c & 1, cx))) break;
      tc_fence_after();
      put_state();
      tmem_st_wait();
      tc_fence_before();
      warp_arrive(&bars[GO], lane);
    }
    float* dst = !ok ? nullptr
                 : kState ? q.sums + ((size_t)unit[4] * p.H + h) * D * D
                 : unit[5] ? la_exit(p, q, unit[3], h, D) : nullptr;
    if (dst) {
      if (kState) {
        float4* v = reinterpret_cast<float4*>(dst) + D / 8 * wg * D + z;
#pragma unroll
        for (int e = 0; e < D / 8; ++e)
          v[e * D] = make_float4(s[2 * e].x, s[2 * e].y, s[2 * e + 1].x, s[2 * e + 1].y);
      } else if (q.s_t) {
#pragma unroll
        for (int e = 0; e < D / 4; ++e) {
          dst[(size_t)(D / 2 * wg + 2 * e) * D + z] = s[e].x;
          dst[(size_t)(D / 2 * wg + 2 * e + 1) * D + z] = s[e].y;
        }
      } else {
        // By way of shared memory, so that a store covers whole rows: 16-byte pieces, those of
        // eight rows on different banks.  The stages after the last chunk's (two at head size
        // 128) are free: what they held has been read (O1 of the chunk before the last came
        // after it), and no copy follows.
        constexpr int PW = D / 8;                       // pieces of a warp's row
        uint8_t* mine = sm + (wg ? (nc + 1) % NS : nc % NS) * M::STAGE + (warp & 3) * 32 * PW * 16;
#pragma unroll
        for (int e = 0; e < PW; ++e)
          *reinterpret_cast<float4*>(mine + (lane * PW + (e ^ (lane & 7))) * 16) =
              make_float4(s[2 * e].x, s[2 * e].y, s[2 * e + 1].x, s[2 * e + 1].y);
        __syncwarp();
        float* o = dst + (size_t)(z - lane + lane / PW) * D + D / 2 * wg + lane % PW * 4;
#pragma unroll
        for (int e = 0; e < PW; ++e) {
          const int row = e * (32 / PW) + lane / PW;
          *reinterpret_cast<float4*>(o) =
              *reinterpret_cast<const float4*>(mine + (row * PW + (lane % PW ^ (row & 7))) * 16);
          o += (size_t)(32 / PW) * D;
        }
      }
    }
    }
  } else if (warp < 16) {
    reg_dealloc<72>();
    if ((warp & 3) < WL) split_rows(0, NE);
  } else {
    // (as launched: 96 registers)
    if (warp == 16) {
      // lam^64, lam^tail and the float on the other side of lam^64, each with what it lacks,
      // relative to it: a state carried over thousands of chunks must not drift by the rounding of
      // one factor
      if (lane < 2) {
        const double v = la_pow(p.decay[h], lane ? tail : C);
        const float f = (float)v, less = (float)(v - (double)f);
        const float g = __int_as_float(__float_as_int(f) + (less < 0.f ? -1 : 1));
        const bool live = v > 1e-30;
        carry[2 * lane] = f;
        carry[2 * lane + 1] = live ? less / f : 0.f;
        if (lane == 0) {
          carry[4] = g;
          carry[5] = live ? (less - (g - f)) / g : 0.f;
        }
      }
      __syncwarp();
      if (lane == 0 && p.tries == 0) mbar_arrive(&bars[TBL]);   // (a test leaves it out)
    }
    // ---------------------------------------------------------------- results
    // A warp takes the 32 columns z of its TMEM lanes, 32 rows at a time, as 8 x 8 tiles: of the
    // row pairs 8 g + 2 (lane % 4), + 1, columns 8 k + lane / 4.
    const uint32_t tl = tm + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t stage = sb + M::OUT + (warp & 3) * 2048;
    const int H = p.H;
    // the lane's row and 16 bytes of a store (eight rows a store)
    const int rr = lane >> 2;
    const uint32_t sw = stage + (lane & 7) * 64 + (((lane >> 3) ^ ((lane >> 1) & 3)) << 4);
    const uint32_t sr = stage + rr * 64 + (((lane & 3) ^ ((rr >> 1) & 3)) << 4);
    const size_t col = (size_t)h * D + 32 * (warp & 3);
    auto walk = [&](auto f32) {
#pragma unroll 1
      for (int c = 0; c < nc; ++c) {
        const bool end = c + 1 == nc;
        const int L = end ? tail : C;
        const int r0 = rev ? s1 - c * C - L : s0 + c * C;
        const float2* f2 = reinterpret_cast<const float2*>(rd + (end ? 64 : 0)) + (lane & 3);
        if (!warp_wait(&bars[ODONE], c & 1, cx)) break;
        tc_fence_after();
        uint32_t v[2][4][4];                            // [hf][g][k]
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
          for (int hz = 0; hz < 2; ++hz) {
            float o1[16], o2[16];
            tmem_ld_16x32(tl + ((uint32_t)(16 * hz) << 16) + TM_O1 + 32 * hf, o1);
            tmem_ld_16x32(tl + ((uint32_t)(16 * hz) << 16) + TM_O2 + 32 * hf, o2);
            tmem_ld_wait();
            if (hf + hz == 2) {
              tc_fence_before();
              warp_arrive(&bars[OFREE], lane);
            }
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              const float2 f = f2[16 * hf + 4 * g];
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const int e = 4 * g + 2 * k;
                const float2 t = fma2(f, make_float2(o1[e], o1[e + 1]), make_float2(o2[e], o2[e + 1]));
                if constexpr (f32.value) {
                  const int row = 32 * hf + 8 * g + 2 * (lane & 3);
                  float* of = reinterpret_cast<float*>(q.out) + (size_t)(r0 + row) * H * D + col +
                              16 * hz + 8 * k + rr;
                  if (row < L) of[0] = t.x;
                  if (row + 1 < L) of[(size_t)H * D] = t.y;
                } else {
                  v[hf][g][2 * hz + k] = pack2(t);
                }
              }
            }
          }
        }
        if constexpr (!f32.value) {
          // turned in shared memory: row 8 g + i of the 64-byte rows, its 16-byte pieces in the
          // order that keeps eight rows on different banks
          uint4* o = reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(q.out) +
                                              (size_t)(r0 + rr) * H * D + col + 8 * (lane & 3));
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            __syncwarp();
#pragma unroll
            for (int g = 0; g < 4; ++g) stmatrix_x4_trans(sw + 512 * g, v[hf][g]);
            __syncwarp();
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint4 w4;
              asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                           : "=r"(w4.x), "=r"(w4.y), "=r"(w4.z), "=r"(w4.w) : "r"(sr + 512 * e) : "memory");
              if (32 * hf + rr + 8 * e < L) *o = w4;    // 8 rows of H D elements
              o += (size_t)H * D;
            }
          }
        }
      }
    };
    if ((warp & 3) >= WL) {
    } else if (kState) {
      split_rows(1, 2);                               // no results: the other buffer's chunks
    } else {
      if (q.out_f32) walk(std::true_type());
      else walk(std::false_type());
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) {
    if (!kState) launch_wait();                       // no launch ends before the ones ahead of it
    tmem_relinquish();
    tmem_dealloc(tm, 512);
    if (lane == 0 && *cx && p.status) {
      atomicCAS(p.status, 0, (int)SF_ERR_TIMEOUT);
      atomicCAS(p.status + 1, 0, (int)(*cx | ((blockIdx.x & 0x3ffffu) << 12)));
    }
  }
}

template <int D>
cudaError_t go(const LaParams& p, bool state_only, cudaStream_t st) {
  const int64_t grid = (int64_t)(state_only ? p.pre_units : p.units) * p.H * p.npass;
  if (grid <= 0) return cudaSuccess;
  if (grid > 0x7fffffff) return cudaErrorInvalidValue;
  Maps maps;
  const int rows = p.B * p.T;
  bool returns = p.pool != nullptr;
  for (int i = 0; i < p.npass; ++i) {
    const LaPass& q = p.pass[i];
    returns = returns || q.s_out;
    if (!make_bf16_map(&maps.m[i][0], q.x, rows, q.hx, D) ||
        !make_bf16_map(&maps.m[i][1], q.y, rows, q.hy, D) ||
        !make_bf16_map(&maps.m[i][2], q.z, rows, q.hz, D))
      return cudaErrorInvalidValue;
  }
  auto kern = state_only ? (returns ? la_tc_kernel<D, true, 3> : la_tc_kernel<D, true, 2>)
                         : (returns ? la_tc_kernel<D, false, 3> : la_tc_kernel<D, false, 2>);
  const cudaError_t e = allow_smem(kern, Mem<D>::SIZE);
  if (e != cudaSuccess) return e;
  return launch_after(!state_only && p.pre_units > 0, kern, (unsigned)grid, NT, Mem<D>::SIZE, st, maps, p);
}

}  // namespace

cudaError_t launch_la_tc(const LaParams& p, int D, bool state_only, cudaStream_t st) {
  return D == 64 ? go<64>(p, state_only, st) : go<128>(p, state_only, st);
}

}  // namespace sfg
