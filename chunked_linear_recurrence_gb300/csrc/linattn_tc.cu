// linattn_tc.cu -- the decayed linear attention's product (linattn.cuh) on tcgen05: BF16 tokens
// with head size 128.
//
// One CTA walks one (segment, head) in 64-row chunks.  Rows r, s of a chunk, the state S [z][y]:
//     QK  = [Y; X] Y^T           M = 128, N = 64, K = 128   (rows 64-127: X Y^T)
//     P   = a QK o lam^|r-s|     BF16, by two warps, to shared memory
//     E   = (lam^f c Z)^T Y      M = 128, N = 128, K = 64   three times (below)
//     O1^T = S X^T               M = 128, N = 64,  K = 128  (S as BF16 in TMEM)
//     O2^T = Z^T P^T             M = 128, N = 64,  K = 64
//     out = b lam^e O1 + O2,     S <- lam^L S + E           (FP32)
// Everything is laid out as the TMA brings it: [rows][128] BF16 tiles of two swizzled 64-column
// panels, read K-major or MN-major as each product needs.
//
// The state stays in the registers of eight warps (64 floats a thread), not in TMEM: every
// chunk's E is a product of its own, so E of the next chunks never waits for S, no FP32 state
// is read and written back around the products, and the sum over the chunks is rounded in
// FP32 to nearest.  E's left operand is exact enough to keep FP32 accuracy of the state: the
// weighted rows are split into three BF16 summands (8 bits each, 24 together), each multiplied
// with the exact Y.  A launch that returns no state takes two of them (16 bits): its state
// only ever reaches BF16 results.
//
// Warps: 0 loads (three chunks in flight), 1 issues, 2-3 form P, 4-11 hold the state and write
// the results (two warpgroups: columns y 0-63 and 64-127 of the state, rows 0-31 and 32-63 of
// the results), 12-15 split the weighted rows.  Per chunk the issuer queues QK, E, then O1 (once
// the state is there), then O2 (once P is there): while the state warps turn E into the next
// entry state, the tensor pipe works on the next chunk's QK and E.  Warps meet through
// mbarriers alone; every wait is bounded, and a thread that gives up writes SF_ERR_TIMEOUT to
// the status word and raises the CTA's abort flag; copies and products in flight land before
// the CTA leaves.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "common.cuh"
#include "f32x2.cuh"
#include "linattn.cuh"
#include "tc_ptx.cuh"
#include "tmap.cuh"

namespace sfg {
namespace {

using namespace tc;

constexpr int D = 128, C = LA_CHUNK, NT = 512, NS = 4;
constexpr uint32_t PANEL = 8192;                 // 64 rows x 128 bytes
constexpr uint32_t B_Y = 0, B_X = PANEL;         // panel 0 of Y and X; panel 1 two panels on
constexpr uint32_t B_Z = 4 * PANEL, STAGE = 6 * PANEL;
constexpr uint32_t O_P = NS * STAGE;             // P [64][64]
constexpr uint32_t O_OUT = O_P + PANEL;          // results, [32 rows][32 columns] of each warp
// b lam^e and c lam^f of a full chunk and of the walk's last one [64] each, a lam^n [64], carry [4]
constexpr uint32_t O_TAB = O_OUT + 16384;
constexpr uint32_t O_BAR = O_TAB + 1536;
constexpr uint32_t SMEM = O_BAR + 256 + 1024;
static_assert(SMEM <= 232448, "shared memory");

// TMEM columns: E, the state's BF16 copy, QK, O1, O2, the weighted rows' parts (32 columns
// each); a launch that computes states alone has two buffers of E and of the parts.
constexpr uint32_t TM_E = 0, TM_SB = 128, TM_P = 192, TM_O1 = 256, TM_O2 = 320;
template <bool kState>
__device__ __forceinline__ uint32_t tm_w(int buf) { return kState ? 256 + 96 * buf : 384; }

constexpr uint32_t ID_QK = idesc_bf16(128, 64, false, false);
constexpr uint32_t ID_E = idesc_bf16(128, 128, false, true);   // A in TMEM
constexpr uint32_t ID_O1 = idesc_bf16(128, 64, false, false);   // A in TMEM
constexpr uint32_t ID_O2 = idesc_bf16(128, 64, true, false);

enum { FULL = 0, LANDED = FULL + NS, FREE = LANDED + NS, QKDONE = FREE + NS, PREADY, SPLIT,
       EDONE = SPLIT + 2, EFREE = EDONE + 2, ODONE = EFREE + 2, GO, TBL, DRAIN, NBAR = DRAIN + 2 };
static_assert(8 * NBAR + 8 <= 256, "barriers");

constexpr long long WAIT_CYCLES = 4000000000ll;   // about 2 s

struct Maps {
  CUtensorMap m[3][3];   // x, y, z of each pass
};

struct Cx {
  int* status;
  volatile int* abort;
};

__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, const Cx& cx) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  while (true) {
    if (mbar_try_wait_sleep(bar, parity, 20000u)) return true;
    if (*cx.abort) return false;
    if (clock64() - t0 > WAIT_CYCLES) {
      *cx.abort = 1;
      if (cx.status) {
        atomicCAS(cx.status, 0, (int)SF_ERR_TIMEOUT);
        atomicCAS(cx.status + 1, 0, (int)(0x40000000u | ((blockIdx.x & 0x3ffffu) << 12) |
                                          ((threadIdx.x >> 5) << 6) | ((smem_u32(bar) & 255u) >> 3)));
      }
      return false;
    }
  }
}
// The lanes of a warp wait together and agree on the outcome.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const Cx& cx) {
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

template <bool kState, int NSP>
__global__ void __launch_bounds__(NT, 1) la_tc_kernel(const __grid_constant__ Maps maps,
                                                      const LaParams p) {
  extern __shared__ __align__(1024) uint8_t raw[];
  uint8_t* sm = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  const uint32_t sb = smem_u32(sm);
  float* rd = reinterpret_cast<float*>(sm + O_TAB);   // [2][64]
  float* wr = rd + 128;                               // [2][64]
  float* pq = rd + 256;                               // [64]
  float* carry = rd + 320;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + O_BAR);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(sm + O_BAR + 8 * NBAR);
  int* abort_s = reinterpret_cast<int*>(sm + O_BAR + 8 * NBAR + 4);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  int id = blockIdx.x;
  const int pi = id % p.npass; id /= p.npass;
  const int h = id % p.H, u = id / p.H;
  const LaPass& q = p.pass[pi];
  int n, w;
  int64_t bos, eos;
  if (!la_locate(u, p, n, w, bos, eos)) return;
  const int64_t len = eos - bos;
  const bool split = p.seg < p.T;
  const bool last = (int64_t)(w + 1) * p.seg >= len;
  if (kState && last) return;                     // nobody enters from its end
  const int64_t off = (int64_t)w * p.seg;
  const int64_t rows = len - off < p.seg ? len - off : p.seg;
  const bool rev = q.reverse != 0;
  const int64_t s0 = rev ? eos - off - rows : bos + off, s1 = s0 + rows;
  bool skip;
  const float* s_in = la_entry(p, q, n, h, D, skip);
  if (skip) {                                     // padding of the paged pool: zero rows
    if (kState) return;
    uint4* o = reinterpret_cast<uint4*>(q.out);
    for (int64_t i = tid; i < rows * 16; i += NT)
      o[((size_t)(s0 + (i >> 4)) * p.H + h) * 16 + (i & 15)] = make_uint4(0, 0, 0, 0);
    return;
  }
  constexpr int NE = kState ? 2 : 1;              // buffers of E and of the weighted rows
  const int nc = (int)((rows + C - 1) / C);
  const int tail = (int)(rows - (int64_t)(nc - 1) * C);   // rows of the walk's last chunk
  const float d = p.decay[h];
  const Cx cx{p.status, abort_s};

  if (tid == 0) {
    for (int i = 0; i < NBAR; ++i)
      mbar_init(&bars[i], i == PREADY ? 2 : i == SPLIT || i == SPLIT + 1 ? 4
                          : i == GO || i == EFREE || i == EFREE + 1 ? 8 : i >= FREE && i < FREE + NS && !kState ? 2 : 1);
    *abort_s = 0;
    fence_mbar_init();
    prefetch_tmap(&maps.m[pi][1]);
    prefetch_tmap(&maps.m[pi][2]);
    if (!kState) prefetch_tmap(&maps.m[pi][0]);
  }
  if (warp == 0) tmem_alloc(tslot, 512);
  auto pw = [&](int e) { return e <= 0 ? 1.f : expf(d * (float)e); };
  if (tid >= 128 && tid < 256) {
    const int i = tid & 63, L = tid < 192 ? C : tail, t = tid - 128;
    rd[t] = i < L ? q.b * pw(rev ? L - 1 - i : i + 1) : 0.f;
    wr[t] = i < L ? q.c * pw(rev ? i + 1 : L - 1 - i) : 0.f;
    if (t < 64) pq[t] = q.a * pw(t);
  }
  if (!kState)   // P on the far side of the diagonal stays zero
    for (int i = tid; i < (int)PANEL / 16; i += NT)
      *reinterpret_cast<uint4*>(sm + O_P + 16 * i) = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = *tslot;

  if (warp < 4) {
    reg_dealloc<104>();
    if (warp == 0) {
      // -------------------------------------------------------------- loader, issuer of E
      const int hx = h / (p.H / q.hx), hy = h / (p.H / q.hy), hz = h / (p.H / q.hz);
      int issued = 0;
      auto load = [&](int c) {
        const int b = c % NS, L = c + 1 == nc ? tail : C;
        const int r0 = (int)(rev ? s1 - (int64_t)c * C - L : s0 + (int64_t)c * C);
        uint8_t* st = sm + b * STAGE;
        uint64_t* bar = L < C ? &bars[LANDED + b] : &bars[FULL + b];   // (the last chunk only)
        if (elect_one()) {
          mbar_arrive_expect_tx(bar, (kState ? 4 : 6) * PANEL);
#pragma unroll
          for (int pp = 0; pp < 2; ++pp) {
            tma_load_3d(st + B_Y + 2 * pp * PANEL, &maps.m[pi][1], bar, 64 * pp, hy, r0);
            tma_load_3d(st + B_Z + pp * PANEL, &maps.m[pi][2], bar, 64 * pp, hz, r0);
            if (!kState) tma_load_3d(st + B_X + 2 * pp * PANEL, &maps.m[pi][0], bar, 64 * pp, hx, r0);
          }
        }
        __syncwarp();
        issued = c + 1;
      };
      // A short last chunk: rows past the end (other tokens, or NaN padding) must not reach the
      // products.
      auto trim = [&]() {
        const int b = (nc - 1) % NS;
        if (!warp_wait(&bars[LANDED + b], 0, cx)) return false;
        uint8_t* st = sm + b * STAGE;
        const int per = (C - tail) * 8;                // 16-byte pieces of a panel
        for (int i = lane; i < 4 * per; i += 32) {
          const int t = i / per, rr = i % per;
          uint8_t* base = st + (t < 2 ? B_Y + 2 * t * PANEL : B_Z + (t - 2) * PANEL);
          *reinterpret_cast<uint4*>(base + (tail + rr / 8) * 128 + (rr % 8) * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        warp_arrive(&bars[FULL + b], lane);
        return true;
      };
      for (int c = 0; c < NS && c < nc; ++c) load(c);
      bool ok = nc != 1 || tail == C || trim();
      for (int c = 0; c < nc && ok; ++c) {
        const int b = c % NS;
        const int eb = c % NE, ph = (c / NE) & 1;
        const uint64_t dy = sdesc_sw128(sb + b * STAGE + B_Y, 2 * PANEL, 1024);
        if (c >= NE && !(ok = warp_wait(&bars[EFREE + eb], ph ^ 1, cx))) break;
        // (the split warps have waited for the rows themselves)
        if (!(ok = warp_wait(&bars[SPLIT + eb], ph, cx))) break;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int sp = 0; sp < NSP; ++sp)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_bf16_ta(tm + TM_E + 128 * eb, tm + tm_w<kState>(eb) + 32 * sp + 8 * kk,
                          dy + kstep_mn(kk), ID_E, kk + sp > 0);
          mma_commit(&bars[EDONE + eb]);
          mma_commit(&bars[FREE + b]);
        }
        __syncwarp();
        if (c + 2 == nc && tail < C && !(ok = trim())) break;
        if (c > 0 && c + NS - 1 < nc) {
          if (!(ok = warp_wait(&bars[FREE + (c - 1) % NS], ((c - 1) / NS) & 1, cx))) break;
          load(c + NS - 1);
        }
      }
      if (!ok)   // let the copies in flight land
        for (int c = issued > NS ? issued - NS : 0; c < issued; ++c) {
          if (c + 1 == nc && tail < C) mbar_wait(&bars[LANDED + c % NS], 0, 100000000ull);
          else mbar_wait(&bars[FULL + c % NS], (c / NS) & 1, 100000000ull);
        }
      if (elect_one()) mma_commit(&bars[DRAIN]);
      mbar_wait(&bars[DRAIN], 0, 100000000ull);
      __syncwarp();
    } else if (warp == 1) {
      // -------------------------------------------------------------- issuer of QK, O1, O2
      // (the whole warp waits; one elected lane issues)
      auto issue_qk = [&](int c) {
        const uint64_t dy = sdesc_sw128(sb + (c % NS) * STAGE + B_Y, 0, 1024);
        const uint32_t t = tm + TM_P;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_bf16(t, dy + kstep_k(kk), dy + kstep_k(kk), ID_QK, kk > 0);
          mma_commit(&bars[QKDONE]);
        }
        __syncwarp();
      };
      auto full = [&](int c) { return warp_wait(&bars[FULL + c % NS], (c / NS) & 1, cx); };
      bool ok = !kState && nc > 0 && full(0);
      if (ok) issue_qk(0);
      for (int c = 0; c < nc && ok; ++c) {
        const int b = c % NS;
        const uint32_t st = sb + b * STAGE;
        if (!(ok = warp_wait(&bars[GO], c & 1, cx))) break;
        tc_fence_after();
        const uint64_t dx = sdesc_sw128(st + B_X, 0, 1024);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_bf16_ta(tm + TM_O1, tm + TM_SB + kk * 8, dx + kstep_k(kk), ID_O1, kk > 0);
        }
        __syncwarp();
        if (!(ok = warp_wait(&bars[PREADY], c & 1, cx))) break;
        tc_fence_after();
        const uint64_t dz = sdesc_sw128(st + B_Z, PANEL, 1024);
        const uint64_t dp = sdesc_sw128(sb + O_P, 0, 1024);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_bf16(tm + TM_O2, dz + kstep_mn(kk), dp + (uint64_t)(kk * 2), ID_O2, kk > 0);
          mma_commit(&bars[ODONE]);
          mma_commit(&bars[FREE + b]);
        }
        __syncwarp();
        // the next chunk's QK, under the state warps' turn
        if (c + 1 < nc) {
          if (!(ok = full(c + 1))) break;
          issue_qk(c + 1);
        }
      }
      if (elect_one()) mma_commit(&bars[DRAIN + 1]);
      mbar_wait(&bars[DRAIN + 1], 0, 100000000ull);
      __syncwarp();
    } else {
      // -------------------------------------------------------------- P
      if (warp == 3) {
        // lam^64 and lam^tail as sums of two floats: a state carried over thousands of chunks
        // must not drift by the rounding of one factor
        if (lane < 2) {
          const double f = la_pow(d, lane ? tail : C);
          carry[2 * lane] = (float)f;
          carry[2 * lane + 1] = (float)(f - (double)(float)f);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[TBL]);
      }
      if (!kState) {
        // row r of P; the factors a lam^|r-s| stay in registers.  The half on the far side of
        // the diagonal (32 columns of one warp) is never touched: it stays zero.
        const int r = (warp - 2) * 32 + lane;          // TMEM lane 64 + r
        float f[2][32];
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const int s = 32 * half + e, gap = rev ? s - r : r - s;
            f[half][e] = gap >= 0 ? pq[gap & 63] : 0.f;
          }
        const uint32_t tl = tm + TM_P + ((uint32_t)(warp * 32) << 16);
        uint8_t* row = sm + O_P + r * 128;
        for (int c = 0; c < nc; ++c) {
          if (!warp_wait(&bars[QKDONE], c & 1, cx)) break;
          tc_fence_after();
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            if (rev ? half == 0 && warp == 3 : half == 1 && warp == 2) continue;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              float x[16];
              tmem_ld16(tl + 32 * half + 16 * k, x);
              tmem_ld_wait();
#pragma unroll
              for (int ch = 0; ch < 2; ++ch) {
                const float* g = &f[half][16 * k + 8 * ch];
                const float* y = x + 8 * ch;
                uint4 v;
                v.x = pack_bf16x2(y[0] * g[0], y[1] * g[1]);
                v.y = pack_bf16x2(y[2] * g[2], y[3] * g[3]);
                v.z = pack_bf16x2(y[4] * g[4], y[5] * g[5]);
                v.w = pack_bf16x2(y[6] * g[6], y[7] * g[7]);
                *reinterpret_cast<uint4*>(row + (((4 * half + 2 * k + ch) ^ (r & 7)) << 4)) = v;
              }
            }
          }
          fence_proxy_async_smem();
          tc_fence_before();
          warp_arrive(&bars[PREADY], lane);
        }
      }
    }
  } else if (warp < 12) {
    reg_alloc<160>();
    // ---------------------------------------------------------------- state and results
    const int wg = (warp - 4) >> 2;
    const int z = ((warp & 3) << 5) + lane;
    const uint32_t tl = tm + ((uint32_t)((warp & 3) * 32) << 16);
    float2 s[32];                                       // columns 64 wg + 2 e, + 1 of row z
    const size_t uoff = ((size_t)u * p.H + h) * D * D;
    {
      const float* src = kState ? nullptr : split ? q.seg_state + uoff : s_in;
      if (!src) {
#pragma unroll
        for (int e = 0; e < 32; ++e) s[e] = make_float2(0.f, 0.f);
      } else if (q.s_t && !split) {                   // stored [y][z]
#pragma unroll
        for (int e = 0; e < 32; ++e)
          s[e] = make_float2(src[(size_t)(64 * wg + 2 * e) * D + z], src[(size_t)(64 * wg + 2 * e + 1) * D + z]);
      } else {
        const float4* v = reinterpret_cast<const float4*>(src + (size_t)z * D + 64 * wg);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float4 f = v[e];
          s[2 * e] = make_float2(f.x, f.y);
          s[2 * e + 1] = make_float2(f.z, f.w);
        }
      }
    }
    auto put_state = [&]() {                          // BF16 copy, the A operand of S X^T
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint32_t v[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = pack_bf16x2(s[16 * k + e].x, s[16 * k + e].y);
        tmem_st16(tl + TM_SB + 32 * wg + 16 * k, v);
      }
    };
    if (!kState && nc > 0) {
      put_state();
      tmem_st_wait();
      tc_fence_before();
      warp_arrive(&bars[GO], lane);
    }
    bool ok = nc == 0 || warp_wait(&bars[TBL], 0, cx);
    const uint32_t stage = sb + O_OUT + (warp - 4) * 2048;
    for (int c = 0; c < nc && ok; ++c) {
      const bool end = c + 1 == nc;
      const int L = end ? tail : C;
      if (!(ok = warp_wait(&bars[EDONE + c % NE], (c / NE) & 1, cx))) break;
      tc_fence_after();
      const float2 fh = make_float2(carry[end ? 2 : 0], carry[end ? 2 : 0]);
      const float2 fl = make_float2(carry[end ? 3 : 1], carry[end ? 3 : 1]);
      float x[2][32];
#pragma unroll
      for (int k = 0; k < 2; ++k) tmem_ld32(tl + TM_E + 128 * (c % NE) + 64 * wg + 32 * k, x[k]);
      tmem_ld_wait();
      tc_fence_before();
      warp_arrive(&bars[EFREE + c % NE], lane);
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        const float* y = &x[e >> 4][2 * (e & 15)];
        s[e] = fma2(fh, s[e], fma2(fl, s[e], make_float2(y[0], y[1])));
      }
      if (kState) continue;
      if (!(ok = warp_wait(&bars[ODONE], c & 1, cx))) break;
      tc_fence_after();
      // O1, O2 rows [32 wg, + 32) as 8 x 8 tiles: of row pairs 8 g + 2 (lane % 4), + 1, columns
      // 16 hz + 8 k + lane / 4 of the warp's 32
      float o1[2][16], o2[2][16];
      if (!end) put_state();                          // S X^T of this chunk has read the old copy
#pragma unroll
      for (int hz = 0; hz < 2; ++hz) {
        tmem_ld_16x32(tl + ((uint32_t)(16 * hz) << 16) + TM_O1 + 32 * wg, o1[hz]);
        tmem_ld_16x32(tl + ((uint32_t)(16 * hz) << 16) + TM_O2 + 32 * wg, o2[hz]);
      }
      tmem_ld_wait();
      if (!end) {
        tmem_st_wait();
        tc_fence_before();
        warp_arrive(&bars[GO], lane);
      }
      const int64_t r0 = (rev ? s1 - (int64_t)c * C - L : s0 + (int64_t)c * C) + 32 * wg;
      const int cnt = L - 32 * wg;                    // rows that exist
      const float2* f2 = reinterpret_cast<const float2*>(rd + (end ? 64 : 0) + 32 * wg) + (lane & 3);
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const float2 f = f2[4 * g];
        uint32_t v[4];                                // tiles of columns 0, 8, 16, 24
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float* y = &o1[k >> 1][4 * g + 2 * (k & 1)];
          const float* y2 = &o2[k >> 1][4 * g + 2 * (k & 1)];
          const float2 t = fma2(f, make_float2(y[0], y[1]), make_float2(y2[0], y2[1]));
          v[k] = pack_bf16x2(t.x, t.y);
          y[0] = t.x;
          y[1] = t.y;
        }
        // row 8 g + i of the 64-byte rows, its 16-byte pieces in the order that keeps eight rows
        // on different banks
        if (!q.out_f32) {
          const int i = lane & 7, m = lane >> 3;
          stmatrix_x4_trans(stage + (8 * g + i) * 64 + ((m ^ ((i >> 1) & 3)) << 4), v);
        }
      }
      if (q.out_f32) {
        float* o = reinterpret_cast<float*>(q.out) +
                   ((size_t)(r0 + 2 * (lane & 3)) * p.H + h) * D + 32 * (warp & 3) + (lane >> 2);
#pragma unroll
        for (int hz = 0; hz < 2; ++hz)
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int row = 8 * (e >> 2) + (e & 1), col = 16 * hz + 8 * ((e >> 1) & 1);
            if (2 * (lane & 3) + row < cnt) o[(size_t)row * p.H * D + col] = o1[hz][e];
          }
        continue;
      }
      __syncwarp();
      const int rr = lane >> 2;
      uint4* o = reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(q.out) +
                                          ((size_t)(r0 + rr) * p.H + h) * D + 32 * (warp & 3) +
                                          8 * (lane & 3));
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint4 v;
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                     : "r"(stage + (8 * e + rr) * 64 + (((lane & 3) ^ ((rr >> 1) & 3)) << 4)) : "memory");
        if (rr + 8 * e < cnt) o[(size_t)e * p.H * D] = v;   // 8 rows of H D elements, 8 a uint4
      }
      __syncwarp();
    }
    float* dst = !ok ? nullptr : kState ? q.seg_state + uoff : last ? la_exit(p, q, n, h, D) : nullptr;
    if (dst) {
      if (q.s_t && !kState) {
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          dst[(size_t)(64 * wg + 2 * e) * D + z] = s[e].x;
          dst[(size_t)(64 * wg + 2 * e + 1) * D + z] = s[e].y;
        }
      } else {
        float4* v = reinterpret_cast<float4*>(dst + (size_t)z * D + 64 * wg);
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = make_float4(s[2 * e].x, s[2 * e].y, s[2 * e + 1].x, s[2 * e + 1].y);
      }
    }
  } else {
    reg_dealloc<88>();
    // ---------------------------------------------------------------- weighted rows in BF16 parts
    // Each warp weights and splits the 32 columns z of its TMEM lanes: 16 at a time, transposed
    // on the way from shared memory (8 x 8 tiles), the rows j along the TMEM columns.  The first
    // 16 are ready before the buffer is free.
    const uint32_t tl = tm + ((uint32_t)((warp & 3) * 32) << 16);
    const int m = lane >> 3, i = lane & 7;
    // lane's source row of K step 0: j = 8 (m / 2) + i, columns z0 + 8 (m % 2) ..; z0 of either
    // half differs in bit 1 of the 16-byte chunk
    const uint32_t ch = (uint32_t)(4 * (warp & 1) + (m & 1));
    const uint32_t src = sb + B_Z + (uint32_t)((warp & 3) >> 1) * PANEL + (uint32_t)(8 * (m >> 1) + i) * 128u;
    const uint32_t c0 = (ch ^ (uint32_t)i) << 4, c1 = ((ch + 2) ^ (uint32_t)i) << 4;
    for (int c = 0; c < nc; ++c) {
      const int b = c % NS, eb = c % NE;
      if (!warp_wait(&bars[FULL + b], (c / NS) & 1, cx)) break;
      const float2* wt = reinterpret_cast<const float2*>(wr + (c + 1 == nc ? 64 : 0)) + (lane & 3);
      float2 wv[8];                                   // rows 8 g + 2 (lane % 4), + 1
#pragma unroll
      for (int g = 0; g < 8; ++g) wv[g] = wt[4 * g];
      bool ok = true;
#pragma unroll
      for (int hz = 0; hz < 2; ++hz) {
        uint32_t o[NSP][16];
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          uint32_t v[4];
          ldmatrix_x4_trans(src + b * STAGE + kk * 2048 + (hz ? c1 : c0), v);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float2 x = mul2(unpack2(v[e]), wv[2 * kk + (e >> 1)]);
#pragma unroll
            for (int sp = 0; sp < NSP; ++sp) {
              o[sp][4 * kk + e] = pack_bf16x2(x.x, x.y);
              if (sp + 1 < NSP) x = sub2(x, unpack2(o[sp][4 * kk + e]));
            }
          }
        }
        // the products of the chunk that had the buffer are done
        if (hz == 0 && c >= NE && !(ok = warp_wait(&bars[EDONE + eb], ((c / NE) & 1) ^ 1, cx))) break;
        if (hz == 0) tc_fence_after();
#pragma unroll
        for (int sp = 0; sp < NSP; ++sp)
          tmem_st_16x32(tl + ((uint32_t)(16 * hz) << 16) + tm_w<kState>(eb) + 32 * sp, o[sp]);
      }
      if (!ok) break;
      tmem_st_wait();
      tc_fence_before();
      warp_arrive(&bars[SPLIT + eb], lane);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) {
    tmem_relinquish();
    tmem_dealloc(tm, 512);
  }
}

}  // namespace

cudaError_t launch_la_tc(const LaParams& p, bool state_only, cudaStream_t st) {
  const int64_t grid = (int64_t)p.units * p.H * p.npass;
  if (grid <= 0) return cudaSuccess;
  if (grid > 0x7fffffff) return cudaErrorInvalidValue;
  Maps maps;
  const int rows = p.B * p.T;
  bool returns = p.pool != nullptr;
  for (int i = 0; i < p.npass; ++i) {
    const LaPass& q = p.pass[i];
    returns = returns || q.s_out;
    if (!make_bf16_map(&maps.m[i][0], q.x, rows, q.hx) || !make_bf16_map(&maps.m[i][1], q.y, rows, q.hy) ||
        !make_bf16_map(&maps.m[i][2], q.z, rows, q.hz))
      return cudaErrorInvalidValue;
  }
  auto kern = state_only ? (returns ? la_tc_kernel<true, 3> : la_tc_kernel<true, 2>)
                         : (returns ? la_tc_kernel<false, 3> : la_tc_kernel<false, 2>);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM);
  if (e != cudaSuccess) return e;
  kern<<<(unsigned)grid, NT, SMEM, st>>>(maps, p);
  return cudaGetLastError();
}

}  // namespace sfg
