// linattn_api.cu -- the C ABI of include/sf_linattn.h: argument checks, workspace layout and
// dispatch.  No entry point allocates memory or synchronises the host.
#include <cmath>
#include <initializer_list>

#include "../../include/sf_linattn.h"
#include "api_checks.cuh"
#include "api_internal.cuh"
#include "linattn.cuh"
#include "simt_chunk.cuh"
#include "tmap.cuh"

using sfg::aligned16;
using sfg::check_heads;
using sfg::cuda_status;
using sfg::eff_hk;
using sfg::eff_scale;
using sfg::report;

namespace {

constexpr size_t kStatusBytes = 256;
thread_local int g_tries = 0;   // sf_testing_inject_linattn_timeout
constexpr int kSms = 152;   // the segment rule's machine: workspace sizes do not ask the device

size_t round_up(size_t x) { return (x + 255) & ~(size_t)255; }

sf_status check_tokens(const sf_gdn_shape* s, bool packed, const char* fn) {
  const sf_status st = check_heads(s, fn);
  if (st != SF_OK) return st;
  if (s->B < 1 || s->T < 0)
    return report(SF_ERR_INVALID_ARG, "%s: need B>=1, T>=0 (got B=%d T=%d)", fn, s->B, s->T);
  const long long elems = (long long)s->B * s->T * s->H * s->K;
  if (elems >= (1LL << 31))
    return report(SF_ERR_UNSUPPORTED, "%s: tensors need int64 element offsets (%lld elements)", fn,
                  elems);
  if (packed) {
    if (s->B != 1) return report(SF_ERR_INVALID_ARG, "%s: cu_seqlens requires B == 1", fn);
    if (s->N < 1) return report(SF_ERR_INVALID_ARG, "%s: cu_seqlens requires N >= 1", fn);
  } else if (s->N != s->B) {
    return report(SF_ERR_INVALID_ARG, "%s: without cu_seqlens N must equal B (N=%d B=%d)", fn, s->N,
                  s->B);
  }
  return SF_OK;
}

// BF16 runs on the tensor-core kernel alone, which needs TMA descriptors.
sf_status check_encoder(const sf_gdn_shape* s, const char* fn) {
  if (s->dtype == SF_BF16 && s->T > 0 && !sfg::tc_fwd_available())
    return report(SF_ERR_UNSUPPORTED,
                  "%s: BF16 needs the tensor-core kernel, but the driver entry "
                  "point cuTensorMapEncodeTiled is unavailable (or disabled by "
                  "SF_GDN_DISABLE_TMA_ENCODER)", fn);
  return SF_OK;
}

// How a launch's walks are cut (linattn.cuh): whole, or into segments whose entry states a
// state-only launch over pieces computes first.
//
// The times are a model of the kernels in microseconds for a 64-row chunk: `t0` a CTA's start
// and end, `walk` and `state` a chunk of the two launches with every SM busy, `walk1` and
// `state1` the same with few CTAs (bound by the chunk's own chain of steps).  `least`: chunks of
// the shortest piece.  The constants only have to order the cuts.  Measured, chunks of a segment
// / of a piece, tcgen05 kernel at D = 128: 24 walks of 300 chunks 50/50 128 us (chosen), 60/60
// 140, 43/43 173, whole 378; 64 walks of 64 chunks 32/16 79 us (chosen), 32/32 85, 16/16 103,
// whole 94; 96 walks of 128 chunks whole 169 us (chosen), 64/64 228; 2 walks of 21 chunks 2/2
// 19.5 us (chosen), 4/4 21.5, whole 38.9.  CUDA-core kernel: 32 walks of 32 chunks at D = 128 16/8
// 245 us (chosen), 8/8 284, 16/16 276; at D = 64 4/4 95 us (chosen), 8/8 110.
struct Cost {
  double slots, t0, walk, walk1, state, state1;
  int least;
};
constexpr Cost kTc128 = {kSms, 4.5, 1.55, 1.35, 0.92, 0.80, 2};
constexpr Cost kTc64 = {kSms, 4.5, 1.20, 1.10, 0.70, 0.65, 2};
// The CUDA-core kernel (one CTA an SM at D = 128, two at 64).
constexpr Cost kSimt128 = {kSms, 4.0, 17.0, 17.0, 6.0, 6.0, 1};
constexpr Cost kSimt64 = {2 * kSms, 4.0, 12.0, 9.0, 5.0, 4.0, 1};

double launch_time(const Cost& c, double ctas, double chunks, bool state) {
  const double busy = ctas < c.slots ? ctas / c.slots : 1.0;
  const double full = state ? c.state : c.walk, few = state ? c.state1 : c.walk1;
  const double per = full * busy > few ? full * busy : few;
  return std::ceil(ctas / c.slots) * (c.t0 + chunks * per);
}

struct Cut {
  int seg, pre;   // rows
};

Cut cut_walks(const sf_gdn_shape* s, bool packed, int npass) {
  const bool tc = s->dtype == SF_BF16;
  const Cost c = tc ? (s->K == 128 ? kTc128 : kTc64) : s->K == 128 ? kSimt128 : kSimt64;
  const int lanes = npass * (tc ? 1 : s->K / 64);            // CTAs of a (sequence, head) walk
  const int64_t chunks = (s->T + 63) / 64;
  const Cut whole = {(int)((chunks > 0 ? chunks : 1) * 64), (int)((chunks > 0 ? chunks : 1) * 64)};
  if (chunks < 2 * c.least) return whole;
  if (packed) {
    // Lengths are on the device; `share` chunks a CTA slot would be even.  With fewer walks than
    // slots nearly all of them are cut and their pieces fill the machine; with more, few are,
    // and smaller pieces spread them.  Measured on the tcgen05 kernel, 65536 tokens, mean of three
    // draws of ragged lengths (1.1 share, 1.2 share in 3 pieces, whole): 5 sequences of 16 heads
    // 266, 309, 508 us; 8 of 32 heads 415, 375, 383 us, with half of the tokens in one of them
    // 480, 390, 635 us.
    const double share = (double)chunks * s->H * lanes / c.slots;
    const double walks = (double)s->N * s->H * lanes;
    const bool many = walks >= c.slots;
    const int k = many ? 3 : 1;
    int64_t seg = (int64_t)std::ceil(share * (many ? 1.2 : 1.1));
    // Short segments only where few walks leave most SMs idle.  Measured, segments of at least 2,
    // 3, 6 chunks: 700 tokens in 2 of 2 heads 17.4, 19.5, 23.6 us, in 5 of 4 23.6, 19.6, 21.5, in
    // 5 of 16 27.6, 27.6, 23.6.
    const int64_t least = !tc ? k : many ? 12 : walks > 32 ? 6 : walks > 16 ? 3 : 2;
    if (seg < least) seg = least;
    seg = (seg + k - 1) / k * k;
    if (seg >= chunks) return whole;
    return {(int)seg * 64, (int)(seg / k) * 64};
  }
  const double walks = (double)s->N * s->H * lanes;
  double best = launch_time(c, walks, (double)chunks, false);
  Cut cut = whole;
  for (int S = 2; S <= 128; ++S) {
    for (int k = 1; k <= 4; ++k) {
      int64_t seg = (chunks + S - 1) / S;
      seg = (seg + k - 1) / k * k;
      if (seg / k < c.least || (S - 1) * seg >= chunks) continue;
      const double units = walks * S, pieces = walks * (S - 1) * k;
      const double t = launch_time(c, units, (double)seg, false) +
                       launch_time(c, pieces, (double)(seg / k), true) + 2.0 +
                       (units + pieces) * s->K * s->K * 4.0 / 5e6;
      if (t < best) {
        best = t;
        cut = {(int)seg * 64, (int)(seg / k) * 64};
      }
    }
  }
  return cut;
}

struct Layout {
  Cut cut;
  int64_t units, pre_units, entries;
  size_t entry, sums, gqa, total;   // segment states of one pass; one FP32 [B,T,H,K] area
};

Layout layout(const sf_gdn_shape* s, bool packed, int npass) {
  Layout l{{64, 64}, 0, 0, 0, 0, 0, 0, kStatusBytes};
  if (!s || s->K < 1 || s->V < 1 || s->H < 1 || s->T < 0 || s->N < 1) return l;
  l.cut = cut_walks(s, packed, npass);
  l.units = sfg::la_units(s->T, s->N, packed, l.cut.seg);
  if (l.cut.seg < s->T) {
    l.pre_units = sfg::la_pre_units(s->T, s->N, packed, l.cut.seg, l.cut.pre);
    const size_t state = (size_t)s->H * s->K * s->V * sizeof(float);
    l.entries = sfg::la_entries(s->T, s->N, packed, l.cut.seg);
    l.entry = round_up(l.entries * state);
    l.sums = round_up(l.pre_units * state);
  }
  if (npass > 1 && eff_hk(s) < s->H)
    l.gqa = round_up((size_t)s->B * s->T * s->H * s->K * sizeof(float));
  l.total = kStatusBytes + npass * (l.entry + l.sums) + 2 * l.gqa;
  return l;
}

cudaError_t run_passes(sfg::LaParams& p, const Layout& l, char* ws, bool bf16, int D,
                       cudaStream_t cs) {
  p.seg = l.cut.seg;
  p.pre = l.cut.pre;
  p.per_seg = p.seg / p.pre;
  p.cuts = p.T > p.seg ? (p.T + p.seg - 1) / p.seg : 1;
  int hk = p.H;
  for (int i = 0; i < p.npass; ++i)
    for (const int n : {p.pass[i].hx, p.pass[i].hy, p.pass[i].hz}) hk = n < hk ? n : hk;
  p.by_pass = sfg::FastDiv::of(p.npass);
  p.by_head = sfg::FastDiv::of(p.H);
  p.by_group = sfg::FastDiv::of(p.H / hk);
  p.by_n = sfg::FastDiv::of(p.N);
  p.by_seg = sfg::FastDiv::of(p.seg);
  p.by_pieces = sfg::FastDiv::of(p.cuts > 1 ? (p.cuts - 1) * p.per_seg : 1);
  p.units = (int)l.units;
  p.pre_units = (int)l.pre_units;
  p.entries = (int)l.entries;
  p.status = reinterpret_cast<int*>(ws);
  for (int i = 0; i < p.npass; ++i) {
    p.pass[i].entry = reinterpret_cast<float*>(ws + kStatusBytes + i * (l.entry + l.sums));
    p.pass[i].sums = p.pass[i].entry + l.entry / sizeof(float);
  }
  // (T = 0: no token is read or written, only the states move; the FP32 kernel does)
  const bool tc = bf16 && p.T > 0;
  if (tc) {
    p.tries = g_tries;
    g_tries = 0;
  }
  auto walk = [&](bool state_only) {
    return tc ? sfg::launch_la_tc(p, D, state_only, cs) : sfg::launch_la_simt(p, D, state_only, cs);
  };
  cudaError_t e = cudaSuccess;
  if (l.pre_units > 0) {
    e = walk(true);
    if (e == cudaSuccess) e = sfg::launch_la_carry(p, D, cs);
  }
  if (e == cudaSuccess) e = walk(false);
  return e;
}

sf_status chunk_fwd(const char* fn, const sf_gdn_shape* shape, const void* q, const void* k,
                    const void* v, const float* decay, const float* initial_state,
                    const int32_t* cu, float* final_state, void* out, float* pool, int num_slots,
                    const int32_t* idx, const uint8_t* has, void* workspace, size_t ws_bytes,
                    sf_stream_t stream) {
  const bool packed = cu != nullptr;
  const sf_status st = check_tokens(shape, packed, fn);
  if (st != SF_OK) return st;
  if (!decay) return report(SF_ERR_INVALID_ARG, "%s: decay must be non-NULL", fn);
  if (shape->T > 0 && (!q || !k || !v || !out))
    return report(SF_ERR_INVALID_ARG, "%s: q, k, v and out must be non-NULL", fn);
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) ||
      !aligned16(initial_state) || !aligned16(final_state))
    return report(SF_ERR_INVALID_ARG, "%s: q, k, v, out and states must be 16-byte aligned", fn);
  const Layout l = layout(shape, packed, 1);
  if (!workspace || !aligned16(workspace) || ws_bytes < l.total)
    return report(SF_ERR_WORKSPACE, "%s: workspace needs %zu bytes, 16-byte aligned", fn, l.total);
  const sf_status enc = check_encoder(shape, fn);
  if (enc != SF_OK) return enc;
  sfg::LaParams p{};
  p.npass = 1;
  p.decay = decay;
  p.cu = cu;
  p.pool = pool; p.state_idx = idx; p.has_init = has; p.num_slots = num_slots;
  p.B = shape->B; p.T = shape->T; p.H = shape->H; p.N = shape->N;
  const float sc = eff_scale(shape);
  const int hk = eff_hk(shape);
  p.pass[0] = sfg::LaPass{q, k, v, out, initial_state, final_state, nullptr, nullptr, hk, hk, shape->H,
                          0, 0, 0, sc, sc, 1.f};
  return cuda_status(run_passes(p, l, static_cast<char*>(workspace), shape->dtype == SF_BF16,
                                shape->K, reinterpret_cast<cudaStream_t>(stream)), fn);
}

sf_status step(const char* fn, const sf_gdn_shape* s, const void* q, const void* k, const void* v,
               const float* decay, const float* gate, const float* beta, float* pool, int num_slots,
               const int32_t* idx, void* out, sf_stream_t stream) {
  const sf_status st = check_heads(s, fn);
  if (st != SF_OK) return st;
  if (s->N < 0 || num_slots < 0 || (!idx && num_slots < s->N))
    return report(SF_ERR_INVALID_ARG,
                  "%s: need N >= 0 and, without state_indices, num_slots >= N (N=%d num_slots=%d)",
                  fn, s->N, num_slots);
  if (s->N == 0) return SF_OK;
  if (!q || !k || !v || !out || !pool || (!decay && (!gate || !beta)))
    return report(SF_ERR_INVALID_ARG, "%s: inputs, state_cache and out must be non-NULL", fn);
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) || !aligned16(pool))
    return report(SF_ERR_INVALID_ARG, "%s: q, k, v, out and state_cache must be 16-byte aligned", fn);
  if ((long long)s->N * s->H * (s->K / 64) > 0x7fffffffLL)
    return report(SF_ERR_UNSUPPORTED, "%s: N * H is too large for one launch", fn);
  sfg::StepParams p{};
  p.q = q; p.k = k; p.v = v; p.decay = decay; p.gate = gate; p.beta = beta; p.pool = pool;
  p.idx = idx; p.out = out; p.N = s->N; p.H = s->H; p.HK = eff_hk(s); p.num_slots = num_slots;
  p.scale = eff_scale(s);
  return cuda_status(sfg::launch_state_step(p, s->dtype == SF_BF16, s->K,
                                            reinterpret_cast<cudaStream_t>(stream)), fn);
}

sf_status check_qk(const sf_qk_shape* s, const void* q, const void* k, const float* qw,
                   const float* kw, const float* cs, const int32_t* pos, const char* fn,
                   sfg::QkParams& p) {
  if (!s) return report(SF_ERR_INVALID_ARG, "%s: shape is NULL", fn);
  if (s->rows < 0 || s->H < 1 || s->HK < 1)
    return report(SF_ERR_INVALID_ARG, "%s: need rows>=0, H>=1, HK>=1", fn);
  if (s->dtype != SF_F32 && s->dtype != SF_BF16)
    return report(SF_ERR_INVALID_ARG, "%s: dtype must be SF_F32 or SF_BF16", fn);
  if (s->norm != SF_NORM_RMS && s->norm != SF_NORM_L2)
    return report(SF_ERR_INVALID_ARG, "%s: norm must be SF_NORM_RMS or SF_NORM_L2", fn);
  if (!(s->eps >= 0.f)) return report(SF_ERR_INVALID_ARG, "%s: eps must be >= 0", fn);
  if (s->D != 64 && s->D != 128)
    return report(SF_ERR_UNSUPPORTED, "%s: head size 64 or 128 only (got %d)", fn, s->D);
  if (s->rotary_dim < 0 || s->rotary_dim > s->D || s->rotary_dim % 8)
    return report(SF_ERR_UNSUPPORTED, "%s: rotary_dim must be a multiple of 8 in [0, D] (got %d)",
                  fn, s->rotary_dim);
  const int el = s->dtype == SF_BF16 ? 8 : 4;   // elements of 16 bytes
  if (s->rows_stride_q % el || s->rows_stride_k % el ||
      s->rows_stride_q < (int64_t)s->H * s->D || s->rows_stride_k < (int64_t)s->HK * s->D)
    return report(SF_ERR_INVALID_ARG,
                  "%s: token strides must be multiples of 16 bytes and hold every head", fn);
  if (s->rows > 0 && (!q || !k)) return report(SF_ERR_INVALID_ARG, "%s: q and k must be non-NULL", fn);
  if (!aligned16(q) || !aligned16(k) || !aligned16(qw) || !aligned16(kw) || !aligned16(cs))
    return report(SF_ERR_INVALID_ARG, "%s: q, k, weights and cos_sin must be 16-byte aligned", fn);
  p.axes = 1;
  p.bound[0] = 0;
  if (s->rotary_dim > 0) {
    if (s->axes < 1 || s->axes > 4)
      return report(SF_ERR_INVALID_ARG, "%s: 1 to 4 position axes (got %d)", fn, s->axes);
    int sum = 0;
    for (int a = 0; a < s->axes; ++a) {
      if (s->sections[a] < 0)
        return report(SF_ERR_INVALID_ARG, "%s: sections[%d] = %d is negative", fn, a, s->sections[a]);
      p.bound[a] = sum += s->sections[a];
    }
    if (sum != s->rotary_dim / 2)
      return report(SF_ERR_INVALID_ARG, "%s: sections sum to %d, rotary_dim / 2 is %d", fn, sum,
                    s->rotary_dim / 2);
    if (s->table_rows < 1 || !cs || (s->rows > 0 && !pos))
      return report(SF_ERR_INVALID_ARG, "%s: cos_sin (table_rows >= 1) and positions needed", fn);
    p.axes = s->axes;
  }
  p.q = q; p.k = k; p.qw = qw; p.kw = kw; p.cs = cs; p.pos = pos;
  p.rows = s->rows; p.sq = s->rows_stride_q; p.sk = s->rows_stride_k;
  p.H = s->H; p.HK = s->HK; p.half = s->rotary_dim / 2; p.inter = s->interleaved != 0;
  p.table_rows = s->table_rows; p.l2 = s->norm == SF_NORM_L2; p.eps = s->eps;
  return SF_OK;
}

}  // namespace

extern "C" {

size_t sf_linattn_fwd_workspace(const sf_gdn_shape* shape, int packed) {
  return layout(shape, packed != 0, 1).total;
}

sf_status sf_linattn_chunk_fwd(const sf_gdn_shape* shape, const void* q, const void* k,
                               const void* v, const float* decay, const float* initial_state,
                               const int32_t* cu_seqlens, int output_final_state, void* out,
                               float* final_state, void* workspace, size_t ws_bytes,
                               sf_stream_t stream) {
  const char* fn = "sf_linattn_chunk_fwd";
  const sfg::Range range(fn);
  if (output_final_state && !final_state)
    return report(SF_ERR_INVALID_ARG, "%s: output_final_state requires final_state", fn);
  return chunk_fwd(fn, shape, q, k, v, decay, initial_state, cu_seqlens,
                   output_final_state ? final_state : nullptr, out, nullptr, 0, nullptr, nullptr,
                   workspace, ws_bytes, stream);
}

sf_status sf_linattn_paged_chunk_fwd(const sf_gdn_shape* shape, const void* q, const void* k,
                                     const void* v, const float* decay, float* state_cache,
                                     int num_slots, const int32_t* state_indices,
                                     const uint8_t* has_initial_state, const int32_t* cu_seqlens,
                                     void* out, void* workspace, size_t ws_bytes,
                                     sf_stream_t stream) {
  const char* fn = "sf_linattn_paged_chunk_fwd";
  const sfg::Range range(fn);
  if (!state_cache || !state_indices || num_slots < 1)
    return report(SF_ERR_INVALID_ARG, "%s: state_cache, state_indices and num_slots >= 1 needed", fn);
  if (!aligned16(state_cache))
    return report(SF_ERR_INVALID_ARG, "%s: state_cache must be 16-byte aligned", fn);
  return chunk_fwd(fn, shape, q, k, v, decay, nullptr, cu_seqlens, nullptr, out, state_cache,
                   num_slots, state_indices, has_initial_state, workspace, ws_bytes, stream);
}

size_t sf_linattn_bwd_workspace(const sf_gdn_shape* shape, int packed) {
  return layout(shape, packed != 0, 3).total;
}

sf_status sf_linattn_chunk_bwd(const sf_gdn_shape* shape, const void* q, const void* k,
                               const void* v, const float* decay, const float* initial_state,
                               const int32_t* cu_seqlens, const void* d_out,
                               const float* d_final_state, void* dq, void* dk, void* dv,
                               float* d_initial_state, void* workspace, size_t ws_bytes,
                               sf_stream_t stream) {
  const char* fn = "sf_linattn_chunk_bwd";
  const sfg::Range range(fn);
  const bool packed = cu_seqlens != nullptr;
  const sf_status st = check_tokens(shape, packed, fn);
  if (st != SF_OK) return st;
  if (!decay) return report(SF_ERR_INVALID_ARG, "%s: decay must be non-NULL", fn);
  if (shape->T > 0 && (!q || !k || !v || !d_out || !dq || !dk || !dv))
    return report(SF_ERR_INVALID_ARG, "%s: inputs and gradient outputs must be non-NULL", fn);
  const void* al[] = {q, k, v, d_out, dq, dk, dv, initial_state, d_final_state, d_initial_state};
  for (const void* a : al)
    if (!aligned16(a))
      return report(SF_ERR_INVALID_ARG, "%s: tensors must be 16-byte aligned", fn);
  const Layout l = layout(shape, packed, 3);
  if (!workspace || !aligned16(workspace) || ws_bytes < l.total)
    return report(SF_ERR_WORKSPACE, "%s: workspace needs %zu bytes, 16-byte aligned", fn, l.total);
  const sf_status enc = check_encoder(shape, fn);
  if (enc != SF_OK) return enc;
  char* ws = static_cast<char*>(workspace);
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  const bool bf16 = shape->dtype == SF_BF16;
  sfg::LaParams p{};
  p.npass = 3;
  p.decay = decay;
  p.cu = cu_seqlens;
  p.B = shape->B; p.T = shape->T; p.H = shape->H; p.N = shape->N;
  const float sc = eff_scale(shape);
  const int hk = eff_hk(shape), H = shape->H;
  float* gq = nullptr;
  float* gk = nullptr;
  if (l.gqa) {   // per-value-head parts in FP32, summed below
    gq = reinterpret_cast<float*>(ws + kStatusBytes + 3 * (l.entry + l.sums));
    gk = reinterpret_cast<float*>(ws + kStatusBytes + 3 * (l.entry + l.sums) + l.gqa);
  }
  const int f32 = gq != nullptr;
  p.pass[0] = sfg::LaPass{d_out, v, k, f32 ? gq : dq, initial_state, nullptr, nullptr, nullptr, H, H, hk,
                          1, f32, 0, sc, sc, 1.f};
  p.pass[1] = sfg::LaPass{k, q, d_out, dv, d_final_state, d_initial_state, nullptr, nullptr, hk, hk, H,
                          0, 0, 1, sc, 1.f, sc};
  p.pass[2] = sfg::LaPass{v, d_out, q, f32 ? gk : dk, d_final_state, nullptr, nullptr, nullptr, H, H, hk,
                          1, f32, 1, sc, 1.f, sc};
  cudaError_t e = run_passes(p, l, ws, bf16, shape->K, cs);
  if (e == cudaSuccess && f32) {
    const int64_t rows = (int64_t)shape->B * shape->T;
    e = sfg::launch_group_sum(gq, gk, dq, dk, bf16, rows, H, hk, shape->K, cu_seqlens, shape->N, cs,
                              true);
  }
  return cuda_status(e, fn);
}

sf_status sf_testing_inject_linattn_timeout(int tries) {
  if (tries < 1 || tries > 10000)
    return report(SF_ERR_INVALID_ARG, "sf_testing_inject_linattn_timeout: need 1 <= tries <= 10000");
  g_tries = tries;
  return SF_OK;
}

sf_status sf_linattn_step(const sf_gdn_shape* shape, const void* q, const void* k, const void* v,
                          const float* decay, float* state_cache, int num_slots,
                          const int32_t* state_indices, void* out, sf_stream_t stream) {
  const char* fn = "sf_linattn_step";
  const sfg::Range range(fn);
  if (!decay) return report(SF_ERR_INVALID_ARG, "%s: decay must be non-NULL", fn);
  return step(fn, shape, q, k, v, decay, nullptr, nullptr, state_cache, num_slots, state_indices,
              out, stream);
}

sf_status sf_gdn_step(const sf_gdn_shape* shape, const void* q, const void* k, const void* v,
                      const float* gate, const float* beta, float* state_cache, int num_slots,
                      const int32_t* state_indices, void* out, sf_stream_t stream) {
  const char* fn = "sf_gdn_step";
  const sfg::Range range(fn);
  return step(fn, shape, q, k, v, nullptr, gate, beta, state_cache, num_slots, state_indices, out,
              stream);
}

sf_status sf_qk_norm_rope_fwd(const sf_qk_shape* shape, const void* q, const void* k,
                              const float* q_weight, const float* k_weight, const float* cos_sin,
                              const int32_t* positions, void* q_out, void* k_out,
                              sf_stream_t stream) {
  const char* fn = "sf_qk_norm_rope_fwd";
  const sfg::Range range(fn);
  sfg::QkParams p{};
  const sf_status st = check_qk(shape, q, k, q_weight, k_weight, cos_sin, positions, fn, p);
  if (st != SF_OK) return st;
  if (shape->rows == 0) return SF_OK;
  if (!q_out || !k_out || !aligned16(q_out) || !aligned16(k_out))
    return report(SF_ERR_INVALID_ARG, "%s: q_out and k_out must be non-NULL, 16-byte aligned", fn);
  if ((q_out == q && shape->rows_stride_q != (int64_t)shape->H * shape->D) ||
      (k_out == k && shape->rows_stride_k != (int64_t)shape->HK * shape->D))
    return report(SF_ERR_INVALID_ARG, "%s: in place needs contiguous q and k", fn);
  p.q_out = q_out;
  p.k_out = k_out;
  return cuda_status(sfg::launch_qk_norm_rope(p, shape->dtype == SF_BF16, shape->D,
                                              reinterpret_cast<cudaStream_t>(stream)), fn);
}

size_t sf_qk_norm_rope_bwd_workspace(const sf_qk_shape* shape) {
  // sums of at most sfg::QK_PARTS CTAs, whatever the device has
  if (!shape || shape->D < 1) return 256;
  return (size_t)sfg::QK_PARTS * shape->D * sizeof(float);
}

sf_status sf_qk_norm_rope_bwd(const sf_qk_shape* shape, const void* q, const void* k,
                              const float* q_weight, const float* k_weight, const float* cos_sin,
                              const int32_t* positions, const void* d_q_out, const void* d_k_out,
                              void* dq, void* dk, float* dq_weight, float* dk_weight,
                              void* workspace, size_t ws_bytes, sf_stream_t stream) {
  const char* fn = "sf_qk_norm_rope_bwd";
  const sfg::Range range(fn);
  sfg::QkParams p{};
  const sf_status st = check_qk(shape, q, k, q_weight, k_weight, cos_sin, positions, fn, p);
  if (st != SF_OK) return st;
  if (shape->rows > 0 && (!d_q_out || !d_k_out || !dq || !dk))
    return report(SF_ERR_INVALID_ARG, "%s: cotangents and gradients must be non-NULL", fn);
  if (!aligned16(d_q_out) || !aligned16(d_k_out) || !aligned16(dq) || !aligned16(dk))
    return report(SF_ERR_INVALID_ARG, "%s: cotangents and gradients must be 16-byte aligned", fn);
  const bool weights = dq_weight || dk_weight;
  if (weights && (!workspace || !aligned16(workspace) || ws_bytes < sf_qk_norm_rope_bwd_workspace(shape)))
    return report(SF_ERR_WORKSPACE, "%s: workspace needs %zu bytes, 16-byte aligned", fn,
                  sf_qk_norm_rope_bwd_workspace(shape));
  p.q_out = dq;
  p.k_out = dk;
  p.dqo = d_q_out;
  p.dko = d_k_out;
  p.part = weights ? static_cast<float*>(workspace) : nullptr;
  return cuda_status(sfg::launch_qk_norm_rope_bwd(p, shape->dtype == SF_BF16, shape->D, dq_weight,
                                                  dk_weight, reinterpret_cast<cudaStream_t>(stream)),
                     fn);
}

}  // extern "C"
