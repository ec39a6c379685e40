// decode_api.cu -- the C ABI of include/sf_decode.h: argument checks and dispatch.  No entry
// point allocates memory or synchronises the host.
#include <initializer_list>

#include "../../include/sf_decode.h"
#include "api_checks.cuh"
#include "api_internal.cuh"
#include "decode.cuh"

using sfg::aligned16;
using sfg::check_heads;
using sfg::cuda_status;
using sfg::overlap;
using sfg::report;

namespace {

static_assert(sfg::DRAFT_MAX == SF_DRAFT_MAX && sfg::MAX_SLOTS == SF_MAX_SLOTS, "limits of the header");

thread_local bool g_give_up = false;   // sf_testing_inject_verify_timeout

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
size_t round_up(size_t x) { return (x + 255) & ~(size_t)255; }

// Fresh tokens (q, out) and pending ones, either of them empty.
sf_status draft(const char* fn, const sf_gdn_shape* s, const sfg::DraftTokens& fresh,
                const sfg::DraftTokens& pend, const float* decay, bool delta, float* pool, int num_slots,
                const int32_t* idx, void* out, sf_stream_t stream) {
  const sf_status st = check_heads(s, fn);
  if (st != SF_OK) return st;
  if (s->N < 0 || num_slots < 0 || (!idx && num_slots < s->N))
    return report(SF_ERR_INVALID_ARG,
                  "%s: need N >= 0 and, without state_indices, num_slots >= N (N=%d num_slots=%d)",
                  fn, s->N, num_slots);
  for (const int rows : {fresh.rows, pend.rows}) {
    if (rows < 0) return report(SF_ERR_INVALID_ARG, "%s: a negative number of tokens (%d)", fn, rows);
    if (rows > SF_DRAFT_MAX)
      return report(SF_ERR_UNSUPPORTED, "%s: at most %d tokens of a sequence (got %d)", fn, SF_DRAFT_MAX, rows);
  }
  if (s->N == 0 || (fresh.rows == 0 && pend.rows == 0)) return SF_OK;
  if (!pool || (!delta && !decay))
    return report(SF_ERR_INVALID_ARG, "%s: state_cache%s must be non-NULL", fn, delta ? "" : " and decay");
  if (fresh.rows > 0 && (!fresh.q || !out))
    return report(SF_ERR_INVALID_ARG, "%s: q and out must be non-NULL", fn);
  for (const sfg::DraftTokens* t : {&fresh, &pend}) {
    if (t->rows == 0) continue;
    if (!t->k || !t->v || (delta && (!t->gate || !t->beta)))
      return report(SF_ERR_INVALID_ARG, "%s: k, v%s must be non-NULL", fn, delta ? ", gate and beta" : "");
    if (!aligned16(t->q) || !aligned16(t->k) || !aligned16(t->v))
      return report(SF_ERR_INVALID_ARG, "%s: q, k and v must be 16-byte aligned", fn);
    if (!aligned4(t->gate) || !aligned4(t->beta) || !aligned4(t->num))
      return report(SF_ERR_INVALID_ARG, "%s: gates and counts must be 4-byte aligned", fn);
  }
  if (!aligned16(out) || (reinterpret_cast<uintptr_t>(pool) & 31) || !aligned4(idx) || !aligned4(decay))
    return report(SF_ERR_INVALID_ARG, "%s: out must be 16-byte aligned, state_cache 32-byte", fn);
  if ((long long)s->N * s->H > 1LL << 27)
    return report(SF_ERR_UNSUPPORTED, "%s: N * H is too large for one launch", fn);
  sfg::DraftParams p{};
  p.fresh = fresh; p.pend = pend; p.decay = delta ? nullptr : decay; p.pool = pool; p.idx = idx; p.out = out;
  p.N = s->N; p.H = s->H; p.HK = sfg::eff_hk(s);
  p.by_head = sfg::FastDiv::of(p.H); p.by_group = sfg::FastDiv::of(p.H / p.HK);
  p.num_slots = num_slots; p.scale = sfg::eff_scale(s);
  return cuda_status(sfg::launch_draft_step(p, s->dtype == SF_BF16, s->K, reinterpret_cast<cudaStream_t>(stream)),
                     fn);
}

sfg::DraftTokens tokens_of(const sf_pending* p) {
  if (!p) return {};
  return {nullptr, p->k, p->v, p->gate, p->beta, p->count, p->P};
}

sf_status check_pool(const sf_state_pool* p, const char* fn) {
  if (!p) return report(SF_ERR_INVALID_ARG, "%s: pool is NULL", fn);
  if (p->num_slots < 1 || p->num_caches < 0 || (p->num_caches > 0 && (!p->caches || !p->slot_bytes)))
    return report(SF_ERR_INVALID_ARG, "%s: need num_slots >= 1 and the caches (num_slots=%d num_caches=%d)", fn,
                  p->num_slots, p->num_caches);
  if (p->num_slots > SF_MAX_SLOTS)
    return report(SF_ERR_UNSUPPORTED, "%s: at most %d slots (got %d)", fn, SF_MAX_SLOTS, p->num_slots);
  for (int c = 0; c < p->num_caches; ++c) {
    if (!p->caches[c] || !aligned16(p->caches[c]) || p->slot_bytes[c] % 16)
      return report(SF_ERR_INVALID_ARG,
                    "%s: cache %d must be non-NULL, 16-byte aligned, its slots a multiple of 16 bytes", fn, c);
    if (p->slot_bytes[c] > (size_t)1 << 38)
      return report(SF_ERR_UNSUPPORTED, "%s: cache %d: a slot of more than 2^38 bytes", fn, c);
  }
  return SF_OK;
}

// A plan over `rows` rows, then the copies it gives.
sf_status planned(const char* fn, const sf_state_pool* pool, sfg::PoolPlan p, int rows, void* ws, size_t ws_bytes,
                  sf_stream_t stream) {
  p.num_slots = pool->num_slots;
  // (a compaction's row is written when its own old index has been read, others' may not have been; a fork
  // reads all indices before, and reserved between its rows)
  const size_t out = (size_t)rows * 4;
  if (p.parents ? overlap(p.out, out, p.reserved, (size_t)p.num_slots)
                : p.out != p.idx && overlap(p.out, out, p.idx, (size_t)p.N * 4))
    return report(SF_ERR_INVALID_ARG, "%s: new_indices overlaps an input that it is not", fn);
  const size_t need = sf_state_workspace(pool->num_slots, rows);
  const bool needs = sfg::pool_move_needs_workspace(p, pool->num_caches), given = ws && aligned16(ws) && ws_bytes >= need;
  if (needs && !given)
    return report(SF_ERR_WORKSPACE, "%s: workspace needs %zu bytes, 16-byte aligned", fn, need);
  if (needs || (given && sfg::pool_move_likes_workspace(p))) {
    char* at = static_cast<char*>(ws);
    p.count = reinterpret_cast<int32_t*>(at);
    p.src = reinterpret_cast<int32_t*>(at + 256);
    p.dst = reinterpret_cast<int32_t*>(at + 256 + round_up((size_t)rows * 4));
    p.first = reinterpret_cast<int32_t*>(at + 256 + 2 * round_up((size_t)rows * 4));
  }
  return cuda_status(sfg::launch_pool_move(p, pool->num_caches, pool->caches, pool->slot_bytes,
                                           reinterpret_cast<cudaStream_t>(stream)), fn);
}

}  // namespace

extern "C" {

sf_status sf_gdn_draft_step(const sf_gdn_shape* shape, const void* q, const void* k, const void* v,
                            const float* gate, const float* beta, const int32_t* num_tokens,
                            const sf_pending* pending, float* state_cache, int num_slots,
                            const int32_t* state_indices, void* out, sf_stream_t stream) {
  const char* fn = "sf_gdn_draft_step";
  const sfg::Range range(fn);
  const int T = shape ? shape->T : 0;
  return draft(fn, shape, {q, k, v, gate, beta, num_tokens, T}, tokens_of(pending), nullptr, true, state_cache,
               num_slots, state_indices, out, stream);
}

sf_status sf_linattn_draft_step(const sf_gdn_shape* shape, const void* q, const void* k,
                                const void* v, const float* decay, const int32_t* num_tokens,
                                const sf_pending* pending, float* state_cache, int num_slots,
                                const int32_t* state_indices, void* out, sf_stream_t stream) {
  const char* fn = "sf_linattn_draft_step";
  const sfg::Range range(fn);
  const int T = shape ? shape->T : 0;
  return draft(fn, shape, {q, k, v, nullptr, nullptr, num_tokens, T}, tokens_of(pending), decay, false, state_cache,
               num_slots, state_indices, out, stream);
}

sf_status sf_gdn_commit(const sf_gdn_shape* shape, const void* k, const void* v, const float* gate,
                        const float* beta, const int32_t* num_tokens, float* state_cache,
                        int num_slots, const int32_t* state_indices, sf_stream_t stream) {
  const char* fn = "sf_gdn_commit";
  const sfg::Range range(fn);
  const int T = shape ? shape->T : 0;
  return draft(fn, shape, {}, {nullptr, k, v, gate, beta, num_tokens, T}, nullptr, true, state_cache, num_slots,
               state_indices, nullptr, stream);
}

sf_status sf_linattn_commit(const sf_gdn_shape* shape, const void* k, const void* v,
                            const float* decay, const int32_t* num_tokens, float* state_cache,
                            int num_slots, const int32_t* state_indices, sf_stream_t stream) {
  const char* fn = "sf_linattn_commit";
  const sfg::Range range(fn);
  const int T = shape ? shape->T : 0;
  return draft(fn, shape, {}, {nullptr, k, v, nullptr, nullptr, num_tokens, T}, decay, false, state_cache, num_slots,
               state_indices, nullptr, stream);
}

sf_status sf_draft_verify(const sf_verify_shape* shape, const void* target_probs,
                          const int32_t* draft_tokens, const float* uniforms,
                          const void* draft_probs, const int32_t* num_drafts, int32_t* tokens,
                          int32_t* num_tokens, sf_stream_t stream) {
  const char* fn = "sf_draft_verify";
  const sfg::Range range(fn);
  if (!shape) return report(SF_ERR_INVALID_ARG, "%s: shape is NULL", fn);
  const sf_verify_shape& s = *shape;
  if (s.dtype != SF_F32 && s.dtype != SF_BF16)
    return report(SF_ERR_INVALID_ARG, "%s: dtype must be SF_F32 or SF_BF16", fn);
  if (s.N < 0 || s.T < 0 || s.V < 1)
    return report(SF_ERR_INVALID_ARG, "%s: need N>=0, T>=0, V>=1 (got N=%d T=%d V=%d)", fn, s.N, s.T, s.V);
  if (s.N > 1 << 24 || s.T > 1 << 20 || s.V > 1 << 30)
    return report(SF_ERR_UNSUPPORTED, "%s: at most 2^24 sequences, 2^20 drafts, 2^30 tokens", fn);
  if (s.target_seq < 0 || s.target_row < 0 || s.draft_seq < 0 || s.draft_row < 0)
    return report(SF_ERR_INVALID_ARG, "%s: strides must not be negative", fn);
  if (s.N == 0) return SF_OK;
  if (!target_probs || !uniforms || !tokens || !num_tokens || (s.T > 0 && !draft_tokens))
    return report(SF_ERR_INVALID_ARG, "%s: inputs and outputs must be non-NULL", fn);
  const uintptr_t el = s.dtype == SF_BF16 ? 1 : 3;
  if ((reinterpret_cast<uintptr_t>(target_probs) & el) || (reinterpret_cast<uintptr_t>(draft_probs) & el) ||
      !aligned4(draft_tokens) || !aligned4(uniforms) || !aligned4(num_drafts) || !aligned4(tokens) ||
      !aligned4(num_tokens))
    return report(SF_ERR_INVALID_ARG, "%s: tensors must be aligned to their elements", fn);
  sfg::VerifyParams p{};
  p.target = target_probs; p.draft = s.T > 0 ? draft_probs : nullptr; p.x = draft_tokens; p.u = uniforms;
  p.num = num_drafts; p.tokens = tokens; p.count = num_tokens;
  p.N = s.N; p.T = s.T; p.V = s.V;
  p.target_seq = s.target_seq; p.target_row = s.target_row;
  p.draft_seq = s.draft_seq; p.draft_row = s.draft_row;
  p.give_up = g_give_up;
  g_give_up = false;
  return cuda_status(sfg::launch_draft_verify(p, s.dtype == SF_BF16, reinterpret_cast<cudaStream_t>(stream)), fn);
}

sf_status sf_testing_inject_verify_timeout(void) {
  g_give_up = true;
  return SF_OK;
}

size_t sf_state_workspace(int num_slots, int rows) {
  if (num_slots < 0 || rows < 0) return 256;
  return 256 + 2 * round_up((size_t)rows * 4) + round_up((size_t)num_slots * 4);
}

sf_status sf_state_copy(const sf_state_pool* pool, const int32_t* src, const int32_t* dst, int M,
                        sf_stream_t stream) {
  const char* fn = "sf_state_copy";
  const sfg::Range range(fn);
  const sf_status st = check_pool(pool, fn);
  if (st != SF_OK) return st;
  if (M < 0) return report(SF_ERR_INVALID_ARG, "%s: need M >= 0 (got %d)", fn, M);
  if (M == 0 || pool->num_caches == 0) return SF_OK;
  if (!src || !dst || !aligned4(src) || !aligned4(dst))
    return report(SF_ERR_INVALID_ARG, "%s: src and dst must be non-NULL, 4-byte aligned", fn);
  return cuda_status(sfg::launch_pool_copy(pool->num_slots, pool->num_caches, pool->caches, pool->slot_bytes, src, dst,
                                           nullptr, M, reinterpret_cast<cudaStream_t>(stream)), fn);
}

sf_status sf_state_fork(const sf_state_pool* pool, const int32_t* state_indices, int N,
                        const int32_t* parents, int M, const uint8_t* reserved,
                        int32_t* new_indices, void* workspace, size_t ws_bytes,
                        sf_stream_t stream) {
  const char* fn = "sf_state_fork";
  const sfg::Range range(fn);
  const sf_status st = check_pool(pool, fn);
  if (st != SF_OK) return st;
  if (N < 0 || M < 0) return report(SF_ERR_INVALID_ARG, "%s: need N >= 0 and M >= 0 (N=%d M=%d)", fn, N, M);
  if (M == 0) return SF_OK;
  if ((N > 0 && !state_indices) || !parents || !new_indices || !aligned4(state_indices) || !aligned4(parents) ||
      !aligned4(new_indices))
    return report(SF_ERR_INVALID_ARG, "%s: indices must be non-NULL, 4-byte aligned", fn);
  sfg::PoolPlan p{};
  p.idx = state_indices; p.N = N; p.parents = parents; p.M = M; p.reserved = reserved; p.out = new_indices;
  return planned(fn, pool, p, M, workspace, ws_bytes, stream);
}

sf_status sf_state_compact(const sf_state_pool* pool, const int32_t* state_indices, int N,
                           const uint8_t* reserved, int32_t* new_indices, void* workspace,
                           size_t ws_bytes, sf_stream_t stream) {
  const char* fn = "sf_state_compact";
  const sfg::Range range(fn);
  const sf_status st = check_pool(pool, fn);
  if (st != SF_OK) return st;
  if (N < 0) return report(SF_ERR_INVALID_ARG, "%s: need N >= 0 (got %d)", fn, N);
  if (N == 0) return SF_OK;
  if (!state_indices || !new_indices || !aligned4(state_indices) || !aligned4(new_indices))
    return report(SF_ERR_INVALID_ARG, "%s: indices must be non-NULL, 4-byte aligned", fn);
  sfg::PoolPlan p{};
  p.idx = state_indices; p.N = N; p.reserved = reserved; p.out = new_indices;
  return planned(fn, pool, p, N, workspace, ws_bytes, stream);
}

}  // extern "C"
