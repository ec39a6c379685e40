// decode.cuh -- launches of the operators of include/sf_decode.h.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "linattn.cuh"

namespace sfg {

constexpr int DRAFT_MAX = 32;

// Tokens of every sequence: the first num[n] of `rows` (clamped; NULL: all of them).
struct DraftTokens {
  const void* q;        // NULL for pending tokens
  const void* k;
  const void* v;
  const float* gate;    // delta rule
  const float* beta;
  const int32_t* num;
  int rows;
};
struct DraftParams {
  DraftTokens pend, fresh;
  const float* decay;   // [H] (linear attention), or NULL
  float* pool;
  const int32_t* idx;   // [N] or NULL
  void* out;
  int N, H, HK, num_slots;
  int run;                      // strips of a head that a warp takes in a row
  FastDiv by_head, by_group;    // of H, H / HK
  float scale;
};
cudaError_t launch_draft_step(const DraftParams& p, bool bf16, int D, cudaStream_t st);

struct VerifyParams {
  const void* target;
  const void* draft;    // or NULL
  const int32_t* x;
  const float* u;
  const int32_t* num;   // or NULL
  int32_t* tokens;
  int32_t* count;
  int N, T, V;
  int64_t target_seq, target_row, draft_seq, draft_row;
  bool give_up;         // failure-detection testing: the first CTA of a sequence gives up its wait at once
};
cudaError_t launch_draft_verify(const VerifyParams& p, bool bf16, cudaStream_t st);

constexpr int MAX_SLOTS = 1 << 18;

struct PoolPlan {
  const int32_t* idx;
  const int32_t* parents;     // of a fork; NULL: compaction
  const uint8_t* reserved;    // or NULL
  int32_t* out;
  int N, M, num_slots;
  // workspace, or NULL
  int32_t* src;               // [rows] pairs to copy ...
  int32_t* dst;
  int32_t* count;             // ... and how many
  int32_t* first;             // fork: [num_slots]
};
inline bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const char *x = static_cast<const char*>(a), *y = static_cast<const char*>(b);
  return x && y && x < y + nb && y < x + na;
}
// The plan, and its copies in every cache: in one launch that needs no workspace, or, if the plan has
// one, in two.  Some plans need it, others are faster with it.
bool pool_move_needs_workspace(const PoolPlan& plan, int num_caches);
bool pool_move_likes_workspace(const PoolPlan& plan);
cudaError_t launch_pool_move(const PoolPlan& plan, int num_caches, void* const* caches,
                             const size_t* slot_bytes, cudaStream_t st);
// Copies of src[i] to dst[i], i < *count (or rows where count is NULL), in every cache.
cudaError_t launch_pool_copy(int num_slots, int num_caches, void* const* caches,
                             const size_t* slot_bytes, const int32_t* src, const int32_t* dst,
                             const int32_t* count, int rows, cudaStream_t st);

}  // namespace sfg
