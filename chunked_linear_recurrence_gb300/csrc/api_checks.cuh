// api_checks.cuh -- argument checks that the translation units of the C ABI share.
#pragma once
#include <cmath>

#include <cuda_runtime.h>

#include "api_internal.cuh"

namespace sfg {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline sf_status cuda_status(cudaError_t e, const char* fn) {
  return e == cudaSuccess ? SF_OK : report(SF_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(e));
}

inline int eff_hk(const sf_gdn_shape* s) { return s->HK > 0 ? s->HK : s->H; }
inline float eff_scale(const sf_gdn_shape* s) {
  return s->scale > 0.f ? s->scale : 1.0f / std::sqrt((float)s->K);
}

// Head counts, head size and type: what the token streams and the steps share.
inline sf_status check_heads(const sf_gdn_shape* s, const char* fn) {
  if (!s) return report(SF_ERR_INVALID_ARG, "%s: shape is NULL", fn);
  if (s->H < 1 || s->K < 1 || s->V < 1)
    return report(SF_ERR_INVALID_ARG, "%s: need H>=1, K>=1, V>=1 (got H=%d K=%d V=%d)", fn, s->H,
                  s->K, s->V);
  if (s->dtype != SF_F32 && s->dtype != SF_BF16)
    return report(SF_ERR_INVALID_ARG, "%s: dtype must be SF_F32 or SF_BF16", fn);
  if (s->HK < 0 || s->H % (s->HK > 0 ? s->HK : s->H))
    return report(SF_ERR_INVALID_ARG, "%s: query/key heads HK = %d must divide H = %d", fn, s->HK,
                  s->H);
  if (s->K != s->V || (s->K != 64 && s->K != 128))
    return report(SF_ERR_UNSUPPORTED, "%s: head sizes K == V in {64, 128} only (got K=%d V=%d)", fn,
                  s->K, s->V);
  return SF_OK;
}

}  // namespace sfg
