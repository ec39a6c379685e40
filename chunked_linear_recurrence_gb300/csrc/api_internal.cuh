// api_internal.cuh -- error reporting and trace ranges shared by the C-ABI translation units.
#pragma once
#if __has_include(<nvtx3/nvToolsExt.h>)
#include <nvtx3/nvToolsExt.h>
#define SF_HAVE_NVTX 1
#endif

#include "../../include/sf_gdn.h"

namespace sfg {
// Records a printf-style message as the calling thread's sf_last_error() and returns s.
sf_status report(sf_status s, const char* fmt, ...);

// An NVTX range around each compute entry point, so that timelines (Nsight Systems, ncu's
// range filters) show the library's calls; without a tool attached it does nothing.
// (Without the NVTX headers it compiles to nothing.)
struct Range {
#ifdef SF_HAVE_NVTX
  explicit Range(const char* name) { nvtxRangePushA(name); }
  ~Range() { nvtxRangePop(); }
#else
  explicit Range(const char*) {}
#endif
  Range(const Range&) = delete;
  Range& operator=(const Range&) = delete;
};
}  // namespace sfg
