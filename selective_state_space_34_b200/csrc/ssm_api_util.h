// ssm_api_util.h -- host helpers of the extern "C" entry points: NVTX ranges and argument checks.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <nvtx3/nvToolsExt.h>

#include "../../include/ssm_scan.h"

namespace {

// An NVTX range named after the entry point around its host work and launches, so a profiler's
// timeline groups each call's kernels under the API call that issued them. Header-only NVTX v3:
// without an attached tool a push or pop is one predictable branch.
struct NvtxRange {
  explicit NvtxRange(const char *name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
};
#define SSM_RANGE(name) NvtxRange ssm_nvtx_range_(name)

[[maybe_unused]] size_t dtype_size(int32_t dt) { return dt == SSM_BF16 ? 2 : 4; }
[[maybe_unused]] bool dtype_ok(int32_t dt) { return dt == SSM_F32 || dt == SSM_BF16; }
[[maybe_unused]] bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

[[maybe_unused]] bool mul_ok(int64_t a, int64_t b, int64_t *out) {
  if (a < 0 || b < 0) return false;
  if (a != 0 && b > INT64_MAX / a) return false;
  *out = a * b;
  return true;
}

}  // namespace
