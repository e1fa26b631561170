// Checks of arguments that the entry points beside the collectives share. Each fails with
// the status and text that the entry point returns.
#pragma once

#include <cstdint>
#include <string>

#include "ccl_internal.h"

namespace ccl {

inline void require(bool ok, const char* what) {
  if (!ok) fail(CCL_ERR_INVALID_ARGUMENT, what);
}

constexpr int64_t kMaxFeatures = int64_t(1) << 20, kMaxLd = int64_t(1) << 22;

inline int elem_size(int dtype) {
  if (dtype == CCL_F32) return 4;
  if (dtype == CCL_BF16) return 2;
  fail(CCL_ERR_UNSUPPORTED, "products take fp32 and bf16");
}

inline int64_t stride_of(int64_t ld, int64_t width, const char* name) {
  if (ld == 0) return width;
  if (ld < width || ld > kMaxLd) fail(CCL_ERR_INVALID_ARGUMENT, std::string(name) + ": a row stride below the row's length or above 2^22");
  return ld;
}

inline int64_t align16(int64_t bytes) { return (bytes + 15) / 16 * 16; }

inline void check_workspace(const void* ws, size_t have, int64_t need) {
  if (need == 0) return;
  if (!ws || int64_t(have) < need)
    fail(CCL_ERR_INVALID_ARGUMENT, "workspace: " + std::to_string(need) + " bytes needed, " + std::to_string(have) + " given");
  require(reinterpret_cast<uintptr_t>(ws) % 16 == 0, "workspace: not 16-byte aligned");
}

inline void launched(int rc, const std::string& err) {
  if (rc) fail(rc, err);
}

inline void elements(int size, const void* p, const char* name) {
  require(p != nullptr, name);
  require(reinterpret_cast<uintptr_t>(p) % size == 0, name);
}

}  // namespace ccl
