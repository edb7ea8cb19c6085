// Argument checks shared by the C ABI's translation units.
#pragma once
#include "common.cuh"

namespace moe {

inline int check_ptr(const void* p, const char* name, size_t align, bool nullable = false) {
  if (!p) return nullable ? MOE_OK : set_error(MOE_EINVAL, "%s is NULL", name);
  if ((uintptr_t)p % align) return set_error(MOE_EINVAL, "%s is not %zu-byte aligned", name, align);
  return MOE_OK;
}

inline int cuda_status(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return MOE_OK;
  return set_error(MOE_ECUDA, "%s: %s", what, cudaGetErrorString(e));
}

}  // namespace moe

#define TRY(expr)            \
  do {                       \
    int _s = (expr);         \
    if (_s != MOE_OK) return _s; \
  } while (0)
