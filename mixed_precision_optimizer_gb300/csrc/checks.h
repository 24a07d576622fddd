// Argument checks that the operators' entry points share.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/mpopt.h"
#include "internal.h"

namespace mpopt {
namespace {

constexpr int64_t kMaxExtent = int64_t(1) << 30;   // rows and columns: TMA coordinates are 32-bit
constexpr int64_t kMaxLd = int64_t(1) << 36;       // TMA row distances stay below 2^40 bytes

opt_status cuda_status(cudaError_t e, const char* where) {
  return e == cudaSuccess ? OPT_OK : static_cast<opt_status>(record_cuda_error(e, where));
}

int elem_size(int32_t dtype) { return dtype == OPT_DTYPE_FP32 ? 4 : dtype == OPT_DTYPE_BF16 ? 2 : 1; }

bool float_dtype(int32_t dtype) { return dtype == OPT_DTYPE_FP32 || dtype == OPT_DTYPE_BF16; }

size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// A matrix argument of `rows` rows: present unless optional, aligned to its
// elements, rows that do not overlap.  With one row the distance is not used.
opt_status check_matrix(const void* p, bool optional, int64_t ld, int64_t rows, int64_t cols, int es) {
  if (!p) return optional ? OPT_OK : OPT_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(es)) return OPT_ERR_MISALIGNED;
  if (rows > 1 && (ld < cols || ld > kMaxLd)) return OPT_ERR_INVALID_ARG;
  return OPT_OK;
}

opt_status check_vector(const void* p, bool optional, int es) {
  if (!p) return optional ? OPT_OK : OPT_ERR_INVALID_ARG;
  return reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(es) ? OPT_ERR_MISALIGNED : OPT_OK;
}

#define MPOPT_TRY(call)                    \
  do {                                     \
    const opt_status s_ = (call);          \
    if (s_ != OPT_OK) return s_;           \
  } while (0)

opt_status check_workspace(const void* ws, size_t have, size_t need) {
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) || have < need) return OPT_ERR_WORKSPACE;
  return OPT_OK;
}

}  // namespace
}  // namespace mpopt
