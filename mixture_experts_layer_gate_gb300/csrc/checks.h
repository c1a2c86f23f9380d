// Argument checks that the host sides of the operators share.
#pragma once

#include <cuda_runtime.h>

#include "../../include/moe.h"
#include "common.cuh"

namespace moe {

inline size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }
inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline size_t size_of(int dtype) { return dtype == MOE_T_F32 ? 4 : 2; }
inline bool is_dtype(int d) { return d == MOE_T_BF16 || d == MOE_T_F16 || d == MOE_T_F32; }

inline moe_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

inline moe_status_t check_header(const void* ws, size_t ws_bytes) {
  if (ws == nullptr || !aligned(ws, 256) || ws_bytes < kHeaderBytes) return MOE_ERR_WORKSPACE;
  return MOE_OK;
}

// A row tensor: present, aligned to its elements, rows that do not overlap.
inline bool rows_ok(const void* p, int64_t stride, int64_t cols, size_t align) {
  return p != nullptr && aligned(p, align) && stride >= cols;
}

#define MOE_TRY(x)                   \
  do {                               \
    const moe_status_t st__ = (x);   \
    if (st__ != MOE_OK) return st__; \
  } while (0)

}  // namespace moe
