// Host-side helpers shared by the library's translation units: errors that
// carry a status code, CUDA call checks and TMA descriptors.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdarg>
#include <cstdio>
#include <stdexcept>
#include <string>

#include "gdit.h"

namespace gdit {

// ------------------------------------------------------------------ errors

struct GditError : std::runtime_error {
  int code;
  GditError(int c, const std::string& m) : std::runtime_error(m), code(c) {}
};

inline std::string fmt(const char* f, ...) {
  char buf[1024];
  va_list ap;
  va_start(ap, f);
  vsnprintf(buf, sizeof(buf), f, ap);
  va_end(ap);
  return buf;
}

#define CUDA_TRY(expr)                                                                                  \
  do {                                                                                                  \
    cudaError_t e_ = (expr);                                                                            \
    if (e_ != cudaSuccess)                                                                              \
      throw GditError(e_ == cudaErrorMemoryAllocation ? GDIT_ENOMEM : GDIT_ECUDA,                       \
                      fmt("%s failed: %s (%s:%d)", #expr, cudaGetErrorString(e_), __FILE__, __LINE__)); \
  } while (0)

#define REQUIRE(cond, ...)                                  \
  do {                                                      \
    if (!(cond)) throw GditError(GDIT_EINVAL, fmt(__VA_ARGS__)); \
  } while (0)

// detail message of the calling thread's last failed call without a handle
inline thread_local std::string g_create_error;

// ------------------------------------------------------------------ TMA descriptors

typedef CUresult (*PFN_encodeTiled_t)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                       const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                       CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// Looked up once, by whichever thread comes first (again after a failure).
inline PFN_encodeTiled_t encode_fn() {
  static const PFN_encodeTiled_t fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    CUDA_TRY(cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q));
    if (p == nullptr || q != cudaDriverEntryPointSuccess)
      throw GditError(GDIT_ECUDA, "cuTensorMapEncodeTiled not available from the driver");
    return reinterpret_cast<PFN_encodeTiled_t>(p);
  }();
  return fn;
}

// bf16 matrix [rows, cols] with row pitch `pitch` elements; boxes of box_rows x 64,
// 128-byte swizzle (the layout the UMMA descriptors expect).
inline CUtensorMap make_tmap(const void* ptr, long long rows, long long cols, long long pitch, int box_rows) {
  REQUIRE(((uintptr_t)ptr & 15u) == 0, "TMA base pointer not 16-byte aligned");
  REQUIRE((pitch * 2) % 16 == 0, "TMA row pitch %lld elements is not a multiple of 16 bytes", pitch);
  REQUIRE(box_rows >= 1 && box_rows <= 256, "TMA box rows %d", box_rows);
  CUtensorMap m;
  cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)std::max<long long>(rows, 1)};
  cuuint64_t strides[1] = {(cuuint64_t)(pitch * 2)};
  cuuint32_t box[2] = {64u, (cuuint32_t)box_rows};
  cuuint32_t estr[2] = {1u, 1u};
  CUresult r = encode_fn()(&m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(ptr), dims, strides, box, estr,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) throw GditError(GDIT_ECUDA, fmt("cuTensorMapEncodeTiled failed (%d)", (int)r));
  return m;
}

}  // namespace gdit
