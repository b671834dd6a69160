// api_internal.h -- host-side helpers shared by the translation units that
// implement the C ABI (attn_api.cu, paged_api.cu): argument checks, the
// per-device status word, the tensor-map encoder and the error record.  Not
// part of the public interface.
#pragma once

#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

namespace gb300_attn {

// Records a CUDA error for attn_last_cuda_error; returns ATTN_ERR_CUDA.
int cuda_fail(cudaError_t e);
// Device address of the status word on the current device; nullptr with *err set on failure.
int* status_ptr(int* err);
// cuTensorMapEncodeTiled, looked up once; nullptr with *err set on failure.
PFN_cuTensorMapEncodeTiled_v12000 encode_fn(int* err);
// The limit of bounded waits, for launches made now.
uint64_t wait_timeout_ns();

inline bool mul_ok(int64_t a, int64_t b, int64_t* out) {
  if (a < 0 || b < 0) return false;
  if (a != 0 && b > (INT64_C(1) << 62) / a) return false;
  *out = a * b;
  return true;
}

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline bool overlaps(const void* a, int64_t abytes, const void* b, int64_t bbytes) {
  if (!a || !b || abytes <= 0 || bbytes <= 0) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a0 < b0 + (uintptr_t)bbytes && b0 < a0 + (uintptr_t)abytes;
}

}  // namespace gb300_attn
