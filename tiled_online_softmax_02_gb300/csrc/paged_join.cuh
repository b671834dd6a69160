// paged_join.cuh -- what the kernels share that join the partial rows of the
// paged attention kernels: a lane's values of a row, and the joined row's way
// out.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "paged_internal.h"

namespace gb300_attn {
namespace {

template <int D>
struct RowVec {
  static constexpr int V = D / 32;  // values of a lane
  float x[V];
  __device__ __forceinline__ void load(const float* row, int lane) {
    if constexpr (V == 4) {
      const float4 v = *reinterpret_cast<const float4*>(row + lane * 4);
      x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
    } else {
      const float2 v = *reinterpret_cast<const float2*>(row + lane * 2);
      x[0] = v.x; x[1] = v.y;
    }
  }
};

template <int D, bool BF16>
__device__ __forceinline__ void store_row(const PagedCut& cut, int r, int Hq, int group, float ml_log2, uint16_t* out,
                                          float* lse, int lane, const float (&acc)[D / 32], float M, float L) {
  constexpr int V = D / 32;
  const float inv = L == 0.0f ? 0.0f : kPagedSumFactor * (1.0f / L);
  const int x = cut.row0 + r;
  const int64_t row = (int64_t)(cut.token0 + x / group) * Hq + cut.head0 + x % group;
  uint32_t packed[V / 2];
#pragma unroll
  for (int v = 0; v < V / 2; ++v) {
    if constexpr (BF16) {
      const __nv_bfloat162 y = __floats2bfloat162_rn(acc[2 * v] * inv, acc[2 * v + 1] * inv);
      packed[v] = *reinterpret_cast<const uint32_t*>(&y);
    } else {
      const __half2 y = __floats2half2_rn(acc[2 * v] * inv, acc[2 * v + 1] * inv);
      packed[v] = *reinterpret_cast<const uint32_t*>(&y);
    }
  }
  uint16_t* dst = out + row * D + lane * V;
  if constexpr (V == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(packed[0], packed[1]);
  else *reinterpret_cast<uint32_t*>(dst) = packed[0];
  if (lse != nullptr && lane == 0)
    lse[row] = L == 0.0f ? -INFINITY : (M + (log2f(L) - ml_log2)) * 0.6931471805599453f;
}

}  // namespace
}  // namespace gb300_attn
