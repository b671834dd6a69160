// paged_mma.cuh -- device helpers of the paged attention kernels: e4m3 tensor
// core descriptors, and values as sums of e4m3 pieces.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "device_common.cuh"

namespace gb300_attn {
namespace {

constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNone = -1e30f;         // running maximum of a row that has seen no key
constexpr float kPieceStep = 32.0f;     // from one e4m3 piece to the next

// Instruction descriptor of tcgen05.mma kind::f8f6f4: fp32 accumulator (bits
// 4-5 = 1), A and B e4m3 (bits 7-9 and 10-12 = 0), major-ness of A / B in bits
// 15 / 16 (1 = MN-major), N >> 3 in 17-22, M >> 4 in 24-28.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N, bool a_mn, bool b_mn) {
  return (1u << 4) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}

// Shared-memory matrix descriptor; layout 2 = 128-byte swizzle, 4 = 64-byte, 0 = none.
__device__ __forceinline__ uint64_t sdesc(uint32_t saddr, uint32_t lbo, uint32_t sbo, uint32_t layout) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | (uint64_t)((lbo >> 4) & 0x3FFFu) << 16 |
         (uint64_t)((sbo >> 4) & 0x3FFFu) << 32 | (uint64_t)1u << 46 | (uint64_t)layout << 61;
}

template <bool BF16>
__device__ __forceinline__ uint16_t to_bits(float x) {
  if constexpr (BF16) return __bfloat16_as_ushort(__float2bfloat16_rn(x));
  else return __half_as_ushort(__float2half_rn(x));
}

}  // namespace
}  // namespace gb300_attn
