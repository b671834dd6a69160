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
constexpr float kMinVScale = 7.9e-31f;  // 2^-100: a block of zeros may have scale 0
constexpr float kPieceStep = 32.0f;     // from one e4m3 piece to the next

// mbar_wait_warp in fewer instructions: these kernels have many waits in many
// roles, and are bound by their instruction fetches before anything else.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, uint64_t timeout_ns, int* status) {
  uint64_t t0 = 0;
  bool ok = true;
  for (uint32_t it = 1; !mbar_try_wait(bar, parity); ++it) {
    if ((it & 15u) != 0u) continue;
    const uint64_t now = global_timer_ns();
    if (t0 == 0) t0 = now;
    if (now - t0 > timeout_ns) {
      atomicOr(status, kStatusTimeout);
      ok = false;
      break;
    }
  }
  return __all_sync(0xffffffffu, ok);
}

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

// e4m3 pieces of two values (lo in bits 0-7): the piece, and what is left of them times 32.
__device__ __forceinline__ uint32_t piece2(float& lo, float& hi) {
  uint16_t b;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(b) : "f"(hi), "f"(lo));
  uint32_t h2;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(b));
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
  lo = (lo - f.x) * kPieceStep;
  hi = (hi - f.y) * kPieceStep;
  return b;
}
__device__ __forceinline__ uint32_t last2(float lo, float hi) {
  uint16_t b;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(b) : "f"(hi), "f"(lo));
  return b;
}

template <bool BF16>
__device__ __forceinline__ uint16_t to_bits(float x) {
  if constexpr (BF16) return __bfloat16_as_ushort(__float2bfloat16_rn(x));
  else return __half_as_ushort(__float2half_rn(x));
}

}  // namespace
}  // namespace gb300_attn
