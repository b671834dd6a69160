// paged4.cuh -- device helpers of the 4-bit cache: e2m1 and e4m3 widened; the
// wait for earlier kernels.
#pragma once

#include <cstdint>

#include <cuda_fp16.h>

namespace gb300_attn {
namespace {

// What launch_early asks of a kernel, before anything else.  What earlier kernels may have written is loaded after it, and
// by ordinary loads or load_written: the read-only path (__ldg) is for memory that nobody writes while the kernel lives, and
// this one may already live while those still write.
__device__ __forceinline__ void after_earlier_kernels() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Eight e2m1 codes as f16 pairs, in order.
__device__ __forceinline__ void widen8(uint32_t w, uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d) {
  asm("{\n\t.reg .b8 x0, x1, x2, x3;\n\tmov.b32 {x0, x1, x2, x3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, x0;\n\tcvt.rn.f16x2.e2m1x2 %1, x1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, x2;\n\tcvt.rn.f16x2.e2m1x2 %3, x3;\n\t}"
      : "=r"(a), "=r"(b), "=r"(c), "=r"(d)
      : "r"(w));
}

// Two e4m3 bytes (the low half of w) as an f16 pair.
__device__ __forceinline__ uint32_t widen_e4m3x2(uint32_t w) {
  uint32_t h;
  asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(h) : "r"(w));
  return h;
}

__device__ __forceinline__ float e4m3_value(uint32_t byte) {
  const uint32_t h = widen_e4m3x2(byte);
  return __half2float(__ushort_as_half((unsigned short)(h & 0xffffu)));
}

__device__ __forceinline__ __half2 as_half2(uint32_t x) { return *reinterpret_cast<const __half2*>(&x); }
__device__ __forceinline__ uint32_t as_bits(__half2 x) { return *reinterpret_cast<const uint32_t*>(&x); }

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

}  // namespace
}  // namespace gb300_attn
