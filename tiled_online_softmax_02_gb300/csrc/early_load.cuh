// early_load.cuh -- the load of kernels that are launched while earlier ones run.
#pragma once

#include <cstdint>

namespace gb300_attn {

// A load of what an earlier kernel wrote, in a kernel launched while that one still runs (after griddepcontrol.wait): the
// read-only path (__ldg) is for memory that nobody writes while a kernel lives.  Volatile, so that it stays behind the
// wait; without a clobber, so that loads of a loop still go out together (by plain ones a merge of 4K keys in 16 ranges
// takes 0.9 us longer).
template <typename T>
__device__ __forceinline__ T load_written(const T* p) {
  static_assert(sizeof(T) == 4 || sizeof(T) == 8 || sizeof(T) == 16, "one load");
  uint32_t w[sizeof(T) / 4];
  if constexpr (sizeof(T) == 4) asm volatile("ld.global.b32 %0, [%1];" : "=r"(w[0]) : "l"(p));
  else if constexpr (sizeof(T) == 8) asm volatile("ld.global.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(p));
  else asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "l"(p));
  T x;
  __builtin_memcpy(&x, w, sizeof(T));
  return x;
}

}  // namespace gb300_attn
