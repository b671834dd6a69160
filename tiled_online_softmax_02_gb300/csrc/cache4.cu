// cache4.cu -- rows into the paged 4-bit cache, and back out of it.
//
// A group is 16 values of a row, with the kv head's factor h (1 where there is
// none) and g the largest finite |x|:
//   s    = e4m3(g / (6 h)), at least 2^-9, at most 448
//   code = e2m1(x / (s h)), to nearest even, cut at 6,
// 6 h, s h and both quotients rounded to fp32.  Where h is a power of two that
// settles e4m3's and e2m1's ties as exact quotients would: one next to a border of
// so few bits is never rounded onto it.  (Under another h, 24 bits of s h against
// 24 of an f32 x, it may be.)
// A group with a NaN gets the scale NaN and zeros.  value = code * s * h.
//
// Under a power-of-two h (1 among them) the quotient x / (s h) is x rh + x rl,
// the inverse of s h as a sum of two: rh rounded down and what is left of it, so
// that the sum is off by 2^-46 of itself and its rounding is the quotient's
// wherever that lies next to a border (the nearest quotients are 0.53 units of
// the last place from one).  rl is kept above 0, for infinities and zeros.  Two
// instructions a value; the fp32 division costs twelve.
//
// Bound: HBM and the issue slots for prompts, and for a few tokens the chain of slot, row, group
// maximum and store.  A thread has one group of K and the same one of V: their
// values are wide loads in flight beside the slot's, no thread waits for another,
// and the 32 lanes of a warp write whole sectors (rows of one head that follow
// one another in a block).
//
// Measured (one GB300, device time): 64 tokens of 8 heads, D = 128, bf16 2.1 us in,
// 2.1 out; 16K tokens 18.4 us in (4.7 TB/s, 70% of a copy's rate), 17.7 out;
// in, 407 instructions a thread take two thirds of the issue slots, DRAM 45%;
// 32.7K tokens out 30.6 us (5.6 TB/s).  With a thread for K and one for V 23.4 and
// 19.3, by fp32 divisions 22.4, 128 and 256 threads a CTA 19.1 and 20 out.
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "../../include/attn.h"
#include "early_load.cuh"
#include "paged4.cuh"
#include "paged4_internal.h"

namespace gb300_attn {
namespace {

constexpr int kThreads = 64;

template <typename T>
__device__ __forceinline__ void widen16(const uint4 (&v)[sizeof(T)], float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < (int)sizeof(T); ++i) {
    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (sizeof(T) == 4) {
        x[4 * i + j] = __uint_as_float(w[j]);
      } else if constexpr (std::is_same<T, __half>::value) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
        x[8 * i + 2 * j] = f.x;
        x[8 * i + 2 * j + 1] = f.y;
      } else {
        x[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
        x[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
      }
    }
  }
}

// The token, head and group of a thread: lanes go over a row's groups, then over tokens.
template <int D>
struct Place {
  static constexpr int kPer = D / kGroup4, kTokens = kThreads / kPer;
  int t, h, part;
  bool there;
  __device__ __forceinline__ Place(const Cache4Params& p, int64_t unit) {
    const int64_t tile = unit / p.Hkv;
    h = (int)(unit - tile * p.Hkv);
    const int64_t tok = tile * kTokens + threadIdx.x / kPer;
    there = tok < p.T;
    t = there ? (int)tok : 0;
    part = threadIdx.x % kPer;
  }
  // index of the row in the cache; -1: no row
  __device__ __forceinline__ int64_t row(const Cache4Params& p) const {
    const int64_t s = load_written(p.slot_map + t);
    if (!there || s < 0 || s >= p.num_slots) return -1;
    return ((s >> p.block_shift) * p.Hkv + h) * p.block_size + (s & (p.block_size - 1));
  }
};

// The largest finite |x| of 16 values, as fp32 bits; 0x7fc00000 where one is NaN.
template <typename T>
__device__ __forceinline__ uint32_t largest(const uint4 (&v)[sizeof(T)], const float (&x)[16]) {
  uint32_t top = 0;  // magnitudes order as their bits; not finite from 0x7f800000 on
  if constexpr (sizeof(T) == 2) {  // 16-bit ones two at a time
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      m = __vmaxu2(m, __vmaxu2(__vmaxu2(v[i].x & 0x7fff7fffu, v[i].y & 0x7fff7fffu),
                               __vmaxu2(v[i].z & 0x7fff7fffu, v[i].w & 0x7fff7fffu)));
    const uint32_t t = max(m & 0xffffu, m >> 16);
    if constexpr (std::is_same<T, __half>::value) top = __float_as_uint(__half2float(__ushort_as_half((unsigned short)t)));
    else top = t << 16;
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) top = max(top, __float_as_uint(x[i]) & 0x7fffffffu);
  }
  if (top >= 0x7f800000u) {  // infinities set no scale
    if (top > 0x7f800000u) return 0x7fc00000u;
    top = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint32_t a = __float_as_uint(x[i]) & 0x7fffffffu;
      top = a < 0x7f800000u ? max(top, a) : top;
    }
  }
  return top;
}

// Eight values as codes, in order.
__device__ __forceinline__ uint32_t narrow8(const float* x) {
  uint32_t w;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(w)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return w;
}

// 16 values as codes and the byte of their scale.
template <typename T>
__device__ __forceinline__ uint2 quantise(const uint4 (&v)[sizeof(T)], float hs, uint32_t& sb) {
  float x[16];
  widen16<T>(v, x);
  const uint32_t top = largest<T>(v, x);
  if (top == 0x7fc00000u) {
    sb = 0x7fu;
    return make_uint2(0u, 0u);
  }
  sb = __nv_cvt_float_to_fp8(__fdiv_rn(__uint_as_float(top), 6.0f * hs), __NV_SATFINITE, __NV_E4M3);
  sb = max(sb & 0x7fu, 1u);
  const float unit = e4m3_value(sb) * hs;
  const uint32_t hb = __float_as_uint(hs);
  if ((hb & 0x7fffffu) == 0u && hb >= (67u << 23) && hb <= (187u << 23)) {  // 2^-60 to 2^60: all of this in range
    const float rh = __frcp_rd(unit), rl = fmaxf(__fmaf_rn(-rh, unit, 1.0f) * rh, rh * 0x1p-60f);
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = __fmaf_rn(x[i], rh, __fmul_rn(x[i], rl));
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = __fdiv_rn(x[i], unit);
  }
  return make_uint2(narrow8(x), narrow8(x + 8));
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) cache4_append_kernel(const __grid_constant__ Cache4Params p, int64_t units) {
  after_earlier_kernels();
  using P = Place<D>;
  for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
    const P at(p, unit);
    uint4 v[2][sizeof(T)];
    float hs[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const T* src = static_cast<const T*>(p.x[k]) + (int64_t)at.t * p.stride[k] + at.h * D + at.part * kGroup4;
#pragma unroll
      for (int i = 0; i < (int)sizeof(T); ++i) v[k][i] = load_written(reinterpret_cast<const uint4*>(src) + i);
      hs[k] = p.heads[k] ? load_written(p.heads[k] + at.h) : 1.0f;
    }
    const int64_t row = at.row(p);
    if (row < 0) continue;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      uint32_t sb;
      const uint2 w = quantise<T>(v[k], hs[k], sb);
      *reinterpret_cast<uint2*>(p.cache[k] + row * (D / 2) + at.part * 8) = w;
      p.scales[k][row * (D / kGroup4) + at.part] = (uint8_t)sb;
    }
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) cache4_read_kernel(const __grid_constant__ Cache4Params p, int64_t units) {
  after_earlier_kernels();
  using P = Place<D>;
  for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
    const P at(p, unit);
    if (!at.there) continue;
    const int64_t row = at.row(p);
    uint2 code[2];
    uint32_t sb[2] = {0u, 0u};
    float hs[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      code[k] = make_uint2(0u, 0u);
      hs[k] = p.heads[k] ? load_written(p.heads[k] + at.h) : 1.0f;
      if (row >= 0) {
        code[k] = load_written(reinterpret_cast<const uint2*>(p.cache[k] + row * (D / 2) + at.part * 8));
        sb[k] = p.scales[k][row * (D / kGroup4) + at.part];
      }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float s = e4m3_value(sb[k]);
      uint32_t h[8];
      widen8(code[k].x, h[0], h[1], h[2], h[3]);
      widen8(code[k].y, h[4], h[5], h[6], h[7]);
      T* dst = static_cast<T*>(p.x[k]) + (int64_t)at.t * p.stride[k] + (int64_t)at.h * p.head_stride[k] + at.part * kGroup4;
      uint32_t o[4 * sizeof(T)];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float2 f = __half22float2(as_half2(h[i]));
        f.x = f.x * s * hs[k];  // code * s is exact
        f.y = f.y * s * hs[k];
        if constexpr (sizeof(T) == 4) {
          o[2 * i] = __float_as_uint(f.x);
          o[2 * i + 1] = __float_as_uint(f.y);
        } else if constexpr (std::is_same<T, __half>::value) {
          o[i] = as_bits(__floats2half2_rn(f.x, f.y));
        } else {
          const __nv_bfloat162 y = __floats2bfloat162_rn(f.x, f.y);
          o[i] = *reinterpret_cast<const uint32_t*>(&y);
        }
      }
#pragma unroll
      for (int i = 0; i < (int)sizeof(T); ++i)
        reinterpret_cast<uint4*>(dst)[i] = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
    }
  }
}

template <typename T, int D>
cudaError_t launch(const Cache4Params& p, bool read, cudaStream_t stream) {
  const int64_t units = ((int64_t)p.T + Place<D>::kTokens - 1) / Place<D>::kTokens * p.Hkv;
  const unsigned grid = (unsigned)std::min<int64_t>(units, 1 << 30);
  return launch_early(read ? cache4_read_kernel<T, D> : cache4_append_kernel<T, D>, grid, kThreads, 0, stream, p, units);
}

template <typename T>
cudaError_t launch_d(const Cache4Params& p, bool read, cudaStream_t stream) {
  return p.D == 128 ? launch<T, 128>(p, read, stream) : launch<T, 64>(p, read, stream);
}

cudaError_t launch_t(const Cache4Params& p, int dtype, bool read, cudaStream_t stream) {
  if (dtype == ATTN_BF16) return launch_d<__nv_bfloat16>(p, read, stream);
  if (dtype == ATTN_F16) return launch_d<__half>(p, read, stream);
  return launch_d<float>(p, read, stream);
}

}  // namespace

cudaError_t launch_cache4_append(const Cache4Params& p, int dtype, cudaStream_t stream) {
  return launch_t(p, dtype, false, stream);
}

cudaError_t launch_cache4_read(const Cache4Params& p, int dtype, cudaStream_t stream) {
  return launch_t(p, dtype, true, stream);
}

}  // namespace gb300_attn
