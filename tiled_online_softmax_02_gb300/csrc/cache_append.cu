// cache_append.cu -- writes new K and V rows into the paged cache as e4m3
// bytes with one scale for each (block, kv head).
//
// The tokens of one block that follow one another in the slot map are a run.
// For a run and a head, over the run's finite values x:
//   need = the smallest power of two s with max|x| <= 448 s (at least 2^-100)
//   s    = max(need, the block's scale)   when the run starts inside the block,
//          need                           when it starts at the block's row 0
//   byte = e4m3(x / s), to nearest even, |x / s| cut at 448, NaN kept
// and where s grew, the block's earlier rows are encoded again for it.
// Powers of two make x / s exact, and a re-encoding loses nothing but what
// falls below the smallest e4m3 value of the new scale.
//
// Bound: HBM for prompts (2 or 4 bytes in and 1 out per value), the latency
// of one load -> maximum -> store chain for a decode step.  One CTA owns the
// runs that begin in its chunk of tokens, for one head of K or of V: short
// runs (a decode step's) take a warp each, long ones the whole CTA, and a
// run's second reading comes out of L1.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "../../include/attn.h"
#include "device_common.cuh"
#include "paged_internal.h"

namespace gb300_attn {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxChunk = 16;
constexpr int kShortRun = 4;  // tokens: up to this many a warp takes alone

// 16 values at src as fp32.
__device__ __forceinline__ void load16(const float* src, float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(src) + i);
    x[4 * i] = v.x; x[4 * i + 1] = v.y; x[4 * i + 2] = v.z; x[4 * i + 3] = v.w;
  }
}
__device__ __forceinline__ float2 widen(uint32_t w, __half) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
__device__ __forceinline__ float2 widen(uint32_t w, __nv_bfloat16) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
}
template <typename T>
__device__ __forceinline__ void load16(const T* src, float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(src) + i);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = widen(w[j], T{});
      x[8 * i + 2 * j] = f.x;
      x[8 * i + 2 * j + 1] = f.y;
    }
  }
}

// 16 e4m3 bytes of x * mul.
__device__ __forceinline__ uint4 encode16(const float (&x)[16], float mul) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i] * mul, x[4 * i + 1] * mul), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i + 2] * mul, x[4 * i + 3] * mul), __NV_SATFINITE, __NV_E4M3);
    w[i] = lo | (hi << 16);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void decode16(uint4 v, float (&x)[16]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[i] >> (16 * j)), __NV_E4M3);
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
      x[4 * i + 2 * j] = f.x;
      x[4 * i + 2 * j + 1] = f.y;
    }
}

// The smallest power of two s >= 2^-100 with amax <= 448 s = 1.75 * 2^8 s, from the bits of amax.
__device__ __forceinline__ float scale_for(float amax) {
  const uint32_t u = __float_as_uint(amax);
  int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  if (amax == 0.0f || e < -100) e = -100;
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

// Run of `len` tokens from token t0, written to rows off0.. of a block, by
// threads tid, tid + NT, ... of one warp (NT = 32) or of the CTA.
template <typename T, int D, int NT>
__device__ __forceinline__ void append_run(const T* x, int64_t stride, uint8_t* tile, float* scale, int off0,
                                           int len, int tid, float* red) {
  constexpr int kVec = D / 16;  // 16-value pieces of a row
  const float old = off0 > 0 ? *scale : 0.0f;
  float amax = 0.0f;
  for (int c = tid; c < len * kVec; c += NT) {
    float v[16];
    load16(x + (int64_t)(c / kVec) * stride + (c % kVec) * 16, v);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float a = fabsf(v[i]);
      amax = a <= 3.4028235e38f ? fmaxf(amax, a) : amax;  // infinities and NaN set no scale
    }
  }
  // non-negative floats order as their bits
  uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(amax));
  if constexpr (NT > 32) {
    __syncthreads();
    if ((tid & 31) == 0) red[tid >> 5] = __uint_as_float(top);
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) top = max(top, __float_as_uint(red[w]));
  }
  const float s = fmaxf(scale_for(__uint_as_float(top)), old);
  const float inv = 1.0f / s;
  for (int c = tid; c < len * kVec; c += NT) {
    float v[16];
    load16(x + (int64_t)(c / kVec) * stride + (c % kVec) * 16, v);
    *reinterpret_cast<uint4*>(tile + (off0 + c / kVec) * D + (c % kVec) * 16) = encode16(v, inv);
  }
  if (off0 > 0 && s > old) {
    const float again = old * inv;
    for (int c = tid; c < off0 * kVec; c += NT) {
      uint4* at = reinterpret_cast<uint4*>(tile + c * 16);
      float v[16];
      decode16(*at, v);
      *at = encode16(v, again);
    }
  }
  if constexpr (NT > 32) __syncthreads(); else __syncwarp();  // every thread has read the old scale
  if (tid == 0) *scale = s;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) cache_append_kernel(const __grid_constant__ AppendParams p) {
  __shared__ int64_t slots[kMaxChunk + 1];  // of tokens first - 1 ..
  __shared__ int begin[kMaxChunk];          // 1 where a run begins
  __shared__ float red[kWarps];
  const int first = blockIdx.x * p.chunk, h = blockIdx.y, which = blockIdx.z;
  const int n = min(p.chunk, p.T - first);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x <= n)
    slots[threadIdx.x] = first + (int)threadIdx.x == 0 ? -1 : __ldg(p.slot_map + first + threadIdx.x - 1);
  __syncthreads();
  const int bs = p.block_size;
  auto valid = [&](int64_t s) { return s >= 0 && s < p.num_slots; };
  if (warp == 0) {
    // a token begins its block's tokens unless the nearest token before it
    // that has a slot is of the same block (that one is almost always the
    // one before; past skipped tokens the warp looks 32 back at a time)
    const int64_t s = lane < n ? slots[lane + 1] : -1, prev = lane < n ? slots[lane] : -1;
    int b = valid(s) && !(valid(prev) && prev / bs == s / bs);
    unsigned look = __ballot_sync(0xffffffffu, b && !valid(prev) && first + lane > 0);
    while (look) {
      const int i = __ffs(look) - 1;
      look &= look - 1;
      const int64_t mine = slots[i + 1] / bs;
      for (int back = first + i - 1; back >= 0; back -= 32) {
        const int64_t t = back - lane >= 0 ? __ldg(p.slot_map + back - lane) : -1;
        const unsigned m = __ballot_sync(0xffffffffu, valid(t));
        if (m) {
          if (__shfl_sync(0xffffffffu, t, __ffs(m) - 1) / bs == mine && lane == i) b = 0;
          break;
        }
      }
    }
    if (lane < n) begin[lane] = b;
  }
  __syncthreads();
  const T* x0 = static_cast<const T*>(which ? p.x[1] : p.x[0]);
  const int64_t stride = which ? p.stride[1] : p.stride[0];
  uint8_t* cache = which ? p.cache[1] : p.cache[0];
  float* scales = which ? p.scales[1] : p.scales[0];

  for (int pass = 0; pass < 2; ++pass) {  // blocks with a short first run by warps, then the others by the CTA
    int mine = 0;
    for (int i = 0; i < n; ++i) {
      if (!begin[i]) continue;
      if (pass == 0 && (mine++ % kWarps) != warp) continue;
      // the block's runs, one after the other (more than one only where skipped tokens lie between them)
      int t = first + i;
      int64_t s = slots[i + 1];
      const int64_t blk = s / bs;
      bool later = false;
      for (;;) {
        const int off = (int)(s - blk * bs);
        // length: tokens t + 1 .. whose slots rise by one inside the block, 32 looked at a time
        int len = 1;
        int64_t next;  // the slot after the run; -1 where it names no row
        for (;;) {
          const int64_t y = t + len + lane < p.T ? __ldg(p.slot_map + t + len + lane) : -1;
          const unsigned m = __ballot_sync(0xffffffffu, off + len + lane < bs && y == s + len + lane);
          const int more = m == 0xffffffffu ? 32 : __ffs(~m) - 1;
          len += more;
          if (more < 32) {
            next = __shfl_sync(0xffffffffu, y, more);
            break;
          }
        }
        if (!later && (len <= kShortRun) != (pass == 0)) break;
        const T* x = x0 + (int64_t)t * stride + h * D;
        const int64_t tile = blk * p.Hkv + h;
        if (pass == 0)
          append_run<T, D, 32>(x, stride, cache + tile * bs * D, scales + tile, off, len, lane, nullptr);
        else
          append_run<T, D, kThreads>(x, stride, cache + tile * bs * D, scales + tile, off, len, threadIdx.x, red);
        t += len;
        while (!valid(next) && t < p.T) {  // over skipped tokens
          const int64_t y = t + lane < p.T ? __ldg(p.slot_map + t + lane) : -1;
          const unsigned m = __ballot_sync(0xffffffffu, valid(y));
          const int skip = m ? __ffs(m) - 1 : 32;
          t += skip;
          if (m) next = __shfl_sync(0xffffffffu, y, skip);
        }
        if (!valid(next) || next / bs != blk) break;
        s = next;
        later = true;
        if (pass == 0) __syncwarp(); else __syncthreads();  // the block's rows and scale are written
      }
    }
  }
}

template <typename T>
cudaError_t launch_t(const AppendParams& p, cudaStream_t stream) {
  const dim3 grid((unsigned)((p.T + p.chunk - 1) / p.chunk), (unsigned)p.Hkv, 2);
  if (p.D == 128) cache_append_kernel<T, 128><<<grid, kThreads, 0, stream>>>(p);
  else cache_append_kernel<T, 64><<<grid, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_append(const AppendParams& in, int dtype, cudaStream_t stream) {
  AppendParams p = in;
  // few tokens: one run a warp and CTA; many: a CTA looks at 16 tokens, a quarter of a usual block
  p.chunk = p.T <= 1024 ? 4 : kMaxChunk;
  if (dtype == ATTN_BF16) return launch_t<__nv_bfloat16>(p, stream);
  if (dtype == ATTN_F16) return launch_t<__half>(p, stream);
  return launch_t<float>(p, stream);
}

}  // namespace gb300_attn
