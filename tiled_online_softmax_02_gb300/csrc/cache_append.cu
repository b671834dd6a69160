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
// runs (a decode step's) take a warp each, long ones the whole CTA.  The slots
// that can matter are read once into shared memory, and a thread keeps its
// first values in registers between finding the maximum and encoding them.  A
// block whose tokens go on behind that window, past skipped ones, is followed by
// the whole CTA, 1024 entries of the map at a time.
//
// Measured (one GB300, device time): 64 new tokens of 8 kv heads 5.1 us; 16K
// tokens of 8 kv heads, D = 128, bf16, 24.8 us, 4.1 TB/s (26.9 without the
// prefetch; 25.6 with one that does not wait for the slots, and reads the rows of
// skipped tokens); 64 tokens in a map of 65536 entries 105 us.  The prompts wait
// for their chain of slots, rows, maximum and stores (leaving out the maximum's or
// the encoding's arithmetic changes nothing).  Ten CTAs an SM leave 48 registers a
// thread (80 and six CTAs for f32), of which the long-run path spills 116 bytes (136);
// 256 threads a CTA (31 us), twice the values in registers (28 us: fewer CTAs
// fit), several heads a CTA (31 to 48 us), 8 or 12 CTAs an SM instead of 10 (26
// and 27 us), 32 or 128 tokens a CTA (26 and 29 us) were all slower.
#include <type_traits>

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
constexpr int kMaxChunk = 64;
constexpr int kWindow = 1 + kMaxChunk + 128;  // slots kept: one before the chunk, and a block after it
constexpr int kWarpPieces = 128;  // up to this many 16-value pieces a warp takes a run alone

// 16 values of a row as they lie in memory: what a thread takes at a time.
template <typename T>
struct Piece {
  static constexpr int kVecs = sizeof(T);  // 16-byte loads
  uint4 v[kVecs];
  __device__ __forceinline__ void load(const T* src) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) v[i] = __ldg(reinterpret_cast<const uint4*>(src) + i);
  }
  __device__ __forceinline__ void widen(float (&x)[16]) const {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (sizeof(T) == 4) {
          x[4 * i + j] = __uint_as_float(w[j]);
        } else {
          const float2 f = pair(w[j], T{});
          x[8 * i + 2 * j] = f.x;
          x[8 * i + 2 * j + 1] = f.y;
        }
      }
    }
  }
  static __device__ __forceinline__ float2 pair(uint32_t w, __half) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  }
  static __device__ __forceinline__ float2 pair(uint32_t w, __nv_bfloat16) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
  static __device__ __forceinline__ float2 pair(uint32_t, float) { return make_float2(0.0f, 0.0f); }
  // The largest finite |x|, as fp32 bits: magnitudes order as their bits, and
  // 16-bit ones are compared two at a time.
  __device__ __forceinline__ uint32_t top() const {
    if constexpr (sizeof(T) == 4) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < kVecs; ++i) {
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t a = w[j] & 0x7fffffffu;
          m = a < 0x7f800000u ? max(m, a) : m;
        }
      }
      return m;
    } else {
      constexpr uint32_t inf = std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < kVecs; ++i)
        m = __vmaxu2(m, __vmaxu2(__vmaxu2(v[i].x & 0x7fff7fffu, v[i].y & 0x7fff7fffu),
                                 __vmaxu2(v[i].z & 0x7fff7fffu, v[i].w & 0x7fff7fffu)));
      uint32_t t = max(m & 0xffffu, m >> 16);
      if (t >= inf) {  // infinities and NaN set no scale
        t = 0;
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
          const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t lo = w[j] & 0x7fffu, hi = (w[j] >> 16) & 0x7fffu;
            t = lo < inf ? max(t, lo) : t;
            t = hi < inf ? max(t, hi) : t;
          }
        }
      }
      return __float_as_uint(pair(t, T{}).x);
    }
  }
};

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
                                           int len, int tid, uint32_t* red) {
  constexpr int kVec = D / 16;  // 16-value pieces of a row
  const float old = off0 > 0 ? *scale : 0.0f;
  const T* x0 = x + (tid % kVec) * 16;  // NT is a multiple of kVec: a thread keeps its column
  constexpr int kKeep = 2;              // pieces kept in registers
  Piece<T> keep[kKeep];
  const int pieces = len * kVec;
#pragma unroll
  for (int k = 0; k < kKeep; ++k)
    if (tid + k * NT < pieces) keep[k].load(x0 + (int64_t)((tid + k * NT) / kVec) * stride);
  uint32_t top = 0;
#pragma unroll
  for (int k = 0; k < kKeep; ++k)
    if (tid + k * NT < pieces) top = max(top, keep[k].top());
#pragma unroll 2
  for (int c = tid + kKeep * NT; c < pieces; c += NT) {
    Piece<T> v;
    v.load(x0 + (int64_t)(c / kVec) * stride);
    top = max(top, v.top());
  }
  top = __reduce_max_sync(0xffffffffu, top);
  if constexpr (NT > 32) {
    __syncthreads();
    if ((tid & 31) == 0) red[tid >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) top = max(top, red[w]);
  }
  const float s = fmaxf(scale_for(__uint_as_float(top)), old);
  const float inv = 1.0f / s;
  uint8_t* out = tile + off0 * D + (tid % kVec) * 16;
#pragma unroll
  for (int k = 0; k < kKeep; ++k)
    if (tid + k * NT < pieces) {
      float v[16];
      keep[k].widen(v);
      *reinterpret_cast<uint4*>(out + (tid + k * NT) / kVec * D) = encode16(v, inv);
    }
#pragma unroll 2
  for (int c = tid + kKeep * NT; c < pieces; c += NT) {
    Piece<T> w;
    w.load(x0 + (int64_t)(c / kVec) * stride);
    float v[16];
    w.widen(v);
    *reinterpret_cast<uint4*>(out + c / kVec * D) = encode16(v, inv);
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

// The first token of [from, end) whose slot names a row (back: the last), or -1.  Called by the whole CTA: a thread has
// eight entries on their way, as a map padded for a captured graph may hold many thousands that name none.
__device__ __noinline__ int find_slot(const int64_t* map, int64_t num_slots, int from, int end, bool back, uint32_t* red) {
  constexpr int kDeep = 8;
  const uint32_t count = (uint32_t)max(end - from, 0);
  for (uint32_t done = 0; done < count; done += kThreads * kDeep) {
    int64_t s[kDeep];
#pragma unroll
    for (int k = 0; k < kDeep; ++k) {
      const uint32_t i = done + k * kThreads + threadIdx.x;
      s[k] = i < count ? __ldg(map + (back ? end - 1 - (int)i : from + (int)i)) : -1;
    }
    uint32_t best = 0xffffffffu;
#pragma unroll
    for (int k = kDeep - 1; k >= 0; --k)
      if (s[k] >= 0 && s[k] < num_slots) best = done + k * kThreads + threadIdx.x;
    if (!__syncthreads_or(best != 0xffffffffu)) continue;
    best = __reduce_min_sync(0xffffffffu, best);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = best;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) best = min(best, red[w]);
    __syncthreads();
    return back ? end - 1 - (int)best : from + (int)best;
  }
  return -1;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 4 ? 6 : 10) cache_append_kernel(const __grid_constant__ AppendParams p) {
  __shared__ int64_t window[kWindow];  // slots of tokens first - 1 ..
  __shared__ uint32_t begin[kMaxChunk / 32];  // a bit where a block's tokens begin
  __shared__ uint32_t red[kWarps];
  __shared__ int unsure, tail;  // a token that may begin a block; where the last block may go on past the window (-1: none)
  __shared__ int64_t tail_block;
  const int first = blockIdx.x * p.chunk, h = blockIdx.y, which = blockIdx.z;
  const int n = min(p.chunk, p.T - first);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int bs = p.block_size, shift = p.block_shift;
  const T* x0 = static_cast<const T*>(which ? p.x[1] : p.x[0]);
  const int64_t stride = which ? p.stride[1] : p.stride[0];
  auto valid = [&](int64_t s) { return s >= 0 && s < p.num_slots; };
  if (threadIdx.x == 0) unsure = tail = -1;
  const int held = 1 + p.chunk + bs;
  const int window_end = min(p.T, first + p.chunk + bs);  // the first token past it
  for (int i = threadIdx.x; i < held; i += kThreads) {
    const int t = first + i - 1;
    window[i] = t >= 0 && t < p.T ? __ldg(p.slot_map + t) : -1;
  }
  __syncthreads();
  // Most rows that this CTA will read are its own tokens': their lines come to L2 while the window is looked at.
  if (p.chunk == kMaxChunk) {
    constexpr int kLines = D * sizeof(T) / 128;
    for (int i = threadIdx.x; i < n * kLines; i += kThreads) {
      const T* line = x0 + (int64_t)(first + i / kLines) * stride + h * D + i % kLines * (D / kLines);
      if (valid(window[1 + i / kLines])) asm volatile("prefetch.global.L2 [%0];" ::"l"(line));
    }
  }
  auto slot_of = [&](int t) -> int64_t {  // -1 past the map
    const int i = t - first + 1;
    return i < held ? window[i] : t < p.T ? __ldg(p.slot_map + t) : -1;
  };
  bool begins = false;
  for (int i0 = warp * 32; i0 < n; i0 += kThreads) {
    // a token begins its block's tokens unless the nearest token before it
    // that has a slot (almost always the one before) is of the same block
    const int i = i0 + lane;
    const int64_t s = i < n ? window[i + 1] : -1;
    int64_t prev = i < n ? window[i] : -1;
    for (unsigned look = __ballot_sync(0xffffffffu, valid(s) && !valid(prev) && first + i > 0); look; look &= look - 1) {
      const int l = __ffs(look) - 1;
      int64_t near = -1;
      for (int j = i0 + l; j >= 0; j -= 32) {  // 32 of the window's tokens at a time, back from the one before
        const int64_t y = j >= lane ? window[j - lane] : -1;
        const unsigned m = __ballot_sync(0xffffffffu, valid(y));
        if (!m) continue;
        near = __shfl_sync(0xffffffffu, y, __ffs(m) - 1);
        break;
      }
      if (lane == l) prev = near;
    }
    const bool b = valid(s) && !(valid(prev) && prev >> shift == s >> shift);
    if (b && !valid(prev) && first > 1) unsure = i;  // only one token has none before it in the window
    const unsigned m = __ballot_sync(0xffffffffu, b);
    if (lane == 0) begin[i0 >> 5] = m;
    begins |= m != 0u;
  }
  if (!__syncthreads_or(begins)) return;
  const int at = unsure;
  if (at >= 0) {  // no slot from one token before the chunk to here: the nearest one lies before that
    const int t = find_slot(p.slot_map, p.num_slots, 0, first - 1, true, red);
    if (threadIdx.x == 0 && t >= 0 && __ldg(p.slot_map + t) >> shift == window[at + 1] >> shift)
      begin[at >> 5] &= ~(1u << (at & 31));
    __syncthreads();
  }
  uint8_t* cache = which ? p.cache[1] : p.cache[0];
  float* scales = which ? p.scales[1] : p.scales[0];

  // Length of the run from token t with slot s: tokens t + 1 .. whose slots rise by one inside the block, 32 looked at a time.
  auto run_length = [&](int t, int64_t s, int64_t* next) {
    const int off = (int)s & (bs - 1);
    for (int len = 1;;) {
      const int64_t y = slot_of(t + len + lane);
      const unsigned m = __ballot_sync(0xffffffffu, off + len + lane < bs && y == s + len + lane);
      const int more = m == 0xffffffffu ? 32 : __ffs(~m) - 1;
      len += more;
      if (more == 32) continue;
      *next = __shfl_sync(0xffffffffu, y, more);
      return len;
    }
  };
  for (int pass = 0; pass < 2; ++pass) {  // blocks with a short first run by warps, then the others by the CTA
    int mine = 0;
    for (int j = 0; j < n; j += 32)
    for (uint32_t todo = begin[j >> 5]; todo != 0; todo &= todo - 1) {
      if (pass == 0 && (mine++ % kWarps) != warp) continue;
      const int i = j + __ffs(todo) - 1;
      // the block's runs, one after the other (more than one only where skipped tokens lie between them)
      int t = first + i;
      int64_t s = window[i + 1];
      const int64_t blk = s >> shift;
      bool later = false;
      for (;;) {
        const int off = (int)s & (bs - 1);
        int64_t next;  // the slot after the run; -1 where it names no row
        const int len = run_length(t, s, &next);
        if (!later && (len * (D / 16) <= kWarpPieces) != (pass == 0)) break;
        const T* x = x0 + (int64_t)t * stride + h * D;
        const int64_t tile = blk * p.Hkv + h;
        if (pass == 0)
          append_run<T, D, 32>(x, stride, cache + tile * bs * D, scales + tile, off, len, lane, nullptr);
        else
          append_run<T, D, kThreads>(x, stride, cache + tile * bs * D, scales + tile, off, len, threadIdx.x, red);
        t += len;
        while (!valid(next) && t < window_end) {  // over skipped tokens
          const int64_t y = t + lane < window_end ? window[t + lane - first + 1] : -1;
          const unsigned m = __ballot_sync(0xffffffffu, valid(y));
          const int skip = m ? __ffs(m) - 1 : min(32, window_end - t);
          t += skip;
          if (m) next = __shfl_sync(0xffffffffu, y, skip);
        }
        if (!valid(next) && t < p.T && lane == 0) {  // it may go on behind the window (as no other block here can)
          tail = t;
          tail_block = blk;
        }
        if (!valid(next) || next >> shift != blk) break;
        s = next;
        later = true;
        if (pass == 0) __syncwarp(); else __syncthreads();  // the block's rows and scale are written
      }
    }
  }

  // the last block's runs behind the window, past any number of skipped tokens
  if (window_end == p.T) return;
  __syncthreads();
  const int64_t blk = tail_block;
  for (int t = tail; t >= 0;) {
    t = find_slot(p.slot_map, p.num_slots, t, p.T, false, red);
    if (t < 0) break;
    const int64_t s = __ldg(p.slot_map + t);
    if (s >> shift != blk) break;
    int64_t next;
    const int len = run_length(t, s, &next);
    const int64_t tile = blk * p.Hkv + h;
    append_run<T, D, kThreads>(x0 + (int64_t)t * stride + h * D, stride, cache + tile * bs * D, scales + tile,
                               (int)s & (bs - 1), len, threadIdx.x, red);
    t += len;
    __syncthreads();  // the block's rows and scale are written
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
  // few tokens: a CTA for every four, to spread single-token runs; many: one for every 64, which a run or two begin in
  p.chunk = p.T <= 1024 ? 4 : kMaxChunk;
  if (dtype == ATTN_BF16) return launch_t<__nv_bfloat16>(p, stream);
  if (dtype == ATTN_F16) return launch_t<__half>(p, stream);
  return launch_t<float>(p, stream);
}

}  // namespace gb300_attn
