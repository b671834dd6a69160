// rope.cu -- rotary positions: pairs of values of a row turned by the angle
// position * frequency of the pair, times a factor.
//   (a, b) -> f (a cos - b sin, b cos + a sin),  (a, b) = (x_i, x_{i + R/2}) or (x_2i, x_2i+1)
// and the inverse (which with the same factor is the transpose, so it takes
// gradients back) with -sin.  Values past the first R of a row are kept.
//
// Angles: position * frequency in fp32 would be off by 2^-24 of itself, whole
// turns for far positions.  A frequency becomes turns a position as a 64-bit
// binary fraction (53 bits of it times 1 / (2 pi)); its product with the
// position, modulo 2^64, is the angle modulo a turn to position * 2^-62 turns,
// of which the upper 32 bits go to sincospi.  Rotation in fp32, rounded once.
//
// Bound: HBM, each value read and written once.  A warp has a token: its lanes
// share out the sines and cosines of the token's pairs, through shared memory,
// and go over its heads, 16-byte pieces of 8 pairs (4 in f32) each, so that the
// 60 instructions of a pair's angle are paid once a token, not once a head.
// With few tokens a token's heads are spread over more warps.
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "../../include/attn.h"
#include "paged4_internal.h"

namespace gb300_attn {
namespace {

constexpr int kThreads = 128;
constexpr int kPairs = 256;  // pairs whose sines and cosines a warp holds at a time

// Turns a position of radians a position, modulo 1, times 2^64.
__device__ __forceinline__ uint64_t turns(double radians) {
  const uint64_t bits = (uint64_t)__double_as_longlong(radians);
  const int e = (int)((bits >> 52) & 2047) - 1023;
  const uint64_t m = (bits << 11) | (1ull << 63);              // radians = m 2^(e - 63)
  const uint64_t hi = __umul64hi(m, 0x28be60db9391054bull);    // 2^64 / (2 pi): turns = hi 2^(e - 63)
  const int up = e + 1;                                        // times 2^64
  uint64_t f = up >= 64 ? 0 : up >= 0 ? hi << up : up > -64 ? hi >> -up : 0;
  if (e == -1023) f = 0;  // zero, or too small to turn anything
  return (bits >> 63) ? 0 - f : f;
}

// The last request whose rows begin at or before row t (as upper bound over q_starts[1 .. B]), by a warp: 32 entries
// a step.  B: none.
__device__ __forceinline__ int find_request(const int32_t* q_starts, int B, int t, int lane) {
  int lo = 0, hi = B;  // the first index i of [lo, hi] with q_starts[i + 1] > t
  while (lo < hi) {
    const int step = (hi - lo + 31) / 32;
    const int i = lo + (lane + 1) * step - 1;  // last entry of lane's part
    const bool past = i >= hi || __ldg(q_starts + i + 1) > t;
    const unsigned m = __ballot_sync(0xffffffffu, past);
    if (m == 0) return hi;
    const int part = __ffs(m) - 1;
    lo += part * step;
    hi = min(hi, lo + step - 1);
  }
  return lo;
}

template <typename T, int VP>
struct Vec;  // 16 bytes of T, or one value
template <typename T, int VP>
struct alignas(VP == 1 ? sizeof(T) : 16) Vec { T x[VP]; };

template <typename T>
__device__ __forceinline__ float to_f(T x) {
  if constexpr (std::is_same<T, float>::value) return x;
  else if constexpr (std::is_same<T, __half>::value) return __half2float(x);
  else return __bfloat162float(x);
}
template <typename T>
__device__ __forceinline__ T from_f(float x) {
  if constexpr (std::is_same<T, float>::value) return x;
  else if constexpr (std::is_same<T, __half>::value) return __float2half_rn(x);
  else return __float2bfloat16_rn(x);
}

// VP pairs a lane: a 16-byte piece of both halves, or two pieces side by side; VP = 1 where rows allow no such pieces.
template <typename T, int VP, bool INTER>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeParams p, int row_lanes, int heads_each,
                                                        int parts) {
  using V = Vec<T, VP>;
  __shared__ __align__(16) float cs[kThreads / 32][2][kPairs];  // cosines and sines of a warp's pairs
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t warps = (int64_t)gridDim.x * (kThreads / 32), all = (int64_t)p.T * parts;
  const int half = p.rotary / 2;
  const int sub = lane / row_lanes, i0 = lane - sub * row_lanes, subs = 32 / row_lanes;
  float* cw = cs[warp][0];
  float* nw = cs[warp][1];
  for (int64_t item = (int64_t)blockIdx.x * (kThreads / 32) + warp; item < all; item += warps) {
    const int t = (int)(item / parts);
    const int h0 = (int)(item - (int64_t)t * parts) * heads_each, h1 = min(h0 + heads_each, p.H[0] + p.H[1]);
    int64_t pos;
    if (p.positions) {
      pos = __ldg(p.positions + t);
    } else {
      const int b = find_request(p.q_starts, p.B, t, lane);
      if (b >= p.B || t < __ldg(p.q_starts)) continue;  // rows of no request
      pos = (int64_t)__ldg(p.totals + b) - __ldg(p.q_starts + b + 1) + t;
    }
    // head h of q and k together lies at in(h) + h D
    const int hq = p.H[0];
    const T* in0 = static_cast<const T*>(p.in[0]) + (int64_t)t * p.in_stride[0];
    const T* in1 = static_cast<const T*>(p.in[1]) + (int64_t)t * p.in_stride[1] - (int64_t)hq * p.D;
    T* out0 = static_cast<T*>(p.out[0]) + (int64_t)t * p.out_stride[0];
    T* out1 = static_cast<T*>(p.out[1]) + (int64_t)t * p.out_stride[1] - (int64_t)hq * p.D;
    auto in = [&](int h) { return (h >= hq ? in1 : in0) + (int64_t)h * p.D; };
    auto out = [&](int h) { return (h >= hq ? out1 : out0) + (int64_t)h * p.D; };
    for (int pair0 = 0; pair0 < half; pair0 += kPairs) {
      const int pairs = min(kPairs, half - pair0);
      __syncwarp();  // the last ones have been read
      for (int i = lane; i < pairs; i += 32) {
        const uint64_t turn = (uint64_t)pos * turns(__ldg(p.freq + pair0 + i));
        float c, n;
        sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &n, &c);
        cw[i] = c * p.scale;
        nw[i] = n * (p.inverse ? -p.scale : p.scale);
      }
      __syncwarp();
      for (int i = i0; i * VP < pairs; i += row_lanes) {
        float c[VP], n[VP];
#pragma unroll
        for (int k = 0; k < VP; ++k) {
          c[k] = cw[i * VP + k];
          n[k] = nw[i * VP + k];
        }
        const int at = INTER ? 2 * (pair0 + i * VP) : pair0 + i * VP, to = INTER ? at + VP : at + half;
#pragma unroll 4
        for (int h = h0 + sub; h < h1; h += subs) {
          const T* src = in(h);
          T* dst = out(h);
          V u = *reinterpret_cast<const V*>(src + at), v = *reinterpret_cast<const V*>(src + to);
#pragma unroll
          for (int k = 0; k < VP; ++k) {
            T& a = INTER && VP > 1 ? (2 * k < VP ? u.x[(2 * k) % VP] : v.x[(2 * k) % VP]) : u.x[k];
            T& b = INTER && VP > 1 ? (2 * k < VP ? u.x[(2 * k + 1) % VP] : v.x[(2 * k + 1) % VP]) : v.x[k];
            const float x = to_f(a), y = to_f(b);
            a = from_f<T>(x * c[k] - y * n[k]);
            b = from_f<T>(y * c[k] + x * n[k]);
          }
          *reinterpret_cast<V*>(dst + at) = u;
          *reinterpret_cast<V*>(dst + to) = v;
        }
      }
    }
    // what is not turned: lanes over the pieces of all heads
    const int rest = (p.D - p.rotary) / VP;
    if (rest == 0 || (p.in_place[0] && p.in_place[1])) continue;
    int h = h0, i = lane;
    while (i >= rest && h < h1) {
      i -= rest;
      ++h;
    }
    while (h < h1) {
      V x[4];
      int hs[4], is[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        hs[k] = h;
        is[k] = i;
        if (h < h1) x[k] = reinterpret_cast<const V*>(in(h) + p.rotary)[i];
        i += 32;
        while (i >= rest && h < h1) {
          i -= rest;
          ++h;
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (hs[k] < h1 && !(hs[k] >= hq ? p.in_place[1] : p.in_place[0]))
          reinterpret_cast<V*>(out(hs[k]) + p.rotary)[is[k]] = x[k];
    }
  }
}

template <typename T, int VP, bool INTER>
cudaError_t launch(const RopeParams& p, cudaStream_t stream) {
  const int nvec = p.rotary / 2 / VP;
  int row_lanes = 1;
  while (row_lanes < nvec && row_lanes < 32) row_lanes *= 2;
  const int H = p.H[0] + p.H[1], subs = 32 / row_lanes;
  int heads_each = H;
  // few tokens: more warps a token, down to one head a lane
  while (heads_each > subs && (int64_t)p.T * ((H + heads_each - 1) / heads_each) < 152 * 16)
    heads_each = std::max(subs, (heads_each + 1) / 2);
  const int parts = (H + heads_each - 1) / heads_each;
  const int64_t blocks = ((int64_t)p.T * parts + kThreads / 32 - 1) / (kThreads / 32);
  rope_kernel<T, VP, INTER><<<(unsigned)std::min<int64_t>(blocks, 1 << 30), kThreads, 0, stream>>>(p, row_lanes, heads_each, parts);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_t(const RopeParams& p, bool inter, cudaStream_t stream) {
  constexpr int VP = 16 / sizeof(T);
  bool wide = p.D % VP == 0 && p.rotary % (2 * VP) == 0;
  for (int i = 0; i < 2; ++i)
    if (p.H[i] > 0)
      wide = wide && p.in_stride[i] % VP == 0 && p.out_stride[i] % VP == 0 &&
             ((reinterpret_cast<uintptr_t>(p.in[i]) | reinterpret_cast<uintptr_t>(p.out[i])) & 15) == 0;
  if (wide) return inter ? launch<T, VP, true>(p, stream) : launch<T, VP, false>(p, stream);
  return inter ? launch<T, 1, true>(p, stream) : launch<T, 1, false>(p, stream);
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, bool interleaved, int dtype, cudaStream_t stream) {
  if (dtype == ATTN_BF16) return launch_t<__nv_bfloat16>(p, interleaved, stream);
  if (dtype == ATTN_F16) return launch_t<__half>(p, interleaved, stream);
  return launch_t<float>(p, interleaved, stream);
}

}  // namespace gb300_attn
