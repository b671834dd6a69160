// rope.cu -- rotary positions: pairs of values of a row turned by the angle
// position * frequency of the pair, times a factor.
//   (a, b) -> f (a cos - b sin, b cos + a sin),  (a, b) = (x_i, x_{i + R/2}) or (x_2i, x_2i+1)
// and the inverse (which with the same factor is the transpose, so it takes
// gradients back) with -sin.  Values past the first R of a row are kept.
//
// Angles: position * frequency in fp32 would be off by 2^-24 of itself, whole
// turns for far positions.  A frequency becomes turns a position as a 64-bit
// binary fraction (53 bits of it times 1 / (2 pi), 64 or 128 bits of that); its
// product with the position, modulo 2^64, is the angle modulo a turn to position
// * 2^-58 turns, of which the upper 32 bits go to sincospi.  Rotation in fp32,
// rounded once.
//
// Bound: HBM, each value read and written once.  A warp has a token: its lanes
// share out the sines and cosines of the token's pairs, through shared memory,
// and go over its heads, 16-byte pieces of 8 pairs (4 in f32) each, so that the
// 60 instructions of a pair's angle are paid once a token, not once a head.
// With few tokens a token's heads are spread over more warps.
//
// Measured (one GB300, device time): 64 tokens of 32 + 8 heads, D = 128, bf16 3.4
// us; 8192 tokens 28.5 us (5.9 TB/s, 88% of a copy's rate), half of each head
// turned, pairs side by side 29.4; f32, 4096 tokens of 24 heads 16.4.  One row of a
// lane in flight in place of two 34.7 us, three 31.3, angles by every lane for
// its own pairs 72.
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "../../include/attn.h"
#include "paged4.cuh"
#include "paged4_internal.h"

namespace gb300_attn {
namespace {

constexpr int kThreads = 32;  // a warp a CTA: with four, 31.1 us in place of 29.3 for 8K rows of 40 heads
constexpr int kBatch = 2;   // rows of a lane in flight
constexpr int kPairs = 256;  // pairs whose sines and cosines a warp holds at a time

// Turns a position of radians a position, modulo 1, times 2^64: off by 2^6 at most for radians below 2^62 in size, so that
// a position's angle is off by 2^-27 turns, less than its rounding.
__device__ __forceinline__ uint64_t turns(double radians) {
  const uint64_t bits = (uint64_t)__double_as_longlong(radians);
  const int e = (int)((bits >> 52) & 2047) - 1023;
  const uint64_t m = (bits << 11) | (1ull << 63);              // radians = m 2^(e - 63)
  uint64_t hi = __umul64hi(m, 0x28be60db9391054bull);          // 2^64 / (2 pi): turns = hi 2^(e - 63)
  const int up = e + 1;                                        // times 2^64
  uint64_t f = up >= 0 ? hi << (up & 63) : up > -64 ? hi >> -up : 0;
  if (up > 6) {  // the shift brings in bits below hi's: 64 more of 1 / (2 pi)
    const uint64_t below = __umul64hi(m, 0x7f09d5f47d4d3770ull), lo = m * 0x28be60db9391054aull + below;
    hi = __umul64hi(m, 0x28be60db9391054aull) + (lo < below ? 1 : 0);
    f = up < 64 ? hi << up | lo >> (64 - up) : up < 128 ? lo << (up - 64) : 0;
  }
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
    const bool past = i >= hi || q_starts[i + 1] > t;
    const unsigned m = __ballot_sync(0xffffffffu, past);
    if (m == 0) return hi;
    const int part = __ffs(m) - 1;
    lo += part * step;
    hi = min(hi, lo + step - 1);
  }
  return lo;
}

// What a lane takes of a row at a time: 16 bytes of T as they lie, or one value.
template <typename T, int VP>
struct Vec { uint32_t w[4]; };
template <typename T>
struct Vec<T, 1> { T x; };

template <typename T, int VP>
__device__ __forceinline__ Vec<T, VP> load_vec(const T* p) {
  Vec<T, VP> v;
  if constexpr (VP == 1) {
    v.x = *p;
  } else {
    const uint4 x = *reinterpret_cast<const uint4*>(p);
    v.w[0] = x.x; v.w[1] = x.y; v.w[2] = x.z; v.w[3] = x.w;
  }
  return v;
}
template <typename T, int VP>
__device__ __forceinline__ void store_vec(T* p, const Vec<T, VP>& v) {
  if constexpr (VP == 1) *p = v.x;
  else *reinterpret_cast<uint4*>(p) = make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]);
}

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
// Two 16-bit values of a word, and back.
template <typename T>
__device__ __forceinline__ float2 unpack(uint32_t w) {
  if constexpr (std::is_same<T, __half>::value) return __half22float2(*reinterpret_cast<const __half2*>(&w));
  else return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <typename T>
__device__ __forceinline__ uint32_t pack(float a, float b) {
  if constexpr (std::is_same<T, __half>::value) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

// Turns the VP pairs of u and v: values of u with those of v, or neighbours (u first).
template <typename T, int VP, bool INTER>
__device__ __forceinline__ void turn_pairs(Vec<T, VP>& u, Vec<T, VP>& v, const float (&c)[VP], const float (&n)[VP]) {
  auto re = [&](float x, float y, int k) { return x * c[k] - y * n[k]; };
  auto im = [&](float x, float y, int k) { return y * c[k] + x * n[k]; };
  if constexpr (VP == 1) {
    const float x = to_f(u.x), y = to_f(v.x);
    u.x = from_f<T>(re(x, y, 0));
    v.x = from_f<T>(im(x, y, 0));
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint32_t& a = !INTER ? u.w[k] : k < 2 ? u.w[2 * k & 3] : v.w[2 * k & 3];
      uint32_t& b = !INTER ? v.w[k] : k < 2 ? u.w[(2 * k & 3) + 1] : v.w[(2 * k & 3) + 1];
      const float x = __uint_as_float(a), y = __uint_as_float(b);
      a = __float_as_uint(re(x, y, k));
      b = __float_as_uint(im(x, y, k));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 x = unpack<T>(u.w[i]), y = unpack<T>(v.w[i]);
      if constexpr (INTER) {
        u.w[i] = pack<T>(re(x.x, x.y, i), im(x.x, x.y, i));
        v.w[i] = pack<T>(re(y.x, y.y, i + 4), im(y.x, y.y, i + 4));
      } else {
        u.w[i] = pack<T>(re(x.x, y.x, 2 * i), re(x.y, y.y, 2 * i + 1));
        v.w[i] = pack<T>(im(x.x, y.x, 2 * i), im(x.y, y.y, 2 * i + 1));
      }
    }
  }
}

// VP pairs a lane: a 16-byte piece of both halves, or two pieces side by side; VP = 1 where rows allow no such pieces.
template <typename T, int VP, bool INTER>
__global__ void __launch_bounds__(kThreads, 32) rope_kernel(const __grid_constant__ RopeParams p, int row_lanes, int rest_lanes,
                                                           int heads_each, int parts) {
  after_earlier_kernels();
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
      pos = p.positions[t];
    } else {
      const int b = find_request(p.q_starts, p.B, t, lane);
      if (b >= p.B || t < p.q_starts[0]) continue;  // rows of no request
      pos = (int64_t)p.totals[b] - p.q_starts[b + 1] + t;
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
        const uint64_t turn = (uint64_t)pos * turns(p.freq[pair0 + i]);
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
        for (int h = h0 + sub; h < h1; h += kBatch * subs) {  // rows in flight together: the outputs may be the inputs
          V u[kBatch], v[kBatch];
#pragma unroll
          for (int m = 0; m < kBatch; ++m) {
            const T* src = in(h + m * subs);
            if (h + m * subs < h1) {
              u[m] = load_vec<T, VP>(src + at);
              v[m] = load_vec<T, VP>(src + to);
            }
          }
#pragma unroll
          for (int m = 0; m < kBatch; ++m) {
            if (h + m * subs >= h1) break;
            turn_pairs<T, VP, INTER>(u[m], v[m], c, n);
            T* dst = out(h + m * subs);
            store_vec<T, VP>(dst + at, u[m]);
            store_vec<T, VP>(dst + to, v[m]);
          }
        }
      }
    }
    // what is not turned, where it has to move
    const int rest = (p.D - p.rotary) / VP, r0 = p.in_place[0] ? max(h0, hq) : h0, r1 = p.in_place[1] ? min(h1, hq) : h1;
    const int rsub = lane / rest_lanes, rsubs = 32 / rest_lanes;
    for (int i = lane - rsub * rest_lanes; i < rest; i += rest_lanes) {
      for (int h = r0 + rsub; h < r1; h += kBatch * rsubs) {
        V x[kBatch];
#pragma unroll
        for (int m = 0; m < kBatch; ++m)
          if (h + m * rsubs < r1) x[m] = load_vec<T, VP>(in(h + m * rsubs) + p.rotary + i * VP);
#pragma unroll
        for (int m = 0; m < kBatch; ++m)
          if (h + m * rsubs < r1) store_vec<T, VP>(out(h + m * rsubs) + p.rotary + i * VP, x[m]);
      }
    }
  }
}

// Lanes that a row's n pieces get: a power of two.
int lanes_for(int n) {
  int lanes = 1;
  while (lanes < n && lanes < 32) lanes *= 2;
  return lanes;
}

template <typename T, int VP, bool INTER>
cudaError_t launch(const RopeParams& p, cudaStream_t stream) {
  const int row_lanes = lanes_for(p.rotary / 2 / VP), rest_lanes = lanes_for((p.D - p.rotary) / VP);
  const int H = p.H[0] + p.H[1], subs = 32 / row_lanes;
  const int64_t sms = paged_sm_count();
  int heads_each = H;
  // few tokens: more warps a token, down to one head a lane
  while (heads_each > subs && (int64_t)p.T * ((H + heads_each - 1) / heads_each) < sms * 16)
    heads_each = std::max(subs, (heads_each + 1) / 2);
  const int parts = (H + heads_each - 1) / heads_each;
  const int64_t blocks = ((int64_t)p.T * parts + kThreads / 32 - 1) / (kThreads / 32);
  return launch_early(rope_kernel<T, VP, INTER>, (unsigned)std::min<int64_t>(blocks, 1 << 30), kThreads, 0, stream, p, row_lanes,
                      rest_lanes, heads_each, parts);
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
