// attn_paged.cu -- attention over the paged 8-bit KV cache.
//
// Row (t, h) of request b, at position pos = total_b - new_b + i:
//   visible keys [lo, hi): lo = window ? max(0, pos + 1 - window) : 0,
//                          hi = causal ? min(total_b, pos + 1) : total_b
//   s_j = scale * k_scale[block(j), h] <q, k8_j>, soft-capped when asked
//   out = sum_j softmax(s)_j v_scale[block(j), h] v8_j, 0 without a visible key
//
// The plainest form: one warp a row, one key at a time, fp32 throughout.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "device_common.cuh"
#include "paged_internal.h"

namespace gb300_attn {
namespace {

__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f32(float x, __half* y) { *y = __float2half_rn(x); }
__device__ __forceinline__ void from_f32(float x, __nv_bfloat16* y) { *y = __float2bfloat16_rn(x); }

__device__ __forceinline__ float e4m3(uint8_t x) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw(x, __NV_E4M3);
  return __half2float(*reinterpret_cast<const __half*>(&h));
}

template <typename T, int D>
__global__ void __launch_bounds__(128) attn_paged_rows(const __grid_constant__ PagedParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (row >= (int64_t)p.T * p.Hq) return;
  const int t = (int)(row / p.Hq), h = (int)(row % p.Hq), kvh = h / p.group;
  int lo = 0, hi = p.B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.q_starts[mid] <= t) lo = mid; else hi = mid - 1;
  }
  const int b = lo;
  if (t < p.q_starts[b] || t >= p.q_starts[b + 1]) return;
  const int64_t pos = (int64_t)p.totals[b] - p.q_starts[b + 1] + t;
  const int64_t cap = (int64_t)p.width * p.block_size;
  int64_t k0 = p.local_window > 0 ? pos + 1 - p.local_window : 0, k1 = p.totals[b];
  if (p.causal && pos + 1 < k1) k1 = pos + 1;
  if (k0 < 0) k0 = 0;
  if (k1 > cap) k1 = cap;
  constexpr int V = D / 32;
  float q[V], o[V];
  const T* qr = static_cast<const T*>(p.q) + (int64_t)t * p.q_stride + h * D + lane * V;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    q[i] = to_f32(qr[i]);
    o[i] = 0.0f;
  }
  float m = -INFINITY, l = 0.0f;
  for (int64_t j = k0; j < k1; ++j) {
    const int blk = p.tables[(int64_t)b * p.width + j / p.block_size];
    const bool ok = blk >= 0 && blk < p.num_blocks;
    if (!ok && lane == 0) atomicOr(p.status, kStatusBadBlock);
    const int64_t tile = (int64_t)blk * p.Hkv + kvh;
    const int64_t at = (tile * p.block_size + j % p.block_size) * D + lane * V;
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) s += ok ? q[i] * e4m3(p.k_cache[at + i]) : 0.0f;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    s *= p.scale * (ok ? p.k_scales[tile] : 1.0f);
    if (p.softcap > 0.0f) s = p.softcap * tanhf(s / p.softcap);
    const float mn = fmaxf(m, s);
    const float keep = mn == -INFINITY ? 1.0f : expf(m - mn), w = mn == -INFINITY ? 0.0f : expf(s - mn);
    l = l * keep + w;
    const float wv = w * (ok ? p.v_scales[tile] : 0.0f);
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = o[i] * keep + (ok ? wv * e4m3(p.v_cache[at + i]) : 0.0f);
    m = mn;
  }
  T* out = static_cast<T*>(p.out) + row * D + lane * V;
#pragma unroll
  for (int i = 0; i < V; ++i) from_f32(l > 0.0f ? o[i] / l : 0.0f, out + i);
  if (p.lse && lane == 0) p.lse[row] = l > 0.0f ? m + logf(l) : -INFINITY;
}

template <typename T>
cudaError_t launch_rows(const PagedParams& p, cudaStream_t stream) {
  const unsigned grid = (unsigned)(((int64_t)p.T * p.Hq + 3) / 4);
  if (p.D == 128) attn_paged_rows<T, 128><<<grid, 128, 0, stream>>>(p);
  else attn_paged_rows<T, 64><<<grid, 128, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_paged(const PagedParams& p, bool bf16, cudaStream_t stream) {
  return bf16 ? launch_rows<__nv_bfloat16>(p, stream) : launch_rows<__half>(p, stream);
}

}  // namespace gb300_attn
