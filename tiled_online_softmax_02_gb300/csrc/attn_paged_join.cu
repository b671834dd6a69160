// attn_paged_join.cu -- joins the partial rows of units that the borders
// between CTAs cut (paged_sched.cuh).  Part k of a row holds O_k = sum of
// 2^(t - m_k) v8, its maximum m_k and L_k = sum of 2^(t - m_k) / v_scale; with
// M = max m_k the row is
//   sum_k 2^(m_k - M) O_k / sum_k 2^(m_k - M) L_k   (0 when the latter is 0).
// Bound: latency; the partial rows lie in L2.  One warp a row, lanes over d;
// the parts' (m, L) are read 32 at a time and their O_k in flight together.
// A programmatic dependent of the attention kernel: it may be scheduled while
// that one drains, and waits for all of it before it reads.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "paged_internal.h"

namespace gb300_attn {
namespace {

constexpr int kWarps = 4;

template <int D, bool BF16>
__global__ void __launch_bounds__(kWarps * 32) attn_paged_join_kernel(const PagedCut* cuts, const float* ws_o,
                                                                      const float2* ws_ml, int unit_rows, int Hq,
                                                                      int group, float ml_log2, uint16_t* out,
                                                                      float* lse) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c = blockIdx.x, lane = threadIdx.x & 31;
  const int r = blockIdx.y * kWarps + (threadIdx.x >> 5);
  const PagedCut cut = cuts[c];
  if (r >= cut.rows || cut.parts == 0) return;
  auto slot = [&](int k) { return (int64_t)(k == 0 ? 2 * c + 1 : 2 * (c + k)) * unit_rows + r; };
  float M = -INFINITY;
  for (int k = lane; k < cut.parts; k += 32) M = fmaxf(M, ws_ml[slot(k)].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  constexpr int V = D / 32;
  float acc[V], L = 0.0f;
#pragma unroll
  for (int v = 0; v < V; ++v) acc[v] = 0.0f;
  for (int k0 = 0; k0 < cut.parts; k0 += 32) {
    float w = 0.0f;
    if (k0 + lane < cut.parts) {
      const float2 ml = ws_ml[slot(k0 + lane)];
      w = exp2f(ml.x - M);
      L = fmaf(w, ml.y, L);
    }
    const int n = min(32, cut.parts - k0);
#pragma unroll 8
    for (int k = 0; k < n; ++k) {
      const float wk = __shfl_sync(0xffffffffu, w, k);
      const float* o = ws_o + slot(k0 + k) * D + lane * V;
      if constexpr (V == 4) {
        const float4 x = *reinterpret_cast<const float4*>(o);
        acc[0] = fmaf(wk, x.x, acc[0]);
        acc[1] = fmaf(wk, x.y, acc[1]);
        acc[2] = fmaf(wk, x.z, acc[2]);
        acc[3] = fmaf(wk, x.w, acc[3]);
      } else {
        const float2 x = *reinterpret_cast<const float2*>(o);
        acc[0] = fmaf(wk, x.x, acc[0]);
        acc[1] = fmaf(wk, x.y, acc[1]);
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
  const float inv = L == 0.0f ? 0.0f : 1.0f / L;
  const int x = cut.row0 + r;
  const int64_t row = (int64_t)(cut.token0 + x / group) * Hq + cut.head0 + x % group;
  uint32_t packed[V / 2];
#pragma unroll
  for (int v = 0; v < V / 2; ++v) {
    if constexpr (BF16) {
      const __nv_bfloat162 y = __floats2bfloat162_rn(acc[2 * v] * inv, acc[2 * v + 1] * inv);
      packed[v] = *reinterpret_cast<const uint32_t*>(&y);
    } else {
      const __half2 y = __floats2half2_rn(acc[2 * v] * inv, acc[2 * v + 1] * inv);
      packed[v] = *reinterpret_cast<const uint32_t*>(&y);
    }
  }
  uint16_t* dst = out + row * D + lane * V;
  if constexpr (V == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(packed[0], packed[1]);
  else *reinterpret_cast<uint32_t*>(dst) = packed[0];
  if (lse != nullptr && lane == 0)
    lse[row] = L == 0.0f ? -INFINITY : (M + (log2f(L) - ml_log2)) * 0.6931471805599453f;
}

template <int D, bool BF16>
cudaError_t launch_t(const PagedLaunch& L, cudaStream_t stream) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)L.grid, (unsigned)((L.rows + kWarps - 1) / kWarps), 1);
  cfg.blockDim = dim3(kWarps * 32, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn_paged_join_kernel<D, BF16>, (const PagedCut*)L.cuts, (const float*)L.ws_o,
                            (const float2*)L.ws_ml, L.rows, L.c.Hq, L.c.group, L.ml_log2,
                            static_cast<uint16_t*>(L.c.out), L.c.lse);
}

}  // namespace

cudaError_t launch_attn_paged_join(const PagedLaunch& L, bool bf16, cudaStream_t stream) {
  if (L.c.D == 128) return bf16 ? launch_t<128, true>(L, stream) : launch_t<128, false>(L, stream);
  return bf16 ? launch_t<64, true>(L, stream) : launch_t<64, false>(L, stream);
}

}  // namespace gb300_attn
