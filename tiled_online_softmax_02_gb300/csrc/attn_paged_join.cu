// attn_paged_join.cu -- joins the partial rows of units that the borders
// between CTAs cut (paged_sched.cuh).  Part k of a row holds O_k = sum of
// 2^(t - m_k) v8, its maximum m_k and L_k = 2^-8 sum of 2^(t - m_k) / v_scale; with
// M = max m_k the row is
//   sum_k 2^(m_k - M) O_k / sum_k 2^(m_k - M) 2^8 L_k   (0 when the latter is 0).
// L_k takes its factor as two halves: it may be as large as the factor is small,
// where the parts' V scales differ.
// Bound: latency; the partial rows lie in L2.  Lanes go over d, and a warp has
// several parts of a row, or several rows, in flight.
// Measured under the profiler (caches flushed): 8 us for 2 MB of partial rows,
// 304 cut units of 8 rows; 13 us for 38 MB, 152 cut units of 256 rows.
// A programmatic dependent of the attention kernel: it may be scheduled while
// that one drains, and waits for all of it before it reads.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "paged_internal.h"

namespace gb300_attn {
namespace {

constexpr int kWarps = 8;
constexpr int kUnitRows = 32;  // rows of a CTA where units have many

template <int D>
struct RowVec {
  static constexpr int V = D / 32;  // values of a lane
  float x[V];
  __device__ __forceinline__ void load(const float* row, int lane) {
    if constexpr (V == 4) {
      const float4 v = *reinterpret_cast<const float4*>(row + lane * 4);
      x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
    } else {
      const float2 v = *reinterpret_cast<const float2*>(row + lane * 2);
      x[0] = v.x; x[1] = v.y;
    }
  }
};

template <int D, bool BF16>
__device__ __forceinline__ void store_row(const PagedCut& cut, int r, int Hq, int group, float ml_log2, uint16_t* out,
                                          float* lse, int lane, const float (&acc)[D / 32], float M, float L) {
  constexpr int V = D / 32;
  const float inv = L == 0.0f ? 0.0f : kPagedSumFactor * (1.0f / L);
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

// Many rows, mostly of two parts (long work: a unit is cut once or twice): a
// warp takes two rows and two parts at a time.  (Four rows at a time: 2 us more
// on 152 cut units of 256 rows, the registers leaving fewer warps.)
template <int D, bool BF16>
__global__ void __launch_bounds__(kWarps * 32) attn_paged_join_kernel(const PagedCut* cuts, const float* ws_o,
                                                                             const float2* ws_ml, int unit_rows,
                                                                             int Hq, int group, float ml_log2,
                                                                             uint16_t* out, float* lse) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int V = D / 32, kRows = 2, kParts = 2;
  const int c = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const PagedCut cut = cuts[c];
  const int end = min(cut.rows, ((int)blockIdx.y + 1) * kUnitRows);
  if (cut.parts == 0) return;
  auto slot = [&](int k, int r) { return (int64_t)(k == 0 ? 2 * c + 1 : 2 * (c + k)) * unit_rows + r; };
  for (int r0 = blockIdx.y * kUnitRows + warp * kRows; r0 < end; r0 += kWarps * kRows) {
    float M[kRows], L[kRows], acc[kRows][V];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      M[i] = -INFINITY;
      L[i] = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) acc[i][v] = 0.0f;
    }
    for (int k0 = 0; k0 < cut.parts; k0 += kParts) {
      // lane 2 i + j holds (m, L) of row i, part j
      const int mr = min(r0 + ((lane >> 1) & 1), cut.rows - 1), mk = k0 + (lane & 1);
      float2 ml = make_float2(-INFINITY, 0.0f);
      if (mk < cut.parts) ml = ws_ml[slot(mk, mr)];
      RowVec<D> o[kRows][kParts];
#pragma unroll
      for (int i = 0; i < kRows; ++i)
#pragma unroll
        for (int j = 0; j < kParts; ++j)
          if (r0 + i < end && k0 + j < cut.parts) o[i][j].load(ws_o + slot(k0 + j, r0 + i) * D, lane);
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const float m0 = __shfl_sync(0xffffffffu, ml.x, 2 * i), m1 = __shfl_sync(0xffffffffu, ml.x, 2 * i + 1);
        const float l0 = __shfl_sync(0xffffffffu, ml.y, 2 * i), l1 = __shfl_sync(0xffffffffu, ml.y, 2 * i + 1);
        const float Mn = fmaxf(fmaxf(M[i], m0), m1);  // finite: part k0 is there
        const float hk = exp2f(0.5f * (M[i] - Mn)), h0 = exp2f(0.5f * (m0 - Mn)), h1 = exp2f(0.5f * (m1 - Mn));
        const float keep = hk * hk, w0 = h0 * h0, w1 = h1 * h1;
        M[i] = Mn;
        L[i] = fmaf(h1, l1 * h1, fmaf(h0, l0 * h0, L[i] * hk * hk));
        const bool two = k0 + 1 < cut.parts;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          acc[i][v] = fmaf(w0, o[i][0].x[v], acc[i][v] * keep);
          if (two) acc[i][v] = fmaf(w1, o[i][1].x[v], acc[i][v]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i)
      if (r0 + i < end) store_row<D, BF16>(cut, r0 + i, Hq, group, ml_log2, out, lse, lane, acc[i], M[i], L[i]);
  }
}

// Few rows and often many parts (decode): one CTA a row, its warps over the
// parts, whose (m, L) and O_k are read at the same time.
template <int D, bool BF16>
__global__ void __launch_bounds__(kWarps * 32) attn_paged_join_rows_kernel(const PagedCut* cuts, const float* ws_o,
                                                                           const float2* ws_ml, int unit_rows, int Hq,
                                                                           int group, float ml_log2, uint16_t* out,
                                                                           float* lse) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int V = D / 32;
  __shared__ float sum_o[kWarps][D];
  __shared__ float2 sum_ml[kWarps];
  const int c = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = blockIdx.y;
  const PagedCut cut = cuts[c];
  if (r >= cut.rows || cut.parts == 0) return;
  auto slot = [&](int k) { return (int64_t)(k == 0 ? 2 * c + 1 : 2 * (c + k)) * unit_rows + r; };
  // this warp's parts: warp, warp + 8, ..., four at a time, under its own maximum
  float M = -INFINITY, L = 0.0f, acc[V];
#pragma unroll
  for (int v = 0; v < V; ++v) acc[v] = 0.0f;
  for (int k0 = warp; k0 < cut.parts; k0 += 4 * kWarps) {
    RowVec<D> o[4];
    float2 ml[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int k = k0 + i * kWarps;
      ml[i] = make_float2(-INFINITY, 0.0f);
      if (k < cut.parts) {
        ml[i] = ws_ml[slot(k)];
        o[i].load(ws_o + slot(k) * D, lane);
      }
    }
    const float Mn = fmaxf(fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x)), M);
    const float hk = exp2f(0.5f * (M - Mn)), keep = hk * hk;  // Mn is finite: part k0 is there
    L = L * hk * hk;
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] *= keep;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (k0 + i * kWarps >= cut.parts) continue;
      const float hw = exp2f(0.5f * (ml[i].x - Mn)), w = hw * hw;
      L = fmaf(hw, ml[i].y * hw, L);
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] = fmaf(w, o[i].x[v], acc[v]);
    }
    M = Mn;
  }
#pragma unroll
  for (int v = 0; v < V; ++v) sum_o[warp][lane * V + v] = acc[v];
  if (lane == 0) sum_ml[warp] = make_float2(M, L);
  __syncthreads();
  if (warp != 0) return;
  float Ma = -INFINITY;
#pragma unroll
  for (int k = 0; k < kWarps; ++k) Ma = fmaxf(Ma, sum_ml[k].x);  // warps without a part hold -inf
  L = 0.0f;
#pragma unroll
  for (int v = 0; v < V; ++v) acc[v] = 0.0f;
#pragma unroll
  for (int k = 0; k < kWarps; ++k) {
    const float hw = exp2f(0.5f * (sum_ml[k].x - Ma)), w = hw * hw;
    L = fmaf(hw, sum_ml[k].y * hw, L);
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] = fmaf(w, sum_o[k][lane * V + v], acc[v]);
  }
  store_row<D, BF16>(cut, r, Hq, group, ml_log2, out, lse, lane, acc, Ma, L);
}

template <int D, bool BF16>
cudaError_t launch_t(const PagedLaunch& L, cudaStream_t stream) {
  const bool by_row = L.rows != kPagedTcRows;  // the decode kernel's units
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)L.grid, (unsigned)(by_row ? L.rows : (L.rows + kUnitRows - 1) / kUnitRows), 1);
  cfg.blockDim = dim3(kWarps * 32, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, by_row ? attn_paged_join_rows_kernel<D, BF16> : attn_paged_join_kernel<D, BF16>,
                            (const PagedCut*)L.cuts, (const float*)L.ws_o, (const float2*)L.ws_ml, L.rows, L.c.Hq,
                            L.c.group, L.ml_log2, static_cast<uint16_t*>(L.c.out), L.c.lse);
}

}  // namespace

cudaError_t launch_attn_paged_join(const PagedLaunch& L, bool bf16, cudaStream_t stream) {
  if (L.c.D == 128) return bf16 ? launch_t<128, true>(L, stream) : launch_t<128, false>(L, stream);
  return bf16 ? launch_t<64, true>(L, stream) : launch_t<64, false>(L, stream);
}

}  // namespace gb300_attn
