// attn_paged4_join.cu -- joins the partial rows that the few-rows kernel over the
// 4-bit cache leaves of units cut between CTAs (paged_sched.cuh), where a unit
// has few parts: a batch of requests, whose units outnumber the borders.  The
// definition is attn_paged_join.cu's: with M = max m_k a row is
//   sum_k 2^(m_k - M) O_k / sum_k 2^(m_k - M) 2^8 L_k   (0 when the latter is 0).
// Bound: latency.  A CTA has a unit, a row's parts are shared out to as many of
// its eight warps as there are to a row, and each has four parts in flight.  (A
// CTA a row, as that kernel has them for the many parts of few units, is eight
// times the CTAs, most of them without a row: 64 requests of 4 kv heads take 41.8 us with it, 39.4 with this.)
// A programmatic dependent of the attention kernel: it may be scheduled while
// that one drains, and waits for all of it before it reads.
#include "paged4_internal.h"
#include "paged_join.cuh"

namespace gb300_attn {
namespace {

constexpr int kWarps = 8, kFlight = 4;

template <int D, bool BF16>
__global__ void __launch_bounds__(kWarps * 32) attn_paged4_join_kernel(const PagedCut* cuts, const float* ws_o,
                                                                       const float2* ws_ml, int unit_rows, int Hq, int group,
                                                                       float ml_log2, uint16_t* out, float* lse) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int V = D / 32;
  __shared__ float sum_o[kWarps][D];
  __shared__ float2 sum_ml[kWarps];
  const int c = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const PagedCut cut = cuts[c];
  if (cut.parts == 0) return;
  const int share = cut.rows > 4 ? 1 : cut.rows > 2 ? 2 : cut.rows > 1 ? 4 : 8;  // warps of a row
  const int sub = warp % share, step = kWarps / share;
  for (int r0 = 0; r0 < cut.rows; r0 += step) {
    const int r = r0 + warp / share;
    float M = -INFINITY, L = 0.0f, acc[V];
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] = 0.0f;
    for (int k0 = sub; r < cut.rows && k0 < cut.parts; k0 += kFlight * share) {
      RowVec<D> o[kFlight];
      float2 ml[kFlight];
#pragma unroll
      for (int i = 0; i < kFlight; ++i) {
        const int k = k0 + i * share;
        ml[i] = make_float2(-INFINITY, 0.0f);
        if (k < cut.parts) {
          const int64_t slot = (int64_t)(k == 0 ? 2 * c + 1 : 2 * (c + k)) * unit_rows + r;
          ml[i] = ws_ml[slot];
          o[i].load(ws_o + slot * D, lane);
        }
      }
      const float Mn = fmaxf(fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x)), M);  // finite: part k0 is there
      const float keep = exp2f(M - Mn);
      L *= keep;
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] *= keep;
#pragma unroll
      for (int i = 0; i < kFlight; ++i) {
        if (k0 + i * share >= cut.parts) continue;
        const float w = exp2f(ml[i].x - Mn);
        L = fmaf(w, ml[i].y, L);
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] = fmaf(w, o[i].x[v], acc[v]);
      }
      M = Mn;
    }
    if (share > 1) {  // the row's warps meet at the first of them (all rows are there in one pass of the loop)
#pragma unroll
      for (int v = 0; v < V; ++v) sum_o[warp][lane * V + v] = acc[v];
      if (lane == 0) sum_ml[warp] = make_float2(M, L);
      __syncthreads();
      if (sub == 0 && r < cut.rows) {
        float Ma = M;  // part 0 is this warp's: finite
        for (int i = 1; i < share; ++i) Ma = fmaxf(Ma, sum_ml[warp + i].x);  // warps without a part hold -inf
        const float keep = exp2f(M - Ma);
        L *= keep;
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] *= keep;
        for (int i = 1; i < share; ++i) {
          const float w = exp2f(sum_ml[warp + i].x - Ma);
          L = fmaf(w, sum_ml[warp + i].y, L);
#pragma unroll
          for (int v = 0; v < V; ++v) acc[v] = fmaf(w, sum_o[warp + i][lane * V + v], acc[v]);
        }
        M = Ma;
      }
    }
    if (sub == 0 && r < cut.rows) store_row<D, BF16>(cut, r, Hq, group, ml_log2, out, lse, lane, acc, M, L);
  }
}

template <int D, bool BF16>
cudaError_t launch_t(const PagedLaunch& L, cudaStream_t stream) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)L.grid, 1, 1);
  cfg.blockDim = dim3(kWarps * 32, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn_paged4_join_kernel<D, BF16>, (const PagedCut*)L.cuts, (const float*)L.ws_o,
                            (const float2*)L.ws_ml, L.rows, L.c.Hq, L.c.group, L.ml_log2, static_cast<uint16_t*>(L.c.out),
                            L.c.lse);
}

}  // namespace

cudaError_t launch_attn_paged4_join(const PagedLaunch& L, bool bf16, cudaStream_t stream) {
  if (L.c.D == 128) return bf16 ? launch_t<128, true>(L, stream) : launch_t<128, false>(L, stream);
  return bf16 ? launch_t<64, true>(L, stream) : launch_t<64, false>(L, stream);
}

}  // namespace gb300_attn
