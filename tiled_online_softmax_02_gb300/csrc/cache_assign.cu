// cache_assign.cu -- who owns which cache block: one step's block tables, row
// starts and token slots from the requests' lengths, on the GPU, so that a
// serving step needs no host round trip and can be captured into a graph.
//
// For request b with past_b cached and new_b added tokens (past_b = 0 when it
// just replaced a finished one, whose blocks go back first):
//   need_b  = ceil((past_b + new_b) / block_size) table entries; those below
//             need_b that hold no block (< 0) take one each from the top of
//             the free stack, in row order
//   start_b = sum of new over earlier requests
//   slot of token start_b + i: block of position past_b + i, row by row.
// Entries already held are kept, so repeating a step changes nothing and a
// request whose length shrank (rejected draft tokens) keeps its blocks.
//
// The work is two prefix sums over a few hundred rows and a scatter of 8
// bytes a token: latency, not bandwidth, is the bound.  So it is one launch:
// one thread-block cluster, whose CTAs each own a range of rows and exchange
// their sums through distributed shared memory.  Blocks are returned before
// any is taken, and every row is complete before a token's slot is read from
// it, by cluster barriers (release / acquire on the global writes too).  The
// order of every list follows the rows, never the timing.
#include <cstdint>

#include "device_common.cuh"
#include "paged_internal.h"

namespace gb300_attn {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;

struct Sums {  // of a CTA's rows
  long long tokens;
  int lacks;   // table entries that need a block
  int given;   // blocks of finished rows
  int flags;   // 1 << AssignResult of every problem met
};

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

__device__ __forceinline__ int peer_i32(const void* ptr, int rank) {
  uint32_t remote;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_u32(ptr)), "r"(rank));
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(remote) : "memory");
  return v;
}

__device__ __forceinline__ long long peer_i64(const void* ptr, int rank) {
  uint32_t remote;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_u32(ptr)), "r"(rank));
  long long v;
  asm volatile("ld.shared::cluster.s64 %0, [%1];" : "=l"(v) : "r"(remote) : "memory");
  return v;
}

template <typename T>
__device__ __forceinline__ T warp_inclusive(T v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// Shared memory: int lacks[rows], int given[rows] (counts, then offsets within
// the CTA), long long tokens[rows] likewise, and the row starts int [B + 1].
__global__ void __launch_bounds__(kThreads) cache_assign_kernel(const AssignParams p, int rows_per_cta, int ctas) {
  extern __shared__ __align__(16) uint8_t smem[];
  long long* tokens = reinterpret_cast<long long*>(smem);
  int* lacks = reinterpret_cast<int*>(tokens + rows_per_cta);
  int* given = lacks + rows_per_cta;
  int* starts = given + rows_per_cta;
  __shared__ Sums sums;
  const int rank = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row0 = min(rank * rows_per_cta, p.B);
  const int rows = min(rows_per_cta, p.B - row0);

  if (threadIdx.x == 0) sums.flags = 0;
  const int count0 = *p.free_count;  // read by every CTA before any barrier, written after the last
  __syncthreads();

  // ---- what every row of this CTA needs and gives
  for (int r = warp; r < rows; r += kWarps) {
    const int b = row0 + r;
    const int past = p.past[b], added = p.added[b];
    const bool fin = p.finished != nullptr && p.finished[b] != 0;
    int flags = (past < 0 || added < 0) ? 1 << kAssignLength : 0;
    const long long total = (fin ? 0ll : (long long)max(past, 0)) + max(added, 0);
    long long need = (total + p.block_size - 1) / p.block_size;
    if (need > p.width || total > INT32_MAX) flags |= 1 << kAssignRowShort;
    if (need > p.width) need = p.width;
    const int32_t* row = p.tables + (int64_t)b * p.width;
    int n_lack = 0, n_given = 0;
    const int upto = fin ? p.width : (int)need;
    for (int c = lane; c < upto; c += 32) {
      const int e = row[c];
      if (e >= p.num_blocks) flags |= 1 << kAssignCorrupt;
      if (fin) {
        n_given += e >= 0;
        n_lack += c < need;
      } else {
        n_lack += e < 0;
      }
    }
    n_lack = __reduce_add_sync(0xffffffffu, n_lack);
    n_given = __reduce_add_sync(0xffffffffu, n_given);
    flags = __reduce_or_sync(0xffffffffu, flags);
    if (lane == 0) {
      lacks[r] = n_lack;
      given[r] = n_given;
      tokens[r] = max(added, 0);
      if (flags) atomicOr(&sums.flags, flags);
    }
  }
  __syncthreads();

  // ---- offsets within the CTA, and the CTA's sums
  if (warp == 0) {
    int l0 = 0, g0 = 0;
    long long t0 = 0;
    for (int r = 0; r < rows; r += 32) {
      const bool in = r + lane < rows;
      const int l = in ? lacks[r + lane] : 0, g = in ? given[r + lane] : 0;
      const long long t = in ? tokens[r + lane] : 0;
      const int li = warp_inclusive(l, lane), gi = warp_inclusive(g, lane);
      const long long ti = warp_inclusive(t, lane);
      if (in) {
        lacks[r + lane] = l0 + li - l;
        given[r + lane] = g0 + gi - g;
        tokens[r + lane] = t0 + ti - t;
      }
      l0 += __shfl_sync(0xffffffffu, li, 31);
      g0 += __shfl_sync(0xffffffffu, gi, 31);
      t0 += __shfl_sync(0xffffffffu, ti, 31);
    }
    if (lane == 0) {
      sums.lacks = l0;
      sums.given = g0;
      sums.tokens = t0;
    }
  }
  if (ctas > 1) cluster_sync(); else __syncthreads();

  // ---- offsets of this CTA, totals, and whether the step can be done
  int lack_base = 0, given_base = 0, flags = 0;
  long long token_base = 0, lack_all = 0, given_all = 0, token_all = 0;
  for (int c = 0; c < ctas; ++c) {
    const int l = ctas > 1 ? peer_i32(&sums.lacks, c) : sums.lacks;
    const int g = ctas > 1 ? peer_i32(&sums.given, c) : sums.given;
    const long long t = ctas > 1 ? peer_i64(&sums.tokens, c) : sums.tokens;
    flags |= ctas > 1 ? peer_i32(&sums.flags, c) : sums.flags;
    if (c < rank) {
      lack_base += l;
      given_base += g;
      token_base += t;
    }
    lack_all += l;
    given_all += g;
    token_all += t;
  }
  const long long count1 = count0 + given_all;
  int res = kAssignOk;
  if (flags & (1 << kAssignLength)) res = kAssignLength;
  else if (flags & (1 << kAssignRowShort)) res = kAssignRowShort;
  else if (token_all > p.T) res = kAssignTokens;
  else if ((flags & (1 << kAssignCorrupt)) || count0 < 0 || count1 > p.num_blocks) res = kAssignCorrupt;
  else if (lack_all > count1) res = kAssignNoBlocks;
  const bool ok = res == kAssignOk;

  // ---- blocks of finished rows go onto the stack; row starts and totals
  for (int r = warp; r < rows; r += kWarps) {
    const int b = row0 + r;
    const bool fin = p.finished != nullptr && p.finished[b] != 0;
    if (lane == 0) {
      p.q_starts[b] = ok ? (int)(token_base + tokens[r]) : 0;
      p.totals[b] = ok ? (fin ? 0 : p.past[b]) + p.added[b] : p.past[b];
    }
    if (!ok || !fin) continue;
    int32_t* row = p.tables + (int64_t)b * p.width;
    long long at = (long long)count0 + given_base + given[r];
    for (int c0 = 0; c0 < p.width; c0 += 32) {
      const int c = c0 + lane;
      const int e = c < p.width ? row[c] : -1;
      const unsigned held = __ballot_sync(0xffffffffu, e >= 0);
      if (e >= 0) p.free_blocks[at + __popc(held & ((1u << lane) - 1u))] = e;
      if (c < p.width) row[c] = -1;
      at += __popc(held);
    }
  }
  if (rank == 0 && threadIdx.x == 0) {
    p.q_starts[p.B] = ok ? (int)token_all : 0;
    *p.result = res;
  }
  if (ctas > 1) cluster_sync(); else __syncthreads();

  // ---- rows take their blocks from the top of the stack
  if (ok) {
    for (int r = warp; r < rows; r += kWarps) {
      const int b = row0 + r;
      const bool fin = p.finished != nullptr && p.finished[b] != 0;
      const int need = (int)(((long long)(fin ? 0 : p.past[b]) + p.added[b] + p.block_size - 1) / p.block_size);
      int32_t* row = p.tables + (int64_t)b * p.width;
      long long nth = (long long)lack_base + lacks[r];
      for (int c0 = 0; c0 < need; c0 += 32) {
        const int c = c0 + lane;
        const bool lack = c < need && __ldcg(row + c) < 0;
        const unsigned m = __ballot_sync(0xffffffffu, lack);
        if (lack) row[c] = __ldcg(p.free_blocks + (count1 - 1 - nth - __popc(m & ((1u << lane) - 1u))));
        nth += __popc(m);
      }
    }
    if (rank == 0 && threadIdx.x == 0) *p.free_count = (int)(count1 - lack_all);
  }
  if (ctas > 1) cluster_sync(); else __syncthreads();

  // ---- slots of the tokens (of this CTA's share of the map)
  for (int i = threadIdx.x; i <= p.B; i += kThreads) starts[i] = __ldcg(p.q_starts + i);
  __syncthreads();
  const int live = starts[p.B];
  for (int64_t t = (int64_t)rank * kThreads + threadIdx.x; t < p.T; t += (int64_t)ctas * kThreads) {
    int64_t slot = -1;
    if (t < live) {
      int lo = 0, hi = p.B - 1;  // the last row whose start is <= t (rows without tokens share a start with the next)
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (starts[mid] <= t) lo = mid; else hi = mid - 1;
      }
      const bool fin = p.finished != nullptr && p.finished[lo] != 0;
      const int pos = (fin ? 0 : p.past[lo]) + (int)t - starts[lo];
      const int blk = __ldcg(p.tables + (int64_t)lo * p.width + pos / p.block_size);
      slot = (int64_t)blk * p.block_size + pos % p.block_size;
    }
    p.slot_map[t] = slot;
  }
}

}  // namespace

cudaError_t launch_cache_assign(const AssignParams& p, cudaStream_t stream) {
  // one CTA where its 16 warps and 512 threads cover the rows and tokens in a few turns, else a cluster of 8
  const int ctas = (p.B <= 2 * kWarps && p.T <= 4 * kThreads) ? 1 : 8;
  const int rows = (p.B + ctas - 1) / ctas;
  const size_t smem = (size_t)rows * 16 + (size_t)(p.B + 1) * 4;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)ctas, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaError_t e = cudaFuncSetAttribute(cache_assign_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (kAssignMaxRequests / 8) * 16 + (kAssignMaxRequests + 1) * 4);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cache_assign_kernel, p, rows, ctas);
}

}  // namespace gb300_attn
