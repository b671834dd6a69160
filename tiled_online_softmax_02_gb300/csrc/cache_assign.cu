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
// The work is a few prefix sums over the rows and a scatter of 8 bytes a token:
// latency, not bandwidth, is the bound.  So it is one launch with as few
// dependent memory accesses as the task has (lengths -> table entries -> free
// list -> slots), everything else in shared memory.  A small step is one CTA; a
// larger one a thread-block cluster of eight, whose CTAs own ranges of rows,
// exchange their sums through distributed shared memory, and order their
// global writes by cluster barriers (release / acquire): blocks are returned
// before any is taken, and every row is complete before a slot is read from
// it.  The order of every list follows the rows, never the timing.
//
// Measured (one GB300, device time): 64 requests, a new token each, 8.0 us on
// one CTA; 48 requests with up to 2048 new tokens, 65536 slots, 15.0 us on the
// cluster.
#include <cstdint>

#include "device_common.cuh"
#include "paged_internal.h"

namespace gb300_attn {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kClusterCtas = 8;

struct Sums {  // of a CTA's rows
  int lacks;   // table entries that need a block
  int given;   // blocks of finished rows
  int flags;   // 1 << AssignResult of every problem met, kListFlag and kResetFlag
  int bad;     // whether a block that they would take is none
};
constexpr int kListFlag = 1 << 16;   // an entry near the top of the free stack names no block
constexpr int kResetFlag = 1 << 17;  // a finished row has an entry that is not -1

__device__ __forceinline__ int peer_i32(const void* ptr, int rank) {
  uint32_t remote;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_u32(ptr)), "r"(rank));
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(remote) : "memory");
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

// Shared memory: int starts[B + 1] (row starts), past[B] (0 for finished
// rows), then of the CTA's own rows lacks[rows] and given[rows] (counts, then
// offsets within the CTA).
template <bool CLUSTER>
__global__ void __launch_bounds__(kThreads) cache_assign_kernel(const __grid_constant__ AssignParams p,
                                                                int rows_per_cta) {
  extern __shared__ __align__(16) int smem[];
  int* starts = smem;
  int* past = starts + p.B + 1;
  int* lacks = past + p.B;
  int* given = lacks + rows_per_cta;
  __shared__ Sums sums;
  __shared__ long long warp_tokens[kWarps];
  const int rank = CLUSTER ? blockIdx.x : 0, ctas = CLUSTER ? kClusterCtas : 1;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int row0 = min(rank * rows_per_cta, p.B);
  const int rows = min(rows_per_cta, p.B - row0);
  auto sync_all = [] {
    if (CLUSTER) asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
    else __syncthreads();
  };
  auto finished = [&](int b) { return p.finished != nullptr && __ldg(p.finished + b) != 0; };

  if (tid == 0) sums.flags = 0;
  const int count0 = __ldcg(p.free_count);  // written after the last barrier but one, when every CTA has read it

  // ---- row starts: a prefix sum over all rows, in every CTA
  const int per = (p.B + kThreads - 1) / kThreads;  // consecutive rows of a thread
  const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
  long long mine = 0;
  int bad = 0;
  for (int b = b0; b < b1; ++b) {
    const int n = __ldg(p.added + b), h = __ldg(p.past + b);
    bad |= (n < 0 || h < 0) ? 1 << kAssignLength : 0;
    past[b] = finished(b) ? 0 : max(h, 0);
    mine += max(n, 0);
  }
  const long long inc = warp_inclusive(mine, lane);
  if (lane == 31) warp_tokens[warp] = inc;
  __syncthreads();
  if (bad) atomicOr(&sums.flags, bad);
  long long tokens = 0, before = inc - mine;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += warp_tokens[w];
    tokens += warp_tokens[w];
  }
  for (int b = b0; b < b1; ++b) {
    starts[b] = (int)min(before, (long long)INT32_MAX);
    before += max(__ldg(p.added + b), 0);
  }
  if (tid == 0) starts[p.B] = (int)min(tokens, (long long)INT32_MAX);
  __syncthreads();

  // ---- what every row of this CTA needs and gives
  // (The free stack's topmost entries, one a thread, come with them: were one taken that names no block, the step could
  // not be done.  Which are taken is known only with the sums; where one of these is bad, or more are taken, that is
  // looked at once more below.)
  const int top = min(max(count0, 0), p.num_blocks) - 1 - (rank * kThreads + tid);
  const int top_entry = top >= 0 ? __ldcg(p.free_blocks + top) : 0;
  auto need_of = [&](int b) {
    return ((long long)past[b] + max(__ldg(p.added + b), 0) + p.block_size - 1) >> p.block_shift;
  };
  // (128 entries of two rows in flight at a time: a row's loads do not wait for one another)
  for (int r0 = warp; r0 < rows; r0 += 2 * kWarps) {
    int need[2], upto[2], n_lack[2] = {0, 0}, n_given[2] = {0, 0}, flags = 0;
    bool fin[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = r0 + i * kWarps, b = row0 + min(r, rows - 1);
      const long long want = need_of(b);
      if (r < rows && (want > p.width || (long long)past[b] + max(__ldg(p.added + b), 0) > INT32_MAX))
        flags = 1 << kAssignRowShort;
      fin[i] = finished(b);
      need[i] = (int)min(want, (long long)p.width);
      upto[i] = r < rows ? (fin[i] ? p.width : need[i]) : 0;
    }
    for (int c0 = 0; c0 < max(upto[0], upto[1]); c0 += 128) {
      int e[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int c = c0 + 32 * k + lane;
          e[i][k] = c < upto[i] ? __ldcg(p.tables + (int64_t)(row0 + r0 + i * kWarps) * p.width + c) : 0;
        }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int c = c0 + 32 * k + lane;
          if (c >= upto[i]) continue;
          flags |= e[i][k] >= p.num_blocks ? 1 << kAssignCorrupt : 0;
          flags |= fin[i] && e[i][k] != -1 ? kResetFlag : 0;
          n_given[i] += fin[i] && e[i][k] >= 0;
          n_lack[i] += fin[i] ? c < need[i] : e[i][k] < 0;
        }
    }
    flags = __reduce_or_sync(0xffffffffu, flags);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int l = __reduce_add_sync(0xffffffffu, n_lack[i]), g = __reduce_add_sync(0xffffffffu, n_given[i]);
      if (lane == 0 && r0 + i * kWarps < rows) {
        lacks[r0 + i * kWarps] = l;
        given[r0 + i * kWarps] = g;
      }
    }
    if (lane == 0 && flags) atomicOr(&sums.flags, flags);
  }
  if (top >= 0 && (top_entry < 0 || top_entry >= p.num_blocks)) atomicOr(&sums.flags, kListFlag);
  __syncthreads();

  // ---- offsets within the CTA, and the CTA's sums
  if (warp == 0) {
    int l0 = 0, g0 = 0;
    for (int r = 0; r < rows; r += 32) {
      const bool in = r + lane < rows;
      const int l = in ? lacks[r + lane] : 0, g = in ? given[r + lane] : 0;
      const int li = warp_inclusive(l, lane), gi = warp_inclusive(g, lane);
      if (in) {
        lacks[r + lane] = l0 + li - l;
        given[r + lane] = g0 + gi - g;
      }
      l0 += __shfl_sync(0xffffffffu, li, 31);
      g0 += __shfl_sync(0xffffffffu, gi, 31);
    }
    if (lane == 0) {
      sums.lacks = l0;
      sums.given = g0;
    }
  }
  sync_all();

  // ---- offsets of this CTA, totals, and whether the step can be done
  int lack_base = 0, given_base = 0, flags = 0;
  long long lack_all = 0, given_all = 0;
  if (CLUSTER) {
    for (int c = 0; c < kClusterCtas; ++c) {
      const int l = peer_i32(&sums.lacks, c), g = peer_i32(&sums.given, c);
      flags |= peer_i32(&sums.flags, c);
      if (c < rank) {
        lack_base += l;
        given_base += g;
      }
      lack_all += l;
      given_all += g;
    }
  } else {
    flags = sums.flags;
    lack_all = sums.lacks;
    given_all = sums.given;
  }
  const long long count1 = count0 + given_all;
  int res = kAssignOk;
  if (flags & (1 << kAssignLength)) res = kAssignLength;
  else if (flags & (1 << kAssignRowShort)) res = kAssignRowShort;
  else if (tokens > p.T) res = kAssignTokens;
  else if ((flags & (1 << kAssignCorrupt)) || count0 < 0 || count1 > p.num_blocks) res = kAssignCorrupt;
  else if (lack_all > count1) res = kAssignNoBlocks;
  if (res == kAssignOk && ((flags & kListFlag) || lack_all - given_all > ctas * kThreads)) {
    bool bad = false;  // among the entries that this CTA's rows take; those of finished rows have been looked at
    for (int n = tid; n < sums.lacks; n += kThreads) {
      const long long at = count1 - 1 - lack_base - n;
      const int e = at < count0 ? __ldcg(p.free_blocks + at) : 0;
      bad |= e < 0 || e >= p.num_blocks;
    }
    bad = __syncthreads_or(bad);
    if (CLUSTER) {
      if (tid == 0) sums.bad = bad;
      sync_all();
      for (int c = 0; c < kClusterCtas; ++c) bad |= peer_i32(&sums.bad, c) != 0;
    }
    if (bad) res = kAssignCorrupt;
  }
  const bool ok = res == kAssignOk;

  // ---- row starts and totals; blocks of finished rows go onto the stack
  for (int r = tid; r < rows; r += kThreads) {
    const int b = row0 + r;
    p.q_starts[b] = ok ? starts[b] : 0;
    p.totals[b] = ok ? past[b] + __ldg(p.added + b) : __ldg(p.past + b);
  }
  if (rank == 0 && tid == 0) {
    p.q_starts[p.B] = ok ? starts[p.B] : 0;
    *p.result = res;
  }
  if (ok && (flags & kResetFlag)) {
    for (int r = warp; r < rows; r += kWarps) {
      const int b = row0 + r;
      if (!finished(b)) continue;
      int32_t* row = p.tables + (int64_t)b * p.width;
      long long at = (long long)count0 + given_base + given[r];
      for (int c0 = 0; c0 < p.width; c0 += 128) {
        int e[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) e[k] = c0 + 32 * k + lane < p.width ? __ldcg(row + c0 + 32 * k + lane) : -1;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const unsigned held = __ballot_sync(0xffffffffu, e[k] >= 0);
          if (e[k] >= 0) p.free_blocks[at + __popc(held & ((1u << lane) - 1u))] = e[k];
          if (c0 + 32 * k + lane < p.width) row[c0 + 32 * k + lane] = -1;
          at += __popc(held);
        }
      }
    }
  }
  if (CLUSTER || (flags & kResetFlag)) sync_all();  // also: every CTA has read free_count

  // ---- rows take their blocks from the top of the stack
  if (ok) {
    for (int r = warp; r < rows; r += kWarps) {
      const int b = row0 + r;
      const int need = (int)need_of(b);
      int32_t* row = p.tables + (int64_t)b * p.width;
      long long nth = (long long)lack_base + lacks[r];
      if ((r + 1 < rows ? lacks[r + 1] : sums.lacks) == lacks[r]) continue;  // it lacks none
      for (int c0 = 0; c0 < need; c0 += 128) {
        int e[4];
        bool lack[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) e[k] = c0 + 32 * k + lane < need ? __ldcg(row + c0 + 32 * k + lane) : 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          lack[k] = e[k] < 0;
          const unsigned m = __ballot_sync(0xffffffffu, lack[k]);
          if (lack[k]) e[k] = __ldcg(p.free_blocks + (count1 - 1 - nth - __popc(m & ((1u << lane) - 1u))));
          nth += __popc(m);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (lack[k]) row[c0 + 32 * k + lane] = e[k];
      }
    }
    if (rank == 0 && tid == 0) *p.free_count = (int)(count1 - lack_all);
  }
  sync_all();

  // ---- slots of the tokens (of this CTA's share of the map), four a thread in flight
  const int live = ok ? starts[p.B] : 0;
  const int step = ctas * kThreads;
  for (int64_t t0 = rank * kThreads + tid; t0 < p.T; t0 += 4 * (int64_t)step) {
    int64_t slot[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t t = t0 + (int64_t)i * step;
      slot[i] = -1;
      if (t >= live) continue;
      int lo = 0, hi = p.B - 1;  // the last row whose start is <= t (rows without tokens share a start with the next)
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (starts[mid] <= t) lo = mid; else hi = mid - 1;
      }
      const int pos = past[lo] + (int)t - starts[lo];
      const int blk = __ldcg(p.tables + (int64_t)lo * p.width + (pos >> p.block_shift));
      slot[i] = ((int64_t)blk << p.block_shift) + (pos & (p.block_size - 1));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t t = t0 + (int64_t)i * step;
      if (t < p.T) p.slot_map[t] = slot[i];
    }
  }
}

template <bool CLUSTER>
cudaError_t launch_t(const AssignParams& p, cudaStream_t stream) {
  const int ctas = CLUSTER ? kClusterCtas : 1;
  const int rows = (p.B + ctas - 1) / ctas;
  const size_t smem = ((size_t)2 * p.B + 1 + 2 * (size_t)rows) * 4;
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(cache_assign_kernel<CLUSTER>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (2 * kAssignMaxRequests + 1 + 2 * kAssignMaxRequests) * 4);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)ctas, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cache_assign_kernel<CLUSTER>, p, rows);
}

}  // namespace

cudaError_t launch_cache_assign(const AssignParams& p, cudaStream_t stream) {
  // one CTA where its 32 warps and 1024 threads cover the rows and tokens in a few turns, else the cluster
  return p.B <= 4 * kWarps && p.T <= 4 * kThreads ? launch_t<false>(p, stream) : launch_t<true>(p, stream);
}

}  // namespace gb300_attn
