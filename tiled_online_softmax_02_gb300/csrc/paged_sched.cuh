// paged_sched.cuh -- how the paged attention kernels share out their work.
//
// A unit is up to NR query rows of one (request, kv head) -- row r of it is
// token r / group, query head r % group of that kv head -- with the key tiles
// (128 keys) some of its rows see.  Units are laid end to end, request by
// request, head by head, row tile by row tile, and the line of all key tiles
// is cut into equal pieces, one a CTA: ragged lengths leave no CTA with more
// than its share, and a unit cut by a border between CTAs leaves partial rows
// that a second kernel joins (a CTA holds at most two: of its first and of
// its last unit).  Everything follows from the lengths and the grid, so equal
// calls give equal bits.
#pragma once

#include <cstdint>

#include "device_common.cuh"
#include "paged_internal.h"

namespace gb300_attn {

constexpr int kPagedKeys = 128;  // keys of a tile

// A request's packed rows and lengths.
struct PagedReq {
  int s0, n;        // first row, rows
  int64_t total;    // cached tokens, these rows' among them
};

__device__ __forceinline__ PagedReq paged_req(const PagedParams& p, int b) {
  PagedReq r;
  r.s0 = min(max(__ldg(p.q_starts + b), 0), p.T);
  r.n = min(max(__ldg(p.q_starts + b + 1), r.s0), p.T) - r.s0;
  r.total = __ldg(p.totals + b);
  return r;
}

// Visible keys [x, y) of the request's row qi; none where y <= x.  Both ends
// rise with qi.
__device__ __forceinline__ int2 paged_limits(const PagedParams& p, const PagedReq& q, int qi) {
  const int64_t pos = q.total - q.n + qi, cap = (int64_t)p.width * p.block_size;
  int64_t lo = p.local_window > 0 ? pos + 1 - p.local_window : 0;
  int64_t hi = q.total < cap ? q.total : cap;
  if (p.causal && pos + 1 < hi) hi = pos + 1;
  return make_int2((int)max(lo, (int64_t)0), (int)max(hi, (int64_t)0));
}

struct PagedUnit {
  PagedReq q;
  int b, kvh, rt;
  int row0, rows;   // rows [row0, row0 + rows) of the kv head's n * group
  int tb, te;       // key tiles some row sees
};

// Row tile rt of (b, kvh): its rows, and the tiles from the first token's
// first key to the last token's last.
template <int NR>
__device__ __forceinline__ void paged_unit_tiles(const PagedParams& p, PagedUnit& u) {
  u.row0 = u.rt * NR;
  u.rows = min(NR, u.q.n * p.group - u.row0);
  const int lo = paged_limits(p, u.q, u.row0 / p.group).x;
  const int hi = paged_limits(p, u.q, (u.row0 + u.rows - 1) / p.group).y;
  u.tb = hi > lo ? lo / kPagedKeys : 0;
  u.te = hi > lo ? (hi + kPagedKeys - 1) / kPagedKeys : 0;
}

__device__ __forceinline__ int paged_cost(const PagedUnit& u) { return max(u.te - u.tb, 1); }

// Tiles of one kv head of request b: the sum over its row tiles.
template <int NR>
__device__ __forceinline__ long long paged_head_cost(const PagedParams& p, int b) {
  PagedUnit u;
  u.q = paged_req(p, b);
  const int64_t rows = (int64_t)u.q.n * p.group;
  long long c = 0;
  for (u.rt = 0; (int64_t)u.rt * NR < rows; ++u.rt) {
    paged_unit_tiles<NR>(p, u);
    c += paged_cost(u);
  }
  return c;
}

// A CTA's piece of the line.
struct PagedShare {
  long long total;    // tiles of all units
  long long w0, w1;   // this CTA's
  int ctas;           // CTAs that have a piece
  int b, kvh, rt, off;  // the unit w0 lies in, and how many of its tiles lie before
};

__device__ __forceinline__ long long paged_cut(long long total, int ctas, int c) { return total * c / ctas; }

// Called by every thread of the CTA (NT threads); sh is shared memory.
struct PagedShareSmem {
  long long warp_sum[32];
  int b, kvh, rt, off;
};
template <int NR, int NT>
__device__ __forceinline__ PagedShare paged_share(const PagedParams& p, PagedShareSmem* sh) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.B + NT - 1) / NT;
  const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) mine += paged_head_cost<NR>(p, b) * p.Hkv;
  long long inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) sh->warp_sum[warp] = inc;
  __syncthreads();
  PagedShare s;
  s.total = 0;
  long long before = inc - mine;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    if (w < warp) before += sh->warp_sum[w];
    s.total += sh->warp_sum[w];
  }
  s.ctas = (int)min((long long)gridDim.x, s.total);
  s.w0 = s.w1 = 0;
  s.b = s.kvh = s.rt = s.off = 0;
  if ((int)blockIdx.x >= s.ctas) return s;
  s.w0 = paged_cut(s.total, s.ctas, blockIdx.x);
  s.w1 = paged_cut(s.total, s.ctas, blockIdx.x + 1);
  if (mine > 0 && s.w0 >= before && s.w0 < before + mine) {
    long long rest = s.w0 - before, c;
    PagedUnit u;
    for (u.b = b0;; ++u.b) {
      c = paged_head_cost<NR>(p, u.b);
      if (rest < c * p.Hkv) break;
      rest -= c * p.Hkv;
    }
    sh->b = u.b;
    sh->kvh = (int)(rest / c);
    rest -= c * sh->kvh;
    u.q = paged_req(p, u.b);
    for (u.rt = 0;; ++u.rt) {
      paged_unit_tiles<NR>(p, u);
      if (rest < paged_cost(u)) break;
      rest -= paged_cost(u);
    }
    sh->rt = u.rt;
    sh->off = (int)rest;
  }
  __syncthreads();
  s.b = sh->b;
  s.kvh = sh->kvh;
  s.rt = sh->rt;
  s.off = sh->off;
  return s;
}

// Walks a CTA's piece, segment by segment: a unit's tiles [t0, t0 + nt).
template <int NR>
struct PagedWalk {
  PagedUnit u;
  long long pos, pos_next, end;  // the segment's ends on the line; the piece's end
  int off;               // tiles of the unit before pos
  int t0, nt;            // key tiles of this segment (nt = 0: a unit without visible keys)
  bool head, whole;      // begins at the unit's first tile; holds all of it
  int index;             // segments walked before this one

  __device__ __forceinline__ void begin(const PagedParams& p, const PagedShare& s) {
    pos = s.w0;
    end = s.w1;
    index = 0;
    if (pos >= end) return;
    u.b = s.b;
    u.kvh = s.kvh;
    u.rt = s.rt;
    u.q = paged_req(p, u.b);
    paged_unit_tiles<NR>(p, u);
    off = s.off;
    segment();
  }
  __device__ __forceinline__ bool done() const { return pos >= end; }
  __device__ __forceinline__ void segment() {
    const int cost = paged_cost(u);
    const int len = (int)min((long long)(cost - off), end - pos);
    head = off == 0;
    whole = head && len == cost;
    t0 = u.tb + off;
    nt = u.te > u.tb ? len : 0;
    pos_next = pos + len;
  }
  __device__ __forceinline__ void next(const PagedParams& p) {
    pos = pos_next;
    ++index;
    if (pos >= end) return;
    off = 0;
    if ((int64_t)(++u.rt) * NR >= (int64_t)u.q.n * p.group) {
      u.rt = 0;
      if (++u.kvh == p.Hkv) {
        u.kvh = 0;
        do u.q = paged_req(p, ++u.b); while (u.q.n == 0);
      }
    }
    paged_unit_tiles<NR>(p, u);
    segment();
  }
};

// CTAs from this one on that hold a part of the unit at the walk's position.
template <int NR>
__device__ __forceinline__ int paged_parts(const PagedWalk<NR>& w, const PagedShare& s) {
  const long long last = w.pos - w.off + paged_cost(w.u) - 1;
  int c = blockIdx.x;
  while (c + 1 < s.ctas && paged_cut(s.total, s.ctas, c + 1) <= last) ++c;
  return c - (int)blockIdx.x + 1;
}

}  // namespace gb300_attn
