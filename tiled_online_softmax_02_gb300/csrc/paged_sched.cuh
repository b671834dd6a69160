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
  int s0, n;   // first row, rows
  int total;   // cached tokens, these rows' among them (at least 0: below it nothing is visible either)
};

__device__ __forceinline__ PagedReq paged_req(const PagedParams& p, int b) {
  PagedReq r;
  r.s0 = min(max(__ldg(p.q_starts + b), 0), p.T);
  r.n = min(max(__ldg(p.q_starts + b + 1), r.s0), p.T) - r.s0;
  r.total = max(__ldg(p.totals + b), 0);
  return r;
}

// Keys that have a slot.
__device__ __forceinline__ int paged_valid(const PagedParams& p, const PagedReq& q) { return min(q.total, p.cap); }

// Visible keys [x, y) of the request's row qi; none where y <= x.  Both ends
// rise with qi.
__device__ __forceinline__ int2 paged_limits(const PagedParams& p, const PagedReq& q, int qi) {
  const int pos = q.total - q.n + qi;  // from -2^31 + 2
  const int lo = p.local_window > 0 && pos >= p.local_window ? pos - p.local_window + 1 : 0;
  const int valid = paged_valid(p, q);
  return make_int2(lo, p.causal && pos < valid ? max(pos + 1, 0) : valid);
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

// What a unit costs besides its tiles, in tiles.
template <int NR>
constexpr int kOver = NR == kPagedTcRows ? 3 : 1;

template <int NR>
__device__ __forceinline__ int paged_cost(const PagedUnit& u) { return max(u.te - u.tb, 1) + kOver<NR>; }

// Tiles of one kv head of request b: the sum over its row tiles.
template <int NR>
__device__ __forceinline__ long long paged_head_cost(const PagedParams& p, int b) {
  PagedUnit u;
  u.q = paged_req(p, b);
  const int rows = u.q.n * p.group;
  long long c = 0;
  for (u.rt = 0; u.rt * NR < rows; ++u.rt) {
    paged_unit_tiles<NR>(p, u);
    c += paged_cost<NR>(u);
  }
  return c;
}

// A CTA's piece of the line, in shared memory.
struct PagedShare {
  long long total;      // length of the line
  long long w0, w1;     // this CTA's piece
  int ctas;             // CTAs that have a piece
  int b, kvh, rt, off;  // the unit w0 lies in, and how far into it: 0, or more than kOver
  long long warp_sum[32];
};

__device__ __forceinline__ long long paged_cut(long long total, int ctas, int c) { return total * c / ctas; }

// Called by every thread of the CTA (NT threads) before a __syncthreads().
template <int NR, int NT>
__device__ __forceinline__ void paged_share(const PagedParams& p, PagedShare* sh) {
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
  long long total = 0, before = inc - mine;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    if (w < warp) before += sh->warp_sum[w];
    total += sh->warp_sum[w];
  }
  const int ctas = (int)min((long long)gridDim.x, total);
  const bool in = (int)blockIdx.x < ctas;
  const long long w0 = in ? paged_cut(total, ctas, blockIdx.x) : 0;
  const long long w1 = in ? paged_cut(total, ctas, blockIdx.x + 1) : 0;
  if (tid == 0) {
    sh->total = total;
    sh->ctas = ctas;
    if (!in) sh->w0 = 0;
    if (!in || w1 == total) sh->w1 = w1;
  }
  // the thread whose requests hold a border finds its unit
  for (int end = 0; end < 2; ++end) {
    const long long at = end ? w1 : w0;
    if (!in || at < before || at >= before + mine) continue;
    long long rest = at - before, c;
    PagedUnit u;
    for (u.b = b0;; ++u.b) {
      c = paged_head_cost<NR>(p, u.b);
      if (rest < c * p.Hkv) break;
      rest -= c * p.Hkv;
    }
    u.kvh = (int)(rest / c);
    rest -= c * u.kvh;
    u.q = paged_req(p, u.b);
    for (u.rt = 0;; ++u.rt) {
      paged_unit_tiles<NR>(p, u);
      if (rest < paged_cost<NR>(u)) break;
      rest -= paged_cost<NR>(u);
    }
    const int off = rest > kOver<NR> ? (int)rest : 0;
    if (end) {
      sh->w1 = at - (rest - off);
    } else {
      sh->w0 = at - (rest - off);
      sh->b = u.b;
      sh->kvh = u.kvh;
      sh->rt = u.rt;
      sh->off = off;
    }
  }
}

// Walks a CTA's piece, segment by segment: a unit's tiles [t0, t0 + nt).
template <int NR>
struct PagedWalk {
  PagedUnit u;
  int left, off;         // what is left of the piece; how far into the unit this segment begins
  int t0, nt;            // key tiles of this segment (nt = 0: a unit without visible keys)
  bool head, whole;      // begins at the unit's first tile; holds all of it
  int index;             // segments walked before this one

  __device__ __forceinline__ void begin(const PagedParams& p, const PagedShare* s) {
    left = (int)(s->w1 - s->w0);
    index = 0;
    if (left <= 0) return;
    u.b = s->b;
    u.kvh = s->kvh;
    u.rt = s->rt;
    u.q = paged_req(p, u.b);
    paged_unit_tiles<NR>(p, u);
    off = s->off;
    segment();
  }
  __device__ __forceinline__ bool done() const { return left <= 0; }
  __device__ __forceinline__ int len() const { return min(paged_cost<NR>(u) - off, left); }
  __device__ __forceinline__ void segment() {
    head = off == 0;
    whole = head && len() == paged_cost<NR>(u);
    const int before = head ? 0 : off - kOver<NR>;
    t0 = u.tb + before;
    nt = u.te > u.tb ? off + len() - kOver<NR> - before : 0;
  }
  __device__ __forceinline__ void next(const PagedParams& p) {
    left -= len();
    ++index;
    if (left <= 0) return;
    off = 0;
    if ((++u.rt) * NR >= u.q.n * p.group) {
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

// CTAs from this one on that hold a part of the walk's unit.
template <int NR>
__device__ __forceinline__ int paged_parts(const PagedWalk<NR>& w, const PagedShare* s) {
  const long long last = s->w1 - w.left - w.off + paged_cost<NR>(w.u) - 1;
  int c = blockIdx.x;
  while (c + 1 < s->ctas && paged_cut(s->total, s->ctas, c + 1) <= last) ++c;
  return c - (int)blockIdx.x + 1;
}

}  // namespace gb300_attn
