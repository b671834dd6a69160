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
#include "early_load.cuh"
#include "paged_internal.h"

namespace gb300_attn {

constexpr int kPagedKeys = 128;  // keys of a tile

// mbar_wait_warp in fewer instructions: these kernels have many waits in many
// roles, and are bound by their instruction fetches before anything else.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, uint64_t timeout_ns, int* status) {
  uint64_t t0 = 0;
  bool ok = true;
  for (uint32_t it = 1; !mbar_try_wait(bar, parity); ++it) {
    if ((it & 15u) != 0u) continue;
    const uint64_t now = global_timer_ns();
    if (t0 == 0) t0 = now;
    if (now - t0 > timeout_ns) {
      atomicOr(status, kStatusTimeout);
      ok = false;
      break;
    }
  }
  return __all_sync(0xffffffffu, ok);
}

// Token of a kv head's row x (x / group; the head is the rest).
__device__ __forceinline__ int paged_token(const PagedParams& p, int x) {
  return p.group_shift >= 0 ? x >> p.group_shift : x / p.group;
}

// A request's packed rows and lengths.
struct PagedReq {
  int s0, n;   // first row, rows
  int total;   // cached tokens, these rows' among them (at least 0: below it nothing is visible either)
};

// How the lengths are read.  A kernel that may begin while earlier ones still write them has to keep off the read-only path
// (see after_earlier_kernels): the few-rows kernel over the 4-bit cache by load_written (8 long requests 42.1 us, by ordinary
// loads 42.6), the many-rows one by ordinary loads (long chunks 557 us, by load_written 563).  The 8-bit kernels, launched
// in order, lose 1 to 2.5% off it.
enum PagedLoad { kReadOnly, kOrdinary, kWritten };

template <PagedLoad LOAD>
__device__ __forceinline__ int paged_length(const int32_t* x) {
  if constexpr (LOAD == kReadOnly) return __ldg(x);
  else if constexpr (LOAD == kWritten) return load_written(x);
  else return *x;
}

template <PagedLoad LOAD>
__device__ __forceinline__ PagedReq paged_req(const PagedParams& p, int b) {
  PagedReq r;
  r.s0 = min(max(paged_length<LOAD>(p.q_starts + b), 0), p.T);
  r.n = min(max(paged_length<LOAD>(p.q_starts + b + 1), r.s0), p.T) - r.s0;
  r.total = max(paged_length<LOAD>(p.totals + b), 0);
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
  const int lo = paged_limits(p, u.q, paged_token(p, u.row0)).x;
  const int hi = paged_limits(p, u.q, paged_token(p, u.row0 + u.rows - 1)).y;
  u.tb = hi > lo ? lo / kPagedKeys : 0;
  u.te = hi > lo ? (hi + kPagedKeys - 1) / kPagedKeys : 0;
}

// What a unit costs besides its tiles, in tiles: the many-rows kernel's Q and output rows, about 10000 cycles.  The
// few-rows kernel's units are given the same (not measured apart; the choice between the kernels counts 2 or 4 for them).
constexpr int kOver = 3;

template <int NR>
__device__ __forceinline__ int paged_cost(const PagedUnit& u) { return max(u.te - u.tb, 1) + kOver; }

// Length on the line of one kv head of a request: the sum over its row tiles; or over first, first + step, ... of them.
template <int NR>
__device__ __forceinline__ long long paged_head_cost(const PagedParams& p, const PagedReq& q, int first = 0, int step = 1) {
  PagedUnit u;
  u.q = q;
  const int rows = u.q.n * p.group;
  long long c = 0;
#pragma unroll 1
  for (u.rt = first; u.rt * NR < rows; u.rt += step) {
    paged_unit_tiles<NR>(p, u);
    c += paged_cost<NR>(u);
  }
  return c;
}

// Where a call may have requests of many row tiles, a warp takes those of more than kLongReq together.  (One prompt of 500
// tokens in 125 row tiles of 16: 44 us a call, 18 of them in one lane's loops; two of 4K in tiles of 256 243 us, 236.)  Single
// tokens would pay 0.2 to 0.7 us for it, so the rows beyond one token a request tell, and the code stands apart: a function
// that the many-rows kernel calls, a kernel of its own for few rows (which lose 2% to the mere call).  The kernels over the
// 8-bit cache do without: the call costs the one for many rows 3%.
constexpr int kLongReq = 8;

template <int NR>
__host__ __device__ inline bool paged_may_be_long(const PagedParams& p) {
  return (long long)(p.T - p.B) * p.group > 4 * kLongReq * NR;
}

template <int NR>
__device__ __forceinline__ int paged_row_tiles(const PagedParams& p, const PagedReq& q) {
  return (int)((q.n * (uint32_t)p.group + NR - 1) / NR);
}

// paged_head_cost of every lane's own request, called by the whole warp: the lanes take the long ones one after the other
// where that is shorter than a lane's own way through the longest.
template <int NR>
__device__ __forceinline__ long long paged_head_costs(const PagedParams& p, const PagedReq& q, int lane) {
  const int tiles = paged_row_tiles<NR>(p, q);
  uint32_t longs = __ballot_sync(0xffffffffu, tiles > kLongReq);
  if (longs != 0 && __reduce_max_sync(0xffffffffu, (uint32_t)tiles) <= (uint32_t)(kLongReq * __popc(longs))) longs = 0;
  long long c = (longs >> lane & 1) != 0 ? 0 : paged_head_cost<NR>(p, q);
  __syncwarp();
  for (; longs != 0; longs &= longs - 1) {
    const int src = __ffs(longs) - 1;
    PagedReq r;
    r.s0 = 0;
    r.n = __shfl_sync(0xffffffffu, q.n, src);
    r.total = __shfl_sync(0xffffffffu, q.total, src);
    long long v = paged_head_cost<NR>(p, r, lane, 32);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (lane == src) c = v;
  }
  return c;
}

// a / b for 0 <= a, 0 < b, in 32 bits where they fit.
__device__ __forceinline__ long long paged_div(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

// A CTA's piece of the line, in shared memory.
struct PagedShare {
  long long per, more;  // length of a piece; the first `more` ones are longer by one
  long long w0, w1;     // this CTA's piece
  int ctas;             // CTAs that have a piece
  int b, kvh, rt, off;  // the unit w0 lies in, and how far into it: 0, or more than kOver
  PagedReq q;           // its request
  long long warp_sum[32];
};

__device__ __forceinline__ long long paged_cut(long long per, long long more, int c) {
  return per * c + min((long long)c, more);
}

// paged_share, below, for such calls.
template <int NR, int NT, int kPiece, PagedLoad LOAD>
__device__ __noinline__ void paged_share_long(const PagedParams& p, PagedShare* sh) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int apart = 0;  // few requests are 2^apart threads apart, so that every warp has some
  while (apart < 5 && p.B <= NT >> (apart + 1)) ++apart;
  const int n = (p.B + NT - 1) / NT;  // requests of a thread
  const int b0 = (tid & ((1 << apart) - 1)) == 0 ? min((tid >> apart) * n, p.B) : p.B, b1 = min(b0 + n, p.B);
  PagedReq q{0, 0, 0};
  long long c = 0, mine = 0;  // of the thread's last request; of all of them
#pragma unroll 1
  for (int i = 0; i < n; ++i) {
    const bool there = b0 + i < b1;
    if (there) q = paged_req<LOAD>(p, b0 + i);
    __syncwarp();
    const long long x = paged_head_costs<NR>(p, there ? q : PagedReq{0, 0, 0}, lane);
    if (there) c = x;
    mine += x * p.Hkv;
  }
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
  const int ctas = (int)min((long long)gridDim.x, (total + kPiece - 1) / kPiece);
  const bool in = (int)blockIdx.x < ctas;
  long long per = 0, more = 0, w0 = 0, w1 = 0;
  if (in) {
    per = paged_div(total, ctas);
    more = total - per * ctas;
    w0 = paged_cut(per, more, blockIdx.x);
    w1 = paged_cut(per, more, blockIdx.x + 1);
  }
  if (tid == 0) {
    sh->per = per;
    sh->more = more;
    sh->ctas = ctas;
    if (!in) sh->w0 = 0;
    if (!in || w1 == total) sh->w1 = w1;
  }
  // the thread whose requests hold a border finds its unit, with its warp's help where the request is long
#pragma unroll 1
  for (int end = 0; end < 2; ++end) {
    const long long at = end ? w1 : w0;
    const bool here = in && at >= before && at < before + mine;
    const int src = __ffs(__ballot_sync(0xffffffffu, here)) - 1;  // one thread of the CTA at most
    if (src < 0) continue;
    long long rest = at - before;
    PagedUnit u;
    u.b = b1 - 1;
    u.q = q;
    u.kvh = u.rt = 0;
    if (n > 1) {  // not the thread's only request
      bool found = false;
#pragma unroll 1
      for (int i = 0; i < n; ++i) {
        PagedReq r{0, 0, 0};
        if (here && !found && b0 + i < b1) r = paged_req<LOAD>(p, b0 + i);
        __syncwarp();
        const long long x = paged_head_costs<NR>(p, r, lane);
        if (!here || found) continue;
        if (rest < x * p.Hkv) {
          found = true;
          u.b = b0 + i;
          u.q = r;
          c = x;
        } else {
          rest -= x * p.Hkv;
        }
      }
    }
    if (here) {
      u.kvh = (int)paged_div(rest, c);
      rest -= c * u.kvh;
    }
    __syncwarp();
    if (__shfl_sync(0xffffffffu, paged_row_tiles<NR>(p, u.q), src) > kLongReq) {  // 32 row tiles at a time
      PagedUnit y;
      y.q.s0 = 0;
      y.q.n = __shfl_sync(0xffffffffu, u.q.n, src);
      y.q.total = __shfl_sync(0xffffffffu, u.q.total, src);
      long long to_go = __shfl_sync(0xffffffffu, rest, src);
      const int tiles = paged_row_tiles<NR>(p, y.q);
#pragma unroll 1
      for (int rt0 = 0; rt0 < tiles; rt0 += 32) {
        y.rt = rt0 + lane;
        int cost = 0;
        if (y.rt < tiles) {
          paged_unit_tiles<NR>(p, y);
          cost = paged_cost<NR>(y);
        }
        long long upto = cost;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const long long v = __shfl_up_sync(0xffffffffu, upto, o);
          if (lane >= o) upto += v;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, to_go < upto);
        if (past != 0) {
          const int first = __ffs(past) - 1;
          const long long begun = __shfl_sync(0xffffffffu, to_go - (upto - cost), first);
          if (here) {
            rest = begun;
            u.rt = rt0 + first;
          }
          break;
        }
        to_go -= __shfl_sync(0xffffffffu, upto, 31);
      }
    } else if (here) {
#pragma unroll 1
      for (u.rt = 0;; ++u.rt) {
        paged_unit_tiles<NR>(p, u);
        if (rest < paged_cost<NR>(u)) break;
        rest -= paged_cost<NR>(u);
      }
    }
    __syncwarp();
    if (!here) continue;
    const int off = rest > kOver ? (int)rest : 0;
    if (end) {
      sh->w1 = at - (rest - off);
    } else {
      sh->w0 = at - (rest - off);
      sh->b = u.b;
      sh->kvh = u.kvh;
      sh->rt = u.rt;
      sh->off = off;
      sh->q = u.q;
    }
  }
}

// Called by every thread of the CTA (NT threads) before a __syncthreads().  Where there is too little for every CTA of the
// grid, those that work have pieces kPiece long or more.
template <int NR, int NT, int kPiece = 1, PagedLoad LOAD = kReadOnly>
__device__ __forceinline__ void paged_share(const PagedParams& p, PagedShare* sh) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = (p.B + NT - 1) / NT;  // requests of a thread
  const int b0 = min(tid * n, p.B), b1 = min(b0 + n, p.B);
  PagedReq q{0, 0, 0};
  long long c = 0, mine = 0;  // of the thread's last request; of all of them
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    q = paged_req<LOAD>(p, b);
    c = paged_head_cost<NR>(p, q);
    mine += c * p.Hkv;
  }
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
  const int ctas = (int)min((long long)gridDim.x, (total + kPiece - 1) / kPiece);
  const bool in = (int)blockIdx.x < ctas;
  long long per = 0, more = 0, w0 = 0, w1 = 0;
  if (in) {
    per = paged_div(total, ctas);
    more = total - per * ctas;
    w0 = paged_cut(per, more, blockIdx.x);
    w1 = paged_cut(per, more, blockIdx.x + 1);
  }
  if (tid == 0) {
    sh->per = per;
    sh->more = more;
    sh->ctas = ctas;
    if (!in) sh->w0 = 0;
    if (!in || w1 == total) sh->w1 = w1;
  }
  // the thread whose requests hold a border finds its unit
#pragma unroll 1
  for (int end = 0; end < 2; ++end) {
    const long long at = end ? w1 : w0;
    if (!in || at < before || at >= before + mine) continue;
    long long rest = at - before;
    PagedUnit u;
    u.b = b1 - 1;
    u.q = q;
    if (n > 1) {  // not the thread's only request
      for (u.b = b0;; ++u.b) {
        u.q = paged_req<LOAD>(p, u.b);
        c = paged_head_cost<NR>(p, u.q);
        if (rest < c * p.Hkv) break;
        rest -= c * p.Hkv;
      }
    }
    u.kvh = (int)paged_div(rest, c);
    rest -= c * u.kvh;
#pragma unroll 1
    for (u.rt = 0;; ++u.rt) {
      paged_unit_tiles<NR>(p, u);
      if (rest < paged_cost<NR>(u)) break;
      rest -= paged_cost<NR>(u);
    }
    const int off = rest > kOver ? (int)rest : 0;
    if (end) {
      sh->w1 = at - (rest - off);
    } else {
      sh->w0 = at - (rest - off);
      sh->b = u.b;
      sh->kvh = u.kvh;
      sh->rt = u.rt;
      sh->off = off;
      sh->q = u.q;
    }
  }
}

// Walks a CTA's piece, segment by segment: a unit's tiles [t0, t0 + nt).
template <int NR, PagedLoad LOAD = kReadOnly>
struct PagedWalk {
  PagedUnit u;
  PagedReq ahead;        // of request u.b + 1, read a unit or more before it is needed
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
    u.q = s->q;
    ahead = paged_req<LOAD>(p, min(u.b + 1, p.B - 1));
    paged_unit_tiles<NR>(p, u);
    off = s->off;
    segment();
  }
  __device__ __forceinline__ bool done() const { return left <= 0; }
  __device__ __forceinline__ int len() const { return min(paged_cost<NR>(u) - off, left); }
  __device__ __forceinline__ void segment() {
    head = off == 0;
    whole = head && len() == paged_cost<NR>(u);
    const int before = head ? 0 : off - kOver;
    t0 = u.tb + before;
    nt = u.te > u.tb ? off + len() - kOver - before : 0;
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
        do {  // the piece goes on, so some later request has rows
          ++u.b;
          u.q = ahead;
          ahead = paged_req<LOAD>(p, min(u.b + 1, p.B - 1));
        } while (u.q.n == 0);
      }
    }
    paged_unit_tiles<NR>(p, u);
    segment();
  }
};

// CTAs from this one on that hold a part of the walk's unit.
template <int NR, PagedLoad LOAD>
__device__ __forceinline__ int paged_parts(const PagedWalk<NR, LOAD>& w, const PagedShare* s) {
  const long long last = s->w1 - w.left - w.off + paged_cost<NR>(w.u) - 1;
  int c = blockIdx.x;
  while (c + 1 < s->ctas && paged_cut(s->per, s->more, c + 1) <= last) ++c;
  return c - (int)blockIdx.x + 1;
}

// The scales of a unit's tiles, from block tables and scale arrays into a ring
// in shared memory, by one warp: lane i < 8 has keys 16 i .. of a tile (a block
// holds 16 or more).  With u = log2 of the V scale, of 2^-100 where that is
// larger, a key's weight is 2^(t - m), t = s log2 e + u, and what it adds to the
// row sum is 2^(t - m) / v_scale.  That holds while 2^(t - m) does not fall below
// fp32's range although 2^(s log2 e) is among the row's largest: while u lies
// at most 90 below the largest one of the unit's tiles so far, m being at most
// that much above t.  Where a tile has a key for which it does not (a block of
// zeros, say, whose scale is 2^-100), or whose scale has no inverse in fp32's
// range, the tile is "far": its keys add 2^(s log2 e - m)
// itself to the sum, and that times the scale is their weight.  It is told by
// borders, not by the largest scale itself, as all tiles pay for that: scales of
// 2^-80 to 2^10, or once there has been one above, of 2^10 to 2^100, are near.
// An entry is (k scale * mul, u, 2^-8 / v scale, u), of far tiles (.., u, 0, log2 v scale).
constexpr int kScaleGroups = kPagedKeys / 16;
constexpr float kMinVLog2 = -100.0f, kNearMin = 0x1p-80f, kNearMax = 0x1p10f, kBigMax = 0x1p100f;

template <int kStages>
struct ScaleFeed {
  int g = 0;  // tiles so far
  template <int NR>
  __device__ __forceinline__ bool unit(const PagedParams& p, const PagedWalk<NR>& w, float mul, float4* ring,
                                       uint32_t full0, uint32_t empty0, int lane) {
    const int valid = paged_valid(p, w.u.q);
    const int32_t* table = p.tables + (int64_t)w.u.b * p.width;
    auto block_of = [&](int n) {
      const uint32_t j = (uint32_t)(w.t0 + n) * kPagedKeys + lane * 16;
      const int b = lane < kScaleGroups && n < w.nt && j < (uint32_t)valid ? __ldg(table + (j >> p.block_shift)) : -1;
      return b >= 0 && b < p.num_blocks ? b : -1;
    };
    float ks, vs;
    bool big = false;  // a scale above kNearMax so far
    auto fetch = [&](int b) {  // a block that is none has key scale 0
      ks = 0.0f;
      vs = 1.0f;
      if (b >= 0) {
        ks = __ldg(p.k_scales + (int64_t)b * p.Hkv + w.u.kvh);
        vs = __ldg(p.v_scales + (int64_t)b * p.Hkv + w.u.kvh);
      }
    };
    const int first = block_of(0);
    int next = block_of(1);
    fetch(first);
    for (int n = 0; n < w.nt; ++n, ++g) {  // scales a tile ahead, blocks two
      const float k0 = ks, v0 = vs;
      fetch(next);
      next = block_of(n + 2);
      const int st = g % kStages;
      if (g >= kStages &&
          !wait_warp(empty0 + st * 8, ((g / kStages) - 1) & 1, p.timeout_ns, p.status))
        return false;
      bool far = false;
      if (__any_sync(0xffffffffu, big || v0 < kNearMin || v0 > kNearMax)) {
        big = __any_sync(0xffffffffu, big || v0 > kNearMax);
        far = __any_sync(0xffffffffu, lane < kScaleGroups && (v0 < (big ? kNearMax : kNearMin) || v0 > kBigMax));
      }
      if (lane < kScaleGroups) {
        const float u = __log2f(v0);
        ring[st * kScaleGroups + lane] = make_float4(k0 * mul, fmaxf(u, kMinVLog2), far ? 0.0f : kPagedSumFactor * (1.0f / v0), u);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(full0 + st * 8);
    }
    return true;
  }
};

}  // namespace gb300_attn
