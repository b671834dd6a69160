// attn_paged4_tc.cu -- attention over the paged 4-bit KV cache for many query
// rows per (request, kv head): prompts and chunks of prompts.
//
// Bound: the tensor cores and the softmax.  A unit is 256 query rows (token /
// head pairs, so the query heads of a kv head share its K and V) in two 128-row
// lanes that alternate: while one lane's softmax runs, the tensor core works on
// the other.
//   S = Q K^T, O += P V   kind::f16.  Four warps widen K and V to f16 (e2m1 *
//   e4m3 is exact there) on their way from the bytes as they lie in the cache
//   to tiles in the tensor core's swizzle: 50 instructions for 32 values, which
//   256 rows share.  P is f16 in tensor memory, over its S.
// Q is f16 as it is, or bf16 times a power of two a row that brings its largest
// element to 2^14, which loses nothing above 2^-31 of that: one product where
// the 8-bit kernel has two or three e4m3 pieces.
//
// One CTA an SM walks its share of the line of key tiles (paged_sched.cuh).
// Roles (512 threads): warps 0-3 and 4-7 the softmax of the two lanes, thread =
// row; they also bring the next unit's Q before they store the last one's rows.
// Warps 8-11 widen; warp 12 loads (bulk copies: a block's rows of a head lie
// together), 13 issues MMAs.
// Tensor memory: S_0, S_1, O_0, O_1, 128 columns each; P over its S.
//
// Measured (one GB300, device time with the join, bf16, 32 query and 8 kv heads,
// D = 128): chunks of about 1.8K tokens at 9K to 14K of context 557 us, 1292
// TFLOP/s, 67% of a 16-bit library product's rate (the 8-bit kernel 591 us); two
// whole prompts of 3.5K to 4K tokens 236 us, 1003 TFLOP/s (257).  The tensor pipe is
// busy 54% of the first's time: a lane's S, softmax and P V follow one another, as
// P takes S's place, and two lanes do not cover that.  Without the widening's
// arithmetic it takes 492 us: its stores, 64 KB a tile, share the memory with the
// products' operands, 192 KB, and its instructions the issue slots.
// Slower: the codes from global memory straight into registers, a tile ahead (601
// us: twice the code), P handed over in halves (no change), the next unit's Q
// prefetched to L2 (no change).
#include <algorithm>
#include <atomic>
#include <cmath>

#include "paged4.cuh"
#include "paged4_internal.h"
#include "paged_mma.cuh"
#include "paged_sched.cuh"

namespace gb300_attn {
namespace {

constexpr int BM = 128, BN = kPagedKeys;
constexpr int kRows = kPagedTcRows;    // rows of a unit: two lanes of 128
constexpr int kThreads = 512;
constexpr int kWidenWarp0 = 8, kWidenWarps = 4, kLoadWarp = 12, kMmaWarp = 13;
constexpr float kRise = 8.0f;          // the maximum moves when a key passes it by 2^8
constexpr float kPLog2 = kPagedTcLog2;  // P is carried as 2^(t - m + 7) <= 2^15
constexpr uint32_t kColO = 256;
// Loops over a tile's four runs of 32 keys.  Their code is what counts: long chunks take 555 us with these, 567 with the
// maximum's loop unrolled once, 577 four times, 602 with the row's scores in registers and no loops, 572 with the next
// run's scores on their way during this one's exponentials.
constexpr int kMaxUnroll = 2, kExpUnroll = 1;

template <int D>
struct Cfg {
  static constexpr int kRow = D / 2, kScRow = D / kGroup4;     // bytes of a row, and of its scales
  static constexpr int kPacked = BN * (kRow + kScRow);         // a tile as it lies in the cache, K or V: codes, then scales
  static constexpr int kTile = BN * D * 2;                     // widened
  static constexpr int kSub = BN * 128;                        // its 64-value blocks: [128 keys][128 bytes]
  static constexpr int kQLane = BM * D * 2;
  static constexpr int kSP = D == 64 ? 6 : 3;                  // packed tiles, K and V in turn
  static constexpr int kSK = D == 64 ? 3 : 2, kSV = kSK;
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = kOffQ + 2 * kQLane;
  static constexpr int kOffV = kOffK + kSK * kTile;
  static constexpr int kOffP = kOffV + kSV * kTile;
  static constexpr int kOffBar = kOffP + kSP * kPacked;
  // p_full, p_empty [kSP], k_full, k_empty [kSK], v_full, v_empty [kSV], q_full, s_full, w_full, o_final [2], drain
  static constexpr int kBars = 2 * (kSP + kSK + kSV) + 9;
  static constexpr int kOffSlot = kOffBar + kBars * 8;
  static constexpr int kOffShare = (kOffSlot + 16 + 15) / 16 * 16;
  static constexpr int kSmem = kOffShare + (int)sizeof(PagedShare) + 1024;
  static_assert(kSmem <= 232448, "shared memory");
  static_assert(kOffBar % 8 == 0 && kPacked % 16 == 0, "alignment");
};

template <int D>
struct Lay {
  using C = Cfg<D>;
  uint8_t* base;
  uint32_t s;
  __device__ uint32_t q(int t) const { return s + C::kOffQ + t * C::kQLane; }
  __device__ uint8_t* q_ptr(int t) const { return base + C::kOffQ + t * C::kQLane; }
  __device__ uint32_t k_tile(int i) const { return s + C::kOffK + i * C::kTile; }
  __device__ uint32_t v_tile(int i) const { return s + C::kOffV + i * C::kTile; }
  __device__ uint8_t* k_ptr(int i) const { return base + C::kOffK + i * C::kTile; }
  __device__ uint8_t* v_ptr(int i) const { return base + C::kOffV + i * C::kTile; }
  __device__ uint32_t packed(int i) const { return s + C::kOffP + i * C::kPacked; }
  __device__ const uint8_t* packed_ptr(int i) const { return base + C::kOffP + i * C::kPacked; }
  __device__ uint32_t bar(int i) const { return s + C::kOffBar + i * 8; }
  __device__ uint32_t p_full(int i) const { return bar(i); }
  __device__ uint32_t p_empty(int i) const { return bar(C::kSP + i); }
  __device__ uint32_t k_full(int i) const { return bar(2 * C::kSP + i); }
  __device__ uint32_t k_empty(int i) const { return bar(2 * C::kSP + C::kSK + i); }
  __device__ uint32_t v_full(int i) const { return bar(2 * C::kSP + 2 * C::kSK + i); }
  __device__ uint32_t v_empty(int i) const { return bar(2 * C::kSP + 2 * C::kSK + C::kSV + i); }
  __device__ uint32_t rest(int i) const { return bar(2 * (C::kSP + C::kSK + C::kSV) + i); }
  __device__ uint32_t q_full(int t) const { return rest(t); }
  __device__ uint32_t s_full(int t) const { return rest(2 + t); }
  __device__ uint32_t w_full(int t) const { return rest(4 + t); }  // P, the weights
  __device__ uint32_t o_final(int t) const { return rest(6 + t); }
  __device__ uint32_t drain() const { return rest(8); }
  __device__ uint32_t* slot() const { return reinterpret_cast<uint32_t*>(base + C::kOffSlot); }
  __device__ PagedShare* share() const { return reinterpret_cast<PagedShare*>(base + C::kOffShare); }
};

struct Paged4TcParams {
  Paged4Params p;
  float scale_log2;    // scale log2 e
  bool aligned32;      // out and ws_o begin on 32-byte boundaries
  float sc_in, sc_out; // soft-cap, from and to log2 units: sc_out tanh(sc_in s)
};

using Walk = PagedWalk<kRows, kOrdinary>;

// Whether lane t of a unit has rows.
__device__ __forceinline__ bool lane_on(const PagedUnit& u, int t) { return t == 0 || u.rows > BM; }

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
               : "memory");
}

// ------------------------------------------------------------------- loads
// One warp: lane 2 i + j copies part j (codes, scales) of block i of a tile, K
// then V.  Blocks past the last key are not read; of an entry that names no block
// the scales become zeros.
template <int D>
__device__ __forceinline__ void load_role(const Paged4Params& P, const Lay<D>& sm, Walk w, int lane) {
  using C = Cfg<D>;
  const PagedParams& p = P.c;
  const int per = BN >> p.block_shift, i = lane >> 1, part = lane & 1;
  const uint32_t bytes = p.block_size * (part ? C::kScRow : C::kRow), block_bytes = p.block_size * (C::kRow + C::kScRow);
  const uint32_t off = (part ? BN * C::kRow : 0) + i * bytes;
  int s = 0;  // packed tiles so far
  bool ok = true;
  for (; ok && !w.done(); w.next(p)) {
    const int valid = paged_valid(p, w.u.q);
    const int32_t* table = p.tables + (int64_t)w.u.b * p.width;
    auto lookup = [&](int t) {  // -1: past the last key; -2: names no block
      const int64_t n = (int64_t)t * per + i;
      if (i >= per || n >= ((int64_t)valid + p.block_size - 1) >> p.block_shift) return -1;
      const int e = table[n];
      return e >= 0 && e < p.num_blocks ? e : -2;
    };
    int next = w.nt > 0 ? lookup(w.t0) : -1;
    for (int n = 0; ok && n < w.nt; ++n) {
      const int blk = next;
      if (n + 1 < w.nt) next = lookup(w.t0 + n + 1);
      if (blk == -2 && part == 0) atomicOr(p.status, kStatusBadBlock);
      const unsigned there = __ballot_sync(0xffffffffu, blk >= 0 && part == 0);
      for (int which = 0; which < 2; ++which, ++s) {
        const int st = s % C::kSP;
        if (s >= C::kSP && !wait_warp(sm.p_empty(st), ((s / C::kSP) - 1) & 1, p.timeout_ns, p.status)) { ok = false; break; }
        if (blk == -2 && part == 1) {
          for (uint32_t o = 0; o < bytes; o += 16)
            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(sm.packed(st) + off + o), "r"(0u) : "memory");
          fence_proxy_async_smem();  // before a later tile's copies to the same place
        }
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(sm.p_full(st), __popc(there) * block_bytes);
        __syncwarp();
        if (blk >= 0) {
          const uint8_t* src = which ? (part ? P.v_sc : p.v_cache) : (part ? P.k_sc : p.k_cache);
          bulk_load(sm.packed(st) + off, src + ((int64_t)blk * p.Hkv + w.u.kvh) * bytes, bytes, sm.p_full(st));
        }
      }
    }
  }
  // every copy lands before the CTA may exit
  for (int n = max(0, s - C::kSP); n < s; ++n) wait_warp(sm.p_full(n % C::kSP), (n / C::kSP) & 1, p.timeout_ns, p.status);
}

// ------------------------------------------------------------------ widening
// Four warps: tiles of K and V in turn, e2m1 times its scale as f16, into
// 64-value blocks of [128 keys][128 bytes] in the 128-byte swizzle; rows past the
// last key as zeros (their slots may hold NaN scales; P is 0 there but 0 * NaN is
// not).  A lane takes 32 values of a row.  Eight neighbours write four rows'
// pieces of the same 128 bytes at a time, so that they never share a bank.
template <int D>
__device__ __forceinline__ void widen_role(const Paged4Params& P, const Lay<D>& sm, Walk w, int warp, int lane) {
  using C = Cfg<D>;
  const PagedParams& p = P.c;
  const int part = D == 128 ? (lane & 1) + ((lane >> 2) & 2) : lane & 1;
  const int r0 = D == 128 ? ((lane >> 1) & 3) + ((lane >> 2) & 4) : lane >> 1;
  constexpr int kStep = D == 128 ? 8 : 16;  // rows of a warp at a time
  int s = 0, g = 0;
  for (; !w.done(); w.next(p)) {
    const int valid = paged_valid(p, w.u.q);
    for (int n = 0; n < w.nt; ++n, ++g) {
      const int rows = min(valid - (w.t0 + n) * BN, BN);
#pragma unroll 1
      for (int which = 0; which < 2; ++which, ++s) {
        const int st = s % C::kSP, to = which ? g % C::kSV : g % C::kSK;
        constexpr int kS = C::kSK;  // as many of V
        if (!wait_warp(sm.p_full(st), (s / C::kSP) & 1, p.timeout_ns, p.status)) return;
        if (g >= kS && !wait_warp(which ? sm.v_empty(to) : sm.k_empty(to), ((g / kS) - 1) & 1, p.timeout_ns, p.status)) return;
        const uint8_t* src = sm.packed_ptr(st);
        uint8_t* dst = (which ? sm.v_ptr(to) : sm.k_ptr(to)) + (part >> 1) * C::kSub;
#pragma unroll 1
        for (int i = 0; i < BN / kStep / kWidenWarps; ++i) {
          const int row = (i * kWidenWarps + warp) * kStep + r0;
          const uint4 v = *reinterpret_cast<const uint4*>(src + row * C::kRow + part * 16);
          uint32_t sc = *reinterpret_cast<const uint16_t*>(src + BN * C::kRow + row * C::kScRow + part * 2);
          if (row >= rows) sc = 0u;
          const uint32_t f = widen_e4m3x2(sc), f0 = __byte_perm(f, 0, 0x1010), f1 = __byte_perm(f, 0, 0x3232);
          const uint32_t code[4] = {v.x, v.y, v.z, v.w};
          uint8_t* out = dst + row * 128;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t h[4];
            widen8(code[j], h[0], h[1], h[2], h[3]);
            const uint32_t m = j < 2 ? f0 : f1;
            *reinterpret_cast<uint4*>(out + ((((part & 1) * 4 + j) ^ (row & 7)) << 4)) =
                make_uint4(mul_f16x2(h[0], m), mul_f16x2(h[1], m), mul_f16x2(h[2], m), mul_f16x2(h[3], m));
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(sm.p_empty(st));
          mbar_arrive(which ? sm.v_full(to) : sm.k_full(to));
        }
      }
    }
  }
}

// --------------------------------------------------------------- MMA issuer
// Lane by lane, per tile: P V of the tile before, then S of this one into the
// columns that P occupied.  A commit covers every earlier MMA of the thread,
// so "S ready" also says "O holds all earlier tiles".
template <int D>
__device__ __forceinline__ void mma_role(const Paged4Params& P, const Lay<D>& sm, Walk w, uint32_t tmem, int lane) {
  using C = Cfg<D>;
  const PagedParams& p = P.c;
  constexpr uint32_t kIdS = make_idesc_f16kind(false, BM, BN, false);
  constexpr uint32_t kIdO = make_idesc_f16kind(false, BM, D, true);
  int g = 0;                          // tiles of the line
  int units[2] = {0, 0}, pc[2] = {0, 0};  // units begun, P tiles used, per lane
  bool ok = true;
  auto issue_s = [&](int t, int ks) {
    const uint64_t a = make_sdesc_sw128(sm.q(t), 16, 1024), b = make_sdesc_sw128(sm.k_tile(ks), 16, 1024);
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {  // 64-value blocks
      const uint32_t o = (i * C::kSub) >> 4;
      mma_ss4_elect(tmem + t * 128, a + o, b + o, a + o + 2, b + o + 2, a + o + 4, b + o + 4, a + o + 6, b + o + 6, kIdS, i > 0 ? 1u : 0u);
    }
    tc_commit_elect(sm.s_full(t));
  };
  auto issue_pv = [&](int t, int vs, bool first) {
    const uint64_t b = make_sdesc_sw128(sm.v_tile(vs), C::kSub, 1024);
    const uint32_t d = tmem + kColO + t * 128, a = tmem + t * 128;
#pragma unroll
    for (int k = 0; k < BN / 16; k += 4)
      mma_ts4_elect(d, a + k * 8, b + (uint32_t)(k * 128), a + (k + 1) * 8, b + (uint32_t)((k + 1) * 128), a + (k + 2) * 8,
                    b + (uint32_t)((k + 2) * 128), a + (k + 3) * 8, b + (uint32_t)((k + 3) * 128), kIdO, first && k == 0 ? 0u : 1u);
  };
  for (; ok && !w.done(); w.next(p)) {
    if (w.nt == 0) continue;  // no S, and no Q was brought
    const bool two = lane_on(w.u, 1);
    for (int n = 0; ok && n <= w.nt; ++n) {
      const int sv = (g + n - 1 + C::kSV) % C::kSV, ks = (g + n) % C::kSK;
      bool k_ready = false;
      if (n >= 1 && !wait_warp(sm.v_full(sv), ((g + n - 1) / C::kSV) & 1, p.timeout_ns, p.status)) { ok = false; break; }
      for (int t = 0; t < (two ? 2 : 1); ++t) {
        if (n >= 1) {
          if (!wait_warp(sm.w_full(t), pc[t] & 1, p.timeout_ns, p.status)) { ok = false; break; }
          tc_fence_after();
          issue_pv(t, sv, n == 1);
          if (n == w.nt) tc_commit_elect(sm.o_final(t));
          ++pc[t];
        }
        if (n < w.nt) {
          if (n == 0) {
            if (!wait_warp(sm.q_full(t), units[t] & 1, p.timeout_ns, p.status)) { ok = false; break; }
            ++units[t];
          }
          if (!k_ready) {
            if (!wait_warp(sm.k_full(ks), ((g + n) / C::kSK) & 1, p.timeout_ns, p.status)) { ok = false; break; }
            k_ready = true;
          }
          tc_fence_after();
          issue_s(t, ks);
        }
        __syncwarp();
      }
      if (!ok) break;
      if (n < w.nt) tc_commit_elect(sm.k_empty(ks));
      if (n >= 1) tc_commit_elect(sm.v_empty(sv));
      __syncwarp();
    }
    g += w.nt;
  }
  tc_commit_elect(sm.drain());
  wait_warp(sm.drain(), 0, p.timeout_ns, p.status);
}

// ------------------------------------------------------------------ softmax
// A lane's rows of Q, K-major in the swizzle; rows past the unit's are zeros.
// Each warp brings its own 32 rows: all of them in flight to their places, and
// bf16 ones are then scaled where they lie, thread = row.  Returns 1 / the scale
// of this thread's own row.
template <int D, bool BF16>
__device__ __forceinline__ float bring_q(const Paged4Params& P, const Lay<D>& sm, const PagedUnit& u, int t, int wq, int lane) {
  using C = Cfg<D>;
  const PagedParams& p = P.c;
  constexpr int kVec = D / 8, kPer = 32 / kVec;  // 16-byte pieces of a row; rows an instruction
  const int c = lane % kVec, sub = lane / kVec, row0 = wq * 32;
  {
    const int row = t * BM + row0 + lane;  // this thread's own; where it lies goes to the threads that load it
    const int tok = paged_token(p, u.row0 + row);
    const int64_t at = row < u.rows ? (int64_t)(u.q.s0 + tok) * p.q_stride +
                                          (int64_t)(u.kvh * p.group + u.row0 + row - tok * p.group) * D : -1;
    const uint16_t* q = static_cast<const uint16_t*>(p.q) + c * 8;
    const uint32_t to = sm.q(t) + (c >> 3) * C::kSub;
#pragma unroll 2
    for (int i = 0; i < kVec; ++i) {
      const int r = row0 + i * kPer + sub;
      const int64_t from = __shfl_sync(0xffffffffu, at, i * kPer + sub);
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + r * 128 + (((c & 7) ^ (r & 7)) << 4)),
                   "l"(q + max(from, (int64_t)0)), "r"(from >= 0 ? 16 : 0) : "memory");
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncwarp();
  const uint32_t sign = p.scale < 0.0f ? 0x80008000u : 0u;  // of the scale: larger raw scores are larger scores
  if (!BF16 && sign == 0u) return 1.0f;
  const int r = row0 + lane;
  uint8_t* mine = sm.q_ptr(t) + r * 128;
  uint32_t top2 = 0;
#pragma unroll 4
  for (int i = 0; i < kVec; ++i) {
    const uint4 v = *reinterpret_cast<const uint4*>(mine + (i >> 3) * C::kSub + (((i & 7) ^ (r & 7)) << 4));
    top2 = __vmaxu2(top2, __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                                   __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu)));
  }
  const uint32_t top = max(top2 & 0xffffu, top2 >> 16);
  // up to [2^14, 2^15); rows of zeros and rows that hold an infinity or NaN stay as they are
  const int e = top == 0u || top >= 0x7f80u ? 0 : min(max(14 - ((int)(top >> 7) - 127), -120), 120);
  const float up = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll 2
  for (int i = 0; i < kVec; ++i) {
    uint4* at = reinterpret_cast<uint4*>(mine + (i >> 3) * C::kSub + (((i & 7) ^ (r & 7)) << 4));
    const uint4 v = *at;
    const uint32_t x[4] = {v.x ^ sign, v.y ^ sign, v.z ^ sign, v.w ^ sign};
    uint32_t y[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      y[k] = BF16 ? as_bits(__floats2half2_rn(__uint_as_float(x[k] << 16) * up, __uint_as_float(x[k] & 0xffff0000u) * up)) : x[k];
    *at = make_uint4(y[0], y[1], y[2], y[3]);
  }
  return BF16 ? __uint_as_float((uint32_t)(127 - e) << 23) : 1.0f;
}

// 32 bytes of a row, which lies apart from other threads' rows: one store of
// a whole sector where the buffer allows it, else two.
__device__ __forceinline__ void store_32b(void* ptr, const uint32_t* v, bool aligned32) {
  if (aligned32) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(ptr), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(ptr)[0] = make_uint4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<uint4*>(ptr)[1] = make_uint4(v[4], v[5], v[6], v[7]);
  }
}

template <int D, bool BF16, bool SOFTCAP>
__device__ __forceinline__ void softmax_role(const Paged4TcParams& TP, const Lay<D>& sm, Walk w, uint32_t tmem, int warp,
                                             int lane) {
  const Paged4Params& P = TP.p;
  const PagedParams& p = P.c;
  const int t = warp >> 2, wq = warp & 3, row = wq * 32 + lane;
  const uint32_t s_addr = tmem + ((uint32_t)(wq * 32) << 16) + t * 128;
  const uint32_t o_addr = s_addr + kColO;
  int sc = 0, oc = 0;  // S tiles and units with tiles of this lane
  // of the unit whose rows are still to be stored
  bool stored = true, whole = false, head = false, mine = false;
  int prev_nt = 0;
  int64_t out_row = 0;
  float m_run = kNone, l_run = 0.0f, vh = 1.0f;
  for (;;) {
    // ---- a unit's Q: this lane's last S has been read, so its Q is free, and the tensor core can
    // begin the unit while the last one's rows are stored
    float qs = 1.0f;  // 1 / the scale of this row's Q
    if (!w.done() && w.nt > 0 && lane_on(w.u, t)) {
      qs = bring_q<D, BF16>(P, sm, w.u, t, wq, lane);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(sm.q_full(t));
    }
    if (!stored) {
      // ---- the last unit's rows
      stored = true;
      if (prev_nt > 0) {
        if (!wait_warp(sm.o_final(t), oc & 1, p.timeout_ns, p.status)) return;
        ++oc;
        tc_fence_after();
      }
      const float inv = l_run == 0.0f ? 0.0f : vh / l_run;
      const int64_t ws_row = (int64_t)(2 * blockIdx.x + (head ? 1 : 0)) * kRows + t * BM + row;
#pragma unroll 1
      for (int k = 0; k < D / 32; ++k) {
        uint32_t o[32];
        if (prev_nt > 0) {
          tmem_ld32(o_addr + k * 32, o);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = 0u;
        }
        if (mine && whole) {
          uint32_t v[16];
#pragma unroll
          for (int i = 0; i < 16; ++i)
            v[i] = (uint32_t)to_bits<BF16>(__uint_as_float(o[2 * i]) * inv) |
                   (uint32_t)to_bits<BF16>(__uint_as_float(o[2 * i + 1]) * inv) << 16;
          uint16_t* dst = static_cast<uint16_t*>(p.out) + out_row * D + k * 32;
          store_32b(dst, &v[0], TP.aligned32);
          store_32b(dst + 16, &v[8], TP.aligned32);
        } else if (mine) {
          float* dst = P.ws_o + ws_row * D + k * 32;
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * vh);
#pragma unroll
          for (int i = 0; i < 4; ++i) store_32b(dst + 8 * i, &o[8 * i], TP.aligned32);
        }
      }
      if (mine && whole && p.lse != nullptr)
        p.lse[out_row] = l_run == 0.0f ? -INFINITY : (m_run + (__log2f(l_run) - kPLog2)) * kLn2;
      if (mine && !whole) P.ws_ml[ws_row] = make_float2(m_run, l_run * kPagedSumFactor);
      tc_fence_before();  // these reads before this lane's next P arrival, which the next P V waits for
    }
    if (w.done()) return;
    const PagedUnit& u = w.u;
    const int nt = w.nt, t0 = w.t0;
    if (!lane_on(u, t)) {
      w.next(p);
      continue;
    }
    mine = t * BM + row < u.rows;
    const int x0 = u.row0 + t * BM;
    const int last = min(x0 + BM, u.row0 + u.rows) - 1;
    const int2 lim = mine ? paged_limits(p, u.q, paged_token(p, x0 + row)) : make_int2(0, 0);
    const int full_lo = paged_limits(p, u.q, paged_token(p, last)).x, full_hi = paged_limits(p, u.q, paged_token(p, x0)).y;
    // positive, so that -inf stays -inf, and finite, so that 0 stays 0.  Under a soft-cap hidden keys do not go through it, and
    // it may be next to nothing: a large cap brings its share back.
    const float kh = P.k_heads ? P.k_heads[u.kvh] : 1.0f;
    const float raw = fminf(fmaxf(qs * kh * (SOFTCAP ? TP.sc_in : TP.scale_log2), SOFTCAP ? 0.0f : 1.2e-38f), 3e38f);
    const float xs = SOFTCAP ? TP.sc_out : raw;  // brings x, the raw score or its tanh, to log2 units
    vh = P.v_heads ? P.v_heads[u.kvh] : 1.0f;
    m_run = kNone;
    l_run = 0.0f;
    for (int n = 0; n < nt; ++n, ++sc) {
      const int key0 = (t0 + n) * BN;
      if (!wait_warp(sm.s_full(t), sc & 1, p.timeout_ns, p.status)) return;
      tc_fence_after();
      if (key0 < full_lo || key0 + BN > full_hi) {  // some key is hidden from some row: -inf over its score
        const int lo = min(max(lim.x - key0, 0), BN), span = max(min(max(lim.y - key0, 0), BN) - lo, 0);
#pragma unroll 1
        for (int ch = 0; ch < 4; ++ch) {
          uint32_t x[32];
          tmem_ld32(s_addr + ch * 32, x);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) x[i] = (uint32_t)(ch * 32 + i - lo) < (uint32_t)span ? x[i] : 0xff800000u;
          tmem_st32(s_addr + ch * 32, x);
        }
        tmem_wait_st();
      }
      // tanh(scale s / c) of a raw score; hidden ones stay -inf.  The hardware tanh: over all fp32 arguments it is off by
      // 2^-16.46 of the value at most, and by 2^-16.93, measured on the GB300 (its specification allows 2^-11), which is what
      // the call promises of capped scores, 2^-16.  With the few-rows kernel's, to 2^-20, the same two long chunks under a
      // cap take 1251 us in place of 844, two values at a time and without a branch.
      auto capped = [&](float x) {
        if constexpr (SOFTCAP) return x == -INFINITY ? x : fast_tanh(x * raw);
        else return x;
      };
      float m_tile = -INFINITY;
#pragma unroll kMaxUnroll
      for (int ch = 0; ch < 4; ++ch) {
        float x[32];
        tmem_ld32(s_addr + ch * 32, reinterpret_cast<uint32_t(&)[32]>(x));
        tmem_wait_ld();
        float a = fmaxf(x[0], x[1]), b = fmaxf(x[2], x[3]);
#pragma unroll
        for (int k = 4; k < 32; k += 4) {
          a = fmax3(a, x[k], x[k + 1]);
          b = fmax3(b, x[k + 2], x[k + 3]);
        }
        m_tile = fmax3(m_tile, a, b);
      }
      m_tile = capped(m_tile) * xs;
      const bool rise = m_tile > m_run + kRise;
      const float m_new = rise ? m_tile : m_run;
      if (n > 0 && __any_sync(0xffffffffu, rise)) {  // O holds every earlier tile
        const float alpha = fast_exp2(m_run - m_new);
        l_run *= alpha;
#pragma unroll 1
        for (int k = 0; k < D / 32; ++k) {
          uint32_t o[32];
          tmem_ld32(o_addr + k * 32, o);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
          tmem_st32(o_addr + k * 32, o);
        }
      }
      m_run = m_new;
      const float off = kPLog2 - m_run;
      const uint64_t mul = f2(xs, xs), add = f2(off, off);
      uint64_t acc[2] = {0ull, 0ull};
#pragma unroll kExpUnroll
      for (int ch = 0; ch < 4; ++ch) {
        float x[32];
        tmem_ld32(s_addr + ch * 32, reinterpret_cast<uint32_t(&)[32]>(x));
        tmem_wait_ld();
        uint32_t pk[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float a, b;
          f2_split(ffma2(f2(capped(x[2 * i]), capped(x[2 * i + 1])), mul, add), a, b);
          a = fast_exp2(a);
          b = fast_exp2(b);
          acc[i & 1] = fadd2(acc[i & 1], f2(a, b));
          pk[i] = as_bits(__floats2half2_rn(a, b));
        }
        tmem_st16(s_addr + ch * 16, pk);  // over columns of S that have been read
      }
      float sa, sb;
      f2_split(fadd2(acc[0], acc[1]), sa, sb);
      l_run += sa + sb;
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(sm.w_full(t));
    }
    stored = false;
    whole = w.whole;
    head = w.head;
    prev_nt = nt;
    const int xr = x0 + row;
    const int tok = paged_token(p, xr);
    out_row = (int64_t)(u.q.s0 + tok) * p.Hq + u.kvh * p.group + xr - tok * p.group;
    if (!whole && head && threadIdx.x == 0) {
      PagedCut c;
      c.parts = paged_parts(w, sm.share());
      c.token0 = u.q.s0;
      c.head0 = u.kvh * p.group;
      c.row0 = u.row0;
      c.rows = u.rows;
      P.cuts[blockIdx.x] = c;
    }
    w.next(p);
  }
}

template <int D, bool BF16, bool SOFTCAP>
__global__ void __launch_bounds__(kThreads, 1) attn_paged4_tc_kernel(const __grid_constant__ Paged4TcParams TP) {
  using C = Cfg<D>;
  const PagedParams& p = TP.p.c;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Lay<D> sm;
  sm.base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  sm.s = smem_u32(sm.base);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  after_earlier_kernels();
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kSP; ++i) {
      mbar_init(sm.p_full(i), 1);
      mbar_init(sm.p_empty(i), kWidenWarps);
    }
    for (int i = 0; i < C::kSK; ++i) {
      mbar_init(sm.k_full(i), kWidenWarps);
      mbar_init(sm.k_empty(i), 1);
    }
    for (int i = 0; i < C::kSV; ++i) {
      mbar_init(sm.v_full(i), kWidenWarps);
      mbar_init(sm.v_empty(i), 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(sm.q_full(t), 4);
      mbar_init(sm.s_full(t), 1);
      mbar_init(sm.w_full(t), 4);
      mbar_init(sm.o_final(t), 1);
    }
    mbar_init(sm.drain(), 1);
    mbar_init_fence();
    TP.p.cuts[blockIdx.x].parts = 0;
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(sm.slot()), 512);
    tmem_relinquish();
  }
  if (paged_may_be_long<kRows>(p)) paged_share_long<kRows, kThreads, kPaged4Piece, kOrdinary>(p, sm.share());
  else paged_share<kRows, kThreads, kPaged4Piece, kOrdinary>(p, sm.share());
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // The joining kernel may be scheduled; it waits.  Where no join follows this may let in any kernel, one with tensor memory
  // of its own among them, so this CTA has its columns by now.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(sm.slot());
  Walk w;
  w.begin(p, sm.share());
  if (warp < kWidenWarp0) {
    softmax_role<D, BF16, SOFTCAP>(TP, sm, w, tmem, warp, lane);
  } else if (warp < kLoadWarp) {
    widen_role<D>(TP.p, sm, w, warp - kWidenWarp0, lane);
  } else {
    if (warp == kLoadWarp) load_role<D>(TP.p, sm, w, lane);
    else if (warp == kMmaWarp) mma_role<D>(TP.p, sm, w, tmem, lane);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, bool BF16, bool SOFTCAP>
cudaError_t launch_tc(const Paged4TcParams& TP, int grid, cudaStream_t stream) {
  auto kernel = attn_paged4_tc_kernel<D, BF16, SOFTCAP>;
  constexpr int smem = Cfg<D>::kSmem;
  static std::atomic<bool> ready[128];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 128 || !ready[dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 128) ready[dev].store(true, std::memory_order_relaxed);
  }
  return launch_early(kernel, (unsigned)grid, kThreads, smem, stream, TP);
}

template <int D, bool BF16>
cudaError_t launch_tc_d(const Paged4TcParams& TP, int grid, cudaStream_t stream) {
  return TP.p.c.softcap > 0.0f ? launch_tc<D, BF16, true>(TP, grid, stream) : launch_tc<D, BF16, false>(TP, grid, stream);
}

}  // namespace

cudaError_t launch_attn_paged4_tc(const Paged4Params& p, int grid, bool bf16, cudaStream_t stream) {
  Paged4TcParams TP{};
  TP.p = p;
  TP.aligned32 = ((reinterpret_cast<uintptr_t>(p.c.out) | reinterpret_cast<uintptr_t>(p.ws_o)) & 31) == 0;
  TP.scale_log2 = (float)std::min(3e38, fabs((double)p.c.scale) * 1.4426950408889634);  // the sign goes into Q
  if (p.c.softcap > 0.0f) {
    TP.sc_in = (float)std::min(3e38, fabs((double)p.c.scale) / (double)p.c.softcap);
    TP.sc_out = (float)((double)p.c.softcap * 1.4426950408889634);
  }
  if (p.c.D == 128) return bf16 ? launch_tc_d<128, true>(TP, grid, stream) : launch_tc_d<128, false>(TP, grid, stream);
  return bf16 ? launch_tc_d<64, true>(TP, grid, stream) : launch_tc_d<64, false>(TP, grid, stream);
}

}  // namespace gb300_attn
