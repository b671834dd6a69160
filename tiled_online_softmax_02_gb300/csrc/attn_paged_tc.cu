// attn_paged_tc.cu -- attention over the paged 8-bit KV cache for many query
// rows per (request, kv head): prompts and chunks of prompts.
//
// Bound: the tensor cores and the softmax's exponentials.  A unit is 256 query
// rows (token / head pairs, so the query heads of a kv head share its K and
// V) in two 128-row lanes that alternate: while one lane's softmax runs, the
// tensor core works on the other.
//   S = Q K^T   kind::f8f6f4 on the cache's e4m3 bytes as TMA brings them; the
//               16-bit Q is two (bf16) or three (f16) e4m3 pieces at one scale,
//               each accumulated into the same S.  e4m3 runs at twice the
//               16-bit rate, so bf16's two pieces cost what one 16-bit product
//               would, f16's three half more, and K needs no conversion.
//   O += P V    kind::f16: P is f16 in tensor memory, V is widened to f16 by
//               four warps on its way from one shared buffer to another.
//               P as e4m3 pieces would cost the softmax warps, which have no
//               slots to spare, about six instructions a value; widening V
//               costs other warps half of one.
// A row of Q carries its own power-of-two scale, which brings its largest element
// into [128, 256), and pieces x0 = e4m3(x), x1 = e4m3(x - x0), ...  One S takes
// them all, so they share that scale, and e4m3's smallest step there, 2^-9: what is
// left is at most 2^-10, 2^-17 of the row's largest element or less.  That holds
// bf16 elements down to 2^-9 of it exactly and f16 ones down to 2^-6; smaller ones
// lose low bits, which their share of the score hardly shows.  (The few-rows kernel
// has a column for each piece, and scales them apart.)
//
// Scales are constant over 16 keys or more (the smallest block).  Per group of
// 16 keys: the largest raw score is found first and scaled once, and
// 2^(s k_scale + log2 v_scale - m) is one FMA and one ex2 a value; the row sum
// takes each group's sum times 1 / v_scale (paged_sched.cuh: in far tiles,
// the sum of 2^(s k_scale - m) itself, in a pass of its own).
//
// One CTA an SM walks its share of the line of key tiles (paged_sched.cuh).
// Roles (512 threads): warps 0-3 and 4-7 the softmax of the two lanes, thread =
// row, which also bring the next unit's Q into pieces before they store the
// last one's rows; warps 8-11 widen V; warp 12 loads (TMA), 13 issues MMAs, 14
// looks up scales and prefetches the next unit's Q rows into L2.
// Tensor memory: S_0, S_1, O_0, O_1, 128 columns each; P over its S.
//
// Measured (one GB300, device time with the join, bf16, 32 query and 8 kv heads,
// D = 128): chunks of about 1.8K tokens at 9K to 14K of context 592 us, 1216
// TFLOP/s, 65% of a 16-bit library product's rate; two whole prompts of 3.5K to
// 4K tokens 257 us, 919 TFLOP/s.  The tensor pipe is busy half of the first's
// time: a lane's S, softmax and P V follow one another, as P takes S's place
// (two of each and two O of 128 columns fill tensor memory), and two lanes do
// not cover that entirely; P V of a tile's first 64 keys at least runs beside
// the exponentials of the others.  A lane's tile is 1240 cycles of waiting for S,
// 700 for the maximum, 100 for what follows it and 1600 for the exponentials.  A unit costs about three
// tiles more than its tiles: 6000 cycles to bring Q, most of them conversions
// to e4m3 and back, and 4000 to store the rows.
#include <algorithm>
#include <atomic>

#include "paged_mma.cuh"
#include "paged_sched.cuh"

namespace gb300_attn {
namespace {

constexpr int BM = 128, BN = kPagedKeys;
constexpr int kRows = kPagedTcRows;    // rows of a unit: two lanes of 128
constexpr int kThreads = 512;
constexpr int kVWarp0 = 8, kTmaWarp = 12, kMmaWarp = 13, kScaleWarp = 14;
constexpr float kRise = 8.0f;          // the maximum moves when a key passes it by 2^8
constexpr float kPLog2 = kPagedTcLog2;  // P is carried as 2^(t - m + 7) <= 2^15
constexpr uint32_t kColO = 256;
// Loops over a tile's four runs of 32 keys.  Two whole prompts took 252 us with these when they were chosen; 258 and 259
// with the maximum's loop unrolled 1 and 4 times, 257 with the exponentials' unrolled twice (instruction fetches).
constexpr int kMaxUnroll = 2, kExpUnroll = 1;

template <int D, bool BF16>
struct Cfg {
  static constexpr int kQP = BF16 ? 2 : 3;
  static constexpr int kTile8 = BN * D;            // e4m3 tile
  static constexpr int kTile16 = BN * D * 2;       // V widened
  static constexpr int kQLane = kQP * BM * D;      // Q pieces of a lane
  static constexpr int kSK = D == 64 ? 4 : (BF16 ? 3 : 2);
  static constexpr int kSV8 = 2;
  static constexpr int kSV = D == 64 ? 3 : 2;
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = kOffQ + 2 * kQLane;
  static constexpr int kOffV8 = kOffK + kSK * kTile8;
  static constexpr int kOffV = kOffV8 + kSV8 * kTile8;
  static constexpr int kOffSc = kOffV + kSV * kTile16;  // float4 [kSK][kScaleGroups]: as the scale warp leaves them
  static constexpr int kOffQe = kOffSc + kSK * kScaleGroups * 16;  // uint32 [256]: the Q rows' scales, as f32 (bf16 Q) or two f16 factors
  static constexpr int kOffBar = kOffQe + kRows * 4;
  // k_full, k_empty [kSK], v8_full, v8_empty [kSV8], v_full, v_empty [kSV], sc_empty [kSK],
  // q_full, s_full, p_half, p_full, o_final [2], drain
  static constexpr int kBars = 2 * (kSK + kSV8 + kSV) + kSK + 11;
  static constexpr int kOffSlot = kOffBar + kBars * 8;
  static constexpr int kOffShare = (kOffSlot + 16 + 15) / 16 * 16;
  static constexpr int kSmem = kOffShare + (int)sizeof(PagedShare) + 1024;
  static_assert(kSmem <= 232448, "shared memory");
  static_assert(kOffBar % 8 == 0 && kQLane % 1024 == 0, "alignment");
};

template <int D, bool BF16>
struct Lay {
  using C = Cfg<D, BF16>;
  uint8_t* base;
  uint32_t s;
  __device__ uint32_t q(int t) const { return s + C::kOffQ + t * C::kQLane; }
  __device__ uint8_t* q_ptr(int t) const { return base + C::kOffQ + t * C::kQLane; }
  __device__ uint32_t k_tile(int i) const { return s + C::kOffK + i * C::kTile8; }
  __device__ uint32_t v8_tile(int i) const { return s + C::kOffV8 + i * C::kTile8; }
  __device__ const uint8_t* v8_ptr(int i) const { return base + C::kOffV8 + i * C::kTile8; }
  __device__ uint32_t v_tile(int i) const { return s + C::kOffV + i * C::kTile16; }
  __device__ uint8_t* v_ptr(int i) const { return base + C::kOffV + i * C::kTile16; }
  __device__ float4* scales(int i) const { return reinterpret_cast<float4*>(base + C::kOffSc) + i * kScaleGroups; }
  __device__ uint32_t bar(int i) const { return s + C::kOffBar + i * 8; }
  __device__ uint32_t k_full(int i) const { return bar(i); }
  __device__ uint32_t k_empty(int i) const { return bar(C::kSK + i); }
  __device__ uint32_t v8_full(int i) const { return bar(2 * C::kSK + i); }
  __device__ uint32_t v8_empty(int i) const { return bar(2 * C::kSK + C::kSV8 + i); }
  __device__ uint32_t v_full(int i) const { return bar(2 * C::kSK + 2 * C::kSV8 + i); }
  __device__ uint32_t v_empty(int i) const { return bar(2 * C::kSK + 2 * C::kSV8 + C::kSV + i); }
  __device__ uint32_t rest(int i) const { return bar(2 * (C::kSK + C::kSV8 + C::kSV) + i); }
  __device__ uint32_t sc_empty(int i) const { return rest(i); }
  __device__ uint32_t q_full(int t) const { return rest(C::kSK + t); }
  __device__ uint32_t s_full(int t) const { return rest(C::kSK + 2 + t); }
  __device__ uint32_t p_half(int t) const { return rest(C::kSK + 4 + t); }
  __device__ uint32_t p_full(int t) const { return rest(C::kSK + 6 + t); }
  __device__ uint32_t o_final(int t) const { return rest(C::kSK + 8 + t); }
  __device__ uint32_t drain() const { return rest(C::kSK + 10); }
  __device__ uint32_t* q_mul() const { return reinterpret_cast<uint32_t*>(base + C::kOffQe); }
  __device__ uint32_t* slot() const { return reinterpret_cast<uint32_t*>(base + C::kOffSlot); }
  __device__ PagedShare* share() const { return reinterpret_cast<PagedShare*>(base + C::kOffShare); }
};

struct PagedTcParams {
  CUtensorMap tmap_k;  // e4m3 [num_blocks * Hkv, block_size, D], box {D, block_size, 1}
  CUtensorMap tmap_v;
  PagedParams c;
  float* ws_o;         // [2 * CTAs][256][D]
  float2* ws_ml;       // [2 * CTAs][256]
  PagedCut* cuts;      // [CTAs]
  float scale_log2;    // |scale| log2 e: its sign goes into Q, so larger raw scores are larger scores
  bool aligned32;      // out and ws_o begin on 32-byte boundaries
  float sc_in, sc_out; // soft-cap, from and to log2 units: sc_out tanh(sc_in s)
};

using Walk = PagedWalk<kRows>;

// Whether lane t of a unit has rows.
__device__ __forceinline__ bool lane_on(const PagedUnit& u, int t) { return t == 0 || u.rows > BM; }

// ------------------------------------------------------------------- loads
// One warp: lane i looks up block i of a tile and loads it, K then V.  Blocks
// past the last key and entries that name no block are read out of range:
// zeros, no memory touched.
template <int D, bool BF16>
__device__ __forceinline__ void load_role(const PagedTcParams& P, const Lay<D, BF16>& sm, Walk w, int lane) {
  using C = Cfg<D, BF16>;
  const PagedParams& p = P.c;
  const int per = BN >> p.block_shift, box = p.block_size * D;
  int g = 0;
  bool ok = true;
  int k_done = 0, v_done = 0;
  for (; ok && !w.done(); w.next(p)) {
    const int valid = paged_valid(p, w.u.q);
    const int32_t* table = p.tables + (int64_t)w.u.b * p.width;
    auto lookup = [&](int t) {  // -1: past the last key; -2: names no block
      const int i = t * per + lane;
      if (lane >= per || i >= (valid + p.block_size - 1) >> p.block_shift) return -1;
      const int e = __ldg(table + i);
      return e >= 0 && e < p.num_blocks ? e : -2;
    };
    int next = w.nt > 0 ? lookup(w.t0) : -1;
    for (int n = 0; n < w.nt; ++n, ++g) {
      const int blk = next;
      if (n + 1 < w.nt) next = lookup(w.t0 + n + 1);
      if (blk == -2) atomicOr(p.status, kStatusBadBlock);
      const int plane = blk >= 0 ? blk * p.Hkv + w.u.kvh : p.num_blocks * p.Hkv;
      const int sk = g % C::kSK, sv = g % C::kSV8;
      if (g >= C::kSK && !wait_warp(sm.k_empty(sk), ((g / C::kSK) - 1) & 1, p.timeout_ns, p.status)) { ok = false; break; }
      if (lane == 0) mbar_arrive_expect_tx(sm.k_full(sk), C::kTile8);
      __syncwarp();
      if (lane < per) tma_load_3d(sm.k_tile(sk) + lane * box, &P.tmap_k, sm.k_full(sk), 0, 0, plane);
      ++k_done;
      if (g >= C::kSV8 && !wait_warp(sm.v8_empty(sv), ((g / C::kSV8) - 1) & 1, p.timeout_ns, p.status)) { ok = false; break; }
      if (lane == 0) mbar_arrive_expect_tx(sm.v8_full(sv), C::kTile8);
      __syncwarp();
      if (lane < per) tma_load_3d(sm.v8_tile(sv) + lane * box, &P.tmap_v, sm.v8_full(sv), 0, 0, plane);
      ++v_done;
    }
  }
  // every copy lands before the CTA may exit
  for (int n = max(0, k_done - C::kSK); n < k_done; ++n)
    wait_warp(sm.k_full(n % C::kSK), (n / C::kSK) & 1, p.timeout_ns, p.status);
  for (int n = max(0, v_done - C::kSV8); n < v_done; ++n)
    wait_warp(sm.v8_full(n % C::kSV8), (n / C::kSV8) & 1, p.timeout_ns, p.status);
}

// ------------------------------------------------------------------ scales
// One warp: the scales of every tile, and the next unit's Q rows into L2.
template <int D, bool BF16>
__device__ __forceinline__ void scale_role(const PagedTcParams& P, const Lay<D, BF16>& sm, Walk w, int lane) {
  const PagedParams& p = P.c;
  ScaleFeed<Cfg<D, BF16>::kSK> feed;
  for (; !w.done(); w.next(p)) {
    Walk x = w;
    x.next(p);
    if (!x.done()) {  // whole tokens of the kv head's query heads
      const int t0 = paged_token(p, x.u.row0), t1 = paged_token(p, x.u.row0 + x.u.rows - 1);
      const uint16_t* q = static_cast<const uint16_t*>(p.q) + (int64_t)x.u.q.s0 * p.q_stride + x.u.kvh * p.group * D;
      for (int i = t0 + lane; i <= t1; i += 32) bulk_prefetch_l2(q + i * p.q_stride, (uint32_t)(p.group * D * 2));
    }
    if (!feed.unit(p, w, P.scale_log2, sm.scales(0), sm.k_full(0), sm.sc_empty(0), lane)) return;
  }
}

// ------------------------------------------------------------------ widen V
// Four warps: V tile rows, e4m3 to f16, rows past the last key as zeros (their
// slots may hold NaN bytes; P is 0 there but 0 * NaN is not).  In: rows of D
// bytes in the swizzle of that width.  Out: 64-value blocks of [128 keys][128
// bytes] in the 128-byte swizzle.  Eight lanes read 128 bytes that lie together
// (a row, or two of 64) and write each 16-byte piece as two: at D = 128 the
// upper four lanes, whose block lies a multiple of 128 bytes further, write
// theirs in the other order, so that the eight never share a bank.
template <int D, bool BF16>
__device__ __forceinline__ void widen_role(const PagedTcParams& P, const Lay<D, BF16>& sm, Walk w, int warp, int lane) {
  using C = Cfg<D, BF16>;
  const PagedParams& p = P.c;
  int g = 0;
  constexpr int kVec = D / 16;  // 16-byte pieces of a row
  const int c = lane % kVec, r0 = lane / kVec;
  const bool swap = c >= 4;
  for (; !w.done(); w.next(p)) {
    const int valid = paged_valid(p, w.u.q);
    for (int n = 0; n < w.nt; ++n, ++g) {
      const int s8 = g % C::kSV8, sv = g % C::kSV;
      if (!wait_warp(sm.v8_full(s8), (g / C::kSV8) & 1, p.timeout_ns, p.status)) return;
      if (g >= C::kSV && !wait_warp(sm.v_empty(sv), ((g / C::kSV) - 1) & 1, p.timeout_ns, p.status)) return;
      const int rows = min(valid - (w.t0 + n) * BN, BN);
      const uint8_t* src = sm.v8_ptr(s8);
      uint8_t* dst = sm.v_ptr(sv);
      constexpr int kIters = BN * kVec / 32 / 4;
#pragma unroll 1
      for (int i = 0; i < kIters; ++i) {
        const int row = (i * 4 + warp) * (32 / kVec) + r0;
        const int at = D == 128 ? c ^ (row & 7) : c ^ ((row >> 1) & 3);
        uint4 v = *reinterpret_cast<const uint4*>(src + row * D + at * 16);
        if (row >= rows) v = make_uint4(0u, 0u, 0u, 0u);
        const uint32_t e[4] = {v.x, v.y, v.z, v.w};
        uint32_t h[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, u;\n\t}"
              : "=r"(h[2 * k]), "=r"(h[2 * k + 1]) : "r"(e[k]));
        }
        uint8_t* out = dst + (c >> 2) * (BN * 128) + row * 128;
        const int lo = (2 * (c & 3)) ^ (row & 7), hi = lo ^ 1;
        const uint4 a = make_uint4(h[0], h[1], h[2], h[3]), b = make_uint4(h[4], h[5], h[6], h[7]);
        *reinterpret_cast<uint4*>(out + ((swap ? hi : lo) << 4)) = swap ? b : a;
        *reinterpret_cast<uint4*>(out + ((swap ? lo : hi) << 4)) = swap ? a : b;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(sm.v8_empty(s8));
        mbar_arrive(sm.v_full(sv));
      }
    }
  }
}

// --------------------------------------------------------------- MMA issuer
__device__ __forceinline__ void mma8x4_elect(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc0) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 a1, b1, a2, b2, a3, b3;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "setp.ne.b32 q, %4, 0;\n\t"
      "add.s64 a1, %1, 2;\n\tadd.s64 b1, %2, 2;\n\tadd.s64 a2, %1, 4;\n\tadd.s64 b2, %2, 4;\n\t"
      "add.s64 a3, %1, 6;\n\tadd.s64 b3, %2, 6;\n\t"
      "@p tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, q;\n\t"
      "@p tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a1, b1, %3, 1;\n\t"
      "@p tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a2, b2, %3, 1;\n\t"
      "@p tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a3, b3, %3, 1;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc0)
      : "memory");
}
__device__ __forceinline__ void mma8x2_elect(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc0) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 a1, b1;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "setp.ne.b32 q, %4, 0;\n\t"
      "add.s64 a1, %1, 2;\n\tadd.s64 b1, %2, 2;\n\t"
      "@p tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, q;\n\t"
      "@p tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a1, b1, %3, 1;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc0)
      : "memory");
}

// Lane by lane, per tile: P V of the tile before, then S of this one into the
// columns that P occupied.  A commit covers every earlier MMA of the thread,
// so "S ready" also says "O holds all earlier tiles".
template <int D, bool BF16>
__device__ __forceinline__ void mma_role(const PagedTcParams& P, const Lay<D, BF16>& sm, Walk w, uint32_t tmem, int lane) {
  using C = Cfg<D, BF16>;
  const PagedParams& p = P.c;
  constexpr uint32_t kIdS = idesc_e4m3(BM, BN, false, false);
  constexpr uint32_t kIdO = make_idesc_f16kind(false, BM, D, true);
  constexpr uint32_t kSwizzle = D == 128 ? 2 : 4;
  int g = 0;                          // tiles of the line
  int units[2] = {0, 0}, pc[2] = {0, 0};  // units begun, P tiles used, per lane
  bool ok = true;
  auto issue_s = [&](int t, int ks) {
    const uint64_t b = sdesc(sm.k_tile(ks), 16, 8 * D, kSwizzle);
#pragma unroll
    for (int i = 0; i < C::kQP; ++i) {
      const uint64_t a = sdesc(sm.q(t) + i * (BM * D), 16, 8 * D, kSwizzle);
      if constexpr (D == 128) mma8x4_elect(tmem + t * 128, a, b, kIdS, i > 0 ? 1u : 0u);
      else mma8x2_elect(tmem + t * 128, a, b, kIdS, i > 0 ? 1u : 0u);
    }
    tc_commit_elect(sm.s_full(t));
  };
  auto issue_pv = [&](int t, int vs, int half, bool first) {  // keys 64 half .. of the tile
    const uint64_t b = make_sdesc_sw128(sm.v_tile(vs), BN * 128, 1024) + (uint32_t)(half * 512);
    const uint32_t d = tmem + kColO + t * 128, a = tmem + t * 128 + half * 32;
    mma_ts4_elect(d, a, b, a + 8, b + 128u, a + 16, b + 256u, a + 24, b + 384u, kIdO, first ? 0u : 1u);
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
          if (!wait_warp(sm.p_half(t), pc[t] & 1, p.timeout_ns, p.status)) { ok = false; break; }
          tc_fence_after();
          issue_pv(t, sv, 0, n == 1);
          if (!wait_warp(sm.p_full(t), pc[t] & 1, p.timeout_ns, p.status)) { ok = false; break; }
          tc_fence_after();
          issue_pv(t, sv, 1, false);
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
// A lane's rows of Q as e4m3 pieces, K-major in the swizzle of the row width;
// rows past the unit's are zeros.  Each warp brings its own 32 rows.  The
// tensor core waits for this between two units, and most of the code comes
// from L2 each time, so it is three small loops:
//   all rows into shared memory as they are, in flight together: a row's first
//   and second half where its first two pieces will lie;
//   thread = row: its largest |x|, on packed 16-bit integers (magnitudes order as
//   their bits), and the power of two that brings it into [128, 256);
//   D / 8 threads a row: 8 values of the row each into pieces, in place, on
//   packed f16, which holds x scaled below 256 exactly down to 2^-24.
// Returns 1 / the scale of this thread's own row.
template <int D, bool BF16>
__device__ __forceinline__ float bring_q(const PagedTcParams& P, const Lay<D, BF16>& sm, const PagedUnit& u, int t,
                                         int wq, int lane) {
  using C = Cfg<D, BF16>;
  const PagedParams& p = P.c;
  constexpr int kVec = D / 8, kPer = 32 / kVec, kHalf = kVec / 2;  // 16-byte pieces of a row; rows an instruction
  constexpr uint32_t kInf = BF16 ? 0x7f80u : 0x7c00u;  // magnitudes from here on are not finite
  static_assert(C::kQP >= 2, "a row lies in the room of two pieces");
  const int c = lane % kVec, sub = lane / kVec, row0 = wq * 32;
  const uint32_t raw0 = (uint32_t)((c / kHalf) * (BM * D) + (row0 + sub) * D + (c % kHalf) * 16);  // + i kPer D
  {
    const int row = t * BM + row0 + lane;  // this thread's own; where it lies goes to the threads that load it
    const int tok = paged_token(p, u.row0 + row);
    const int64_t at = row < u.rows ? (int64_t)(u.q.s0 + tok) * p.q_stride +
                                          (u.kvh * p.group + u.row0 + row - tok * p.group) * D : -1;
    const uint16_t* q = static_cast<const uint16_t*>(p.q) + c * 8;
    const uint32_t to = sm.q(t) + raw0;
#pragma unroll 2
    for (int i = 0; i < kVec; ++i) {
      const int64_t from = __shfl_sync(0xffffffffu, at, i * kPer + sub);
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + i * (kPer * D)),
                   "l"(q + max(from, (int64_t)0)), "r"(from >= 0 ? 16 : 0) : "memory");
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncwarp();
  float inv;
  {
    const uint8_t* mine = sm.q_ptr(t) + (row0 + lane) * D;
    const int turn = D == 128 ? lane : lane >> 1;  // eight rows' pieces in eight banks' groups
    uint32_t top2 = 0;
#pragma unroll 4
    for (int i = 0; i < kVec; ++i) {
      const uint4 v = *reinterpret_cast<const uint4*>(mine + i / kHalf * (BM * D) + ((i + turn) % kHalf) * 16);
      top2 = __vmaxu2(top2, __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                                     __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu)));
    }
    const uint32_t top = max(top2 & 0xffffu, top2 >> 16);
    int ex;
    if constexpr (BF16) ex = (int)(top >> 7) - 127;
    else ex = (int)(__float_as_uint(__half2float(__ushort_as_half((unsigned short)top))) >> 23) - 127;
    const bool odd = top >= kInf;  // the row holds an infinity or NaN: its scores become NaN
    ex = top == 0u || odd ? 0 : min(max(7 - ex, -120), BF16 ? 120 : 30);
    if constexpr (BF16) {
      sm.q_mul()[t * BM + row0 + lane] = odd ? 0x7fc00000u : (uint32_t)(ex + 127) << 23;
    } else {
      const int e0 = min(ex, 15), e1 = ex - e0;  // ex is -8 .. 30
      sm.q_mul()[t * BM + row0 + lane] = (uint32_t)(odd ? 0x7e00 : (e0 + 15) << 10) | (uint32_t)(e1 + 15) << 26;
    }
    inv = __uint_as_float((uint32_t)(127 - ex) << 23);
  }
  __syncwarp();
  const uint32_t sign = p.scale < 0.0f ? 0x80008000u : 0u;
  uint8_t* base = sm.q_ptr(t);
#pragma unroll 1
  for (int i = 0; i < kVec; ++i) {
    const int r = row0 + i * kPer + sub;
    const uint4 v = *reinterpret_cast<const uint4*>(base + raw0 + i * (kPer * D));
    const uint32_t mbits = sm.q_mul()[t * BM + r];
    const float mul = __uint_as_float(mbits);                                 // bf16: the scale
    const uint32_t m0 = __byte_perm(mbits, 0, 0x1010), m1 = __byte_perm(mbits, 0, 0x3232);  // f16: its two factors
    __syncwarp();  // the row has been read
    const uint32_t e[4] = {v.x ^ sign, v.y ^ sign, v.z ^ sign, v.w ^ sign};
    uint32_t h[4];  // scaled, f16 pairs
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (BF16) {
        float a, b2;
        f2_split(fmul2(f2(__uint_as_float(e[k] << 16), __uint_as_float(e[k] & 0xffff0000u)), f2(mul, mul)), a, b2);
        const __half2 hh = __floats2half2_rn(a, b2);
        h[k] = *reinterpret_cast<const uint32_t*>(&hh);
      } else {  // two powers of two that f16 holds
        asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(h[k]) : "r"(e[k]), "r"(m0));
        asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(h[k]) : "r"(m1));
      }
    }
    // 8 bytes of chunk c / 2 of the row, whose index the swizzle XORs
    const int at = D == 128 ? ((c >> 1) ^ (r & 7)) : ((c >> 1) ^ ((r >> 1) & 3));
    uint8_t* out = base + r * D + at * 16 + (c & 1) * 8;
#pragma unroll
    for (int j = 0; j < C::kQP; ++j) {
      uint32_t w[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint16_t b0, b1;
        asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(b0) : "r"(h[2 * k]));
        asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(b1) : "r"(h[2 * k + 1]));
        asm("mov.b32 %0, {%1, %2};" : "=r"(w[k]) : "h"(b0), "h"(b1));
        if (j + 1 < C::kQP) {
          uint32_t f0, f1;
          asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(f0) : "h"(b0));
          asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(f1) : "h"(b1));
          asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(h[2 * k]) : "r"(h[2 * k]), "r"(f0));
          asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(h[2 * k + 1]) : "r"(h[2 * k + 1]), "r"(f1));
        }
      }
      *reinterpret_cast<uint2*>(out + j * (BM * D)) = make_uint2(w[0], w[1]);
    }
  }
  return inv;
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
__device__ __forceinline__ void softmax_role(const PagedTcParams& P, const Lay<D, BF16>& sm, Walk w, uint32_t tmem,
                                             int warp, int lane) {
  using C = Cfg<D, BF16>;
  const PagedParams& p = P.c;
  const int t = warp >> 2, wq = warp & 3, row = wq * 32 + lane;
  const uint32_t s_addr = tmem + ((uint32_t)(wq * 32) << 16) + t * 128;
  const uint32_t o_addr = s_addr - t * 128 + kColO + t * 128;
  int g = 0, sc = 0, oc = 0;  // tiles of the line, S tiles and units with tiles of this lane
  // of the unit whose rows are still to be stored
  bool stored = true, whole = false, head = false, mine = false;
  int prev_nt = 0;
  int64_t out_row = 0;
  float m_run = kNone, l_run = 0.0f;
  for (;;) {
    // ---- a unit's Q: this lane's last S has been read, so its Q is free, and the tensor core can
    // begin the unit while the last one's rows are stored
    float qs = 1.0f;  // 1 / the scale of this row's Q pieces
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
      const float inv = l_run == 0.0f ? 0.0f : kPagedSumFactor * (1.0f / l_run);
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
          store_32b(dst, &v[0], P.aligned32);
          store_32b(dst + 16, &v[8], P.aligned32);
        } else if (mine) {
          float* dst = P.ws_o + ws_row * D + k * 32;
#pragma unroll
          for (int i = 0; i < 4; ++i) store_32b(dst + 8 * i, &o[8 * i], P.aligned32);
        }
      }
      if (mine && whole && p.lse != nullptr)
        p.lse[out_row] = l_run == 0.0f ? -INFINITY : (m_run + (__log2f(l_run) + (kPagedSumLog2 - kPLog2))) * kLn2;
      if (mine && !whole) P.ws_ml[ws_row] = make_float2(m_run, l_run);
      tc_fence_before();  // these reads before this lane's next P arrival, which the next P V waits for
    }
    if (w.done()) return;
    const PagedUnit& u = w.u;
    const int nt = w.nt, t0 = w.t0;
    if (!lane_on(u, t)) {  // the other lane's tiles pass by; their scales too
      for (int n = 0; n < nt; ++n, ++g) {
        if (!wait_warp(sm.k_full(g % C::kSK), (g / C::kSK) & 1, p.timeout_ns, p.status)) return;
        if (lane == 0) mbar_arrive(sm.sc_empty(g % C::kSK));
      }
      w.next(p);
      continue;
    }
    mine = t * BM + row < u.rows;
    const int x0 = u.row0 + t * BM;
    const int last = min(x0 + BM, u.row0 + u.rows) - 1;
    const int2 lim = mine ? paged_limits(p, u.q, paged_token(p, x0 + row)) : make_int2(0, 0);
    const int full_lo = paged_limits(p, u.q, paged_token(p, last)).x, full_hi = paged_limits(p, u.q, paged_token(p, x0)).y;
    m_run = kNone;
    l_run = 0.0f;
    for (int n = 0; n < nt; ++n, ++g, ++sc) {
      const int key0 = (t0 + n) * BN;
      // a group's k scale |scale| log2 e and what follows of its V scale; raw scores times the row's
      // factor and the first are in log2 units.  The product stays above 0, so that -inf stays -inf
      // (they lie there once S does: K's barrier, which S waited for, takes the scale warp's arrival too)
      const float4* scl = sm.scales(g % C::kSK);
      if (!wait_warp(sm.s_full(t), sc & 1, p.timeout_ns, p.status)) return;
      const bool far_tile = scl[0].z == 0.0f;
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
      // tanh(scale s / c) of a raw score, c log2 e being the factor.  The hardware tanh: over all fp32 arguments on the
      // GB300 its error is at most 1.11e-5 of the value, 2^-16.46 (its specification allows 2^-11): at scores of 50 a weight is off by less
      // than half a step of f16.  As 1 - 2 / (e^2y + 1), two prompts with a cap take 433 us instead of 353.
      auto capped = [&](float x, float k) {
        if constexpr (SOFTCAP) return x == -INFINITY ? x : fast_tanh(x * fminf(k * qs * P.sc_in, 3e38f));
        return x;
      };
      auto factor = [&](float k) { return SOFTCAP ? P.sc_out : fmaxf(k * qs, 1.2e-38f); };
      // The row's largest score, 32 keys at a time: the loops stay rolled and S is read a second
      // time below, which costs less than the instruction fetches of code four times the size
      float m_tile = -INFINITY;
#pragma unroll kMaxUnroll
      for (int ch = 0; ch < 4; ++ch) {
        float x[32];
        tmem_ld32(s_addr + ch * 32, reinterpret_cast<uint32_t(&)[32]>(x));
        tmem_wait_ld();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float2 kl = *reinterpret_cast<const float2*>(scl + 2 * ch + h);
          float a = fmaxf(x[16 * h], x[16 * h + 1]), b = fmaxf(x[16 * h + 2], x[16 * h + 3]);
#pragma unroll
          for (int k = 4; k < 16; k += 4) {
            a = fmax3(a, x[16 * h + k], x[16 * h + k + 1]);
            b = fmax3(b, x[16 * h + k + 2], x[16 * h + k + 3]);
          }
          a = fmaxf(a, b);
          m_tile = fmaxf(m_tile, fmaf(capped(a, kl.x), factor(kl.x), kl.y));
        }
      }
      const bool rise = m_tile > m_run + kRise;
      const float m_new = rise ? m_tile : m_run;
      if (n > 0 && __any_sync(0xffffffffu, rise)) {  // O holds every earlier tile
        // the sum takes the factor in two steps: it may be as large as that is small, where V scales differ
        const float half = fast_exp2(0.5f * (m_run - m_new)), alpha = half * half;
        l_run = l_run * half * half;
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
      uint64_t sum = 0ull;
      if (__builtin_expect(far_tile, 0)) {  // a far tile
        float own = 0.0f;
#pragma unroll 1
        for (int c = 0; c < BN; c += 4) {
          float x[4];
          asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]) : "r"(s_addr + c) : "memory");
          tmem_wait_ld();
          const float kx = scl[c >> 4].x, kf = factor(kx);
#pragma unroll
          for (int k = 0; k < 4; ++k) own += fast_exp2(fmaf(capped(x[k], kx), kf, off));
        }
        sum = f2(own * kPagedSumFactor, 0.0f);
      }
#pragma unroll kExpUnroll
      for (int ch = 0; ch < 4; ++ch) {
        float x[32];
        tmem_ld32(s_addr + ch * 32, reinterpret_cast<uint32_t(&)[32]>(x));
        tmem_wait_ld();
        uint32_t pk[16];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float4 s4 = scl[2 * ch + h];
          const float kf = factor(s4.x);
          const uint64_t mul = f2(kf, kf), add = f2(s4.w + off, s4.w + off);
          uint64_t part[2] = {0ull, 0ull};
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            float a, b;
            f2_split(ffma2(f2(capped(x[16 * h + 2 * k], s4.x), capped(x[16 * h + 2 * k + 1], s4.x)), mul, add), a, b);
            a = fast_exp2(a);
            b = fast_exp2(b);
            part[k & 1] = fadd2(part[k & 1], f2(a, b));
            const __half2 hh = __floats2half2_rn(a, b);
            pk[8 * h + k] = *reinterpret_cast<const uint32_t*>(&hh);
          }
          sum = ffma2(fadd2(part[0], part[1]), f2(s4.z, s4.z), sum);
        }
        tmem_st16(s_addr + ch * 16, pk);  // over columns of S that have been read
        if (ch == 1) {  // P V of the first 64 keys runs during the others' exponentials
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(sm.p_half(t));
        }
      }
      float sa, sb;
      f2_split(sum, sa, sb);
      l_run += sa + sb;
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(sm.sc_empty(g % C::kSK));
        mbar_arrive(sm.p_full(t));
      }
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
__global__ void __launch_bounds__(kThreads, 1) attn_paged_tc_kernel(const __grid_constant__ PagedTcParams P) {
  using C = Cfg<D, BF16>;
  const PagedParams& p = P.c;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Lay<D, BF16> sm;
  sm.base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  sm.s = smem_u32(sm.base);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kSK; ++i) {
      mbar_init(sm.k_full(i), 2);  // the TMA's, and the scale warp's
      mbar_init(sm.k_empty(i), 1);
      mbar_init(sm.sc_empty(i), 8);
    }
    for (int i = 0; i < C::kSV8; ++i) {
      mbar_init(sm.v8_full(i), 1);
      mbar_init(sm.v8_empty(i), 4);
    }
    for (int i = 0; i < C::kSV; ++i) {
      mbar_init(sm.v_full(i), 4);
      mbar_init(sm.v_empty(i), 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(sm.q_full(t), 4);
      mbar_init(sm.s_full(t), 1);
      mbar_init(sm.p_half(t), 4);
      mbar_init(sm.p_full(t), 4);
      mbar_init(sm.o_final(t), 1);
    }
    mbar_init(sm.drain(), 1);
    mbar_init_fence();
    P.cuts[blockIdx.x].parts = 0;
  }
  if (warp == kTmaWarp && lane == 0) {
    tma_prefetch_desc(&P.tmap_k);
    tma_prefetch_desc(&P.tmap_v);
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(sm.slot()), 512);
    tmem_relinquish();
  }
  paged_share<kRows, kThreads>(p, sm.share());
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // The joining kernel may be scheduled; it waits.  Where no join follows this may let in any kernel, one with tensor memory
  // of its own among them, so this CTA has its columns by now.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(sm.slot());
  Walk w;
  w.begin(p, sm.share());
  if (warp < kVWarp0) softmax_role<D, BF16, SOFTCAP>(P, sm, w, tmem, warp, lane);
  else if (warp < kTmaWarp) widen_role<D, BF16>(P, sm, w, warp - kVWarp0, lane);
  else if (warp == kTmaWarp) load_role<D, BF16>(P, sm, w, lane);
  else if (warp == kMmaWarp) mma_role<D, BF16>(P, sm, w, tmem, lane);
  else if (warp == kScaleWarp) scale_role<D, BF16>(P, sm, w, lane);
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, bool BF16, bool SOFTCAP>
cudaError_t launch_tc(const PagedTcParams& P, int grid, cudaStream_t stream) {
  auto kernel = attn_paged_tc_kernel<D, BF16, SOFTCAP>;
  constexpr int smem = Cfg<D, BF16>::kSmem;
  static std::atomic<bool> ready[128];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 128 || !ready[dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 128) ready[dev].store(true, std::memory_order_relaxed);
  }
  kernel<<<grid, kThreads, smem, stream>>>(P);
  return cudaGetLastError();
}

template <int D, bool BF16>
cudaError_t launch_tc_d(const PagedTcParams& P, int grid, cudaStream_t stream) {
  return P.c.softcap > 0.0f ? launch_tc<D, BF16, true>(P, grid, stream) : launch_tc<D, BF16, false>(P, grid, stream);
}

}  // namespace

cudaError_t launch_attn_paged_tc(const PagedLaunch& L, bool bf16, cudaStream_t stream) {
  PagedTcParams P{};
  P.tmap_k = L.tmap_k;
  P.tmap_v = L.tmap_v;
  P.c = L.c;
  P.ws_o = L.ws_o;
  P.ws_ml = L.ws_ml;
  P.cuts = L.cuts;
  P.aligned32 = ((reinterpret_cast<uintptr_t>(L.c.out) | reinterpret_cast<uintptr_t>(L.ws_o)) & 31) == 0;
  P.scale_log2 = (float)(fabs((double)L.c.scale) * 1.4426950408889634);
  if (L.c.softcap > 0.0f) {
    P.sc_in = (float)std::min(3e38, 0.6931471805599453 / (double)L.c.softcap);
    P.sc_out = (float)((double)L.c.softcap * 1.4426950408889634);
  }
  if (L.c.D == 128) return bf16 ? launch_tc_d<128, true>(P, L.grid, stream) : launch_tc_d<128, false>(P, L.grid, stream);
  return bf16 ? launch_tc_d<64, true>(P, L.grid, stream) : launch_tc_d<64, false>(P, L.grid, stream);
}

}  // namespace gb300_attn
