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
//               would, and K needs no conversion.
//   O += P V    kind::f16: P is f16 in tensor memory, V is widened to f16 by
//               four warps on its way from one shared buffer to another.
//               P as e4m3 pieces would cost the softmax warps, which have no
//               slots to spare, about six instructions a value; widening V
//               costs other warps half of one.
// A row of Q carries its own power-of-two scale, the largest that keeps it in
// e4m3's range, and pieces x0 = e4m3(x), x1 = e4m3(x - x0), ...: what is left
// is below 2^-18 of the row's largest element.
//
// Scales are constant over 16 keys or more (the smallest block).  Per group of
// 16 keys: the largest raw score is found first and scaled once, and
// 2^(s k_scale + log2 v_scale - m) is one FMA and one ex2 a value; the row sum
// takes each group's sum times 1 / v_scale.
//
// One CTA an SM walks its share of the line of key tiles (paged_sched.cuh).
// Roles (512 threads): warps 0-3 and 4-7 the softmax of the two lanes, thread =
// row, which also bring the next unit's Q rows into pieces before they finish
// the last; warps 8-11 widen V; warp 12 loads (TMA), 13 issues MMAs, 14 looks
// up scales.  Registers move from the latter eight warps to the softmax.
// Tensor memory: S_0, S_1, O_0, O_1, 128 columns each; P over its S.
#include <atomic>

#include "paged_mma.cuh"
#include "paged_sched.cuh"

namespace gb300_attn {
namespace {

constexpr int BM = 128, BN = kPagedKeys;
constexpr int kRows = kPagedTcRows;    // rows of a unit: two lanes of 128
constexpr int kThreads = 512;
constexpr int kVWarp0 = 8, kTmaWarp = 12, kMmaWarp = 13, kScaleWarp = 14;
constexpr int kGroups = BN / 16;       // scale groups of a tile
constexpr float kRise = 8.0f;          // the maximum moves when a key passes it by 2^8
constexpr float kPLog2 = kPagedTcLog2;  // P is carried as 2^(t - m + 7) <= 2^15
constexpr uint32_t kColO = 256;
constexpr int kSC = 4;                 // stages of the scale ring

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
  static constexpr int kOffSc = kOffV + kSV * kTile16;  // float4 [kSC][kGroups]: k scale, log2 v scale, 1 / v scale
  static constexpr int kOffBar = kOffSc + kSC * kGroups * 16;
  // k_full, k_empty [kSK], v8_full, v8_empty [kSV8], v_full, v_empty [kSV], sc_full, sc_empty [kSC],
  // q_full, s_full, p_full, o_final [2], drain
  static constexpr int kBars = 2 * (kSK + kSV8 + kSV + kSC) + 9;
  static constexpr int kOffSlot = kOffBar + kBars * 8;
  static constexpr int kOffShare = (kOffSlot + 16 + 15) / 16 * 16;
  static constexpr int kSmem = kOffShare + (int)sizeof(PagedShareSmem) + 1024;
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
  __device__ float4* scales(int i) const { return reinterpret_cast<float4*>(base + C::kOffSc) + i * kGroups; }
  __device__ uint32_t bar(int i) const { return s + C::kOffBar + i * 8; }
  __device__ uint32_t k_full(int i) const { return bar(i); }
  __device__ uint32_t k_empty(int i) const { return bar(C::kSK + i); }
  __device__ uint32_t v8_full(int i) const { return bar(2 * C::kSK + i); }
  __device__ uint32_t v8_empty(int i) const { return bar(2 * C::kSK + C::kSV8 + i); }
  __device__ uint32_t v_full(int i) const { return bar(2 * C::kSK + 2 * C::kSV8 + i); }
  __device__ uint32_t v_empty(int i) const { return bar(2 * C::kSK + 2 * C::kSV8 + C::kSV + i); }
  __device__ uint32_t rest(int i) const { return bar(2 * (C::kSK + C::kSV8 + C::kSV) + i); }
  __device__ uint32_t sc_full(int i) const { return rest(i); }
  __device__ uint32_t sc_empty(int i) const { return rest(kSC + i); }
  __device__ uint32_t q_full(int t) const { return rest(2 * kSC + t); }
  __device__ uint32_t s_full(int t) const { return rest(2 * kSC + 2 + t); }
  __device__ uint32_t p_full(int t) const { return rest(2 * kSC + 4 + t); }
  __device__ uint32_t o_final(int t) const { return rest(2 * kSC + 6 + t); }
  __device__ uint32_t drain() const { return rest(2 * kSC + 8); }
  __device__ uint32_t* slot() const { return reinterpret_cast<uint32_t*>(base + C::kOffSlot); }
  __device__ PagedShareSmem* share() const { return reinterpret_cast<PagedShareSmem*>(base + C::kOffShare); }
};

struct PagedTcParams {
  CUtensorMap tmap_k;  // e4m3 [num_blocks * Hkv, block_size, D], box {D, block_size, 1}
  CUtensorMap tmap_v;
  PagedParams c;
  float* ws_o;         // [2 * CTAs][256][D]
  float2* ws_ml;       // [2 * CTAs][256]
  PagedCut* cuts;      // [CTAs]
  float scale_abs;     // |scale|: its sign goes into Q, so larger raw scores are larger scores
  float sc_in, sc_out; // soft-cap: sc_out tanh(sc_in s), log2 units
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
  const int per = BN / p.block_size, box = p.block_size * D;
  int g = 0;
  bool ok = true;
  int k_done = 0, v_done = 0;
  for (; ok && !w.done(); w.next(p)) {
    const int64_t cap = min(w.u.q.total, (int64_t)p.width * p.block_size);
    const int32_t* table = p.tables + (int64_t)w.u.b * p.width;
    auto lookup = [&](int t) {  // -1: past the last key; -2: names no block
      const int64_t i = (int64_t)t * per + lane;
      if (lane >= per || i * p.block_size >= cap) return -1;
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
      if (g >= C::kSK && !mbar_wait_warp(sm.k_empty(sk), ((g / C::kSK) - 1) & 1, p.timeout_ns, p.status)) { ok = false; break; }
      if (lane == 0) mbar_arrive_expect_tx(sm.k_full(sk), C::kTile8);
      __syncwarp();
      if (lane < per) tma_load_3d(sm.k_tile(sk) + lane * box, &P.tmap_k, sm.k_full(sk), 0, 0, plane);
      ++k_done;
      if (g >= C::kSV8 && !mbar_wait_warp(sm.v8_empty(sv), ((g / C::kSV8) - 1) & 1, p.timeout_ns, p.status)) { ok = false; break; }
      if (lane == 0) mbar_arrive_expect_tx(sm.v8_full(sv), C::kTile8);
      __syncwarp();
      if (lane < per) tma_load_3d(sm.v8_tile(sv) + lane * box, &P.tmap_v, sm.v8_full(sv), 0, 0, plane);
      ++v_done;
    }
  }
  // every copy lands before the CTA may exit
  for (int n = max(0, k_done - C::kSK); n < k_done; ++n)
    mbar_wait_warp(sm.k_full(n % C::kSK), (n / C::kSK) & 1, p.timeout_ns, p.status);
  for (int n = max(0, v_done - C::kSV8); n < v_done; ++n)
    mbar_wait_warp(sm.v8_full(n % C::kSV8), (n / C::kSV8) & 1, p.timeout_ns, p.status);
}

// ------------------------------------------------------------------ scales
// One warp: lane i < 8 holds the scales of keys 16 i .. of a tile.
template <int D, bool BF16>
__device__ __forceinline__ void scale_role(const PagedTcParams& P, const Lay<D, BF16>& sm, Walk w, int lane) {
  const PagedParams& p = P.c;
  int g = 0;
  for (; !w.done(); w.next(p)) {
    const int64_t valid = min(w.u.q.total, (int64_t)p.width * p.block_size);
    const int32_t* table = p.tables + (int64_t)w.u.b * p.width;
    auto block_of = [&](int n) {
      const int64_t j = (int64_t)(w.t0 + n) * BN + lane * 16;
      const int b = lane < kGroups && n < w.nt && j < valid ? __ldg(table + (int)j / p.block_size) : -1;
      return b >= 0 && b < p.num_blocks ? b : -1;
    };
    int blk = block_of(0), blk1 = block_of(1);
    float ks = 0.0f, vs = 1.0f;
    auto fetch = [&](int b) {
      ks = 0.0f;
      vs = 1.0f;
      if (b >= 0) {
        ks = __ldg(p.k_scales + (int64_t)b * p.Hkv + w.u.kvh);
        vs = __ldg(p.v_scales + (int64_t)b * p.Hkv + w.u.kvh);
      }
    };
    fetch(blk);
    for (int n = 0; n < w.nt; ++n, ++g) {
      const float k0 = ks, v0 = fmaxf(vs, kMinVScale);
      fetch(blk1);
      blk1 = block_of(n + 2);
      const int st = g % kSC;
      if (g >= kSC && !mbar_wait_warp(sm.sc_empty(st), ((g / kSC) - 1) & 1, p.timeout_ns, p.status)) return;
      if (lane < kGroups) sm.scales(st)[lane] = make_float4(k0 * P.scale_abs, __log2f(v0), 1.0f / v0, 0.0f);
      __syncwarp();
      if (lane == 0) mbar_arrive(sm.sc_full(st));
    }
  }
}

// ------------------------------------------------------------------ widen V
// Four warps: V tile rows, e4m3 to f16, rows past the last key as zeros (their
// slots may hold NaN bytes; P is 0 there but 0 * NaN is not).  In: rows of D
// bytes in the swizzle of that width.  Out: 64-value blocks of [128 keys][128
// bytes] in the 128-byte swizzle.  A quarter-warp takes the four 16-byte pieces
// of 64 values of rows k and k ^ 5: the in-swizzle puts those in disjoint banks
// (bit 2 differs), and so does the out-swizzle (bit 0 differs).
template <int D, bool BF16>
__device__ __forceinline__ void widen_role(const PagedTcParams& P, const Lay<D, BF16>& sm, Walk w, int warp, int lane) {
  using C = Cfg<D, BF16>;
  const PagedParams& p = P.c;
  int g = 0;
  const int c = lane & 3, r8 = (lane >> 3) ^ ((lane & 4) ? 5 : 0);  // row of a group of 8
  for (; !w.done(); w.next(p)) {
    const int64_t valid = min(w.u.q.total, (int64_t)p.width * p.block_size);
    for (int n = 0; n < w.nt; ++n, ++g) {
      const int s8 = g % C::kSV8, sv = g % C::kSV;
      if (!mbar_wait_warp(sm.v8_full(s8), (g / C::kSV8) & 1, p.timeout_ns, p.status)) return;
      if (g >= C::kSV && !mbar_wait_warp(sm.v_empty(sv), ((g / C::kSV) - 1) & 1, p.timeout_ns, p.status)) return;
      const int64_t left = valid - (int64_t)(w.t0 + n) * BN;
      const int rows = left < BN ? (int)left : BN;
      const uint8_t* src = sm.v8_ptr(s8);
      uint8_t* dst = sm.v_ptr(sv);
      constexpr int kIters = BN / 8 * (D / 64) / 4;
#pragma unroll
      for (int i = 0; i < kIters; ++i) {
        const int it = i * 4 + warp;
        const int row = (it / (D / 64)) * 8 + r8, half = it % (D / 64);
        const int piece = half * 4 + c;
        const int at = D == 128 ? piece ^ (row & 7) : piece ^ ((row >> 1) & 3);
        uint4 v = *reinterpret_cast<const uint4*>(src + row * D + at * 16);
        if (row >= rows) v = make_uint4(0u, 0u, 0u, 0u);
        const uint32_t e[4] = {v.x, v.y, v.z, v.w};
        uint32_t h[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, u;\n\t}"
              : "=r"(h[2 * k]), "=r"(h[2 * k + 1]) : "r"(e[k]));
        }
        uint8_t* out = dst + half * (BN * 128) + row * 128;
        *reinterpret_cast<uint4*>(out + (((2 * c) ^ (row & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
        *reinterpret_cast<uint4*>(out + (((2 * c + 1) ^ (row & 7)) << 4)) = make_uint4(h[4], h[5], h[6], h[7]);
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
  auto issue_pv = [&](int t, int vs, bool first) {
    const uint64_t b = make_sdesc_sw128(sm.v_tile(vs), BN * 128, 1024);
    const uint32_t d = tmem + kColO + t * 128, a = tmem + t * 128;
#pragma unroll
    for (int k = 0; k < BN / 16; k += 4)
      mma_ts4_elect(d, a + k * 8, b + (uint32_t)(k * 128), a + (k + 1) * 8, b + (uint32_t)((k + 1) * 128),
                    a + (k + 2) * 8, b + (uint32_t)((k + 2) * 128), a + (k + 3) * 8, b + (uint32_t)((k + 3) * 128), kIdO,
                    (!first || k > 0) ? 1u : 0u);
  };
  for (; ok && !w.done(); w.next(p)) {
    if (w.nt == 0) continue;  // no S: the softmax warps take no Q of it either
    const bool two = lane_on(w.u, 1);
    for (int n = 0; ok && n <= w.nt; ++n) {
      const int sv = (g + n - 1 + C::kSV) % C::kSV, ks = (g + n) % C::kSK;
      bool k_ready = false;
      if (n >= 1 && !mbar_wait_warp(sm.v_full(sv), ((g + n - 1) / C::kSV) & 1, p.timeout_ns, p.status)) { ok = false; break; }
      for (int t = 0; t < (two ? 2 : 1); ++t) {
        if (n >= 1) {
          if (!mbar_wait_warp(sm.p_full(t), pc[t] & 1, p.timeout_ns, p.status)) { ok = false; break; }
          tc_fence_after();
          issue_pv(t, sv, n == 1);
          if (n == w.nt) tc_commit_elect(sm.o_final(t));
          ++pc[t];
        }
        if (n < w.nt) {
          if (n == 0) {
            if (!mbar_wait_warp(sm.q_full(t), units[t] & 1, p.timeout_ns, p.status)) { ok = false; break; }
            ++units[t];
          }
          if (!k_ready) {
            if (!mbar_wait_warp(sm.k_full(ks), ((g + n) / C::kSK) & 1, p.timeout_ns, p.status)) { ok = false; break; }
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
  mbar_wait_warp(sm.drain(), 0, p.timeout_ns, p.status);
}

// ------------------------------------------------------------------ softmax
// This thread's row of Q as e4m3 pieces into its lane's buffer.  Returns
// 1 / the row's scale.
template <int D, bool BF16>
__device__ __forceinline__ float bring_q(const PagedTcParams& P, const Lay<D, BF16>& sm, const PagedUnit& u, int t, int row) {
  using C = Cfg<D, BF16>;
  const PagedParams& p = P.c;
  const int x = u.row0 + t * BM + row;
  const bool in = t * BM + row < u.rows;
  uint4 raw[D / 8];
  if (in) {
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) +
                                                    (int64_t)(u.q.s0 + x / p.group) * p.q_stride +
                                                    (u.kvh * p.group + x % p.group) * D);
#pragma unroll
    for (int i = 0; i < D / 8; ++i) raw[i] = __ldg(q + i);
  } else {
#pragma unroll
    for (int i = 0; i < D / 8; ++i) raw[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  auto widen = [&](uint32_t v, float& a, float& b) {
    if constexpr (BF16) {
      a = __uint_as_float(v << 16);
      b = __uint_as_float(v & 0xffff0000u);
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&v));
      a = f.x;
      b = f.y;
    }
  };
  float top = 0.0f;
#pragma unroll
  for (int i = 0; i < D / 8; ++i) {
    const uint32_t e[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float a, b;
      widen(e[k], a, b);
      a = fabsf(a);
      b = fabsf(b);
      top = a < INFINITY ? fmaxf(top, a) : top;
      top = b < INFINITY ? fmaxf(top, b) : top;
    }
  }
  // the power of two that brings the largest element into [128, 256)
  int ex = (int)(__float_as_uint(top) >> 23) - 127;
  ex = top > 0.0f ? min(max(7 - ex, -120), 120) : 0;
  const float up = __uint_as_float((uint32_t)(ex + 127) << 23);
  const float mul = P.c.scale < 0.0f ? -up : up;
  uint8_t* dst = sm.q_ptr(t) + row * D;
#pragma unroll
  for (int c = 0; c < D / 16; ++c) {
    uint32_t w[3][4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint4 r = raw[2 * c + (k >> 1)];
      const uint32_t e0 = (k & 1) ? r.z : r.x, e1 = (k & 1) ? r.w : r.y;
      float v[4];
      widen(e0, v[0], v[1]);
      widen(e1, v[2], v[3]);
      bool odd = false;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        odd |= !(fabsf(v[i]) < INFINITY);
        v[i] *= mul;
      }
#pragma unroll
      for (int i = 0; i < C::kQP; ++i) {
        uint32_t two[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          uint16_t b;
          asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(b) : "f"(v[2 * j + 1]), "f"(v[2 * j]));
          two[j] = b;
          if (i + 1 < C::kQP) {
            uint32_t h2;
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(b));
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
            v[2 * j] -= f.x;
            v[2 * j + 1] -= f.y;
          }
        }
        w[i][k] = two[0] | (two[1] << 16);
      }
      if (odd) w[0][k] = 0x7f7f7f7fu;  // an element that is not finite makes its row's scores NaN
    }
    const int at = D == 128 ? (c ^ (row & 7)) : (c ^ ((row >> 1) & 3));
#pragma unroll
    for (int i = 0; i < C::kQP; ++i)
      *reinterpret_cast<uint4*>(dst + i * (BM * D) + at * 16) = make_uint4(w[i][0], w[i][1], w[i][2], w[i][3]);
  }
  return 1.0f / up;
}

template <int D, bool BF16, bool SOFTCAP>
__device__ __forceinline__ void softmax_role(const PagedTcParams& P, const Lay<D, BF16>& sm, Walk w, const PagedShare& share,
                                             uint32_t tmem, int warp, int lane) {
  const PagedParams& p = P.c;
  const int t = warp >> 2, wq = warp & 3, row = wq * 32 + lane;
  const uint32_t s_addr = tmem + ((uint32_t)(wq * 32) << 16) + t * 128;
  const uint32_t o_addr = s_addr - t * 128 + kColO + t * 128;
  int g = 0, sc = 0, oc = 0;  // tiles of the line, S tiles and finished units of this lane
  float qinv = 0.0f;
  auto q_ready = [&](const Walk& x) {
    if (x.done() || x.nt == 0 || !lane_on(x.u, t)) return;
    qinv = bring_q<D, BF16>(P, sm, x.u, t, row);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(sm.q_full(t));
  };
  q_ready(w);
  while (!w.done()) {
    const PagedUnit u = w.u;
    const int nt = w.nt, t0 = w.t0;
    const bool on = lane_on(u, t), mine = t * BM + row < u.rows;
    if (!on) {  // the other lane's tiles pass by; their scales too
      for (int n = 0; n < nt; ++n, ++g) {
        if (!mbar_wait_warp(sm.sc_full(g % kSC), (g / kSC) & 1, p.timeout_ns, p.status)) return;
        if (lane == 0) mbar_arrive(sm.sc_empty(g % kSC));
      }
      w.next(p);
      q_ready(w);
      continue;
    }
    const int x0 = u.row0 + t * BM;
    const int last = min(x0 + BM, u.row0 + u.rows) - 1;
    const int2 lim = mine ? paged_limits(p, u.q, (x0 + row) / p.group) : make_int2(0, 0);
    const int full_lo = paged_limits(p, u.q, last / p.group).x, full_hi = paged_limits(p, u.q, x0 / p.group).y;
    const float qs = qinv;
    float m_run = kNone, l_run = 0.0f;
    for (int n = 0; n < nt; ++n, ++g, ++sc) {
      const int key0 = (t0 + n) * BN;
      if (!mbar_wait_warp(sm.sc_full(g % kSC), (g / kSC) & 1, p.timeout_ns, p.status)) return;
      // raw score -> log2 units: x km + lv.  km stays above 0, so that -inf does
      float km[kGroups], lv[kGroups], iv[kGroups];
#pragma unroll
      for (int i = 0; i < kGroups; ++i) {
        const float4 s = sm.scales(g % kSC)[i];
        km[i] = fmaxf(s.x * qs, 1.2e-38f);
        lv[i] = s.y;
        iv[i] = s.z;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(sm.sc_empty(g % kSC));
      if (!mbar_wait_warp(sm.s_full(t), sc & 1, p.timeout_ns, p.status)) return;
      tc_fence_after();
      float x[BN];
#pragma unroll
      for (int k = 0; k < 4; ++k) tmem_ld32(s_addr + k * 32, *reinterpret_cast<uint32_t(*)[32]>(&x[k * 32]));
      tmem_wait_ld();
      if constexpr (SOFTCAP) {
        // tanh(scale s / c) as the raw value, c log2 e the factor.  The hardware tanh: its error, 2^-11 of c, is
        // below what a 16-bit output holds of scores that c caps
#pragma unroll
        for (int i = 0; i < BN; ++i) x[i] = fast_tanh(x[i] * (km[i / 16] * P.sc_in));
#pragma unroll
        for (int i = 0; i < kGroups; ++i) km[i] = P.sc_out;
      } else {
#pragma unroll
        for (int i = 0; i < kGroups; ++i) km[i] = fmaxf(km[i] * 1.4426950408889634f, 1.2e-38f);
      }
      if (key0 < full_lo || key0 + BN > full_hi) {
        const int lo = min(max(lim.x - key0, 0), BN), hi = min(max(lim.y - key0, 0), BN);
        const uint32_t span = hi > lo ? (uint32_t)(hi - lo) : 0u;
#pragma unroll
        for (int i = 0; i < BN; ++i) x[i] = (uint32_t)(i - lo) < span ? x[i] : -INFINITY;
      }
      float m_tile = -INFINITY;
#pragma unroll
      for (int i = 0; i < kGroups; ++i) {
        float a = fmaxf(x[16 * i], x[16 * i + 1]), b = fmaxf(x[16 * i + 2], x[16 * i + 3]);
#pragma unroll
        for (int k = 4; k < 16; k += 4) {
          a = fmax3(a, x[16 * i + k], x[16 * i + k + 1]);
          b = fmax3(b, x[16 * i + k + 2], x[16 * i + k + 3]);
        }
        m_tile = fmaxf(m_tile, fmaf(fmaxf(a, b), km[i], lv[i]));
      }
      float alpha = 1.0f;
      const bool rise = m_tile > m_run + kRise;
      if (rise) {
        alpha = fast_exp2(m_run - m_tile);
        m_run = m_tile;
        l_run *= alpha;
      }
      const float off = kPLog2 - m_run;
      uint64_t sum = 0ull;
#pragma unroll
      for (int ch = 0; ch < 4; ++ch) {
        uint32_t pk[16];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int i = ch * 2 + h;
          const uint64_t mul = f2(km[i], km[i]), add = f2(lv[i] + off, lv[i] + off);
          uint64_t part[2] = {0ull, 0ull};
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            float a, b;
            f2_split(ffma2(f2(x[16 * i + 2 * k], x[16 * i + 2 * k + 1]), mul, add), a, b);
            a = fast_exp2(a);
            b = fast_exp2(b);
            part[k & 1] = fadd2(part[k & 1], f2(a, b));
            const __half2 hh = __floats2half2_rn(a, b);
            pk[8 * h + k] = *reinterpret_cast<const uint32_t*>(&hh);
          }
          sum = ffma2(fadd2(part[0], part[1]), f2(iv[i], iv[i]), sum);
        }
        tmem_st16(s_addr + ch * 16, pk);
      }
      float sa, sb;
      f2_split(sum, sa, sb);
      l_run += sa + sb;
      if (n > 0 && __any_sync(0xffffffffu, rise)) {  // O holds every earlier tile
#pragma unroll
        for (int k = 0; k < D / 32; ++k) {
          uint32_t o[32];
          tmem_ld32(o_addr + k * 32, o);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
          tmem_st32(o_addr + k * 32, o);
        }
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(sm.p_full(t));
    }
    // ---- the next unit's Q (this lane's S of the last tile has been read, so its Q is free), then this unit's rows
    const bool whole = w.whole, head = w.head;
    if (!whole && head && threadIdx.x == 0) {
      PagedCut c;
      c.parts = paged_parts(w, share);
      c.token0 = u.q.s0;
      c.head0 = u.kvh * p.group;
      c.row0 = u.row0;
      c.rows = u.rows;
      P.cuts[blockIdx.x] = c;
    }
    w.next(p);
    q_ready(w);
    if (nt > 0) {
      if (!mbar_wait_warp(sm.o_final(t), oc & 1, p.timeout_ns, p.status)) return;
      ++oc;
      tc_fence_after();
    }
    const float inv = l_run == 0.0f ? 0.0f : 1.0f / l_run;
    const int xr = x0 + row;
    const int64_t out_row = (int64_t)(u.q.s0 + xr / p.group) * p.Hq + u.kvh * p.group + xr % p.group;
    const int64_t ws_row = (int64_t)(2 * blockIdx.x + (head ? 1 : 0)) * kRows + t * BM + row;
#pragma unroll
    for (int k = 0; k < D / 32; ++k) {
      uint32_t o[32];
      if (nt > 0) {
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
        uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + out_row * D + k * 32);
#pragma unroll
        for (int i = 0; i < 4; ++i) dst[i] = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
      } else if (mine) {
        uint4* dst = reinterpret_cast<uint4*>(P.ws_o + ws_row * D + k * 32);
#pragma unroll
        for (int i = 0; i < 8; ++i) dst[i] = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
      }
    }
    if (mine && whole && p.lse != nullptr)
      p.lse[out_row] = l_run == 0.0f ? -INFINITY : (m_run + (__log2f(l_run) - kPLog2)) * kLn2;
    if (mine && !whole) P.ws_ml[ws_row] = make_float2(m_run, l_run);
    tc_fence_before();  // these reads before this lane's next P arrival, which the next P V waits for
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
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the joining kernel may be scheduled; it waits
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kSK; ++i) {
      mbar_init(sm.k_full(i), 1);
      mbar_init(sm.k_empty(i), 1);
    }
    for (int i = 0; i < C::kSV8; ++i) {
      mbar_init(sm.v8_full(i), 1);
      mbar_init(sm.v8_empty(i), 4);
    }
    for (int i = 0; i < C::kSV; ++i) {
      mbar_init(sm.v_full(i), 4);
      mbar_init(sm.v_empty(i), 1);
    }
    for (int i = 0; i < kSC; ++i) {
      mbar_init(sm.sc_full(i), 1);
      mbar_init(sm.sc_empty(i), 8);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(sm.q_full(t), 4);
      mbar_init(sm.s_full(t), 1);
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
  const PagedShare share = paged_share<kRows, kThreads>(p, sm.share());
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(sm.slot());
  // 512 threads of 128 registers at launch: 256 x 200 + 256 x 56 = 512 x 128
  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    Walk w;
    w.begin(p, share);
    softmax_role<D, BF16, SOFTCAP>(P, sm, w, share, tmem, warp, lane);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    Walk w;
    w.begin(p, share);
    if (warp < kTmaWarp) widen_role<D, BF16>(P, sm, w, warp - kVWarp0, lane);
    else if (warp == kTmaWarp) load_role<D, BF16>(P, sm, w, lane);
    else if (warp == kMmaWarp) mma_role<D, BF16>(P, sm, w, tmem, lane);
    else if (warp == kScaleWarp) scale_role<D, BF16>(P, sm, w, lane);
  }
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
  P.scale_abs = fabsf(L.c.scale);
  if (L.c.softcap > 0.0f) {
    P.sc_in = 1.0f / L.c.softcap;
    P.sc_out = (float)((double)L.c.softcap * 1.4426950408889634);
  }
  if (L.c.D == 128) return bf16 ? launch_tc_d<128, true>(P, L.grid, stream) : launch_tc_d<128, false>(P, L.grid, stream);
  return bf16 ? launch_tc_d<64, true>(P, L.grid, stream) : launch_tc_d<64, false>(P, L.grid, stream);
}

}  // namespace gb300_attn
