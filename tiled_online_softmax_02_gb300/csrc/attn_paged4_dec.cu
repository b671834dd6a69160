// attn_paged4_dec.cu -- attention over the paged 4-bit KV cache for few query
// rows per (request, kv head): decode steps and drafted tokens.
//
// Floor: HBM, 4.5 bits a value.  At that rate every clock brings 41 values to
// an SM, which has 128 lanes of arithmetic for them, so instructions a value count:
//   S^T = K Q^T, O^T = V^T P^T   mma m16n8k16 in f16, keys (d for V) in M, the
//   query rows in N.  Its operands are registers, so the bytes go from shared
//   memory straight into them: one conversion and one multiplication for two
//   values.  (On the tcgen05 path widened values would have to be written to
//   shared memory and read again: 2 + 2 bytes a value, above what shared memory
//   moves.  Products on K as it lies, with block scales, were not tried.)
//   e2m1 * e4m3 is exact in f16 (6 bits, 2^-10 to 2688).  Q is f16 as it is, or
//   bf16 times a power of two a row that brings its largest element to 2^14,
//   which loses nothing above 2^-31 of that.  P is f16: 11 bits, 2^-29 of the
//   row's largest weight or less.
// Which value lies at which place of an operand is free as long as both sides
// agree, so every lane reads whole pieces of a row: 16 bytes of a key's K
// (values 32 t ..), 8 bytes of a key's V, whose 16 values share a scale.
// Two keys' V codes are put side by side in a byte before they are widened:
// four instructions for 16 values.
//
// Work sharing as in the 8-bit kernel (paged_sched.cuh); a CTA's warps take 32
// keys each in turn, with their own maximum, sum and O^T, and meet once a unit.
// Every warp brings its own keys by 16-byte asynchronous copies, a sub-tile
// ahead, the next unit's before the last one's rows are joined: no warp waits for
// another between two meetings, and nothing waits on a barrier in memory.
//
// Measured (one GB300, device time with the join, D = 128): 8 requests of 9K to
// 33K tokens, 32 query and 8 kv heads, bf16, 42.5 us, 4.5 TB/s, 67% of a copy's
// rate (the 8-bit kernel 58); 64 requests of up to 8K, 4 kv heads, f16, blocks of
// 16 slots, 39.1 us (54); one request of 3.5K 9.0 us (11.6).  About 8 us of each
// are the launch, the shares, the first keys and the join.  32 keys cost 540
// instructions: 128 conversions and 128 multiplications, on two pipes that take
// one every other cycle, 32 products, which with those alone take 138 cycles
// (a loop of nothing else), some 60 for the softmax, 45 for the loads.  The first
// case took 46.8 us with 38.4 of them left when its loads were left out, 36.3 when
// its arithmetic was.
// Slower: a ring of bulk copies fed by a ninth warp (51 us, its registers spill),
// K and V in stages apart (49), three stages (46.1), the next sub-tile's first
// product beside this one's second (46.1), V's rows in an order without bank
// conflicts (46.4 against 45.8).  Two accumulators for S: no change.
// No unit is full in that case: 2.4 of 4 issue slots a cycle, ALU 48%, DRAM 58%,
// tensor 21%.  16 warps an SM is what 128 registers allow (bf16 spills 24 bytes, 48
// under a soft-cap), so the rest of the time is latency that four warps a scheduler
// leave open.
#include <algorithm>
#include <atomic>
#include <cmath>

#include "paged4.cuh"
#include "paged4_internal.h"
#include "paged_mma.cuh"
#include "paged_sched.cuh"

namespace gb300_attn {
namespace {

constexpr int kSub = 32;                   // keys a warp takes at a time
constexpr float kRise = 8.0f;              // the maximum moves when a key passes it by 2^8
constexpr float kPLog2 = kPaged4DecLog2;   // P is carried as 2^(t - m + 5) <= 2^13

template <int D, int NT>
struct Cfg {
  static constexpr int NR = 8 * NT;                      // query rows of a unit
  static constexpr int kWarps = 8, kThreads = 32 * kWarps;
  static constexpr int kCtas = NT == 1 ? kPaged4DecCtas : 1;
  static constexpr int kStages = NT == 1 ? 2 : 4;        // sub-tiles in a warp's ring
  static constexpr int kLeft = NT == 1 ? 1 : 0;          // its last stages, which take the warp's O when a unit ends (0: a buffer apart)
  static constexpr int kRow = D / 2, kScRow = D / kGroup4;  // bytes of a row, and of its scales
  static constexpr int kData = kSub * kRow, kSc = kSub * kScRow;
  static constexpr int kStage = 2 * (kData + kSc);       // K, V, K scales, V scales
  static constexpr int kOffMerge = kWarps * kStages * kStage, kOwn = NR * D * 4;
  static constexpr int kOffMl = kOffMerge + (kLeft ? 0 : kWarps * kOwn);
  static constexpr int kOffShare = kOffMl + kWarps * NR * 8;
  static constexpr int kSmem = kOffShare + (int)sizeof(PagedShare);
  static_assert(kCtas * (kSmem + 1024) <= 228 * 1024 && kSmem <= 232448, "shared memory");
  static_assert((kLeft == 0 || kOwn <= kLeft * kStage) && kLeft < kStages && kStage % 16 == 0, "a warp's O");
};

struct Paged4DecParams {
  Paged4Params p;
  float scale_log2;     // |scale| log2 e
  float sc_in, sc_out;  // soft-cap: sc_out tanh(sc_in s) in log2 units
};

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint32_t select_bits(uint32_t a, uint32_t b, uint32_t mask) { return (a & mask) | (b & ~mask); }

// 16 bytes to shared memory: `bytes` of them copied, the others zeros.
__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// tanh to 2^-20 of itself: 1 - 2 / (e^2|y| + 1), and below 0.3 the Taylor series (the next term is 2^-24 of y).
__device__ __forceinline__ float tanh20(float y) {
  const float a = fabsf(y), z = y * y;
  const float big = copysignf(1.0f - 2.0f * fast_rcp(fast_exp2(a * 2.8853900817779268f) + 1.0f), y);
  float s = fmaf(z, 62.0f / 2835.0f, -17.0f / 315.0f);
  s = fmaf(z, s, 2.0f / 15.0f);
  s = fmaf(z, s, -1.0f / 3.0f);
  return a < 0.3f ? fmaf(y * z, s, y) : big;
}

// ------------------------------------------------------------------- loads
// A warp's sub-tiles of a unit's segment: first, first + kWarps, ... below end (in sub-tiles of the request's keys).
struct Subs {
  int first, count;
};

template <int NT, int W>
__device__ __forceinline__ Subs subs_of(const PagedParams& p, const PagedWalk<8 * NT, kWritten>& w, int warp) {
  const PagedUnit& u = w.u;
  const int lo = paged_limits(p, u.q, paged_token(p, u.row0)).x, hi = paged_limits(p, u.q, paged_token(p, u.row0 + u.rows - 1)).y;
  const int a = max(w.t0 * (kPagedKeys / kSub), lo / kSub) + warp;
  const int e = min((w.t0 + w.nt) * (kPagedKeys / kSub), (int)(((int64_t)hi + kSub - 1) / kSub));
  return Subs{a, w.nt > 0 && a < e ? (e - a + W - 1) / W : 0};
}

// The block-table entry of this lane's half of a sub-tile (lanes 0-15: its first 16 keys): -1 past the last key, -2 names
// no block.
__device__ __forceinline__ int entry_of(const PagedParams& p, const int32_t* table, int valid, int sub, int lane) {
  const int64_t key = (int64_t)sub * kSub + (lane & 16);
  if (key >= valid) return -1;
  const int e = load_written(table + (key >> p.block_shift));
  return e >= 0 && e < p.num_blocks ? e : -2;
}

// Copies a sub-tile into a stage: codes and scales as they lie, zeros for what has no block, and for the scales of keys past
// the last (their slots may hold NaN, and a weight of 0 times that is not 0).
template <int D, int NT>
__device__ __forceinline__ void load_sub(const Paged4Params& P, uint32_t stage, int kvh, int sub, int entry, int valid,
                                         int lane) {
  using C = Cfg<D, NT>;
  const PagedParams& p = P.c;
  if (entry == -2 && (lane & 15) == 0) atomicOr(p.status, kStatusBadBlock);
  // rows of the cache, of the sub-tile's first key as each half of it sees them
  const int e0 = __shfl_sync(0xffffffffu, entry, 0);
  const bool there0 = e0 >= 0;
  bool there1 = there0;
  int64_t row0 = ((int64_t)max(e0, 0) * p.Hkv + kvh) * p.block_size, row1;
  if (p.block_size < kSub) {  // two blocks of 16
    const int e1 = __shfl_sync(0xffffffffu, entry, 16);
    there1 = e1 >= 0;
    row1 = there1 ? ((int64_t)e1 * p.Hkv + kvh) * 16 - 16 : -16;
  } else {
    row0 += there0 ? (sub * kSub) & (p.block_size - 1) : 0;
    row1 = row0;
  }
  constexpr int kN = C::kData / 512;  // pieces of 16 bytes a lane takes of K, and of V
  const int at = lane * 16;
  const int64_t off0 = row0 * C::kRow + at, off1 = row1 * C::kRow + at;
#pragma unroll
  for (int j = 0; j < kN; ++j) {
    const int64_t off = (j < kN / 2 ? off0 : off1) + j * 512;
    const int bytes = (j < kN / 2 ? there0 : there1) ? 16 : 0;
    copy16(stage + j * 512 + at, p.k_cache + off, bytes);
    copy16(stage + C::kData + j * 512 + at, p.v_cache + off, bytes);
  }
  constexpr int kL = C::kSc / 16;  // lanes for K's scales, and for V's
  if (lane < 2 * kL) {
    const int l = lane & (kL - 1);
    const bool second = l >= kL / 2;
    const int bytes = min(max(valid - sub * kSub, 0), kSub) * C::kScRow - l * 16;
    copy16(stage + 2 * C::kData + at, (lane < kL ? P.k_sc : P.v_sc) + (second ? row1 : row0) * C::kScRow + l * 16,
           (second ? there1 : there0) ? min(max(bytes, 0), 16) : 0);
  }
}

// ----------------------------------------------------------------- compute
template <int D, int NT, bool BF16, bool SOFTCAP>
__device__ __forceinline__ void compute_role(const Paged4DecParams& DP, uint8_t* smem, const PagedShare* share,
                                             PagedWalk<8 * NT, kWritten> w, int warp, int lane) {
  using C = Cfg<D, NT>;
  const Paged4Params& P = DP.p;
  const PagedParams& p = P.c;
  constexpr int KS = D / 16, MT = D / 16, NR = C::NR, S = C::kStages, E = S - C::kLeft, W = C::kWarps;
  const int g = lane >> 2, t = lane & 3;
  uint8_t* ring = smem + warp * (S * C::kStage);
  const uint32_t ring_s = smem_u32(ring);
  const uint32_t sign = p.scale < 0.0f ? 0x80008000u : 0u;  // of the scale, into Q: larger raw scores are larger scores
  Subs subs;
  int first[S + 1];  // entries of the unit's first sub-tiles
  int entry;         // and of the one that is loaded next
  uint32_t raw[NT][2 * KS];  // this lane's part of Q: row g of every 8, values (D / 4) t ..
  // What a unit begins with, in the order in which it waits for memory: which blocks hold its first keys, its Q, the keys
  // themselves, all but those whose place still holds the last unit's O.
  auto look_up = [&]() {
    subs = subs_of<NT, W>(p, w, warp);
    const int valid = paged_valid(p, w.u.q);
    const int32_t* table = p.tables + (int64_t)w.u.b * p.width;
#pragma unroll
    for (int s = 0; s <= S; ++s) first[s] = s < subs.count ? entry_of(p, table, valid, subs.first + s * W, lane) : -1;
  };
  auto load_q = [&]() {
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
      for (int i = 0; i < 2 * KS; ++i) raw[j][i] = 0u;
      if (j * 8 + g < w.u.rows) {
        const int x = w.u.row0 + j * 8 + g, tok = paged_token(p, x);
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + (int64_t)(w.u.q.s0 + tok) * p.q_stride +
                                                          (int64_t)(w.u.kvh * p.group + x - tok * p.group) * D + t * (D / 4));
#pragma unroll
        for (int i = 0; i < KS / 2; ++i) {
          const uint4 v = load_written(src + i);
          raw[j][4 * i] = v.x; raw[j][4 * i + 1] = v.y; raw[j][4 * i + 2] = v.z; raw[j][4 * i + 3] = v.w;
        }
      }
    }
  };
  auto load_keys = [&](int from, int to) {
#pragma unroll
    for (int s = 0; s < S; ++s) {
      if (s < from || s >= to) continue;
      if (s < subs.count) load_sub<D, NT>(P, ring_s + s * C::kStage, w.u.kvh, subs.first + s * W, first[s], paged_valid(p, w.u.q), lane);
      copies_commit();
    }
  };
  if (!w.done()) {
    look_up();
    load_q();
    load_keys(0, S);
  }
  while (!w.done()) {
    const PagedUnit& u = w.u;
    entry = first[S];
    uint32_t qf[NT][KS][2];
    float fac[NT][2];  // what brings the raw scores of rows 2 t, 2 t + 1 to log2 units
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
      for (int i = 0; i < 2 * KS; ++i) raw[j][i] ^= sign;
      float down = 1.0f;  // 1 / the power of two that row g's Q carries
      if constexpr (BF16) {
        uint32_t top2 = 0;
#pragma unroll
        for (int i = 0; i < 2 * KS; ++i) top2 = __vmaxu2(top2, raw[j][i] & 0x7fff7fffu);
        uint32_t top = max(top2 & 0xffffu, top2 >> 16);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // up to [2^14, 2^15); rows of zeros and rows that hold an infinity or NaN stay as they are
        const int e = top == 0u || top >= 0x7f80u ? 0 : min(max(14 - ((int)(top >> 7) - 127), -120), 120);
        const float up = __uint_as_float((uint32_t)(127 + e) << 23);
        down = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
        for (int i = 0; i < 2 * KS; ++i)
          raw[j][i] = as_bits(__floats2half2_rn(__uint_as_float(raw[j][i] << 16) * up, __uint_as_float(raw[j][i] & 0xffff0000u) * up));
      }
      const float kh = P.k_heads ? P.k_heads[u.kvh] : 1.0f;
      // positive, so that -inf stays -inf, and finite, so that 0 stays 0.  Under a soft-cap hidden keys do not go through it, and
      // it may be next to nothing: a large cap brings its share back.
      down = fminf(fmaxf(down * (SOFTCAP ? DP.sc_in : DP.scale_log2) * kh, SOFTCAP ? 0.0f : 1.2e-38f), 3e38f);
      fac[j][0] = __shfl_sync(0xffffffffu, down, 8 * t);
      fac[j][1] = __shfl_sync(0xffffffffu, down, 8 * t + 4);
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        qf[j][s][0] = raw[j][2 * s];
        qf[j][s][1] = raw[j][2 * s + 1];
      }
    }
    float o[NT][MT][4], m[NT][2];
    uint64_t l2[NT];  // the rows' sums, a pair
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[j][i][k] = 0.0f;
      m[j][0] = m[j][1] = kNone;
      l2[j] = 0ull;
    }
    const int valid = paged_valid(p, u.q);
    const int full_lo = paged_limits(p, u.q, paged_token(p, u.row0 + u.rows - 1)).x;
    const int full_hi = paged_limits(p, u.q, paged_token(p, u.row0)).y;
    // ---- this warp's keys
    const int32_t* table = p.tables + (int64_t)u.b * p.width;
    int at = 0;  // n % S
    for (int n = 0; n < subs.count; ++n) {
      const int key0 = (subs.first + n * W) * kSub;
      uint32_t pf[NT][2][2];
      copies_wait<S - 1>();
      __syncwarp();
      const uint8_t* stage = ring + at * C::kStage;
      {
        const uint8_t* kd = stage;
        const uint8_t* ksc = stage + 2 * C::kData;
        float s[NT][2][4];
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int k = 0; k < 4; ++k) s[j][mt][k] = 0.0f;
          uint32_t wd[2][KS / 2];  // rows g and g + 8: codes, and their scales
          __half2 sc[2];
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int row = mt * 16 + x * 8 + g;
            if constexpr (D == 128) {
              const uint4 v = *reinterpret_cast<const uint4*>(kd + row * C::kRow + t * 16);
              wd[x][0] = v.x; wd[x][1] = v.y; wd[x][2] = v.z; wd[x][3] = v.w;
              sc[x] = as_half2(widen_e4m3x2(*reinterpret_cast<const uint16_t*>(ksc + row * C::kScRow + t * 2)));
            } else {
              const uint2 v = *reinterpret_cast<const uint2*>(kd + row * C::kRow + t * 8);
              wd[x][0] = v.x; wd[x][1] = v.y;
              sc[x] = as_half2(widen_e4m3x2(ksc[row * C::kScRow + t]));
            }
          }
#pragma unroll
          for (int i = 0; i < KS / 2; ++i) {  // eight values a lane: two steps of 16
            uint32_t a[2][4];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              widen8(wd[x][i], a[x][0], a[x][1], a[x][2], a[x][3]);
              const __half2 f = D == 128 && i >= KS / 4 ? __high2half2(sc[x]) : __low2half2(sc[x]);
#pragma unroll
              for (int k = 0; k < 4; ++k) a[x][k] = as_bits(__hmul2(as_half2(a[x][k]), f));
            }
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              mma16816(s[j][mt], a[0][0], a[1][0], a[0][1], a[1][1], qf[j][2 * i][0], qf[j][2 * i][1]);
              mma16816(s[j][mt], a[0][2], a[1][2], a[0][3], a[1][3], qf[j][2 * i + 1][0], qf[j][2 * i + 1][1]);
            }
          }
        }
        if constexpr (SOFTCAP) {
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
              for (int k = 0; k < 4; ++k) s[j][mt][k] = tanh20(s[j][mt][k] * fac[j][k & 1]);
        }
        if (key0 < full_lo || key0 + kSub > full_hi) {  // some key is hidden from some row
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const int r = j * 8 + 2 * t + x;
              const int2 lim = r < u.rows ? paged_limits(p, u.q, paged_token(p, u.row0 + r)) : make_int2(0, 0);
#pragma unroll
              for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                  const int key = key0 + mt * 16 + k * 8 + g;
                  if (key < lim.x || key >= lim.y) s[j][mt][2 * k + x] = -INFINITY;
                }
            }
        }
        // ---- the running maxima, which all lanes of a row share, move only when a key passes them by far
        float mx[NT][2];
        bool rise = false;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            mx[j][x] = fmaxf(fmax3(s[j][0][x], s[j][0][x + 2], s[j][1][x]), s[j][1][x + 2]) * (SOFTCAP ? DP.sc_out : fac[j][x]);
            rise |= mx[j][x] > m[j][x] + kRise;
          }
        if (__any_sync(0xffffffffu, rise)) {
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            float al[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              float v = mx[j][x];
              v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
              v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
              v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
              v = v > m[j][x] + kRise ? v : m[j][x];
              al[x] = fast_exp2(m[j][x] - v);
              m[j][x] = v;
            }
            l2[j] = fmul2(l2[j], f2(al[0], al[1]));
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
              for (int k = 0; k < 4; ++k) o[j][i][k] *= al[k & 1];
          }
        }
        // ---- weights, transposed into the second product's operand
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const uint64_t mul = SOFTCAP ? f2(DP.sc_out, DP.sc_out) : f2(fac[j][0], fac[j][1]);
          const uint64_t off = f2(kPLog2 - m[j][0], kPLog2 - m[j][1]);
#pragma unroll
          for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              float a, b;
              f2_split(ffma2(f2(s[j][mt][2 * k], s[j][mt][2 * k + 1]), mul, off), a, b);
              a = fast_exp2(a);
              b = fast_exp2(b);
              l2[j] = fadd2(l2[j], f2(a, b));
              pf[j][mt][k] = transpose8x8(as_bits(__floats2half2_rn(a, b)));
            }
        }
        // ---- O^T += V^T P^T: lane (g, t) has values (D / 8) g .. of keys 2 t, 2 t + 1, 2 t + 8, 2 t + 9
        const uint8_t* vd = stage + C::kData;
        const uint8_t* vsc = stage + 2 * C::kData + C::kSc;
        constexpr int VW = D / 64;  // words of a lane's values of a key
        const int gs = D == 128 ? g : g >> 1;
#pragma unroll
        for (int kt = 0; kt < 2; ++kt) {
          uint32_t wv[4][VW], sb[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int row = kt * 16 + (x >> 1) * 8 + 2 * t + (x & 1);
            if constexpr (D == 128) {
              const uint2 v = *reinterpret_cast<const uint2*>(vd + row * C::kRow + g * 8);
              wv[x][0] = v.x;
              wv[x][1] = v.y;
            } else {
              wv[x][0] = *reinterpret_cast<const uint32_t*>(vd + row * C::kRow + g * 4);
            }
            sb[x] = vsc[row * C::kScRow + gs];
          }
          const uint32_t s0 = widen_e4m3x2(sb[0] | sb[1] << 8), s1 = widen_e4m3x2(sb[2] | sb[3] << 8);
#pragma unroll
          for (int i = 0; i < VW; ++i) {
            uint32_t a0[4], a1[4], a2[4], a3[4];
            widen8(select_bits(wv[0][i], wv[1][i] << 4, 0x0f0f0f0fu), a0[0], a0[1], a0[2], a0[3]);
            widen8(select_bits(wv[0][i] >> 4, wv[1][i], 0x0f0f0f0fu), a1[0], a1[1], a1[2], a1[3]);
            widen8(select_bits(wv[2][i], wv[3][i] << 4, 0x0f0f0f0fu), a2[0], a2[1], a2[2], a2[3]);
            widen8(select_bits(wv[2][i] >> 4, wv[3][i], 0x0f0f0f0fu), a3[0], a3[1], a3[2], a3[3]);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              a0[k] = mul_f16x2(a0[k], s0);
              a1[k] = mul_f16x2(a1[k], s0);
              a2[k] = mul_f16x2(a2[k], s1);
              a3[k] = mul_f16x2(a3[k], s1);
            }
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
              for (int k = 0; k < 4; ++k) mma16816(o[j][4 * i + k], a0[k], a1[k], a2[k], a3[k], pf[j][kt][0], pf[j][kt][1]);
          }
        }
      }
      __syncwarp();  // the stage has been read
      if (n + S < subs.count) {
        const int next = subs.first + (n + S) * W;
        load_sub<D, NT>(P, ring_s + at * C::kStage, u.kvh, next, entry, valid, lane);
        if (n + S + 1 < subs.count) entry = entry_of(p, table, valid, next + W, lane);
      }
      copies_commit();
      at = at + 1 == S ? 0 : at + 1;
    }

    // ---- the unit's rows: the warps leave their maxima, sums and O, and the next unit's Q and first keys are on their way
    // while they meet.  A row's 16-byte pieces lie in an order that keeps eight writing lanes out of each other's banks.
    const int s0 = u.q.s0, head0 = u.kvh * p.group, kvh = u.kvh, row0 = u.row0, rows = u.rows;
    const bool whole = w.whole, head = w.head;
    if (!whole && head && threadIdx.x == 0) {
      PagedCut c;
      c.parts = paged_parts(w, share);
      c.token0 = s0;
      c.head0 = head0;
      c.row0 = row0;
      c.rows = rows;
      P.cuts[blockIdx.x] = c;
    }
    w.next(p);
    if (!w.done()) look_up();
    auto left = [&](int c) { return reinterpret_cast<float*>(smem + (C::kLeft ? (c * S + E) * C::kStage : C::kOffMerge + c * C::kOwn)); };
    auto turn = [](int r) { return D == 128 ? (r >> 1) & 3 : ((r >> 1) & 1) | ((r >> 2) & 1) << 2; };
    float2* ml = reinterpret_cast<float2*>(smem + C::kOffMl);
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      float l[2];
      f2_split(l2[j], l[0], l[1]);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        l[x] += __shfl_xor_sync(0xffffffffu, l[x], 4);
        l[x] += __shfl_xor_sync(0xffffffffu, l[x], 8);
        l[x] += __shfl_xor_sync(0xffffffffu, l[x], 16);
        const int r = j * 8 + 2 * t + x;
        if (r >= rows) continue;
        if (g == 0) ml[warp * NR + r] = make_float2(m[j][x], l[x]);
        float4* dst = reinterpret_cast<float4*>(left(warp) + r * D);
#pragma unroll
        for (int i = 0; i < MT / 2; ++i)
          dst[(g * (D / 32) + i) ^ turn(r)] = make_float4(o[j][2 * i][x], o[j][2 * i][x + 2], o[j][2 * i + 1][x], o[j][2 * i + 1][x + 2]);
      }
    }
    if (!w.done()) {
      load_q();
      load_keys(0, E);
    }

    // ---- the warps meet: rows' maxima, sums and O, joined in the order of the warps
    asm volatile("bar.sync 1, %0;" ::"n"(C::kThreads) : "memory");
    const float vh = P.v_heads ? P.v_heads[kvh] : 1.0f;
#pragma unroll 1
    for (int r = warp; r < rows; r += W) {
      constexpr int V = D / 32;
      const int d = lane * V;
      float M = kNone, L = 0.0f, acc[V];
#pragma unroll
      for (int c = 0; c < W; ++c) M = fmaxf(M, ml[c * NR + r].x);
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] = 0.0f;
#pragma unroll
      for (int c = 0; c < W; ++c) {
        const float2 y = ml[c * NR + r];
        const float wgt = fast_exp2(y.x - M);
        L = fmaf(wgt, y.y, L);
        const float* src = left(c) + r * D + ((d >> 2) ^ turn(r)) * 4 + (d & 3);
        float y4[4];
        if constexpr (V == 4) *reinterpret_cast<float4*>(y4) = *reinterpret_cast<const float4*>(src);
        else *reinterpret_cast<float2*>(y4) = *reinterpret_cast<const float2*>(src);
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] = fmaf(wgt, y4[v], acc[v]);
      }
      if (whole) {
        const int x = row0 + r, tok = paged_token(p, x);
        const int64_t row = (int64_t)(s0 + tok) * p.Hq + head0 + x - tok * p.group;
        const float inv = L == 0.0f ? 0.0f : vh / L;
        uint16_t* dst = static_cast<uint16_t*>(p.out) + row * D + d;
        uint32_t y[V / 2];
#pragma unroll
        for (int v = 0; v < V / 2; ++v)
          y[v] = (uint32_t)to_bits<BF16>(acc[2 * v] * inv) | (uint32_t)to_bits<BF16>(acc[2 * v + 1] * inv) << 16;
        if constexpr (V == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(y[0], y[1]);
        else *reinterpret_cast<uint32_t*>(dst) = y[0];
        if (p.lse != nullptr && d == 0) p.lse[row] = L == 0.0f ? -INFINITY : (M + (__log2f(L) - kPLog2)) * kLn2;
      } else {
        const int64_t row = (int64_t)(2 * blockIdx.x + (head ? 1 : 0)) * NR + r;
        float* dst = P.ws_o + row * D + d;
        if constexpr (V == 4) *reinterpret_cast<float4*>(dst) = make_float4(acc[0] * vh, acc[1] * vh, acc[2] * vh, acc[3] * vh);
        else *reinterpret_cast<float2*>(dst) = make_float2(acc[0] * vh, acc[1] * vh);
        if (d == 0) P.ws_ml[row] = make_float2(M, L * kPagedSumFactor);
      }
    }
    if (!w.done()) {
      asm volatile("bar.sync 2, %0;" ::"n"(C::kThreads) : "memory");  // the rows have been read
      load_keys(E, S);
    }
  }
  copies_wait<0>();
}

template <int D, int NT, bool BF16, bool SOFTCAP, bool LONG>
__global__ void __launch_bounds__(Cfg<D, NT>::kThreads, Cfg<D, NT>::kCtas)
    attn_paged4_dec_kernel(const __grid_constant__ Paged4DecParams DP) {
  using C = Cfg<D, NT>;
  const PagedParams& p = DP.p.c;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  PagedShare* share = reinterpret_cast<PagedShare*>(smem + C::kOffShare);
  after_earlier_kernels();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the joining kernel may be scheduled; it waits
  if (threadIdx.x == 0) DP.p.cuts[blockIdx.x].parts = 0;
  if constexpr (LONG) paged_share_long<8 * NT, C::kThreads, kPaged4Piece, kWritten>(p, share);
  else paged_share<8 * NT, C::kThreads, kPaged4Piece, kWritten>(p, share);
  __syncthreads();
  PagedWalk<8 * NT, kWritten> w;
  w.begin(p, share);
  compute_role<D, NT, BF16, SOFTCAP>(DP, smem, share, w, warp, lane);
}

template <int D, int NT, bool BF16, bool SOFTCAP, bool LONG>
cudaError_t launch_k(const Paged4DecParams& DP, int grid, cudaStream_t stream) {
  auto kernel = attn_paged4_dec_kernel<D, NT, BF16, SOFTCAP, LONG>;
  constexpr int smem = Cfg<D, NT>::kSmem;
  static std::atomic<bool> ready[128];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 128 || !ready[dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 128) ready[dev].store(true, std::memory_order_relaxed);
  }
  return launch_early(kernel, (unsigned)grid, Cfg<D, NT>::kThreads, smem, stream, DP);
}

template <int D, int NT, bool BF16, bool SOFTCAP>
cudaError_t launch_l(const Paged4DecParams& DP, int grid, cudaStream_t stream) {
  return paged_may_be_long<8 * NT>(DP.p.c) ? launch_k<D, NT, BF16, SOFTCAP, true>(DP, grid, stream)
                                           : launch_k<D, NT, BF16, SOFTCAP, false>(DP, grid, stream);
}

template <int D, int NT>
cudaError_t launch_n(const Paged4DecParams& DP, int grid, bool bf16, cudaStream_t stream) {
  if (DP.p.c.softcap > 0.0f) return bf16 ? launch_l<D, NT, true, true>(DP, grid, stream) : launch_l<D, NT, false, true>(DP, grid, stream);
  return bf16 ? launch_l<D, NT, true, false>(DP, grid, stream) : launch_l<D, NT, false, false>(DP, grid, stream);
}

}  // namespace

cudaError_t launch_attn_paged4_dec(const Paged4Params& p, int rows, int grid, bool bf16, cudaStream_t stream) {
  Paged4DecParams DP{};
  DP.p = p;
  DP.scale_log2 = (float)std::min(3e38, fabs((double)p.c.scale) * 1.4426950408889634);  // the sign goes into Q
  if (p.c.softcap > 0.0f) {
    DP.sc_in = (float)std::min(3e38, fabs((double)p.c.scale) / (double)p.c.softcap);
    DP.sc_out = (float)((double)p.c.softcap * 1.4426950408889634);
  }
  if (p.c.D == 128) return rows == 8 ? launch_n<128, 1>(DP, grid, bf16, stream) : launch_n<128, 2>(DP, grid, bf16, stream);
  return rows == 8 ? launch_n<64, 1>(DP, grid, bf16, stream) : launch_n<64, 2>(DP, grid, bf16, stream);
}

}  // namespace gb300_attn
