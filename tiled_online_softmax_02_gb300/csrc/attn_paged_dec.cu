// attn_paged_dec.cu -- attention over the paged 8-bit KV cache for few query
// rows per (request, kv head): decode steps, drafted tokens to verify.
//
// Bound: HBM.  Every cached byte is read once, and the e4m3 bytes go from the
// cache to the tensor cores as they are -- TMA into shared memory, tcgen05
// kind::f8f6f4 from there -- so no lane converts a K or V value.  As few rows
// would leave a 128-row tile empty, keys stand in M and rows in N:
//   S^T[key, row] = K_tile Q^T           M = 128 keys, N = pieces * NR, K = D
//   O^T[d, row]  += V_tile^T P^T         M = 128 (d),  N = 3 * NR, K = 128 keys
// The 16-bit and fp32 factors are carried as sums of e4m3 pieces, each piece
// its own rows of N:  x = x0 + x1 / 32 + x2 / 1024, x0 = e4m3(x),
// x1 = e4m3(32 (x - x0)), ...  A piece's rest is at most 2^-4 of it, so two
// pieces hold a bf16 Q exactly and three an f16 Q (down to 2^-23 and 2^-28 of
// the row's largest element, which a power of two brings into e4m3's range), and
// three hold a P of 11 bits (it is rounded to f16 first, as packed f16
// arithmetic splits it in half the instructions; 16-bit outputs have no more
// bits, the row sum takes the unrounded weights), down to 2^-25 of its largest.
//
// Scales: a key's K scale multiplies its scores (the thread that owns the key
// holds it).  Its V scale enters the exponent, t = s log2 e + log2 v_scale,
// so O accumulates 2^(t - m) v8 whatever the scales are, m being the running
// maximum of t, and the row sum takes 2^(t - m) / v_scale (paged_sched.cuh: in
// far tiles, without the detour by 2^(t - m)).
//
// One CTA walks its share of the line of key tiles (paged_sched.cuh).  Roles
// (256 threads): warps 0-3 softmax, thread = key; warp 4 K loads, warp 5 V
// loads (block table lookup by lanes, one TMA box a block), warp 6 MMA issue,
// warp 7 the next unit's Q into pieces, and the scales of its tiles.
//
// Measured (one GB300, device time with the join): 8 requests of 9K to 32.7K
// tokens, 8 kv heads, 4 rows each, bf16, D = 128: 58.2 us, 5.9 TB/s, 87% of a
// copy's rate; 64 requests of 100 to 8000 tokens, 4 kv heads, 8 rows, f16,
// blocks of 16: 54.1 us, 4.9 TB/s, 73%; one request of 3.5K tokens: 11.3 us,
// which is the way to the first result.  Two CTAs an SM, each with a ring of
// 80 KB (64 KB at D = 64), keep about 24 MB on their way; a warp's
// instructions, not registers or shared memory, are what these roles run out
// of, so loops stay rolled where they can.  Units of 16 rows spill about 120
// bytes a thread at the 128 registers that two CTAs leave.
#include <algorithm>
#include <atomic>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "paged_mma.cuh"
#include "paged_sched.cuh"

namespace gb300_attn {
namespace {

constexpr int kThreads = 256;
constexpr int kKWarp = 4, kVWarp = 5, kMmaWarp = 6;  // warp 7: Q
constexpr float kInvStep = 1.0f / kPieceStep;
// P is carried as 32 * 2^(t - m); the maximum moves when a key passes it by
// more than 3 (log2 units), so the first piece stays below 256 < 448.
constexpr float kRise = 3.0f, kPLog2 = kPagedDecLog2;

template <int D, int NR, bool BF16>
struct Cfg {
  static constexpr int kQP = BF16 ? 2 : 3;                        // pieces of Q
  static constexpr int kPP = 3;                                   // pieces of P
  static constexpr int kNQ = (kQP * NR + 15) / 16 * 16;           // N of S^T
  static constexpr int kNP = (kPP * NR + 15) / 16 * 16;           // N of O^T
  static constexpr int kTile = kPagedKeys * D;                    // bytes of a K or V tile
  static constexpr int kSK = D == 64 ? 4 : 3;                     // K stages
  static constexpr int kSV = D == 64 ? 4 : 2;                     // V stages
  static constexpr int kQBytes = (kNQ * D + 1023) / 1024 * 1024;
  static constexpr int kPBytes = kNP * kPagedKeys;
  static constexpr int kOffK = 0;
  static constexpr int kOffV = kOffK + kSK * kTile;
  static constexpr int kOffQ = kOffV + kSV * kTile;               // two buffers
  static constexpr int kOffP = kOffQ + 2 * kQBytes;               // two buffers
  static constexpr int kOffLim = kOffP + 2 * kPBytes;             // int2 [2][NR]
  static constexpr int kOffRed = kOffLim + 2 * NR * 8;            // float [2][4][NR]: maxima, sums
  static constexpr int kOffQs = kOffRed + 2 * 4 * NR * 4;         // float [2][NR]: 1 / scale of a row's Q pieces
  static constexpr int kOffSc = kOffQs + 2 * NR * 4;                      // float4 [kSK][kScaleGroups]
  static constexpr int kOffBar = kOffSc + kSK * kScaleGroups * 16;
  // k_full, k_empty [kSK], v_full, v_empty [kSV], s_full, p_full, pv_done, q_full, q_empty [2],
  // sc_empty [kSK], drain
  static constexpr int kBars = 2 * kSK + 2 * kSV + 11 + kSK;
  static constexpr int kOffSlot = kOffBar + kBars * 8;
  static constexpr int kOffShare = (kOffSlot + 16 + 15) / 16 * 16;
  static constexpr int kSmem = kOffShare + (int)sizeof(PagedShare) + 1024;  // + alignment slack
  static constexpr int kColO = 2 * kNQ;                           // TMEM: S^T twice, then O^T
  static constexpr int kCols = 2 * kNQ + kNP;
  static constexpr uint32_t kTmem = kCols <= 32 ? 32 : kCols <= 64 ? 64 : kCols <= 128 ? 128 : kCols <= 256 ? 256 : 512;
  static_assert(kTmem * kPagedDecCtas <= 512, "tensor memory");
  static_assert(kSmem <= 115200, "shared memory of two CTAs on an SM");
  static_assert(kOffBar % 8 == 0 && kOffQ % 1024 == 0 && kOffP % 1024 == 0, "alignment");
};

template <int D, int NR, bool BF16>
struct Lay {
  using C = Cfg<D, NR, BF16>;
  uint8_t* base;
  uint32_t s;
  __device__ uint32_t k_tile(int i) const { return s + C::kOffK + i * C::kTile; }
  __device__ uint32_t v_tile(int i) const { return s + C::kOffV + i * C::kTile; }
  __device__ uint8_t* v_ptr(int i) const { return base + C::kOffV + i * C::kTile; }
  __device__ uint32_t q(int i) const { return s + C::kOffQ + i * C::kQBytes; }
  __device__ uint8_t* q_ptr(int i) const { return base + C::kOffQ + i * C::kQBytes; }
  __device__ uint32_t p(int i) const { return s + C::kOffP + i * C::kPBytes; }
  __device__ uint8_t* p_ptr(int i) const { return base + C::kOffP + i * C::kPBytes; }
  __device__ int2* lim(int i) const { return reinterpret_cast<int2*>(base + C::kOffLim) + i * NR; }
  __device__ float* red(int i) const { return reinterpret_cast<float*>(base + C::kOffRed) + i * 4 * NR; }
  __device__ float* qs(int i) const { return reinterpret_cast<float*>(base + C::kOffQs) + i * NR; }
  __device__ uint32_t bar(int i) const { return s + C::kOffBar + i * 8; }
  __device__ uint32_t k_full(int i) const { return bar(i); }
  __device__ uint32_t k_empty(int i) const { return bar(C::kSK + i); }
  __device__ uint32_t v_full(int i) const { return bar(2 * C::kSK + i); }
  __device__ uint32_t v_empty(int i) const { return bar(2 * C::kSK + C::kSV + i); }
  __device__ uint32_t rest(int i) const { return bar(2 * C::kSK + 2 * C::kSV + i); }
  __device__ uint32_t s_full(int i) const { return rest(i); }
  __device__ uint32_t p_full(int i) const { return rest(2 + i); }
  __device__ uint32_t pv_done(int i) const { return rest(4 + i); }
  __device__ uint32_t q_full(int i) const { return rest(6 + i); }
  __device__ uint32_t q_empty(int i) const { return rest(8 + i); }
  __device__ uint32_t sc_empty(int i) const { return rest(10 + i); }
  __device__ uint32_t drain() const { return rest(10 + C::kSK); }
  __device__ float4* scales(int i) const { return reinterpret_cast<float4*>(base + C::kOffSc) + i * kScaleGroups; }
  __device__ uint32_t* slot() const { return reinterpret_cast<uint32_t*>(base + C::kOffSlot); }
  __device__ PagedShare* share() const { return reinterpret_cast<PagedShare*>(base + C::kOffShare); }
};

__device__ __forceinline__ void mma8_elect(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "setp.ne.b32 q, %4, 0;\n\t"
      "@p tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, q;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// n consecutive 32-bit columns of this thread's TMEM lane (n = 4, 8 or 16).
__device__ __forceinline__ void tld(uint32_t a, float (&r)[4]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
               : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void tld(uint32_t a, float (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7])
               : "r"(a) : "memory");
}
__device__ __forceinline__ void tld(uint32_t a, float (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15}, [%16];"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
        "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
      : "r"(a) : "memory");
}
__device__ __forceinline__ void tst16(uint32_t a, const float (&r)[16]) {
  tmem_st16(a, reinterpret_cast<const uint32_t(&)[16]>(r));
}

// e4m3 pieces of four values in two packed f16 pairs: the piece's bytes, and
// the pairs become what is left of them times 32 (exact).
__device__ __forceinline__ uint32_t last4(uint32_t h0, uint32_t h1) {
  uint16_t b0, b1;
  uint32_t w;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(b0) : "r"(h0));
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(b1) : "r"(h1));
  asm("mov.b32 %0, {%1, %2};" : "=r"(w) : "h"(b0), "h"(b1));
  return w;
}
__device__ __forceinline__ uint32_t piece4(uint32_t& h0, uint32_t& h1) {
  const uint32_t w = last4(h0, h1);
  uint32_t f0, f1;
  asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, u;\n\t}"
      : "=r"(f0), "=r"(f1) : "r"(w));
  asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(h0) : "r"(f0));
  asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(h1) : "r"(f1));
  asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(h0) : "r"(0x50005000u));
  asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(h1) : "r"(0x50005000u));
  return w;
}

__device__ __forceinline__ uint64_t fsub2(uint64_t a, uint64_t b) { return ffma2(b, f2(-1.0f, -1.0f), a); }

// Reduce-scatter over the warp: on entry each lane holds NR values; on exit
// lane l holds the max (sum) over all lanes of value row_of_lane<NR>(l).
template <int NR>
__device__ __forceinline__ int row_of_lane(int lane) {
  int r = 0, half = NR / 2;
#pragma unroll
  for (int bit = 4; half >= 1; --bit, half >>= 1)
    if (lane & (1 << bit)) r += half;
  return r;
}
template <int NR, bool MAX>
__device__ __forceinline__ float reduce_scatter(float (&v)[NR], int lane) {
#pragma unroll
  for (int half = NR / 2, bit = 4; half >= 1; half >>= 1, --bit) {
    const bool upper = (lane >> bit) & 1;
#pragma unroll
    for (int k = 0; k < half; ++k) {
      const float send = upper ? v[k] : v[k + half];
      const float keep = upper ? v[k + half] : v[k];
      const float got = __shfl_xor_sync(0xffffffffu, send, 1 << bit);
      v[k] = MAX ? fmaxf(keep, got) : keep + got;
    }
  }
  float x = v[0];
#pragma unroll
  for (int bit = 0; (1 << bit) < 32 / NR; ++bit) {
    const float got = __shfl_xor_sync(0xffffffffu, x, 1 << bit);
    x = MAX ? fmaxf(x, got) : x + got;
  }
  return x;
}

struct DecParams {
  CUtensorMap tmap_k;  // e4m3 [num_blocks * Hkv, block_size, D], box {D, block_size, 1}
  CUtensorMap tmap_v;
  PagedParams c;
  float* ws_o;         // [2 * CTAs][NR][D]: partial rows, sum of 2^(t - m) v8
  float2* ws_ml;       // [2 * CTAs][NR]: m, 2^-8 sum of 2^(t - m) / v_scale
  PagedCut* cuts;      // [CTAs]
  float k1, k2, k3;    // soft-cap in log2 units: k2 / (2^(k1 s) + 1) + k3; k3 tanh(k1 s) where k2 is 0
  float scale_log2;
};

// ------------------------------------------------------------------ loaders
// One warp; lane i looks up and loads block i of a tile.  Blocks past the
// request's last key, and entries that name no block, are read out of range,
// which fills their rows with zeros and touches no memory.
template <int D, int NR, int NS>
__device__ __forceinline__ void load_role(const DecParams& P, const CUtensorMap* tmap, PagedWalk<NR> w, uint32_t ring,
                                          uint32_t full0, uint32_t empty0, int lane, bool report) {
  const PagedParams& p = P.c;
  constexpr int kTile = kPagedKeys * D;
  const int per = kPagedKeys >> p.block_shift, box = p.block_size * D;
  int g = 0;
  bool ok = true;
  auto lookup = [&](const PagedWalk<NR>& x, int n) {  // tile n of x's segment.  -1: past the last key; -2: names no block
    const int i = (x.t0 + n) * per + lane;
    if (lane >= per || i >= (paged_valid(p, x.u.q) + p.block_size - 1) >> p.block_shift) return -1;
    const int e = __ldg(p.tables + (int64_t)x.u.b * p.width + i);
    return e >= 0 && e < p.num_blocks ? e : -2;
  };
  int next = w.done() ? -1 : lookup(w, 0);
  while (ok && !w.done()) {
    PagedWalk<NR> y = w;  // the next unit, its first blocks looked up while this one's stream
    y.next(p);
    const int first = y.done() ? -1 : lookup(y, 0);
    for (int n = 0; n < w.nt; ++n, ++g) {
      const int st = g % NS, blk = next;
      if (n + 1 < w.nt) next = lookup(w, n + 1);
      if (g >= NS && !wait_warp(empty0 + st * 8, ((g / NS) - 1) & 1, p.timeout_ns, p.status)) {
        ok = false;
        break;
      }
      if (lane == 0) mbar_arrive_expect_tx(full0 + st * 8, kTile);
      __syncwarp();
      if (lane < per) {
        if (report && blk == -2) atomicOr(p.status, kStatusBadBlock);
        tma_load_3d(ring + st * kTile + lane * box, tmap, full0 + st * 8, 0, 0,
                    blk >= 0 ? blk * p.Hkv + w.u.kvh : p.num_blocks * p.Hkv);
      }
    }
    w = y;
    next = first;
  }
  // every copy lands before the CTA may exit
  for (int n = g > NS ? g - NS : 0; n < g; ++n) wait_warp(full0 + (n % NS) * 8, (n / NS) & 1, p.timeout_ns, p.status);
}

// ------------------------------------------------------- Q pieces and scales
// One warp: the unit's rows as e4m3 pieces, piece i of row r at row i * NR + r,
// K-major in the swizzle of the row width; rows past the unit's are zeros (the
// rows of N past the pieces were zeroed once).  Then the scales of the unit's
// tiles.  A row is D / 8 lanes wide (16 bytes each).  The next unit waits for
// this, and at the kernel's start every instruction comes from L2 first, so it
// is a loop of at most four steps' code, the next rows on their way: a row's
// largest |x| on packed 16-bit integers (magnitudes order as
// their bits), pieces and rests on packed f16, which holds x scaled below 256
// exactly down to 2^-24.
template <int D, int NR, bool BF16>
__device__ __forceinline__ void q_role(const DecParams& P, const Lay<D, NR, BF16>& sm, PagedWalk<NR> w, int lane) {
  using C = Cfg<D, NR, BF16>;
  const PagedParams& p = P.c;
  constexpr int kVec = D / 8, kPer = 32 / kVec;  // rows an instruction
  constexpr int kLoads = NR / kPer > 0 ? NR / kPer : 1;
  constexpr uint32_t kInf = BF16 ? 0x7f80u : 0x7c00u;  // magnitudes from here on are not finite
  const int c = lane % kVec, sub = lane / kVec;
  ScaleFeed<C::kSK> feed;
  for (; !w.done(); w.next(p)) {
    const int buf = w.index & 1;
    if (w.index >= 2 && !wait_warp(sm.q_empty(buf), ((w.index >> 1) - 1) & 1, p.timeout_ns, p.status)) return;
    const PagedUnit& u = w.u;
    const uint16_t* q = static_cast<const uint16_t*>(p.q) + (int64_t)u.q.s0 * p.q_stride + u.kvh * p.group * D + c * 8;
    const int tok0 = paged_token(p, u.row0 + sub);
    int tok = tok0, head = u.row0 + sub - tok0 * p.group;
    auto load = [&](int i) {  // rows i * kPer ..; called in order
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (i * kPer + sub < u.rows) v = __ldg(reinterpret_cast<const uint4*>(q + (int64_t)tok * p.q_stride + head * D));
      for (head += kPer; head >= p.group; head -= p.group) ++tok;
      return v;
    };
    uint8_t* dst = sm.q_ptr(buf) + (c & 1) * 8;
    uint4 next = load(0);
#pragma unroll 4
    for (int i = 0; i < kLoads; ++i) {
      const int r = i * kPer + sub;
      const uint32_t e[4] = {next.x, next.y, next.z, next.w};
      next = load(i + 1);
      const uint32_t top2 = __vmaxu2(__vmaxu2(e[0] & 0x7fff7fffu, e[1] & 0x7fff7fffu),
                                     __vmaxu2(e[2] & 0x7fff7fffu, e[3] & 0x7fff7fffu));
      uint32_t top = max(top2 & 0xffffu, top2 >> 16);
#pragma unroll
      for (int o = 1; o < kVec; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      const bool odd = top >= kInf;  // the row holds an infinity or NaN: its scores become NaN
      // the power of two that brings the row's largest element into [128, 256)
      int ex;
      if constexpr (BF16) ex = (int)(top >> 7) - 127;
      else ex = (int)(__float_as_uint(__half2float(__ushort_as_half((unsigned short)top))) >> 23) - 127;
      ex = top == 0u || odd ? 0 : min(max(7 - ex, -120), 120);
      const float mul = __uint_as_float((uint32_t)(ex + 127) << 23);
      if (c == 0 && r < NR) sm.qs(buf)[r] = __uint_as_float((uint32_t)(127 - ex) << 23);
      uint32_t h[4];  // scaled, f16 pairs
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float x, y;
        if constexpr (BF16) {
          x = __uint_as_float(e[k] << 16);
          y = __uint_as_float(e[k] & 0xffff0000u);
        } else {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&e[k]));
          x = f.x;
          y = f.y;
        }
        f2_split(fmul2(f2(x, y), f2(mul, mul)), x, y);
        const __half2 hh = __floats2half2_rn(x, y);
        h[k] = *reinterpret_cast<const uint32_t*>(&hh);
      }
#pragma unroll
      for (int j = 0; j < C::kQP; ++j) {
        uint32_t w2[2];
#pragma unroll
        for (int k = 0; k < 2; ++k)
          w2[k] = j + 1 < C::kQP ? piece4(h[2 * k], h[2 * k + 1]) : last4(h[2 * k], h[2 * k + 1]);
        if (odd) w2[0] = w2[1] = j == 0 ? 0x7f7f7f7fu : 0u;
        // 8 bytes of chunk c / 2 of row n, the chunk's index XORed as the swizzle does
        const int n = j * NR + r;
        const int at = D == 128 ? ((c >> 1) ^ (n & 7)) : ((c >> 1) ^ ((n >> 1) & 3));
        if (NR >= kPer || r < NR) *reinterpret_cast<uint2*>(dst + n * D + at * 16) = make_uint2(w2[0], w2[1]);
      }
    }
    for (int r = lane; r < NR; r += 32)
      sm.lim(buf)[r] = r < u.rows ? paged_limits(p, u.q, paged_token(p, u.row0 + r)) : make_int2(0, 0);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(sm.q_full(buf));
    if (!feed.unit(p, w, 1.0f, sm.scales(0), sm.k_full(0), sm.sc_empty(0), lane)) return;
  }
}

// ---------------------------------------------------------------- MMA issuer
// Tile i of the CTA's line: S^T(i) into buffer i % 2, then O^T += V^T P^T of
// tile i - 1.  That buffer is free: P(i - 2), written after S(i - 2) was read,
// was waited for in the step before.
template <int D, int NR, bool BF16>
__device__ __forceinline__ void mma_role(const DecParams& P, const Lay<D, NR, BF16>& sm, PagedWalk<NR> w, uint32_t tmem,
                                         int lane) {
  using C = Cfg<D, NR, BF16>;
  const PagedParams& p = P.c;
  constexpr uint32_t kIdS = idesc_e4m3(128, C::kNQ, false, false);
  constexpr uint32_t kIdO = idesc_e4m3(128, C::kNP, true, true);
  constexpr uint32_t kSwizzle = D == 128 ? 2 : 4;
  constexpr uint32_t kGroup8 = 8 * D;  // bytes of 8 rows
  int g = 0;
  bool pending = false;   // a tile whose P V is still to be issued
  bool pend_first = false;
  int pend_valid = kPagedKeys;  // valid keys from its first one on
  bool ok = true;
  auto pv = [&](int t) -> bool {
    if (!wait_warp(sm.p_full(t & 1), (t >> 1) & 1, p.timeout_ns, p.status)) return false;
    const int vs = t % C::kSV;
    if (!wait_warp(sm.v_full(vs), (t / C::kSV) & 1, p.timeout_ns, p.status)) return false;
    if (pend_valid < kPagedKeys) {
      // slots past the request's last key may hold NaN bytes: P is 0 there but 0 * NaN is not
      for (int c = max(pend_valid, 0) * (D / 16) + lane; c < kPagedKeys * (D / 16); c += 32)
        *reinterpret_cast<uint4*>(sm.v_ptr(vs) + c * 16) = make_uint4(0u, 0u, 0u, 0u);  // whole rows: the swizzle does not matter
      fence_proxy_async_smem();
      __syncwarp();
    }
    tc_fence_after();
    // A = V^T: M-major, one swizzle atom of 128 (64: repeated, LBO 0) d's by 8 keys, SBO apart
    const uint64_t a0 = sdesc(sm.v_tile(vs), 0, kGroup8, kSwizzle);
    // B = P^T: N-major without swizzle, 16 rows of N by 8 keys in 128 bytes; LBO to the next 8 keys, SBO to the next 16 rows
    const uint64_t b0 = sdesc(sm.p(t & 1), 128, 16 * kPagedKeys, 0);
#pragma unroll
    for (int k = 0; k < kPagedKeys / 32; ++k)
      mma8_elect(tmem + C::kColO, a0 + (uint32_t)((k * 4 * kGroup8) >> 4), b0 + (uint32_t)((k * 512) >> 4), kIdO,
                 (!pend_first || k > 0) ? 1u : 0u);
    tc_commit_elect(sm.pv_done(t & 1));
    tc_commit_elect(sm.v_empty(vs));
    return true;
  };
  for (; ok && !w.done(); w.next(p)) {
    const int buf = w.index & 1;
    if (pending) {  // a unit's last P V does not wait for the next one's Q
      if (!pv(g - 1)) { ok = false; break; }
      pending = false;
    }
    if (!wait_warp(sm.q_full(buf), (w.index >> 1) & 1, p.timeout_ns, p.status)) { ok = false; break; }
    const int valid = paged_valid(p, w.u.q);
    for (int n = 0; ok && n < w.nt; ++n, ++g) {
      const int ks = g % C::kSK;
      if (!wait_warp(sm.k_full(ks), (g / C::kSK) & 1, p.timeout_ns, p.status)) { ok = false; break; }
      tc_fence_after();
      const uint64_t a0 = sdesc(sm.k_tile(ks), 16, kGroup8, kSwizzle);
      const uint64_t b0 = sdesc(sm.q(buf), 16, kGroup8, kSwizzle);
#pragma unroll
      for (int k = 0; k < D / 32; ++k)
        mma8_elect(tmem + (g & 1) * C::kNQ, a0 + (uint32_t)(k * 2), b0 + (uint32_t)(k * 2), kIdS, k > 0 ? 1u : 0u);
      tc_commit_elect(sm.s_full(g & 1));
      tc_commit_elect(sm.k_empty(ks));
      if (pending && !pv(g - 1)) { ok = false; break; }
      pending = true;
      pend_first = n == 0;
      pend_valid = valid - (w.t0 + n) * kPagedKeys;
    }
    // Q and the limits are free once this unit's S^T products are done and its rows' softmax has read
    // them: the softmax arrives for itself
    if (ok) tc_commit_elect(sm.q_empty(buf));
  }
  if (ok && pending) pv(g - 1);
  // every MMA done before tensor memory is given back
  tc_commit_elect(sm.drain());
  wait_warp(sm.drain(), 0, p.timeout_ns, p.status);
}

// ------------------------------------------------------------------ softmax
// Thread tid of warps 0-3 owns key tid of every tile (lane tid of S^T) and, at
// a unit's end, d = tid of O^T.
template <int D, int NR, bool BF16, bool SOFTCAP>
__device__ __forceinline__ void softmax_role(const DecParams& P, const Lay<D, NR, BF16>& sm, PagedWalk<NR> w,
                                             uint32_t tmem, int warp, int lane) {
  using C = Cfg<D, NR, BF16>;
  const PagedParams& p = P.c;
  const int tid = warp * 32 + lane;
  const uint32_t tq = tmem + ((uint32_t)(warp * 32) << 16);
  int g = 0;  // tiles so far
  // The four warps meet at a hardware barrier, so none of them may leave early: one whose bounded
  // wait has run out goes on without waiting (the status word has the timeout; the rows are not valid).
  bool dead = false;
  auto wait = [&](uint32_t bar, uint32_t parity) {
    if (!dead) dead = !wait_warp(bar, parity, p.timeout_ns, p.status);
  };
  auto meet = [] { asm volatile("barrier.cta.sync 1, 128;" ::: "memory"); };
  auto meet_any = [](bool x) {  // ... and learn whether x holds for some thread
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %1, 0;\n\tbarrier.cta.red.or.pred p, 1, 128, q;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r) : "r"((uint32_t)x) : "memory");
    return r != 0;
  };
  for (; !w.done(); w.next(p)) {
    const PagedUnit& u = w.u;
    const int buf = w.index & 1;
    wait(sm.q_full(buf), (w.index >> 1) & 1);
    const int2* lim = sm.lim(buf);
    const uint64_t* qs2 = reinterpret_cast<const uint64_t*>(sm.qs(buf));  // two rows each
    const int full_lo = lim[u.rows - 1].x, full_hi = lim[0].y;  // keys every row sees
    // rows two by two (packed fp32): row sums, and the running maxima less kPLog2, the same in every thread
    uint64_t l2[NR / 2], m2[NR / 2];
#pragma unroll
    for (int r = 0; r < NR / 2; ++r) {
      l2[r] = 0ull;
      m2[r] = f2(kNone, kNone);
    }
    if (w.nt == 0) meet();  // a unit without a tile has no other meeting before its sums

    for (int n = 0; n < w.nt; ++n, ++g) {
      const int key0 = (w.t0 + n) * kPagedKeys, j = key0 + tid;
      wait(sm.s_full(g & 1), (g >> 1) & 1);
      tc_fence_after();
      // the scales of this thread's key lie there once S^T does: K's barrier takes the scale warp's arrival too
      const float4 scl = sm.scales(g % C::kSK)[tid >> 4];
      const float lv = scl.y;
      // scores in log2 units plus log2 v_scale, then less the maxima: t - m + 5
      float t[NR];
      {
        float x1[NR], x2[C::kQP > 2 ? NR : 1];
        const uint32_t a = tq + (uint32_t)((g & 1) * C::kNQ);
        tld(a, t);
        tld(a + NR, x1);
        if constexpr (C::kQP > 2) tld(a + 2 * NR, x2);
        tmem_wait_ld();
        const uint64_t step = f2(kInvStep, kInvStep);
        float km = P.scale_log2 * scl.x;
        if constexpr (SOFTCAP) km = fminf(fmaxf(P.k1 * scl.x, -3e38f), 3e38f);  // times a score of 0 is 0
        const uint64_t km2 = f2(km, km), lv2 = f2(lv, lv);
#pragma unroll
        for (int r = 0; r < NR; r += 2) {
          uint64_t s = f2(x1[r], x1[r + 1]);
          if constexpr (C::kQP > 2) s = ffma2(f2(x2[r], x2[r + 1]), step, s);
          s = ffma2(s, step, f2(t[r], t[r + 1]));
          s = fmul2(s, qs2[r / 2]);
          if constexpr (SOFTCAP) {
            float a0, a1;
            f2_split(fmul2(s, km2), a0, a1);
            if (P.k2 != 0.0f) {
              t[r] = fmaf(P.k2, fast_rcp(fast_exp2(a0) + 1.0f), P.k3 + lv);
              t[r + 1] = fmaf(P.k2, fast_rcp(fast_exp2(a1) + 1.0f), P.k3 + lv);
            } else {
              t[r] = fmaf(P.k3, fast_tanh(a0), lv);
              t[r + 1] = fmaf(P.k3, fast_tanh(a1), lv);
            }
          } else {
            f2_split(ffma2(s, km2, lv2), t[r], t[r + 1]);
          }
        }
      }
      if (key0 < full_lo || key0 + kPagedKeys > full_hi) {
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          const int2 e = lim[r];
          t[r] = (j >= e.x && j < e.y) ? t[r] : -INFINITY;
        }
      }
      // does any key pass its row's maximum by more than kRise?
      float over = -INFINITY;
#pragma unroll
      for (int r = 0; r < NR; r += 2) {
        float a, b;
        f2_split(fsub2(f2(t[r], t[r + 1]), m2[r / 2]), a, b);
        over = fmax3(over, a, b);
      }
      if (n == 0 || meet_any(over > kRise + kPLog2)) {
        float x[NR];
#pragma unroll
        for (int r = 0; r < NR; ++r) x[r] = t[r];
        const float wm = reduce_scatter<NR, true>(x, lane);
        float* red = sm.red(0);
        if ((lane & (32 / NR - 1)) == 0) red[warp * NR + row_of_lane<NR>(lane)] = wm;
        meet();
        float* alpha = x;
#pragma unroll
        for (int r = 0; r < NR; r += 2) {
          float old[2];
          f2_split(m2[r / 2], old[0], old[1]);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float top = fmaxf(fmaxf(red[r + i], red[NR + r + i]), fmaxf(red[2 * NR + r + i], red[3 * NR + r + i])) - kPLog2;
            const float mn = top > old[i] + kRise ? top : old[i];
            alpha[r + i] = fast_exp2(0.5f * (old[i] - mn));
            old[i] = mn;
          }
          m2[r / 2] = f2(old[0], old[1]);
          // in two steps: the sum of earlier keys may be as large as the factor is small, where V scales differ
          const uint64_t half = f2(alpha[r], alpha[r + 1]);
          l2[r / 2] = fmul2(fmul2(l2[r / 2], half), half);
          alpha[r] *= alpha[r];
          alpha[r + 1] *= alpha[r + 1];
        }
        if (n > 0) {  // O^T holds the unit's earlier tiles once their P V is done
          wait(sm.pv_done((g - 1) & 1), ((g - 1) >> 1) & 1);
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < C::kNP; c += 16) {
            float o[16];
            tld(tq + (uint32_t)(C::kColO + c), o);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] *= alpha[(c + i) % NR];
            tst16(tq + (uint32_t)(C::kColO + c), o);
          }
          tmem_wait_st();
          tc_fence_before();
        }
      }
      // P buffer g % 2 was last read by the P V of tile g - 2, issued before S^T(g): S^T(g) ready says it is done
      // weights, rounded to f16 (11 bits) and carried on as three e4m3 pieces
      uint32_t words[C::kNP / 4];
#pragma unroll
      for (int i = 0; i < C::kNP / 4; ++i) words[i] = 0u;
      const float iv = scl.z;
      if (__builtin_expect(iv == 0.0f, 0)) {  // a far tile
        const float rest = scl.w - lv;  // not 0 for scales below 2^-100 only
#pragma unroll
        for (int r = 0; r < NR; r += 2) {
          float a, b;
          f2_split(fsub2(f2(t[r], t[r + 1]), m2[r / 2]), a, b);
          l2[r / 2] = ffma2(f2(fast_exp2(a - lv), fast_exp2(b - lv)), f2(kPagedSumFactor, kPagedSumFactor), l2[r / 2]);
          t[r] += rest;
          t[r + 1] += rest;
        }
      }
      const uint64_t iv2 = f2(iv, iv);
#pragma unroll
      for (int r = 0; r < NR; r += 4) {
        uint32_t h[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float a, b;
          f2_split(fsub2(f2(t[r + 2 * i], t[r + 2 * i + 1]), m2[r / 2 + i]), a, b);
          a = fast_exp2(a);
          b = fast_exp2(b);
          l2[r / 2 + i] = ffma2(f2(a, b), iv2, l2[r / 2 + i]);
          const __half2 hh = __floats2half2_rn(a, b);
          h[i] = *reinterpret_cast<const uint32_t*>(&hh);
        }
        words[r / 4] = piece4(h[0], h[1]);
        words[(NR + r) / 4] = piece4(h[0], h[1]);
        words[(2 * NR + r) / 4] = last4(h[0], h[1]);
      }
      uint8_t* pb = sm.p_ptr(g & 1) + tid * 16;
#pragma unroll
      for (int c = 0; c < C::kNP / 16; ++c)
        *reinterpret_cast<uint4*>(pb + c * 16 * kPagedKeys) =
            make_uint4(words[4 * c], words[4 * c + 1], words[4 * c + 2], words[4 * c + 3]);
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(sm.p_full(g & 1));
        mbar_arrive(sm.sc_empty(g % C::kSK));
      }
    }

    // ---- the segment's rows: sums over the threads, O^T, and out (or a partial row)
    float x[NR], m[NR];
#pragma unroll
    for (int r = 0; r < NR; r += 2) {
      f2_split(l2[r / 2], x[r], x[r + 1]);
      f2_split(m2[r / 2], m[r], m[r + 1]);
    }
    const float ws = reduce_scatter<NR, false>(x, lane);
    float* red = sm.red(1);  // not the maxima's, which a slower warp may still read
    if ((lane & (32 / NR - 1)) == 0) red[warp * NR + row_of_lane<NR>(lane)] = ws;
    meet();
    float o[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) o[r] = 0.0f;
    if (w.nt > 0) {
      wait(sm.pv_done((g - 1) & 1), ((g - 1) >> 1) & 1);
      tc_fence_after();
      float o1[NR], o2[NR];
      tld(tq + (uint32_t)C::kColO, o);
      tld(tq + (uint32_t)(C::kColO + NR), o1);
      tld(tq + (uint32_t)(C::kColO + 2 * NR), o2);
      tmem_wait_ld();
      tc_fence_before();
#pragma unroll
      for (int r = 0; r < NR; ++r) o[r] = fmaf(fmaf(o2[r], kInvStep, o1[r]), kInvStep, o[r]);
    }
    const int slot = 2 * blockIdx.x + (w.head ? 1 : 0);
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      if (r >= u.rows) break;
      const float L = red[r] + red[NR + r] + red[2 * NR + r] + red[3 * NR + r];
      if (w.whole) {
        const int xr = u.row0 + r;
        const int tok = paged_token(p, xr);
        const int64_t row = (int64_t)(u.q.s0 + tok) * p.Hq + u.kvh * p.group + xr - tok * p.group;
        const float inv = L == 0.0f ? 0.0f : kPagedSumFactor * (1.0f / L);
        if (tid < D) static_cast<uint16_t*>(p.out)[row * D + tid] = to_bits<BF16>(o[r] * inv);
        if (p.lse != nullptr && tid == r)
          p.lse[row] = L == 0.0f ? -INFINITY : (m[r] + (__log2f(L) + kPagedSumLog2)) * kLn2;
      } else {
        if (tid < D) P.ws_o[((int64_t)slot * NR + r) * D + tid] = o[r];
        if (tid == r) P.ws_ml[slot * NR + r] = make_float2(m[r], L);
      }
    }
    if (!w.whole && w.head && tid == 0) {
      PagedCut c;
      c.parts = paged_parts(w, sm.share());
      c.token0 = u.q.s0;
      c.head0 = u.kvh * p.group;
      c.row0 = u.row0;
      c.rows = u.rows;
      P.cuts[blockIdx.x] = c;
    }
    // the limits and the Q scale may be replaced once every warp is here
    __syncwarp();
    if (lane == 0) mbar_arrive(sm.q_empty(buf));
  }
}

template <int D, int NR, bool BF16, bool SOFTCAP>
__global__ void __launch_bounds__(kThreads, kPagedDecCtas)
    attn_paged_dec_kernel(const __grid_constant__ DecParams P) {
  using C = Cfg<D, NR, BF16>;
  const PagedParams& p = P.c;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Lay<D, NR, BF16> sm;
  sm.base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  sm.s = smem_u32(sm.base);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kSK; ++i) {
      mbar_init(sm.k_full(i), 2);  // the TMA's, and the scale warp's
      mbar_init(sm.k_empty(i), 1);
      mbar_init(sm.sc_empty(i), 4);
    }
    for (int i = 0; i < C::kSV; ++i) {
      mbar_init(sm.v_full(i), 1);
      mbar_init(sm.v_empty(i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(sm.s_full(i), 1);
      mbar_init(sm.p_full(i), 4);
      mbar_init(sm.pv_done(i), 1);
      mbar_init(sm.q_full(i), 1);
      mbar_init(sm.q_empty(i), 5);  // four softmax warps and the MMA warp's commit
    }
    mbar_init(sm.drain(), 1);
    mbar_init_fence();
    P.cuts[blockIdx.x].parts = 0;
  }
  if constexpr (C::kQP * NR < C::kNQ) {  // rows of N that no piece fills
    for (int i = threadIdx.x; i < 2 * C::kQBytes / 16; i += kThreads)
      *reinterpret_cast<uint4*>(sm.q_ptr(0) + i * 16) = make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async_smem();
  }
  if (warp == kKWarp && lane == 0) tma_prefetch_desc(&P.tmap_k);
  if (warp == kVWarp && lane == 0) tma_prefetch_desc(&P.tmap_v);
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(sm.slot()), C::kTmem);
    tmem_relinquish();
  }
  paged_share<NR, kThreads>(p, sm.share());
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // The joining kernel may be scheduled; it waits.  Where no join follows this may let in any kernel, one with tensor memory
  // of its own among them, so this CTA has its columns by now.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(sm.slot());
  PagedWalk<NR> w;
  w.begin(p, sm.share());
  if (warp < 4) {
    softmax_role<D, NR, BF16, SOFTCAP>(P, sm, w, tmem, warp, lane);
  } else if (warp == kKWarp) {
    load_role<D, NR, C::kSK>(P, &P.tmap_k, w, sm.k_tile(0), sm.k_full(0), sm.k_empty(0), lane, true);
  } else if (warp == kVWarp) {
    load_role<D, NR, C::kSV>(P, &P.tmap_v, w, sm.v_tile(0), sm.v_full(0), sm.v_empty(0), lane, false);
  } else if (warp == kMmaWarp) {
    mma_role<D, NR, BF16>(P, sm, w, tmem, lane);
  } else {
    q_role<D, NR, BF16>(P, sm, w, lane);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmem);
  }
}


template <int D, int NR, bool BF16, bool SOFTCAP>
cudaError_t launch_dec(const DecParams& P, int grid, cudaStream_t stream) {
  auto kernel = attn_paged_dec_kernel<D, NR, BF16, SOFTCAP>;
  constexpr int smem = Cfg<D, NR, BF16>::kSmem;
  static std::atomic<bool> ready[128];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 128 || !ready[dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 128) ready[dev].store(true, std::memory_order_relaxed);
  }
  kernel<<<grid, kThreads, smem, stream>>>(P);
  return cudaGetLastError();
}

template <int D, int NR>
cudaError_t launch_dec_d(const DecParams& P, bool bf16, int grid, cudaStream_t stream) {
  if (P.c.softcap > 0.0f)
    return bf16 ? launch_dec<D, NR, true, true>(P, grid, stream) : launch_dec<D, NR, false, true>(P, grid, stream);
  return bf16 ? launch_dec<D, NR, true, false>(P, grid, stream) : launch_dec<D, NR, false, false>(P, grid, stream);
}

template <int NR>
cudaError_t launch_dec_nr(const DecParams& P, bool bf16, int grid, cudaStream_t stream) {
  return P.c.D == 128 ? launch_dec_d<128, NR>(P, bf16, grid, stream) : launch_dec_d<64, NR>(P, bf16, grid, stream);
}

}  // namespace

cudaError_t launch_attn_paged_dec(const PagedLaunch& L, bool bf16, cudaStream_t stream) {
  DecParams P{};
  P.tmap_k = L.tmap_k;
  P.tmap_v = L.tmap_v;
  P.c = L.c;
  P.ws_o = L.ws_o;
  P.ws_ml = L.ws_ml;
  P.cuts = L.cuts;
  const double l2e = 1.4426950408889634;
  P.scale_log2 = (float)((double)L.c.scale * l2e);
  if (L.c.softcap > 0.0f) {
    // The quotient's error is 2^-21 of the cap, as it is the difference of two numbers of the cap's size; the hardware
    // tanh's is 2^-16 of the score.  Caps in use, 20 to 50, are better off with the first, large ones with the second.
    const bool quotient = L.c.softcap <= 512.0f;
    P.k1 = (float)std::max(-3e38, std::min(3e38, (quotient ? 2.0 * l2e : 1.0) * (double)L.c.scale / (double)L.c.softcap));
    P.k2 = quotient ? (float)(-2.0 * (double)L.c.softcap * l2e) : 0.0f;
    P.k3 = (float)((double)L.c.softcap * l2e);
  }
  switch (L.rows) {
    case 4: return launch_dec_nr<4>(P, bf16, L.grid, stream);
    case 8: return launch_dec_nr<8>(P, bf16, L.grid, stream);
    case 16: return launch_dec_nr<16>(P, bf16, L.grid, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace gb300_attn
