// paged4_api.cu -- the C ABI of the paged 4-bit KV cache and of the rotary
// positions (attn_cache_append_fp4, attn_cache_read_fp4, attn_fwd_paged_fp4,
// attn_rope in include/attn.h): argument validation, then the launches.  A
// request the kernels cannot run is refused with a status before anything is
// launched.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>

#include "../../include/attn.h"
#include "api_internal.h"
#include "paged4_internal.h"

using namespace gb300_attn;

namespace {

int block_shift(int bs) { return bs == 16 ? 4 : bs == 32 ? 5 : bs == 64 ? 6 : bs == 128 ? 7 : -1; }

// Pieces of `width` bytes: `inner` of them `inner_stride` apart, that `n` times, `stride` apart.  Neither strides nor pieces
// overlap within a set.
struct Rows {
  const void* p;
  int64_t n, width, stride, inner = 1, inner_stride = 0;
};

int64_t span(const Rows& r) {
  return r.n <= 0 || r.width <= 0 ? 0 : (r.n - 1) * r.stride + (r.inner - 1) * r.inner_stride + r.width;
}

// Whether two sets of pieces share a byte.  Sets of the same strides may lie between each other (slices of a fused
// projection, K and V of a head side by side); others may not even have spans in common.
bool share(const Rows& a, const Rows& b) {
  if (!overlaps(a.p, span(a), b.p, span(b))) return false;
  const bool once = a.n <= 1 && b.n <= 1;
  if ((!once && (a.stride != b.stride || a.stride <= 0)) || a.inner != b.inner || a.inner_stride != b.inner_stride) return true;
  int64_t d = (int64_t)(reinterpret_cast<uintptr_t>(b.p) - reinterpret_cast<uintptr_t>(a.p));
  if (!once && (d %= a.stride) < 0) d += a.stride;
  // pieces of b lie d + j inner_stride from pieces of a, |j| < inner, and that a stride lower
  for (int low = 0; low < (once ? 1 : 2); ++low) {
    const int64_t x = d - (low ? a.stride : 0);
    const int64_t near = a.inner > 1 ? -x / a.inner_stride : 0;
    for (int64_t j = std::max(near - 1, 1 - a.inner); j <= std::min(near + 1, a.inner - 1); ++j) {
      const int64_t at = x + j * a.inner_stride;
      if (at > -b.width && at < a.width) return true;
    }
  }
  return false;
}

// One-level sets that are the same rows (of a single one the stride says nothing).
bool same(const Rows& a, const Rows& b) {
  return a.p == b.p && a.n == b.n && a.width == b.width && (a.n <= 1 || a.stride == b.stride);
}

Rows flat(const void* p, int64_t bytes) { return Rows{p, p && bytes > 0 ? 1 : 0, bytes, bytes}; }

template <int NW, int NR>
bool clash(const Rows (&w)[NW], const Rows (&r)[NR]) {
  for (int i = 0; i < NW; ++i) {
    for (int j = i + 1; j < NW; ++j)
      if (share(w[i], w[j])) return true;
    for (int j = 0; j < NR; ++j)
      if (share(w[i], r[j])) return true;
  }
  return false;
}

// Bytes of the cache (one of K, V): its codes, half of D a row; false where they pass 2^60.
bool cache_bytes(int num_blocks, int Hkv, int block_size, int D, int64_t* codes) {
  int64_t tiles, t;
  return mul_ok(num_blocks, Hkv, &tiles) && tiles <= INT32_MAX && mul_ok(tiles, (int64_t)block_size * D, &t) &&
         t <= (INT64_C(1) << 60) && (*codes = t / 2, true);
}

bool dtype_ok(int dtype) { return dtype == ATTN_F32 || dtype == ATTN_F16 || dtype == ATTN_BF16; }

// Whether `n` rows of `width` values, `stride` apart, are ones (n > 0) whose span fits 2^60 bytes.
bool stride_ok(int64_t n, int64_t stride, int64_t width) {
  int64_t t;
  return n <= 0 || (stride >= width && mul_ok(n, stride, &t) && t <= (INT64_C(1) << 57));
}

// What append and read have in common: 0 where there is nothing to do, -1 where p is ready, else a status.
int cache4_check(Cache4Params& p, void* k, void* v, const int64_t* slot_map, void* k_cache, void* v_cache, void* k_scales,
                 void* v_scales, const float* k_heads, const float* v_heads, int T, int Hkv, int D, const int64_t (&ts)[2],
                 const int64_t (&hs)[2], int num_blocks, int block_size, int dtype, bool read) {
  if (!dtype_ok(dtype)) return ATTN_ERR_INVALID_ARG;
  if (T < 0 || Hkv <= 0 || D <= 0 || num_blocks < 0 || block_size <= 0) return ATTN_ERR_INVALID_ARG;
  const int64_t esize = dtype == ATTN_F32 ? 4 : 2;
  int64_t codes, row;
  if (!cache_bytes(num_blocks, Hkv, block_size, D, &codes)) return ATTN_ERR_INVALID_ARG;
  Rows x[2];
  for (int i = 0; i < 2; ++i) {
    // rows of a token's heads one after the other, or of a head's tokens
    const bool tokens_out = Hkv == 1 || ts[i] >= hs[i];
    const int64_t inner = tokens_out ? hs[i] : ts[i], outer = tokens_out ? ts[i] : hs[i];
    const int64_t n_in = tokens_out ? Hkv : T, n_out = tokens_out ? T : Hkv;
    if (!mul_ok(std::max<int64_t>(n_in, 1) - 1, inner, &row) || row > (INT64_C(1) << 57)) return ATTN_ERR_INVALID_ARG;
    row += D;
    if (T > 0 && (!stride_ok(n_in > 1 ? n_in : 0, inner, D) || !stride_ok(n_out > 1 ? n_out : 0, outer, row)))
      return ATTN_ERR_INVALID_ARG;
    x[i] = n_in > 1 ? Rows{i ? v : k, n_out, D * esize, outer * esize, n_in, inner * esize}
                    : Rows{i ? v : k, n_out, D * esize, outer * esize};
  }
  if (T == 0) return 0;
  if (!k || !v || !slot_map) return ATTN_ERR_INVALID_ARG;
  if (num_blocks == 0 && !read) return 0;  // nowhere to write
  if (num_blocks > 0 && (!k_cache || !v_cache || !k_scales || !v_scales)) return ATTN_ERR_INVALID_ARG;
  const Rows c[] = {flat(k_cache, codes), flat(v_cache, codes), flat(k_scales, codes / 8), flat(v_scales, codes / 8)};
  const Rows heads[] = {flat(k_heads, (int64_t)Hkv * 4), flat(v_heads, (int64_t)Hkv * 4)};
  const Rows map = flat(slot_map, (int64_t)T * 8);
  if (read) {
    const Rows r[] = {c[0], c[1], c[2], c[3], heads[0], heads[1], map};
    if (clash(x, r)) return ATTN_ERR_INVALID_ARG;
  } else {
    const Rows r[] = {x[0], x[1], heads[0], heads[1], map};
    if (clash(c, r)) return ATTN_ERR_INVALID_ARG;
  }
  if (block_shift(block_size) < 0 || (D != 64 && D != 128)) return ATTN_ERR_UNSUPPORTED;
  for (int i = 0; i < 2; ++i)
    if (!aligned(x[i].p, 16) || (T > 1 && (ts[i] * esize) % 16 != 0) || (Hkv > 1 && (hs[i] * esize) % 16 != 0))
      return ATTN_ERR_UNSUPPORTED;
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(k_scales, 16) || !aligned(v_scales, 16) ||
      !aligned(k_heads, 4) || !aligned(v_heads, 4) || !aligned(slot_map, 8))
    return ATTN_ERR_UNSUPPORTED;
  p.x[0] = k; p.x[1] = v;
  for (int i = 0; i < 2; ++i) {
    p.stride[i] = ts[i];
    p.head_stride[i] = hs[i];
  }
  p.slot_map = slot_map;
  p.cache[0] = static_cast<uint8_t*>(k_cache); p.cache[1] = static_cast<uint8_t*>(v_cache);
  p.scales[0] = static_cast<uint8_t*>(k_scales); p.scales[1] = static_cast<uint8_t*>(v_scales);
  p.heads[0] = k_heads; p.heads[1] = v_heads;
  p.num_slots = (int64_t)num_blocks * block_size;
  p.T = T; p.Hkv = Hkv; p.D = D; p.block_size = block_size;
  p.block_shift = block_shift(block_size);
  return -1;
}

}  // namespace

extern "C" int attn_cache_append_fp4(const void* k, const void* v, const int64_t* slot_map, void* k_cache, void* v_cache,
                                     void* k_scales, void* v_scales, const float* k_head_scales,
                                     const float* v_head_scales, int num_tokens, int Hkv, int D, int64_t k_token_stride,
                                     int64_t v_token_stride, int num_blocks, int block_size, int dtype, void* stream) {
  Cache4Params p{};
  const int64_t ts[2] = {k_token_stride, v_token_stride}, hs[2] = {D, D};
  // a token's heads lie together: strides below their width are no rows of tokens
  if (num_tokens > 0 && Hkv > 0 && D > 0 && std::min(ts[0], ts[1]) < (int64_t)Hkv * D) return ATTN_ERR_INVALID_ARG;
  const int rc = cache4_check(p, const_cast<void*>(k), const_cast<void*>(v), slot_map, k_cache, v_cache, k_scales, v_scales,
                              k_head_scales, v_head_scales, num_tokens, Hkv, D, ts, hs, num_blocks, block_size, dtype, false);
  if (rc >= 0) return rc;
  const cudaError_t e = launch_cache4_append(p, dtype, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ATTN_OK : cuda_fail(e);
}

extern "C" int attn_cache_read_fp4(const void* k_cache, const void* v_cache, const void* k_scales, const void* v_scales,
                                   const float* k_head_scales, const float* v_head_scales, const int64_t* slot_map, void* k,
                                   void* v, int num_tokens, int Hkv, int D, int64_t k_token_stride, int64_t k_head_stride,
                                   int64_t v_token_stride, int64_t v_head_stride, int num_blocks, int block_size, int dtype,
                                   void* stream) {
  Cache4Params p{};
  const int64_t ts[2] = {k_token_stride, v_token_stride}, hs[2] = {k_head_stride, v_head_stride};
  const int rc = cache4_check(p, k, v, slot_map, const_cast<void*>(k_cache), const_cast<void*>(v_cache),
                              const_cast<void*>(k_scales), const_cast<void*>(v_scales), k_head_scales, v_head_scales,
                              num_tokens, Hkv, D, ts, hs, num_blocks, block_size, dtype, true);
  if (rc >= 0) return rc;
  const cudaError_t e = launch_cache4_read(p, dtype, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ATTN_OK : cuda_fail(e);
}

extern "C" int attn_rope(const void* q, const void* k, void* q_out, void* k_out, const double* inv_freq,
                         const int32_t* positions, const int32_t* q_starts, const int32_t* total_lengths, int num_tokens,
                         int B, int Hq, int Hk, int D, int rotary_dim, int64_t q_token_stride, int64_t k_token_stride,
                         int64_t q_out_token_stride, int64_t k_out_token_stride, int interleaved, int inverse, float scale,
                         int dtype, void* stream) {
  if (!dtype_ok(dtype)) return ATTN_ERR_INVALID_ARG;
  if (num_tokens < 0 || B < 0 || Hq <= 0 || Hk < 0 || D <= 0) return ATTN_ERR_INVALID_ARG;
  if (rotary_dim < 0 || rotary_dim > D || rotary_dim % 2 != 0) return ATTN_ERR_INVALID_ARG;
  if ((interleaved != 0 && interleaved != 1) || (inverse != 0 && inverse != 1) || !std::isfinite(scale)) return ATTN_ERR_INVALID_ARG;
  const int64_t T = num_tokens, esize = dtype == ATTN_F32 ? 4 : 2;
  const int64_t wq = (int64_t)Hq * D, wk = (int64_t)Hk * D;
  if (!stride_ok(T, q_token_stride, wq) || !stride_ok(T, q_out_token_stride, wq)) return ATTN_ERR_INVALID_ARG;
  if (Hk > 0 && (!stride_ok(T, k_token_stride, wk) || !stride_ok(T, k_out_token_stride, wk))) return ATTN_ERR_INVALID_ARG;
  // positions as they are, or those of the requests' newest tokens
  if (positions ? q_starts || total_lengths : B > 0 && T > 0 && (!q_starts || !total_lengths)) return ATTN_ERR_INVALID_ARG;
  if (T == 0 || (!positions && B == 0)) return ATTN_OK;  // no row, or none that belongs to a request
  if (!q || !q_out || (Hk > 0 && (!k || !k_out)) || (rotary_dim > 0 && !inv_freq)) return ATTN_ERR_INVALID_ARG;
  const Rows in[2] = {{q, T, wq * esize, q_token_stride * esize}, {k, Hk > 0 ? T : 0, wk * esize, k_token_stride * esize}};
  const Rows out[2] = {{q_out, T, wq * esize, q_out_token_stride * esize},
                       {k_out, Hk > 0 ? T : 0, wk * esize, k_out_token_stride * esize}};
  const Rows rest[] = {flat(inv_freq, (int64_t)rotary_dim * 4), flat(positions, T * 4), flat(q_starts, (int64_t)B * 4 + 4),
                       flat(total_lengths, (int64_t)B * 4)};
  if (clash(out, rest)) return ATTN_ERR_INVALID_ARG;
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2; ++j)
      if (!(i == j && same(out[i], in[j])) && share(out[i], in[j])) return ATTN_ERR_INVALID_ARG;  // in place, or apart
  for (int i = 0; i < 2; ++i)
    if (!aligned(in[i].n ? in[i].p : nullptr, esize) || !aligned(out[i].n ? out[i].p : nullptr, esize)) return ATTN_ERR_UNSUPPORTED;
  if (!aligned(inv_freq, 8) || !aligned(positions, 4) || !aligned(q_starts, 4) || !aligned(total_lengths, 4))
    return ATTN_ERR_UNSUPPORTED;
  if ((int64_t)Hq + Hk > 65535) return ATTN_ERR_UNSUPPORTED;
  RopeParams p{};
  p.in[0] = q; p.in[1] = k;
  p.out[0] = q_out; p.out[1] = k_out;
  p.in_stride[0] = q_token_stride; p.in_stride[1] = k_token_stride;
  p.out_stride[0] = q_out_token_stride; p.out_stride[1] = k_out_token_stride;
  p.H[0] = Hq; p.H[1] = Hk;
  p.freq = inv_freq;
  p.positions = positions; p.q_starts = q_starts; p.totals = total_lengths;
  p.T = num_tokens; p.B = B; p.D = D; p.rotary = rotary_dim;
  p.inverse = inverse != 0;
  for (int i = 0; i < 2; ++i) p.in_place[i] = p.H[i] == 0 || same(out[i], in[i]);
  p.scale = scale;
  if (rotary_dim == 0 && p.in_place[0] && p.in_place[1]) return ATTN_OK;  // nothing turns, nothing moves
  const cudaError_t e = launch_rope(p, interleaved != 0, dtype, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ATTN_OK : cuda_fail(e);
}

namespace {

// How a call of attn_fwd_paged_fp4 runs: rows of a unit, CTAs, and the parts of the workspace.
struct Plan4 {
  int rows, grid;
  size_t ml_at, cuts_at, bytes;
};

// `max_tiles`: key tiles that a unit may see, as far as the host knows; the workspace does not depend on it.
Plan4 plan4(int64_t T, int64_t B, int Hq, int Hkv, int D, int64_t max_tiles) {
  Plan4 pl{};
  if (T <= 0 || B <= 0 || Hkv <= 0 || Hq < Hkv || D <= 0) return pl;
  const int group = Hq / Hkv, sms = paged_sm_count();
  // Rows per (request, kv head) of an even batch; a request with more takes several units.  The lengths are on the device,
  // so the mean is all there is to go by.  A unit of 16 rows costs 1.5 times one of 8.  48 requests of up to 8K tokens, 4 kv
  // heads, D = 128, in units of 8 and of 16 rows: 12 rows 53 and 48 us, 16 rows 49 and 44, 24 rows 69 and 74, 32 rows 89 and
  // 77; 4 requests, 16 rows 14.1 and 13.7.
  const int64_t rows = std::max<int64_t>(1, (T + B / 2) / B) * group, eights = (rows + 7) / 8;
  pl.rows = eights == 1 || eights == 3 ? 8 : 16;
  const size_t slots = 2 * (size_t)sms * (rows <= 16 ? 16 : kPagedTcRows);  // the choice below needs no more
  const size_t cuts = (size_t)sms * kPaged4DecCtas;
  // The few-rows kernel takes 300 tiles a microsecond in units of 8 rows, 200 in units of 16, the many-rows kernel 100 of its
  // 256 rows; a unit costs some tiles more; and what one unit's tiles leave on many SMs takes the latter up to 13 us to join.
  // Of the tiles that there may be to read (the tables' width, or the window) 0.7 are taken to be there.  Few and many: 4 kv
  // heads, 48 requests of up to 8K, 24 rows 69 and 85 us, 32 rows 77 and 86; 8 requests, 32 rows 25 and 32, 64 rows 40 and
  // 33; one of 4K, 64 rows 13 and 30, 128 rows 17 and 31, 512 rows 35 and 28; 8 kv heads, 4 requests of 32K, 32 rows 85 and
  // 102, 200 tokens over 800 34 and 25; prompts of 4 kv heads: one of 500 tokens 26 and 22, 4 of 120 19 and 11.  D = 64: the
  // same order.
  auto time = [&](int unit, int64_t over, int64_t rate) {
    return (double)(B * Hkv * ((rows + unit - 1) / unit)) * (0.7 * max_tiles + over) / rate;
  };
  const double few = pl.rows == 8 ? time(8, 2, 300) : time(16, 4, 200);
  const double many = time(kPagedTcRows, 3, 100) + std::min<int64_t>(13, 3 + 3 * max_tiles);
  if (rows > 16 && few >= many) pl.rows = kPagedTcRows;
  const int64_t most = (int64_t)sms * (pl.rows == 8 ? kPaged4DecCtas : 1);
  const int64_t units = (T * group / pl.rows + B) * Hkv;  // no more CTAs than there can be tiles
  pl.grid = (int)(units >= most || units * max_tiles >= most ? most : units * max_tiles);
  pl.ml_at = slots * D * 4;
  pl.cuts_at = pl.ml_at + slots * 8;
  pl.bytes = pl.cuts_at + cuts * sizeof(PagedCut);
  return pl;
}

}  // namespace

extern "C" size_t attn_paged_fp4_workspace_bytes(int num_tokens, int B, int Hq, int Hkv, int D) {
  return plan4(num_tokens, B, Hq, Hkv, D, 1).bytes;
}

extern "C" int attn_fwd_paged_fp4(const void* q, const void* k_cache, const void* v_cache, const void* k_scales,
                                  const void* v_scales, const float* k_head_scales, const float* v_head_scales,
                                  const int32_t* block_tables, const int32_t* q_starts, const int32_t* total_lengths,
                                  void* out, float* lse, int num_tokens, int B, int Hq, int Hkv, int D,
                                  int64_t q_token_stride, int num_blocks, int block_size, int max_blocks, int causal,
                                  int local_window, float scale, float softcap, int dtype, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  if (!dtype_ok(dtype)) return ATTN_ERR_INVALID_ARG;
  if (num_tokens < 0 || B < 0 || Hq <= 0 || Hkv <= 0 || D <= 0 || Hq % Hkv != 0) return ATTN_ERR_INVALID_ARG;
  if (num_blocks < 0 || block_size <= 0 || max_blocks < 0) return ATTN_ERR_INVALID_ARG;
  if (causal != 0 && causal != 1) return ATTN_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || !std::isfinite(softcap)) return ATTN_ERR_INVALID_ARG;
  int64_t codes, rows, out_elems, table_bytes;
  if (!cache_bytes(num_blocks, Hkv, block_size, D, &codes)) return ATTN_ERR_INVALID_ARG;
  const int64_t T = num_tokens, wq = (int64_t)Hq * D;
  if (!stride_ok(T, q_token_stride, wq)) return ATTN_ERR_INVALID_ARG;
  if (!mul_ok(T, Hq, &rows) || rows > INT32_MAX - 1024 || !mul_ok(rows, D, &out_elems)) return ATTN_ERR_INVALID_ARG;
  if (!mul_ok((int64_t)B * 4, max_blocks, &table_bytes)) return ATTN_ERR_INVALID_ARG;
  if ((int64_t)max_blocks * block_size > INT32_MAX - 127) return ATTN_ERR_INVALID_ARG;  // rounded up to a tile of 128
  if (T == 0 || B == 0) return ATTN_OK;  // no row belongs to a request
  if (!q || !out || !q_starts || !total_lengths) return ATTN_ERR_INVALID_ARG;
  if (num_blocks == 0 || !k_cache || !v_cache || !k_scales || !v_scales || (max_blocks > 0 && !block_tables))
    return ATTN_ERR_INVALID_ARG;
  const size_t need = attn_paged_fp4_workspace_bytes(num_tokens, B, Hq, Hkv, D);
  if (need > 0 && (!workspace || workspace_bytes < need)) return ATTN_ERR_INVALID_ARG;
  const int64_t n = (int64_t)B * 4, hb = (int64_t)Hkv * 4;
  const Rows w[] = {flat(out, out_elems * 2), flat(lse, rows * 4), flat(workspace, (int64_t)need)};
  const Rows r[] = {{q, T, wq * 2, q_token_stride * 2}, flat(k_cache, codes), flat(v_cache, codes), flat(k_scales, codes / 8),
                    flat(v_scales, codes / 8), flat(k_head_scales, hb), flat(v_head_scales, hb), flat(block_tables, table_bytes),
                    flat(q_starts, n + 4), flat(total_lengths, n)};
  if (clash(w, r)) return ATTN_ERR_INVALID_ARG;
  if (dtype == ATTN_F32 || (D != 64 && D != 128) || block_shift(block_size) < 0 || B > kPagedMaxRequests || Hq > 65535)
    return ATTN_ERR_UNSUPPORTED;
  if (!aligned(q, 16) || (q_token_stride * 2) % 16 != 0 || !aligned(out, 16) || !aligned(k_cache, 16) ||
      !aligned(v_cache, 16) || !aligned(k_scales, 16) || !aligned(v_scales, 16) || (need > 0 && !aligned(workspace, 16)))
    return ATTN_ERR_UNSUPPORTED;
  if (!aligned(lse, 4) || !aligned(k_head_scales, 4) || !aligned(v_head_scales, 4) || !aligned(block_tables, 4) ||
      !aligned(q_starts, 4) || !aligned(total_lengths, 4))
    return ATTN_ERR_UNSUPPORTED;

  int err = ATTN_OK;
  int* status = status_ptr(&err);
  if (!status) return err;
  Paged4Params P{};
  PagedParams& p = P.c;
  p.q = q;
  p.q_stride = q_token_stride;
  p.k_cache = static_cast<const uint8_t*>(k_cache);
  p.v_cache = static_cast<const uint8_t*>(v_cache);
  P.k_sc = static_cast<const uint8_t*>(k_scales);
  P.v_sc = static_cast<const uint8_t*>(v_scales);
  P.k_heads = k_head_scales;
  P.v_heads = v_head_scales;
  p.tables = block_tables;
  p.q_starts = q_starts;
  p.totals = total_lengths;
  p.out = out;
  p.lse = lse;
  p.T = num_tokens; p.B = B; p.Hq = Hq; p.Hkv = Hkv; p.D = D; p.group = Hq / Hkv;
  p.num_blocks = num_blocks; p.block_size = block_size; p.width = max_blocks;
  p.block_shift = block_shift(block_size);
  p.cap = max_blocks * block_size;
  p.group_shift = -1;
  for (int i = 0; i < 31; ++i)
    if (p.group == 1 << i) p.group_shift = i;
  p.causal = causal;
  p.local_window = local_window > 0 ? local_window : 0;
  p.scale = scale;
  // caps that leave fp32 scores as they are, and caps that leave nothing of them: their factors would pass fp32's range
  p.softcap = softcap > 0.0f && softcap < 0x1p100f ? std::max(softcap, 0x1p-100f) : 0.0f;
  p.timeout_ns = wait_timeout_ns();
  p.status = status;
  const int64_t max_tiles = std::max<int64_t>(1, ((int64_t)max_blocks * block_size + 127) / 128);
  // tiles that a unit of an even batch can see
  const int64_t seen = p.local_window > 0 ? std::min(max_tiles, (p.local_window + T / B) / 128 + 2) : max_tiles;
  const Plan4 plan = plan4(T, B, Hq, Hkv, D, seen);
  P.ws_o = static_cast<float*>(workspace);
  P.ws_ml = reinterpret_cast<float2*>(static_cast<char*>(workspace) + plan.ml_at);
  P.cuts = reinterpret_cast<PagedCut*>(static_cast<char*>(workspace) + plan.cuts_at);
  const bool bf16 = dtype == ATTN_BF16;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = plan.rows == kPagedTcRows ? launch_attn_paged4_tc(P, plan.grid, bf16, st)
                                            : launch_attn_paged4_dec(P, plan.rows, plan.grid, bf16, st);
  if (e == cudaSuccess && max_tiles > 1) {
    PagedLaunch L{};
    L.c = p;
    L.rows = plan.rows;
    L.grid = plan.grid;
    L.ws_o = P.ws_o;
    L.ws_ml = P.ws_ml;
    L.cuts = P.cuts;
    L.ml_log2 = (plan.rows == kPagedTcRows ? kPagedTcLog2 : kPaged4DecLog2) - kPagedSumLog2;
    // Parts a unit, about: CTAs over units.  64 requests (three) take 41.8 us with a CTA a row and 39.4 with one a unit, one
    // request of 4K (39) 8.9 and 9.3, 4 of 16 rows (ten) 13.8 and 15.9.
    const int64_t parts = plan.grid / ((int64_t)B * Hkv * std::max<int64_t>(1, (T / B * p.group + plan.rows - 1) / plan.rows)) + 1;
    e = plan.rows == kPagedTcRows || parts > 8 ? launch_attn_paged_join(L, bf16, st) : launch_attn_paged4_join(L, bf16, st);
  }
  return e == cudaSuccess ? ATTN_OK : cuda_fail(e);
}
