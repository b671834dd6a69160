// paged_api.cu -- the C ABI of the paged 8-bit KV cache (attn_cache_assign,
// attn_cache_append_fp8, attn_fwd_paged_fp8 in include/attn.h): argument
// validation, then one launcher call each.  As for attn_fwd, a request the
// kernels cannot run is refused with a status before anything is launched.
#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>
#include <cstdint>

#include "../../include/attn.h"
#include "api_internal.h"
#include "paged_internal.h"

using namespace gb300_attn;

namespace {

bool block_size_ok(int bs) { return bs == 16 || bs == 32 || bs == 64 || bs == 128; }

int block_shift(int bs) { return bs == 16 ? 4 : bs == 32 ? 5 : bs == 64 ? 6 : 7; }

struct Span {
  const void* p;
  int64_t bytes;
};

// Whether any written span overlaps another span.
template <int NW, int NR>
bool clash(const Span (&w)[NW], const Span (&r)[NR]) {
  for (int i = 0; i < NW; ++i) {
    for (int j = i + 1; j < NW; ++j)
      if (overlaps(w[i].p, w[i].bytes, w[j].p, w[j].bytes)) return true;
    for (int j = 0; j < NR; ++j)
      if (overlaps(w[i].p, w[i].bytes, r[j].p, r[j].bytes)) return true;
  }
  return false;
}

// Bytes of the cache (one of K, V); false when they pass 2^60 or the tiles pass a tensor map's 2^31 planes.
bool cache_bytes(int num_blocks, int Hkv, int block_size, int D, int64_t* bytes) {
  int64_t tiles, t;
  return mul_ok(num_blocks, Hkv, &tiles) && tiles <= INT32_MAX && mul_ok(tiles, (int64_t)block_size * D, &t) &&
         t <= (INT64_C(1) << 60) && (*bytes = t, true);
}

// Elements spanned by n rows of `width` values, `stride` apart; false unless width <= stride.
bool strided_span(int64_t n, int64_t stride, int64_t width, int64_t* elems) {
  if (n <= 0) return *elems = 0, true;
  int64_t t;
  if (stride < width || !mul_ok(n - 1, stride, &t) || t > (INT64_C(1) << 58)) return false;
  *elems = t + width;
  return true;
}

}  // namespace

extern "C" int attn_cache_assign(const int32_t* past_lengths, const int32_t* new_lengths, const uint8_t* finished,
                                 int32_t* block_tables, int32_t* free_blocks, int32_t* free_count,
                                 int32_t* q_starts, int32_t* total_lengths, int64_t* slot_map, int32_t* result,
                                 int B, int max_blocks, int block_size, int num_blocks, int num_tokens,
                                 void* stream) {
  if (B < 0 || max_blocks < 0 || num_blocks < 0 || num_tokens < 0) return ATTN_ERR_INVALID_ARG;
  if (block_size <= 0) return ATTN_ERR_INVALID_ARG;
  if (!q_starts || !result || !free_count || (num_tokens > 0 && !slot_map) || (num_blocks > 0 && !free_blocks))
    return ATTN_ERR_INVALID_ARG;
  if (B > 0 && (!past_lengths || !new_lengths || !total_lengths || (max_blocks > 0 && !block_tables)))
    return ATTN_ERR_INVALID_ARG;
  const int64_t n = (int64_t)B * 4;
  int64_t table_bytes;
  if (!mul_ok(n, max_blocks, &table_bytes)) return ATTN_ERR_INVALID_ARG;
  const Span w[] = {{block_tables, table_bytes}, {free_blocks, (int64_t)num_blocks * 4}, {free_count, 4},
                    {q_starts, n + 4}, {total_lengths, n}, {slot_map, (int64_t)num_tokens * 8}, {result, 4}};
  const Span r[] = {{past_lengths, n}, {new_lengths, n}, {finished, B}};
  if (clash(w, r)) return ATTN_ERR_INVALID_ARG;
  if (!block_size_ok(block_size) || B > kAssignMaxRequests) return ATTN_ERR_UNSUPPORTED;
  for (const Span& s : w)
    if (!aligned(s.p, s.p == slot_map ? 8 : 4)) return ATTN_ERR_UNSUPPORTED;
  if (!aligned(past_lengths, 4) || !aligned(new_lengths, 4)) return ATTN_ERR_UNSUPPORTED;
  AssignParams p{past_lengths, new_lengths, finished, block_tables, free_blocks, free_count, q_starts, total_lengths,
                 slot_map, result, B, max_blocks, block_size, block_shift(block_size), num_blocks, num_tokens};
  const cudaError_t e = launch_cache_assign(p, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ATTN_OK : cuda_fail(e);
}

extern "C" int attn_cache_append_fp8(const void* k, const void* v, const int64_t* slot_map, void* k_cache,
                                     void* v_cache, float* k_scales, float* v_scales, int num_tokens, int Hkv, int D,
                                     int64_t k_token_stride, int64_t v_token_stride, int num_blocks, int block_size,
                                     int dtype, void* stream) {
  if (dtype != ATTN_F32 && dtype != ATTN_F16 && dtype != ATTN_BF16) return ATTN_ERR_INVALID_ARG;
  if (num_tokens < 0 || Hkv <= 0 || D <= 0 || num_blocks < 0 || block_size <= 0) return ATTN_ERR_INVALID_ARG;
  const int64_t esize = dtype == ATTN_F32 ? 4 : 2, width = (int64_t)Hkv * D;
  int64_t cbytes, kspan, vspan;
  if (!cache_bytes(num_blocks, Hkv, block_size, D, &cbytes)) return ATTN_ERR_INVALID_ARG;
  if (!strided_span(num_tokens, k_token_stride, width, &kspan) ||
      !strided_span(num_tokens, v_token_stride, width, &vspan))
    return ATTN_ERR_INVALID_ARG;
  if (num_tokens == 0 || num_blocks == 0) return ATTN_OK;  // nothing to write, or nowhere
  if (!k || !v || !slot_map || !k_cache || !v_cache || !k_scales || !v_scales) return ATTN_ERR_INVALID_ARG;
  const int64_t sbytes = (int64_t)num_blocks * Hkv * 4;
  const Span w[] = {{k_cache, cbytes}, {v_cache, cbytes}, {k_scales, sbytes}, {v_scales, sbytes}};
  const Span r[] = {{k, kspan * esize}, {v, vspan * esize}, {slot_map, (int64_t)num_tokens * 8}};
  if (clash(w, r)) return ATTN_ERR_INVALID_ARG;
  if (!block_size_ok(block_size) || (D != 64 && D != 128) || Hkv > 65535) return ATTN_ERR_UNSUPPORTED;
  if (!aligned(k, 16) || !aligned(v, 16) || (k_token_stride * esize) % 16 != 0 ||
      (v_token_stride * esize) % 16 != 0 || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      !aligned(k_scales, 4) || !aligned(v_scales, 4) || !aligned(slot_map, 8))
    return ATTN_ERR_UNSUPPORTED;
  AppendParams p{};
  p.x[0] = k; p.x[1] = v;
  p.stride[0] = k_token_stride; p.stride[1] = v_token_stride;
  p.slot_map = slot_map;
  p.cache[0] = static_cast<uint8_t*>(k_cache); p.cache[1] = static_cast<uint8_t*>(v_cache);
  p.scales[0] = k_scales; p.scales[1] = v_scales;
  p.num_slots = (int64_t)num_blocks * block_size;
  p.T = num_tokens; p.Hkv = Hkv; p.D = D; p.block_size = block_size;
  p.block_shift = block_shift(block_size);
  const cudaError_t e = launch_cache_append(p, dtype, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ATTN_OK : cuda_fail(e);
}

namespace {

// SMs of the current device, looked up once for each.
int sm_count() {
  static std::atomic<int> cache[128];
  int dev = 0, sms = 152;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 128) return sms;
  const int known = cache[dev].load(std::memory_order_relaxed);
  if (known > 0) return known;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 152;
  cache[dev].store(sms, std::memory_order_relaxed);
  return sms;
}

// How a call of attn_fwd_paged_fp8 runs: rows of a unit, CTAs, and the parts of the workspace.
struct PagedPlan {
  int rows, grid;
  size_t ml_at, cuts_at, bytes;
};

PagedPlan paged_plan(int64_t T, int64_t B, int Hq, int Hkv, int D, int64_t max_tiles) {
  PagedPlan pl{};
  if (T <= 0 || B <= 0 || Hkv <= 0 || Hq < Hkv || D <= 0) return pl;
  const int group = Hq / Hkv;
  // Rows per (request, kv head) of an even batch; a request with more takes several units.  The few-rows kernel's
  // time a tile grows with the rows it holds, the many-rows kernel's does not.  48 requests of up to 8K tokens, 4 kv
  // heads, D = 128: 9, 12, 16 rows take 64, 70, 74 us in units of 16 and 93 in the many-rows kernel; 20 and 32 rows
  // 110 and 125 us as two units of 16 each, 94 there.
  // Lengths are on the device, so the mean is all there is to go by, padding rows in it: 64 single tokens at 4K take 87
  // us, in a T of 2048 rows 204; 63 of them with one chunk of 2048 332 us, where the two alone take 86 and 116.
  const int64_t rows = std::max<int64_t>(1, (T + B / 2) / B) * group;
  pl.rows = rows <= 4 ? 4 : rows <= 8 ? 8 : rows <= 16 ? 16 : kPagedTcRows;
  int64_t most = (int64_t)sm_count() * (pl.rows == kPagedTcRows ? 1 : kPagedDecCtas);
  const size_t slots = 2 * (size_t)most * pl.rows;  // the choice below needs no more
  // With little to read a call is the way to the first result and the join of the parts, both shorter in units of 8
  // rows, and reading the keys once a unit costs nothing yet.  What there may be to read: the tables' width.
  // 4 kv heads: 12 rows, 4 requests of up to 8K tokens 14.8 us against 18.8; 16 rows, 4 of 100K 125 against 84.  32
  // rows, 8 requests of up to 8K 27 against 30 (4 of them 18 against 28); 16 of them 48 against 41.  8 kv heads: 128
  // rows, one request of 4K 27 against 31; two of them 37 against 26.
  const int64_t eights = B * Hkv * ((rows + 7) / 8), small = (int64_t)1 << 13;  // key tiles
  if (pl.rows == 16 ? eights * max_tiles <= 2 * small
                    : pl.rows == kPagedTcRows && eights <= sm_count() && eights * max_tiles <= small) {
    pl.rows = 8;
    most = (int64_t)sm_count() * kPagedDecCtas;
  }
  // no more CTAs than there can be tiles
  const int64_t units = (T * group / pl.rows + B) * Hkv;
  pl.grid = (int)(units >= most || units * max_tiles >= most ? most : units * max_tiles);
  pl.ml_at = slots * D * 4;
  pl.cuts_at = pl.ml_at + slots * 8;
  pl.bytes = pl.cuts_at + (size_t)sm_count() * kPagedDecCtas * sizeof(PagedCut);
  return pl;
}

// The cache as a 3-D map of bytes [num_blocks * Hkv, block_size, D]; a box is one block of one head, its rows in
// the swizzle that the tensor cores read; planes out of range read as zero.
int encode_cache(CUtensorMap* map, const void* base, int64_t planes, int block_size, int D) {
  int err = ATTN_OK;
  auto fn = encode_fn(&err);
  if (!fn) return err;
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)block_size, (cuuint64_t)planes};
  const cuuint64_t strides[2] = {(cuuint64_t)D, (cuuint64_t)block_size * (cuuint64_t)D};
  const cuuint32_t box[3] = {(cuuint32_t)D, (cuuint32_t)block_size, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  auto encode = [&] {
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  };
  if (encode() == CUDA_SUCCESS) return ATTN_OK;
  // a host thread that has made no runtime call yet has no context current, which the driver call needs
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaSetDevice(dev);
  if (e != cudaSuccess) return cuda_fail(e);
  return encode() == CUDA_SUCCESS ? ATTN_OK : cuda_fail(cudaErrorInvalidValue);
}

}  // namespace

extern "C" size_t attn_paged_workspace_bytes(int num_tokens, int B, int Hq, int Hkv, int D) {
  return paged_plan(num_tokens, B, Hq, Hkv, D, 1).bytes;
}

extern "C" int attn_fwd_paged_fp8(const void* q, const void* k_cache, const void* v_cache, const float* k_scales,
                                  const float* v_scales, const int32_t* block_tables, const int32_t* q_starts,
                                  const int32_t* total_lengths, void* out, float* lse, int num_tokens, int B, int Hq,
                                  int Hkv, int D, int64_t q_token_stride, int num_blocks, int block_size,
                                  int max_blocks, int causal, int local_window, float scale, float softcap, int dtype,
                                  void* workspace, size_t workspace_bytes, void* stream) {
  if (dtype != ATTN_F32 && dtype != ATTN_F16 && dtype != ATTN_BF16) return ATTN_ERR_INVALID_ARG;
  if (num_tokens < 0 || B < 0 || Hq <= 0 || Hkv <= 0 || D <= 0 || Hq % Hkv != 0) return ATTN_ERR_INVALID_ARG;
  if (num_blocks < 0 || block_size <= 0 || max_blocks < 0) return ATTN_ERR_INVALID_ARG;
  if (causal != 0 && causal != 1) return ATTN_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || !std::isfinite(softcap)) return ATTN_ERR_INVALID_ARG;
  int64_t cbytes, qspan, rows, out_elems, table_bytes;
  if (!cache_bytes(num_blocks, Hkv, block_size, D, &cbytes)) return ATTN_ERR_INVALID_ARG;
  if (!strided_span(num_tokens, q_token_stride, (int64_t)Hq * D, &qspan)) return ATTN_ERR_INVALID_ARG;
  if (!mul_ok(num_tokens, Hq, &rows) || rows > INT32_MAX - 1024 || !mul_ok(rows, D, &out_elems))
    return ATTN_ERR_INVALID_ARG;
  if (!mul_ok((int64_t)B * 4, max_blocks, &table_bytes)) return ATTN_ERR_INVALID_ARG;
  if ((int64_t)max_blocks * block_size > INT32_MAX - 127) return ATTN_ERR_INVALID_ARG;  // rounded up to a tile of 128
  if (num_tokens == 0 || B == 0) return ATTN_OK;  // no row belongs to a request
  if (!q || !out || !q_starts || !total_lengths) return ATTN_ERR_INVALID_ARG;
  if (num_blocks == 0 || !k_cache || !v_cache || !k_scales || !v_scales || (max_blocks > 0 && !block_tables))
    return ATTN_ERR_INVALID_ARG;
  const size_t need = attn_paged_workspace_bytes(num_tokens, B, Hq, Hkv, D);
  if (need > 0 && (!workspace || workspace_bytes < need)) return ATTN_ERR_INVALID_ARG;
  const int64_t sbytes = (int64_t)num_blocks * Hkv * 4, n = (int64_t)B * 4;
  const Span w[] = {{out, out_elems * 2}, {lse, rows * 4}, {workspace, (int64_t)need}};
  const Span r[] = {{q, qspan * 2}, {k_cache, cbytes}, {v_cache, cbytes}, {k_scales, sbytes}, {v_scales, sbytes},
                    {block_tables, table_bytes}, {q_starts, n + 4}, {total_lengths, n}};
  if (clash(w, r)) return ATTN_ERR_INVALID_ARG;
  if (dtype == ATTN_F32 || (D != 64 && D != 128) || !block_size_ok(block_size) || B > kPagedMaxRequests ||
      Hq > 65535)
    return ATTN_ERR_UNSUPPORTED;
  if (!aligned(q, 16) || (q_token_stride * 2) % 16 != 0 || !aligned(out, 16) || !aligned(k_cache, 16) ||
      !aligned(v_cache, 16) || (need > 0 && !aligned(workspace, 16)))
    return ATTN_ERR_UNSUPPORTED;
  if (!aligned(lse, 4) || !aligned(k_scales, 4) || !aligned(v_scales, 4) || !aligned(block_tables, 4) ||
      !aligned(q_starts, 4) || !aligned(total_lengths, 4))
    return ATTN_ERR_UNSUPPORTED;

  int err = ATTN_OK;
  int* status = status_ptr(&err);
  if (!status) return err;
  PagedParams p{};
  p.q = q;
  p.q_stride = q_token_stride;
  p.k_cache = static_cast<const uint8_t*>(k_cache);
  p.v_cache = static_cast<const uint8_t*>(v_cache);
  p.k_scales = k_scales;
  p.v_scales = v_scales;
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
  const bool bf16 = dtype == ATTN_BF16;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int64_t max_tiles = std::max<int64_t>(1, ((int64_t)max_blocks * block_size + 127) / 128);
  const PagedPlan plan = paged_plan(num_tokens, B, Hq, Hkv, D, max_tiles);
  PagedLaunch L{};
  L.c = p;
  int rc = encode_cache(&L.tmap_k, k_cache, (int64_t)num_blocks * Hkv, block_size, D);
  if (rc == ATTN_OK) rc = encode_cache(&L.tmap_v, v_cache, (int64_t)num_blocks * Hkv, block_size, D);
  if (rc != ATTN_OK) return rc;
  L.rows = plan.rows;
  L.grid = plan.grid;
  L.ws_o = static_cast<float*>(workspace);
  L.ws_ml = reinterpret_cast<float2*>(static_cast<char*>(workspace) + plan.ml_at);
  L.cuts = reinterpret_cast<PagedCut*>(static_cast<char*>(workspace) + plan.cuts_at);
  cudaError_t e;
  if (plan.rows == kPagedTcRows) {
    L.ml_log2 = kPagedTcLog2 - kPagedSumLog2;
    e = launch_attn_paged_tc(L, bf16, st);
  } else {
    L.ml_log2 = -kPagedSumLog2;  // its maxima already hold P's factor
    e = launch_attn_paged_dec(L, bf16, st);
  }
  if (e == cudaSuccess && max_tiles > 1) e = launch_attn_paged_join(L, bf16, st);
  return e == cudaSuccess ? ATTN_OK : cuda_fail(e);
}
