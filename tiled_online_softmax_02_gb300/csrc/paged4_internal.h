// paged4_internal.h -- parameter blocks and launchers of the paged 4-bit KV
// cache and of the rotary positions, shared between the C ABI layer
// (paged4_api.cu) and the kernels.  Not part of the public interface.
//
// The 4-bit cache has the blocks, slots and block tables of the 8-bit one.  A
// row of D values is D / 2 bytes of e2m1 (value 2 i in the low half of byte i)
// and D / 16 bytes of e4m3, one scale for every 16 values; a kv head may carry
// an f32 factor besides: value = e2m1 * e4m3 * head.
#pragma once

#include "paged_internal.h"

namespace gb300_attn {

constexpr int kGroup4 = 16;  // values that share a scale

// attn_cache_append_fp4 and attn_cache_read_fp4: rows x[0] = k, x[1] = v.
struct Cache4Params {
  void* x[2];               // [T, Hkv, D]: token t, head h at x + t * stride + h * head_stride elements
  int64_t stride[2], head_stride[2];
  const int64_t* slot_map;  // [T]
  uint8_t* cache[2];        // [num_blocks, Hkv, block_size, D / 2]
  uint8_t* scales[2];       // [num_blocks, Hkv, block_size, D / 16]
  const float* heads[2];    // [Hkv] or nullptr
  int64_t num_slots;        // num_blocks * block_size
  int T, Hkv, D, block_size, block_shift;
};

struct RopeParams {
  const void* in[2];        // q [T, Hq, D], k [T, Hk, D]: token t at in + t * in_stride elements
  void* out[2];
  int64_t in_stride[2], out_stride[2];
  int H[2];
  const double* freq;       // [rotary / 2] radians a position
  const int32_t* positions; // [T], or nullptr: from the next two
  const int32_t* q_starts;  // [B + 1]
  const int32_t* totals;    // [B]
  int T, B, D, rotary;
  bool inverse, in_place[2];
  float scale;
};

// attn_fwd_paged_fp4: c.k_cache and c.v_cache hold e2m1 bytes, c.k_scales and c.v_scales are not used.
struct Paged4Params {
  PagedParams c;
  const uint8_t* k_sc;      // e4m3 [num_blocks, Hkv, block_size, D / 16]
  const uint8_t* v_sc;
  const float* k_heads;     // [Hkv] or nullptr
  const float* v_heads;
  float* ws_o;              // [2 * grid][rows][D]: partial rows
  float2* ws_ml;            // [2 * grid][rows]: m, 2^-8 of the sum
  PagedCut* cuts;           // [grid]
};

constexpr int kPaged4DecCtas = 2;        // CTAs of the few-rows kernel on an SM, in units of 8 rows
// Length of a CTA's piece of the work line, at least, in tiles (and in the kOver that a unit's head takes of the line, so the
// pieces of short units may hold one tile or none): the few-rows kernel's eight warps have 256 keys between them in the time of
// 32, and every part of a unit is one more to join.  One request of 3.5K in pieces of 1, 2, 3, 4 tiles 9.8, 8.9, 9.2 and 9.4 us; 512 rows over
// 4K, 4 kv heads, in the many-rows kernel 33, 28, 26 and 26; a prompt of 500 tokens there 21.3, 21.2, 22.4 and 22.1.
constexpr int kPaged4Piece = 2;
constexpr float kPaged4DecLog2 = 5.0f;   // log2 of the factor that P carries

// A launch that may begin while the kernel before it on the stream drains: every kernel launched so waits for all of that
// one (after_earlier_kernels) before it reads or writes anything.
template <typename... KArgs, typename... Args>
cudaError_t launch_early(void (*kernel)(KArgs...), unsigned grid, unsigned block, size_t smem, cudaStream_t stream, Args&&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(block, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

cudaError_t launch_cache4_append(const Cache4Params& p, int dtype, cudaStream_t stream);
cudaError_t launch_cache4_read(const Cache4Params& p, int dtype, cudaStream_t stream);
cudaError_t launch_rope(const RopeParams& p, bool interleaved, int dtype, cudaStream_t stream);
cudaError_t launch_attn_paged4_dec(const Paged4Params& p, int rows, int grid, bool bf16, cudaStream_t stream);  // rows 8 or 16
cudaError_t launch_attn_paged4_tc(const Paged4Params& p, int grid, bool bf16, cudaStream_t stream);  // rows kPagedTcRows

cudaError_t launch_attn_paged4_join(const PagedLaunch& L, bool bf16, cudaStream_t stream);  // rows 8 or 16, few parts a unit

}  // namespace gb300_attn
