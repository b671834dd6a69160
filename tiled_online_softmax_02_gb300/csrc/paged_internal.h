// paged_internal.h -- parameter blocks and launchers of the paged 8-bit KV
// cache, shared between the C ABI layer (paged_api.cu) and the kernels.  Not
// part of the public interface.
//
// The cache is num_blocks blocks of block_size token slots; a block holds
// every kv head: [num_blocks, Hkv, block_size, D] e4m3 bytes, one fp32 scale
// for each (block, head).  Slot s is row s % block_size of block
// s / block_size; a request's block table maps position p to block
// table[p / block_size].
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace gb300_attn {

// Status bit: an attention call met a block-table entry that names no block.
constexpr int kStatusBadBlock = 2;

// Codes attn_cache_assign leaves in `result`.
enum AssignResult {
  kAssignOk = 0,
  kAssignNoBlocks = 1,   // fewer free blocks than needed
  kAssignRowShort = 2,   // a request needs more table entries than a row has
  kAssignTokens = 3,     // more new tokens than the slot map holds
  kAssignLength = 4,     // a negative length
  kAssignCorrupt = 5     // free_count, a table entry or a free-list entry to be taken out of range
};

constexpr int kAssignMaxRequests = 8192;
constexpr int kPagedMaxRequests = 8192;

struct AssignParams {
  const int32_t* past;      // [B] tokens in the cache
  const int32_t* added;     // [B] tokens this step adds
  const uint8_t* finished;  // [B] or nullptr: rows that give their blocks back first
  int32_t* tables;          // [B, width]
  int32_t* free_blocks;     // [num_blocks] stack
  int32_t* free_count;      // [1]
  int32_t* q_starts;        // [B + 1]
  int32_t* totals;          // [B]
  int64_t* slot_map;        // [T]
  int32_t* result;          // [1]
  int B, width, block_size, block_shift, num_blocks, T;
};

struct AppendParams {
  const void* x[2];         // k, v: [T, Hkv, D], token t at x + t * stride elements
  int64_t stride[2];
  const int64_t* slot_map;  // [T]
  uint8_t* cache[2];        // [num_blocks, Hkv, block_size, D]
  float* scales[2];         // [num_blocks, Hkv]
  int64_t num_slots;        // num_blocks * block_size
  int T, Hkv, D, block_size, block_shift;
  int chunk;                // tokens whose runs one CTA owns
};

struct PagedParams {
  const void* q;            // [T, Hq, D], token t at q + t * q_stride elements
  int64_t q_stride;
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  const float* k_scales;
  const float* v_scales;
  const int32_t* tables;    // [B, width]
  const int32_t* q_starts;  // [B + 1]
  const int32_t* totals;    // [B]
  void* out;                // [T, Hq, D]
  float* lse;               // [T, Hq] or nullptr
  int T, B, Hq, Hkv, D, group, num_blocks, block_size, block_shift, width;
  int cap;                  // width * block_size: keys a block table can name
  int group_shift;          // log2 of group, -1 where it is no power of two
  int causal, local_window;
  float scale, softcap;
  uint64_t timeout_ns;
  int* status;
};

int paged_sm_count();  // SMs of the current device
cudaError_t launch_cache_assign(const AssignParams& p, cudaStream_t stream);
cudaError_t launch_cache_append(const AppendParams& p, int dtype, cudaStream_t stream);

// What the joining kernel is told of a unit that begins in a CTA's share and
// goes on in the next ones: its partial rows are slot 2 c + 1 of that CTA and
// slots 2 (c + k) of the CTAs after it.
struct PagedCut {
  int parts;      // CTAs that hold a part; 0: no such unit
  int token0;     // packed row of the request's first token
  int head0;      // first query head of the kv head
  int row0, rows; // rows [row0, row0 + rows): token row / group, head row % group
  int pad[3];
};

// A launch of one of the attention kernels, and of the kernel that joins the
// partial rows of units cut between CTAs.
constexpr int kPagedDecCtas = 2;     // CTAs of the few-rows kernel on an SM
constexpr int kPagedTcRows = 256;
constexpr float kPagedDecLog2 = 5.0f;  // log2 of the factor that P carries, in each of the kernels
constexpr float kPagedTcLog2 = 7.0f;
// Row sums are carried as 2^-8 of themselves: 2^31 keys of scale 2^-100 stay below fp32's range, keys of scale 2^105 above it.
constexpr float kPagedSumLog2 = 8.0f, kPagedSumFactor = 0x1p-8f;

struct PagedLaunch {
  PagedParams c;
  CUtensorMap tmap_k, tmap_v;  // e4m3 [num_blocks * Hkv, block_size, D], box {D, block_size, 1}
  int rows;                    // query rows of a unit
  int grid;
  float* ws_o;                 // [2 * grid][rows][D]: partial rows, sum of 2^(t - m) v8
  float2* ws_ml;               // [2 * grid][rows]: m, 2^-8 sum of 2^(t - m) / v_scale
  PagedCut* cuts;              // [grid]
  float ml_log2;               // the kernel's sums carry this factor (log2)
};

cudaError_t launch_attn_paged_dec(const PagedLaunch& L, bool bf16, cudaStream_t stream);  // rows 4, 8 or 16
cudaError_t launch_attn_paged_tc(const PagedLaunch& L, bool bf16, cudaStream_t stream);   // rows kPagedTcRows
cudaError_t launch_attn_paged_join(const PagedLaunch& L, bool bf16, cudaStream_t stream);

}  // namespace gb300_attn
