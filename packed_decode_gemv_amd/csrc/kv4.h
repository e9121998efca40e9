// Internal definitions of the 4-bit key/value cache (not public).
#pragma once

#include "vbq_common.h"

namespace vbq {

constexpr int kKvBlock = VBQ_KV4_BLOCK_TOKENS;
constexpr int kKvGroupBytes = 2304;   // a block's bytes per 64 channels

// Byte offsets inside a block of G groups.
__host__ __device__ constexpr int kv_value_codes(int G) { return 1024 * G; }
__host__ __device__ constexpr int kv_key_so(int G) { return 2048 * G; }
__host__ __device__ constexpr int kv_value_so(int G) { return 2176 * G; }

// What a kernel needs of a cache. Blocks are found as
// ((page * heads + head) << block_shift) + block in the page.
struct KvCache {
  uint8_t* data;
  uint32_t* flags;
  int32_t n_pages;
  int32_t heads;
  int32_t block_shift;   // log2(page_tokens / 32)
  int32_t groups;        // head_dim / 64
};

struct KvRange {
  int32_t batch, width, total, max_tokens;
  const int32_t* table;
  const int32_t* start;
  const int32_t* cu;
};

__device__ inline void kv_flag(const KvCache& c, uint32_t bits) {
  if (c.flags) atomicOr(c.flags, bits);
}

// Address of a block of a valid page.
__device__ inline uint8_t* kv_block(const KvCache& c, int G, uint32_t page, int head, uint32_t block_in_page) {
  const uint64_t n = (((uint64_t)page * (uint32_t)c.heads + (uint32_t)head) << c.block_shift) + block_in_page;
  return c.data + n * (uint32_t)(kKvGroupBytes * G);
}

struct KvAttn {
  KvCache cache;
  const int32_t* table;
  const int32_t* lens;
  const int32_t* cu;
  const uint16_t* q;
  int64_t q_ts, q_hs;
  uint16_t* out;
  float* lse;
  uint32_t* counters;   // per (sequence, head): parts done; zero between calls
  float* acc;           // sums of parts, by workgroup: [rows][head_dim]
  float* ml;            // their bases (powers of two) and sums of p: [rows][2]
  int32_t width, total_q, max_q, max_kv;
  int32_t n_heads, ratio;      // query heads, and how many share a key/value head
  int32_t bf16, causal, window, sinks;
  int32_t ratio_inv;           // ceil(65536 / ratio)
  int32_t batch;
  int32_t parts;               // up to 32 rows: that long tiles are cut into in all, about (0: no cuts, a
                               // workgroup a tile); more rows: that each tile is cut into, at most
  float scale_log2;            // scale * log2(e)
};

// A launch's first dimension holds 2^32 - 1 threads, and more are cut off without an error.
constexpr bool kv_grid_fits(int64_t groups, int64_t threads) { return groups * threads <= (int64_t)UINT32_MAX; }

hipError_t launch_kv4_append(const KvCache& c, const KvRange& r, const void* k, const void* v, int dtype,
                             int64_t k_ts, int64_t k_hs, int64_t v_ts, int64_t v_hs, hipStream_t s);
hipError_t launch_kv4_read(const KvCache& c, const KvRange& r, void* k, void* v, int dtype, hipStream_t s);
// Sizes of an attention launch, from the call's sizes alone: rows of a tile,
// parts (as above), tiles, workgroups and their threads, and places for sums in
// the workspace.
struct KvAttnPlan {
  int32_t rows, parts, threads;
  int64_t tiles, grid, places;
};
KvAttnPlan kv4_attn_plan(int batch, int heads, int ratio, int groups, int total_q, int max_q, int max_kv, int window,
                         int sinks);
hipError_t launch_kv4_attention(const KvAttn& a, const KvAttnPlan& p, hipStream_t s);

}  // namespace vbq
