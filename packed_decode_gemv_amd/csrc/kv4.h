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
  // With shared tokens (see Part in kvattn_kernels.h); batch, max_q and max_kv are then those
  // of a launch: groups with their rows and shared tokens, or sequences with their own.
  const int32_t* groups;       // [n_groups + 1] sequences before each
  const int32_t* shared;       // [n_groups] tokens
  float* sums;                 // of a launch's rows: [total_q][n_heads][head_dim]
  float* sums_ml;              // their bases and sums of p
  int32_t n_groups, sequences, max_shared, max_group_q;
};

// A fork (see kvfork.hip): the call's arguments, and places in its workspace.
struct KvFork {
  KvCache cache;
  const int32_t* table_in;
  const int32_t* lens_in;
  const int32_t* refs_in;
  const int32_t* parents;
  const int32_t* reserve;   // NULL: none
  int32_t* table_out;
  int32_t* lens_out;
  int32_t* refs_out;
  int32_t batch_in, batch_out, width;
  int32_t* head;     // pages that were found; copies
  int4* copies;      // [batch_out] page, which of the pages to take, blocks
  int32_t* offset;   // [batch_out] pages taken by the sequences before, sign bit: a first continuation
  int32_t* kids;     // [batch_in] continuations
  int32_t* first;    // [batch_in] (used where they do not fit LDS)
  int32_t* free;     // the pages to take
  uint32_t copiers;  // workgroups that copy (set by the launch)
};
hipError_t launch_kv4_fork(const KvFork& f, hipStream_t s);

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
// (see kvshared.h) for heads of 64, 128, 192 and 256 channels. each: one launch, `own` over all tokens.
hipError_t launch_kv4_attention_shared_g1(const KvAttn& shared, const KvAttnPlan& sp, const KvAttn& own,
                                          const KvAttnPlan& op, bool each, hipStream_t s);
hipError_t launch_kv4_attention_shared_g2(const KvAttn& shared, const KvAttnPlan& sp, const KvAttn& own,
                                          const KvAttnPlan& op, bool each, hipStream_t s);
hipError_t launch_kv4_attention_shared_g3(const KvAttn& shared, const KvAttnPlan& sp, const KvAttn& own,
                                          const KvAttnPlan& op, bool each, hipStream_t s);
hipError_t launch_kv4_attention_shared_g4(const KvAttn& shared, const KvAttnPlan& sp, const KvAttn& own,
                                          const KvAttnPlan& op, bool each, hipStream_t s);

}  // namespace vbq
