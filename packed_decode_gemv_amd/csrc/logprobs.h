// Internal definitions of token_logprobs (not public).
#pragma once

#include "vbq_common.h"

namespace vbq {

constexpr int kLogprobStep = 1024;   // logits of one step of a wavefront
constexpr int kLogprobSplits = 32;   // workgroups that share a row, at most

// What a workgroup leaves of its part of a row, beside its best keys.
struct LogprobPart {
  float m, s, t;     // maximum, sum of e = exp(x - m), sum of e log2(e)
  int32_t before;    // logits that stand before the given token's
};

struct Logprobs {
  const void* logits;
  const void* tokens;      // NULL: none
  int64_t row_stride;
  float* logprob;
  int32_t* rank;
  float* entropy;
  float* lse;
  float* top_logprob;
  int32_t* top_index;
  uint32_t* counters;      // per row: parts done; zero between calls
  uint64_t* keys;          // [row][split][top]
  LogprobPart* parts;      // [row][split]
  int32_t rows, vocab, top, long_tokens, splits;
};

// Workgroups that share a row, from the sizes alone.
int logprob_splits(int rows, int vocab);
hipError_t launch_token_logprobs(const Logprobs& a, int dtype, hipStream_t s);

}  // namespace vbq
