// Internal definitions of head_norm_rotary (not public).
#pragma once

#include "vbq_common.h"

namespace vbq {

// One of the two tensors: rows [token][head][channel], strides in elements.
struct HeadRows {
  const void* in;
  void* out;
  const float* weight;   // NULL: not normed
  int64_t in_ts, in_hs, out_ts, out_hs;
  int32_t heads, out_dtype;
};

struct HeadRotary {
  HeadRows q, k;
  const int32_t* positions;
  const float* inv_freq;
  const uint8_t* axis;     // NULL: one axis
  int64_t position_stride;
  int64_t tokens;
  int32_t head_dim, rotary_dim, axes, interleaved;
  float eps;
  int32_t passes;          // wavefronts that share a token (set by the launch)
};

hipError_t launch_head_norm_rotary(HeadRotary a, int dtype, hipStream_t s);

}  // namespace vbq
