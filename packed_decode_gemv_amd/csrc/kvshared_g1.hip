// Attention with shared tokens, heads of 64 channels.
#include "kvshared.h"

namespace vbq {
hipError_t launch_kv4_attention_shared_g1(const KvAttn& shared, const KvAttnPlan& sp, const KvAttn& own,
                                          const KvAttnPlan& op, bool each, hipStream_t s) {
  return launch_shared<1>(shared, sp, own, op, each, s);
}
}  // namespace vbq
